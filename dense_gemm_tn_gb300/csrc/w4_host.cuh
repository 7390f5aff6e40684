// Host side of the products with 4-bit weights and of their quantiser (included by
// w4.cu, inside its anonymous namespace).

bool w4_group_ok(int64_t group) { return group == 32 || group == 64 || group == 128 || group == 256; }

void record_w4(const char *name, const DeviceState &dev, int64_t tiles)
{
    t_rec = LaunchRecord{};
    t_rec.name = name;
    t_rec.grouped = 1;
    t_rec.cluster = 1;
    t_rec.grid = t_rec.tiles = static_cast<int>(tiles);
    t_rec.slots = dev.sms;
}

template <typename Kernel>
gemm_status_t allow_smem(Kernel *kernel, size_t bytes, bool &set)
{
    std::lock_guard<std::mutex> lock(g_mutex);
    if (!set) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
        if (e != cudaSuccess) return fail(GEMM_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
        set = true;
    }
    return GEMM_OK;
}

template <bool kBf16, int kTilesM, int kTilesN>
gemm_status_t launch_w4(const char *name, DeviceState &dev, w4::ProductParams &p, bool aligned, cudaStream_t stream)
{
    const bool whole = p.group_shift >= 7;
    auto kernel = whole ? (aligned ? w4::product_kernel<kBf16, kTilesM, kTilesN, true, true>
                                   : w4::product_kernel<kBf16, kTilesM, kTilesN, true, false>)
                        : (aligned ? w4::product_kernel<kBf16, kTilesM, kTilesN, false, true>
                                   : w4::product_kernel<kBf16, kTilesM, kTilesN, false, false>);
    p.token_tiles = static_cast<int32_t>((int64_t(p.N) + 8 * kTilesN - 1) / (8 * kTilesN));
    const int64_t tiles = (int64_t(p.M) + 16 * kTilesM - 1) / (16 * kTilesM) * p.token_tiles;
    if (tiles > INT32_MAX) return fail(GEMM_ERR_UNSUPPORTED, "%s: too many tiles", name);
    const int part = w4::part_floats(kTilesM, kTilesN), ring = aligned ? w4::ring_floats(kTilesM) : 0;
    const size_t smem = size_t(w4::kWarps) * (part > ring ? part : ring) * sizeof(float);
    if (smem > 48 * 1024) {                       // (only an aligned kernel's ring)
        const gemm_status_t st = allow_smem(kernel, smem, dev.w4_attr[0][kBf16][whole][kTilesM][kTilesN]);
        if (st != GEMM_OK) return st;
    }
    record_w4(name, dev, tiles);
    return launch_plain(name, kernel, dim3(static_cast<unsigned>(tiles), 1, 1), w4::kThreads, smem, stream, p);
}

template <bool kBf16, int kTilesM, int kTilesN, bool kWhole>
gemm_status_t launch_w4_wide(const char *name, DeviceState &dev, w4::ProductParams &p, cudaStream_t stream)
{
    using Cfg = w4::WideCfg<kTilesM, kTilesN, kWhole>;
    auto kernel = w4::wide_kernel<kBf16, kTilesM, kTilesN, kWhole>;
    p.token_tiles = static_cast<int32_t>((int64_t(p.N) + Cfg::kTokens - 1) / Cfg::kTokens);
    const int64_t tiles = (int64_t(p.M) + Cfg::kRows - 1) / Cfg::kRows * p.token_tiles;
    if (tiles > INT32_MAX) return fail(GEMM_ERR_UNSUPPORTED, "%s: too many tiles", name);
    const gemm_status_t st = allow_smem(kernel, Cfg::kBytes, dev.w4_attr[1][kBf16][kWhole][kTilesM][kTilesN]);
    if (st != GEMM_OK) return st;
    record_w4(name, dev, tiles);
    return launch_plain(name, kernel, dim3(static_cast<unsigned>(tiles), 1, 1), w4::kThreads, Cfg::kBytes, stream, p);
}

template <bool kBf16, int kTilesM, int kTilesN>
gemm_status_t launch_w4_wide(const char *name, DeviceState &dev, w4::ProductParams &p, cudaStream_t stream)
{
    return p.group_shift >= 7 ? launch_w4_wide<kBf16, kTilesM, kTilesN, true>(name, dev, p, stream)
                              : launch_w4_wide<kBf16, kTilesM, kTilesN, false>(name, dev, p, stream);
}

// Up to 8 tokens, few rows and rows that are not aligned: warps split the sum, each with two
// tiles of 16 rows where these still make three CTAs for four SMs.  Measured on GB300, groups of
// 128, one tile / two: 8192 x 8192 and one token 13.7 / 11.8 us, 28672 x 4096 19.0 / 19.0, with
// eight 23.9 / 20.2, 4096 x 4096 with one 5.9 / 5.2, 1024 x 4096 3.0 / 3.9.  More tokens over rows
// that give nearly every SM a tile of 64: warps share the tokens.  At K = 4096, split / shared:
// 16 tokens, 4096 rows 7.0 / 10.6 us, 8192 12.6 / 11.0, 28672 34.6 / 24.1; 64 tokens 17.7 / 25.4,
// 33.2 / 25.8, 96.3 / 74.5.
template <bool kBf16>
gemm_status_t launch_w4_tokens(const char *name, DeviceState &dev, w4::ProductParams &p, bool aligned, cudaStream_t stream)
{
    const int64_t M = p.M, sms = dev.sms;
    if (aligned && p.N > 8 && M >= 53 * sms) {
        if (p.N <= 16) return launch_w4_wide<kBf16, 1, 2>(name, dev, p, stream);
        if (p.N <= 32) return launch_w4_wide<kBf16, 1, 4>(name, dev, p, stream);
        return launch_w4_wide<kBf16, 1, 8>(name, dev, p, stream);
    }
    const bool many = M >= 24 * sms;
    if (p.N <= 8)
        return many ? launch_w4<kBf16, 2, 1>(name, dev, p, aligned, stream) : launch_w4<kBf16, 1, 1>(name, dev, p, aligned, stream);
    if (p.N <= 16)
        return many ? launch_w4<kBf16, 2, 2>(name, dev, p, aligned, stream) : launch_w4<kBf16, 1, 2>(name, dev, p, aligned, stream);
    return launch_w4<kBf16, 2, 4>(name, dev, p, aligned, stream);
}

gemm_status_t run_w4(int type, int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, const void *scale, int64_t lds,
                     int64_t group, const void *B, int64_t ldb, void *C, int64_t ldc, cudaStream_t stream)
{
    const char *name = "gemm_w4_tn";
    if (type != GEMM_IN_F16 && type != GEMM_IN_BF16)
        return fail(GEMM_ERR_INVALID_ARG, "%s: unknown or unsupported type %d (GEMM_IN_F16 or GEMM_IN_BF16)", name, type);
    if (M < 0 || N < 0 || K < 0)
        return fail(GEMM_ERR_INVALID_ARG, "%s: negative size (M=%lld N=%lld K=%lld)", name, (long long)M, (long long)N,
                    (long long)K);
    if (!w4_group_ok(group)) return fail(GEMM_ERR_INVALID_ARG, "%s: the group is not 32, 64, 128 or 256 terms", name);
    const int64_t bytes = (K + 1) / 2, groups = (K + group - 1) / group;
    if (lda < 1 || lda < bytes || lds < 1 || lds < groups || ldb < 1 || ldb < K || ldc < 1 || ldc < M)
        return fail(GEMM_ERR_INVALID_ARG, "%s: a leading dimension is below its row's length", name);
    if (M > kMaxDim || N > kMaxDim || K > kMaxDim || lda > kMaxDim || lds > kMaxDim || ldb > kMaxDim || ldc > kMaxDim)
        return fail(GEMM_ERR_UNSUPPORTED, "%s: a size or leading dimension is too large", name);
    if (M == 0 || N == 0) return GEMM_OK;
    if (!C) return fail(GEMM_ERR_INVALID_ARG, "%s: the result is NULL", name);
    if (!aligned_to(C, 2)) return fail(GEMM_ERR_INVALID_ARG, "%s: the result is not 2-byte aligned", name);
    if (K > 0) {
        if (!A || !scale || !B) return fail(GEMM_ERR_INVALID_ARG, "%s: an operand is NULL", name);
        if (!aligned_to(scale, 2) || !aligned_to(B, 2))
            return fail(GEMM_ERR_INVALID_ARG, "%s: an operand is not aligned to its element size", name);
    }
    gemm_status_t st = check_apart(name, "C", Span(C, 1, 0, N, ldc * 2, M * 2),
                                   {Span(A, 1, 0, M, lda, bytes), Span(scale, 1, 0, M, lds * 2, groups * 2),
                                    Span(B, 1, 0, N, ldb * 2, K * 2)});
    if (st != GEMM_OK) return st;
    DeviceState *dev = nullptr;
    st = device_state(&dev, nullptr);
    if (st != GEMM_OK) return st;
    w4::ProductParams p;
    memset(&p, 0, sizeof(p));
    p.a = static_cast<const uint8_t *>(A);
    p.lda = lda;
    p.scale = static_cast<const uint16_t *>(scale);
    p.lds = lds;
    p.b = static_cast<const uint16_t *>(B);
    p.ldb = ldb;
    p.c = static_cast<uint16_t *>(C);
    p.ldc = ldc;
    p.M = static_cast<int32_t>(M);
    p.N = static_cast<int32_t>(N);
    p.K = static_cast<int32_t>(K);
    while ((int64_t(1) << p.group_shift) < group) ++p.group_shift;
    p.groups = static_cast<int32_t>(groups);
    p.words = aligned_to(A, 4) && aligned_to(B, 4);
    const bool aligned = aligned_to(A, 16) && (M == 1 || lda % 16 == 0) && aligned_to(B, 16) && (N == 1 || ldb % 8 == 0);
    return type == GEMM_IN_BF16 ? launch_w4_tokens<true>(name, *dev, p, aligned, stream)
                                : launch_w4_tokens<false>(name, *dev, p, aligned, stream);
}

gemm_status_t run_quant_w4(const void *x, int x_type, int64_t rows, int64_t cols, int64_t ldx, int64_t group, void *q,
                           int64_t ldq, int scale_type, void *scale, int64_t lds, cudaStream_t stream)
{
    const char *name = "gemm_quantize_w4_rows";
    if (x_type < w4::kF32 || x_type > w4::kBF16)
        return fail(GEMM_ERR_INVALID_ARG, "%s: unknown input type %d", name, x_type);
    if (scale_type != GEMM_IN_F16 && scale_type != GEMM_IN_BF16)
        return fail(GEMM_ERR_INVALID_ARG, "%s: unknown or unsupported scale type %d (GEMM_IN_F16 or GEMM_IN_BF16)", name,
                    scale_type);
    if (rows < 0 || cols < 0) return fail(GEMM_ERR_INVALID_ARG, "%s: negative size", name);
    if (!w4_group_ok(group)) return fail(GEMM_ERR_INVALID_ARG, "%s: the group is not 32, 64, 128 or 256 terms", name);
    if (ldx < 1 || ldx < cols || ldq < 1 || ldq < (cols + 1) / 2 || lds < 1 || lds < (cols + group - 1) / group)
        return fail(GEMM_ERR_INVALID_ARG, "%s: a leading dimension is below its row's length", name);
    if (cols > kMaxDim || rows > (int64_t(1) << 40) / (cols > 1 ? cols : 1))
        return fail(GEMM_ERR_UNSUPPORTED, "%s: more than 2^40 elements", name);
    const int64_t seg = x_type == w4::kF32 ? w4::QuantCfg<w4::kF32>::kSeg : w4::QuantCfg<w4::kF16>::kSeg;
    const int64_t segs = (cols + seg - 1) / seg;  // a launch's second index
    if (segs > 65535) return fail(GEMM_ERR_UNSUPPORTED, "%s: too many columns", name);
    if (rows == 0 || cols == 0) return GEMM_OK;
    if (!x || !q || !scale) return fail(GEMM_ERR_INVALID_ARG, "%s: x, q or scale is NULL", name);
    const int64_t esz = x_type == w4::kF32 ? 4 : 2;
    if (!aligned_to(x, esz)) return fail(GEMM_ERR_INVALID_ARG, "%s: x is not aligned to its element size", name);
    if (!aligned_to(scale, 2)) return fail(GEMM_ERR_INVALID_ARG, "%s: scale is not 2-byte aligned", name);
    const Span sX(x, 1, 0, rows, ldx * esz, cols * esz), sQ(q, 1, 0, rows, ldq, (cols + 1) / 2);
    const Span sS(scale, 1, 0, rows, lds * 2, (cols + group - 1) / group * 2);
    gemm_status_t st = check_apart(name, "q", sQ, {sX, sS});
    if (st == GEMM_OK) st = check_apart(name, "scale", sS, {sX});
    if (st != GEMM_OK) return st;
    DeviceState *dev = nullptr;
    st = device_state(&dev, nullptr);
    if (st != GEMM_OK) return st;
    w4::QuantParams p;
    memset(&p, 0, sizeof(p));
    p.x = x;
    p.ldx = ldx;
    p.q = static_cast<uint8_t *>(q);
    p.ldq = ldq;
    p.scale = static_cast<uint16_t *>(scale);
    p.lds = lds;
    p.rows = rows;
    p.cols = static_cast<int32_t>(cols);
    p.group = static_cast<int32_t>(group);
    p.bf16 = scale_type == GEMM_IN_BF16;
    p.vec = aligned_to(x, 16) && aligned_to(q, 8) && (rows == 1 || (ldx * esz % 16 == 0 && ldq % 8 == 0));
    const int64_t per = w4::kQuantThreads / 32;
    int64_t grid = (rows + per - 1) / per;
    // CTAs that stay, a row ahead in their reads: about four an SM.  Measured on GB300, 8192 x
    // 8192 bf16: 51.4 us with a CTA for every 8 rows and 512 terms, 43.6 with these.
    const int64_t most = (int64_t(dev->sms) * 4 + segs - 1) / segs;
    if (grid > most) grid = most;
    t_rec = LaunchRecord{};
    t_rec.name = name;
    t_rec.quant = true;
    t_rec.qgrid = grid * segs;
    t_rec.qunits = rows * segs;
    t_rec.vec = p.vec;
    auto kernel = x_type == w4::kF32 ? w4::quant_kernel<w4::kF32>
                  : x_type == w4::kF16 ? w4::quant_kernel<w4::kF16> : w4::quant_kernel<w4::kBF16>;
    return launch_plain(name, kernel, dim3(static_cast<unsigned>(grid), static_cast<unsigned>(segs), 1), w4::kQuantThreads, 0,
                        stream, p);
}
