// Host side of the gated projections and of the vocabulary's loss (included by
// layers.cu, inside its anonymous namespace).  Like the grouped products these
// calls keep nothing in the library: all their buffers are the caller's workspace.

// Sections of a workspace, each from a 256-byte boundary on.
struct Sections {
    uint8_t *base;
    size_t at = 0;
    template <typename T>
    T *take(size_t n)
    {
        T *p = reinterpret_cast<T *>(base + at);
        at += (n * sizeof(T) + 255) & ~size_t(255);
        return p;
    }
};

gemm_status_t check_workspace(const char *name, const void *workspace, int64_t bytes, size_t need, const char *query)
{
    if (need == 0) return GEMM_OK;
    if (!workspace || bytes < static_cast<int64_t>(need))
        return fail(GEMM_ERR_INVALID_ARG, "%s: the workspace has %lld bytes, %zu are needed (%s)", name,
                    (long long)(workspace ? bytes : 0), need, query);
    if (reinterpret_cast<uintptr_t>(workspace) % 256)
        return fail(GEMM_ERR_INVALID_ARG, "%s: the workspace is not 256-byte aligned", name);
    return GEMM_OK;
}

tn::GroupedParams sink_params(const GroupedCall &c, int64_t l_extent, int64_t red, void *out, int64_t ldo)
{
    tn::GroupedParams prm;
    memset(&prm, 0, sizeof(prm));
    prm.offsets = c.offsets;
    prm.out = static_cast<uint16_t *>(out);
    prm.out_ld = ldo;
    prm.E = static_cast<int32_t>(c.E);
    prm.T = static_cast<int32_t>(c.T);
    prm.l_extent = static_cast<int32_t>(l_extent);
    prm.red = static_cast<int32_t>(red);
    prm.fmt = prm.out_fmt = c.type == GEMM_IN_BF16 ? 1u : 0u;
    prm.out_vec = aligned_to(out, 16) && ldo % 8 == 0;
    prm.split = 1;
    prm.flags = stall_flags(g_inject_stall.load());
    prm.wait_limit_ns = g_wait_limit_ns.load();
    return prm;
}

// The operands of a call as the TMA reads them: in place, or copied into the workspace.
struct SinkOperands {
    const void *x, *y;
    int64_t ldx, stride_x, ldy, in_x, in_y;
};

gemm_status_t place_operands(const char *name, DeviceState &dev, const GroupedPlan &plan, Sections &ws,
                             const int32_t *offsets, cudaStream_t stream, SinkOperands &o)
{
    o = {plan.x.base, plan.y.base, plan.x.ld, plan.x.stride, plan.y.ld, plan.x.inner, plan.y.inner};
    if (plan.x.copy) {
        o.x = ws.take<uint8_t>(plan.x.copy_bytes);
        o.ldx = o.in_x = plan.x.copy_ld;
        o.stride_x = plan.x.rows * o.ldx;
    }
    if (plan.y.copy) {
        o.y = ws.take<uint8_t>(plan.y.copy_bytes);
        o.ldy = o.in_y = plan.y.copy_ld;
    }
    if (!plan.x.copy && !plan.y.copy) return GEMM_OK;
    return launch_widen<uint16_t>(name, dev, plan, const_cast<void *>(o.x), const_cast<void *>(o.y), offsets, stream);
}

// ------------------------------------------------------------------ token gradients in parts
// The cut of one group's token gradient: T rows of K, sums of `red` terms.
ProductCut token_grad_cut(int64_t T, int64_t K, int64_t red)
{
    const int group = T <= kSumFewRows ? 1 : 2;
    return cut_product(group, T, (K + 128 * group - 1) / (128 * group), (red + 63) / 64, T * K, true);
}

// Floats of the parts' sums: none where a tile's sum is whole when it is stored.
size_t token_grad_floats(const ProductCut &cut, int64_t pieces, int64_t T, int64_t K)
{
    return cut.parts > 1 || pieces > 1 ? size_t(cut.parts) * size_t(T) * size_t(K) : 0;
}

// Piece i of `pieces` of dB = scale (d A): A's `c.M` rows (x), d's rows of `red` gradients.
gemm_status_t launch_token_grad(const GroupedCall &c, DeviceState &dev, const ProductCut &cut, const void *x, int64_t ldx,
                                int64_t in_x, const uint16_t *d, int64_t ldd, int64_t red, void *dB, int64_t lddb,
                                const float *scale, float *sum, int64_t i, int64_t pieces)
{
    tn::GroupedParams prm = sink_params(c, c.K, red, dB, lddb);
    prm.tile_rows = cut.rows;
    prm.parts = cut.parts;
    prm.sink.sum = sum;
    prm.sink.sum_ld = c.K;
    prm.sink.sum_stride = c.T * c.K;
    prm.sink.out_scale = scale;
    prm.sink.add = cut.parts == 1 && pieces == 1         ? tn::kAddOnly
                   : i == 0                              ? tn::kAddFirst
                   : cut.parts == 1 && i + 1 == pieces   ? tn::kAddLast
                                                         : tn::kAddMore;
    gemm_status_t st = launch_grouped_op<tn::kGrGradBAdd>(c, dev, prm, x, d, ldx, 0, ldd, in_x, (red + 7) / 8 * 8);
    if (st != GEMM_OK || cut.parts == 1 || i + 1 < pieces) return st;
    tn::PartsParams p{sum, c.K, c.T * c.K, static_cast<uint16_t *>(dB), lddb, scale, c.T, static_cast<int32_t>(c.K), cut.parts,
                      c.type == GEMM_IN_BF16, c.K % 4 == 0 && lddb % 4 == 0 && aligned_to(dB, 8)};
    const int64_t units = p.vec ? c.K / 4 : c.K;
    const int64_t gx = (units + tn::kPartsThreads - 1) / tn::kPartsThreads;
    int64_t gy = (int64_t(dev.sms) * 16 + gx - 1) / gx;
    if (gy > c.T) gy = c.T;
    if (gy > 65535) gy = 65535;
    return launch_plain(c.name, tn::parts_join_kernel, dim3(static_cast<unsigned>(gx), static_cast<unsigned>(gy), 1),
                        tn::kPartsThreads, 0, c.stream, p);
}

// ------------------------------------------------------------------ gated projections
bool gated_sizes_fit(int64_t E, int64_t M, int64_t K, int64_t T, int64_t lda, int64_t ldb, int64_t stride)
{
    return M <= kMaxDim / 2 && grouped_sizes_fit(E, 2 * M, K, T, lda, ldb, stride);
}

struct GatedPlan {
    GroupedPlan g;               // the copies (and the backward pass's tensor maps)
    int64_t ldd, units;          // the backward pass's rows of 2 M gradients: padded, and up to a whole 16-byte unit
    ProductCut cut;              // without experts: of the token gradient
    size_t floats;               // ... and its parts' sums
    size_t entries;              // ... of the room (layers_kernels.cuh) where dP's rows have none to spare
    size_t bytes;
    bool fits;
};

// A is read along its rows in the forward pass and across them in the backward pass.
GatedPlan gated_plan(bool grad, bool dense, int64_t E, int64_t M, int64_t K, int64_t T, const void *A, int64_t lda,
                     int64_t stride_a, const void *B, int64_t ldb)
{
    GatedPlan p{};
    p.fits = true;
    p.units = (2 * M + 7) / 8 * 8;
    p.ldd = (2 * M + 63) / 64 * 64;
    if (grouped_idle(E, M, K, T)) return p;
    if (!grad) {
        p.g = grouped_plan(GEMM_GROUPED_PRODUCT, E, 2 * M, K, T, A, lda, stride_a, B, ldb);
        p.bytes = p.g.bytes();
        p.fits = p.g.fits;
        return p;
    }
    p.g.x = grouped_operand(A, 2 * M, E, K, lda, stride_a, false, false);
    p.g.y = grouped_operand(B, T, 1, K, ldb, 0, false, false);
    p.g.map_bytes = dense ? 0 : size_t(E) * 2 * sizeof(CUtensorMap);
    p.fits = grouped_copy(p.g.x, false, false) && grouped_copy(p.g.y, false, false) && T <= (int64_t(1) << 60) / p.ldd;
    p.bytes = p.g.bytes() + ((size_t(T) * size_t(p.ldd) * 2 + 255) & ~size_t(255));
    if (dense) {
        p.cut = token_grad_cut(T, K, 2 * M);
        p.floats = token_grad_floats(p.cut, 1, T, K);
        p.bytes += (p.floats * sizeof(float) + 255) & ~size_t(255);
    }
    if ((p.ldd - p.units) * 2 < int64_t(tn::kGatedEntry * sizeof(float))) {
        p.entries = size_t(T < tn::kGatedTops ? T : tn::kGatedTops);
        p.bytes += (p.entries * tn::kGatedEntry * sizeof(float) + 255) & ~size_t(255);
    }
    return p;
}

int64_t gated_workspace(int grad, int dense, int64_t E, int64_t M, int64_t K, int64_t T, const void *A, int64_t lda,
                        int64_t stride_a, const void *B, int64_t ldb)
{
    if (E < 0 || M < 0 || K < 0 || T < 0 || lda < 1 || ldb < 1 || lda < K || ldb < K || stride_a < 0 || (dense && E != 1) ||
        !gated_sizes_fit(E, M, K, T, lda, ldb, stride_a))
        return -1;
    const GatedPlan p = gated_plan(grad != 0, dense != 0, E, M, K, T, A, lda, stride_a, B, ldb);
    return p.fits ? static_cast<int64_t>(p.bytes) : -1;
}

// What the forward and the backward call check alike.
gemm_status_t check_gated(const char *name, int type, int act, int64_t E, int64_t M, int64_t K, int64_t T, int64_t lda,
                          int64_t stride_a, int64_t ldb, const int32_t *offsets)
{
    if (type != GEMM_IN_F16 && type != GEMM_IN_BF16)
        return fail(GEMM_ERR_INVALID_ARG, "%s: unknown or unsupported type %d (GEMM_IN_F16 or GEMM_IN_BF16)", name, type);
    if (act < GEMM_ACT_SILU || act > GEMM_ACT_GELU_TANH)
        return fail(GEMM_ERR_INVALID_ARG, "%s: unknown activation %d", name, act);
    if (E < 0 || M < 0 || K < 0 || T < 0)
        return fail(GEMM_ERR_INVALID_ARG, "%s: negative size (E=%lld M=%lld K=%lld rows=%lld)", name, (long long)E,
                    (long long)M, (long long)K, (long long)T);
    if (lda < 1 || lda < K || ldb < 1 || ldb < K)
        return fail(GEMM_ERR_INVALID_ARG, "%s: a leading dimension is below its row's length", name);
    if (stride_a < 0) return fail(GEMM_ERR_INVALID_ARG, "%s: negative stride", name);
    if (!offsets && E != 1) return fail(GEMM_ERR_INVALID_ARG, "%s: offsets is NULL, and there is not one expert", name);
    if (!aligned_to(offsets, 4)) return fail(GEMM_ERR_INVALID_ARG, "%s: offsets is not 4-byte aligned", name);
    if (!gated_sizes_fit(E, M, K, T, lda, ldb, stride_a))
        return fail(GEMM_ERR_UNSUPPORTED, "%s: more than %d experts, or a size, leading dimension or stride too large", name,
                    tn::kGrMaxExperts);
    return GEMM_OK;
}

// A decode step's tokens go to a kernel of their own (where the general one would read
// the operands in place) up to two of its CTAs an SM: there the general kernel's tiles are
// too few, beyond it their wider loads win.  Measured on GB300, general / this: 512 x 1024
// with one token 6.8 / 3.0 us, 2048 x 2048 9.8 / 6.0, with 16 tokens 10.0 / 6.7, 4096 x 2048 11.3 / 10.5
// and 11.6 / 9.3, 4096 x 4096 16.7 / 18.3 and 16.9 / 16.2 (256 CTAs); 8192 x 2048 15.4 / 17.2,
// 14336 x 4096 42.5 / 44.9 (896).  By expert: 2 of 8 of 1024 x 2048 10.5 / 7.2, 8 of 8 (512
// CTAs) 15.8 / 18.4.
constexpr int64_t kGatedFewRows = 16;

int64_t gated_few_ctas(bool dense, int64_t E, int64_t M, int64_t T) { return (M + 15) / 16 * (dense || E < T ? E : T); }

template <bool kBf16, int kTilesN>
gemm_status_t launch_gated_few(const char *name, DeviceState &dev, const tn::GatedFewParams &p, cudaStream_t stream)
{
    auto kernel = tn::gated_few_kernel<kBf16, kTilesN>;
    const int64_t ctas = gated_few_ctas(!p.offsets, p.E, p.M, p.T);
    {
        std::lock_guard<std::mutex> lock(g_mutex);
        bool &set = dev.few_attr[kBf16][kTilesN - 1];
        if (!set) {
            const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, tn::kFewRingBytes);
            if (e != cudaSuccess) return fail(GEMM_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
            set = true;
        }
    }
    t_rec = LaunchRecord{};
    t_rec.name = name;
    t_rec.grouped = 1;
    t_rec.cluster = 1;
    t_rec.grid = static_cast<int>(ctas);
    t_rec.slots = dev.sms;
    t_rec.tiles = static_cast<int>(ctas);
    return launch_plain(name, kernel, dim3(static_cast<unsigned>(ctas), 1, 1), tn::kFewThreads, tn::kFewRingBytes, stream, p);
}

gemm_status_t run_gated(int type, int act, int64_t E, int64_t M, int64_t K, int64_t T, const void *A, int64_t lda,
                        int64_t stride_a, const void *B, int64_t ldb, const int32_t *offsets, void *H, int64_t ldh, float *P,
                        int64_t ldp, void *workspace, int64_t workspace_bytes, cudaStream_t stream)
{
    const char *name = "gemm_tn_gated";
    gemm_status_t st = check_gated(name, type, act, E, M, K, T, lda, stride_a, ldb, offsets);
    if (st != GEMM_OK) return st;
    if (ldh < 1 || ldh < M || (P && (ldp < 1 || ldp < 2 * M)))
        return fail(GEMM_ERR_INVALID_ARG, "%s: a leading dimension is below its row's length", name);
    if (ldh > kMaxDim || (P && ldp > kMaxDim))
        return fail(GEMM_ERR_UNSUPPORTED, "%s: a leading dimension is too large", name);
    if (E == 0 || M == 0 || T == 0) return GEMM_OK;
    if (!H) return fail(GEMM_ERR_INVALID_ARG, "%s: the result is NULL", name);
    if (!aligned_to(H, 2) || !aligned_to(P, 4))
        return fail(GEMM_ERR_INVALID_ARG, "%s: a result is not aligned to its element size", name);
    if (K > 0 && (!A || !B)) return fail(GEMM_ERR_INVALID_ARG, "%s: an operand is NULL", name);
    if (K > 0 && (!aligned_to(A, 2) || !aligned_to(B, 2)))
        return fail(GEMM_ERR_INVALID_ARG, "%s: an operand is not aligned to its element size", name);
    const GatedPlan plan = gated_plan(false, !offsets, E, M, K, T, A, lda, stride_a, B, ldb);
    if (!plan.fits) return fail(GEMM_ERR_UNSUPPORTED, "%s: the operands' copies are too large", name);
    if ((st = check_workspace(name, workspace, workspace_bytes, plan.bytes, "gemm_gated_workspace")) != GEMM_OK) return st;
    const Span sA(A, E, stride_a * 2, 2 * M, lda * 2, K * 2), sB(B, 1, 0, T, ldb * 2, K * 2);
    const Span sO(offsets, (E + 1) * 4), sW(workspace, static_cast<int64_t>(plan.bytes)), sH(H, 1, 0, T, ldh * 2, M * 2);
    const Span sP(P, 1, 0, T, ldp * 4, 2 * M * 4);
    if ((st = check_apart(name, "H", sH, {sA, sB, sO, sP, sW})) != GEMM_OK) return st;
    if ((st = check_apart(name, "P", sP, {sA, sB, sO, sW})) != GEMM_OK) return st;
    if ((st = check_apart(name, "the workspace", sW, {sA, sB, sO})) != GEMM_OK) return st;
    DeviceState *dev = nullptr;
    if ((st = device_state(&dev, nullptr)) != GEMM_OK) return st;
    if (K > 0 && T <= kGatedFewRows && !plan.g.x.copy && !plan.g.y.copy && gated_few_ctas(!offsets, E, M, T) <= 2 * dev->sms) {
        const tn::GatedFewParams p{static_cast<const uint16_t *>(A), lda, stride_a, static_cast<const uint16_t *>(B), ldb, offsets,
                                   static_cast<uint16_t *>(H), ldh, P, ldp, static_cast<int32_t>(E), static_cast<int32_t>(T),
                                   static_cast<int32_t>(M), static_cast<int32_t>(K), static_cast<int32_t>((M + 15) / 16), act};
        if (type == GEMM_IN_BF16)
            return T <= 8 ? launch_gated_few<true, 1>(name, *dev, p, stream) : launch_gated_few<true, 2>(name, *dev, p, stream);
        return T <= 8 ? launch_gated_few<false, 1>(name, *dev, p, stream) : launch_gated_few<false, 2>(name, *dev, p, stream);
    }

    Sections ws{static_cast<uint8_t *>(workspace)};
    SinkOperands o{};
    if (K > 0 && (st = place_operands(name, *dev, plan.g, ws, offsets, stream, o)) != GEMM_OK) return st;
    GroupedCall c{name, GEMM_GROUPED_PRODUCT, type, type, E, M, K, T};
    c.offsets = offsets;
    c.stream = stream;
    tn::GroupedParams prm = sink_params(c, M, K, H, ldh);
    prm.sink.act = act;
    prm.sink.pre = P;
    prm.sink.pre_ld = ldp;
    st = launch_grouped_op<tn::kGrGated>(c, *dev, prm, o.x, o.y, o.ldx, o.stride_x, o.ldy, o.in_x, o.in_y);
    t_rec.copied = (plan.g.x.copy ? 1 : 0) | (plan.g.y.copy ? 2 : 0);
    return st;
}

template <int kAct>
gemm_status_t launch_gated_grad(const char *name, DeviceState &dev, tn::GatedGradParams p, bool bf16, cudaStream_t stream)
{
    const bool vec = p.M % 8 == 0 && p.pre_ld % 4 == 0 && p.dh_ld % 8 == 0 && aligned_to(p.pre, 16) && aligned_to(p.dh, 16);
    const int64_t units = vec ? int64_t(p.M) / 8 : p.M;
    p.lanes = 32;
    while (p.lanes < tn::kGatedGradThreads && p.lanes < units) p.lanes *= 2;
    const int64_t across = (units + p.lanes - 1) / p.lanes, rows = tn::kGatedGradThreads / p.lanes;
    // about eight CTAs an SM, whole rows of them
    const int64_t want = int64_t(dev.sms) * 8;
    const int64_t gx = across < want ? across : want;
    int64_t gy = (want + gx - 1) / gx;
    if (gy > (p.T + rows - 1) / rows) gy = (p.T + rows - 1) / rows;
    if (gy > 65535) gy = 65535;
    const dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>(gy), 1);
    auto kernel = bf16 ? (vec ? tn::gated_grad_kernel<kAct, true, true> : tn::gated_grad_kernel<kAct, true, false>)
                       : (vec ? tn::gated_grad_kernel<kAct, false, true> : tn::gated_grad_kernel<kAct, false, false>);
    if (bf16) return launch_plain(name, kernel, grid, tn::kGatedGradThreads, 0, stream, p);
    // fp16: the size of dH first, and the pass once more where dP's is another
    p.tops = p.T < tn::kGatedTops ? p.T : tn::kGatedTops;
    p.top_vec = p.dh_ld % 8 == 0 && aligned_to(p.dh, 16);
    p.top_lanes = tn::kGatedTopThreads;           // (short rows share a CTA, and all where there are more than CTAs)
    while (p.top_lanes > 32 && (p.top_lanes / 2 >= p.M / 8 || int64_t(p.tops) * (tn::kGatedTopThreads / p.top_lanes) < p.T))
        p.top_lanes /= 2;
    gemm_status_t st = launch_plain(name, tn::gated_top_kernel, dim3(static_cast<unsigned>(p.tops), 1, 1), tn::kGatedTopThreads, 0,
                                    stream, p);
    if (st == GEMM_OK) st = launch_plain(name, kernel, grid, tn::kGatedGradThreads, 0, stream, p);
    p.again = true;
    if (st == GEMM_OK) st = launch_plain(name, kernel, grid, tn::kGatedGradThreads, 0, stream, p);
    return st;
}

gemm_status_t run_gated_grad(int type, int act, int64_t E, int64_t M, int64_t K, int64_t T, const void *A, int64_t lda,
                             int64_t stride_a, const void *B, int64_t ldb, const int32_t *offsets, const float *P,
                             int64_t ldp, const void *dH, int64_t lddh, void *dA, int64_t ldda, int64_t stride_da, void *dB,
                             int64_t lddb, void *workspace, int64_t workspace_bytes, cudaStream_t stream)
{
    const char *name = "gemm_tn_gated_grad";
    gemm_status_t st = check_gated(name, type, act, E, M, K, T, lda, stride_a, ldb, offsets);
    if (st != GEMM_OK) return st;
    if (ldp < 1 || ldp < 2 * M || lddh < 1 || lddh < M || (dA && (ldda < 1 || ldda < K)) || (dB && (lddb < 1 || lddb < K)))
        return fail(GEMM_ERR_INVALID_ARG, "%s: a leading dimension is below its row's length", name);
    if (dA && stride_da < 0) return fail(GEMM_ERR_INVALID_ARG, "%s: negative stride", name);
    if (ldp > kMaxDim || lddh > kMaxDim || (dA && (ldda > kMaxDim || stride_da > (int64_t(1) << 38))) ||
        (dB && lddb > kMaxDim))
        return fail(GEMM_ERR_UNSUPPORTED, "%s: a leading dimension or stride is too large", name);
    if (E == 0 || K == 0) return GEMM_OK;         // no gradient has an element
    if (M == 0) dA = nullptr;
    if (T == 0) dB = nullptr;
    if (!dA && !dB) return GEMM_OK;
    if (!aligned_to(dA, 2) || !aligned_to(dB, 2))
        return fail(GEMM_ERR_INVALID_ARG, "%s: a result is not 2-byte aligned", name);
    if (dA && E > 1 && stride_da < (2 * M - 1) * ldda + K && (stride_da < K || ldda < (E - 1) * stride_da + K))
        return fail(GEMM_ERR_INVALID_ARG, "%s: the experts' results overlap", name);
    const bool idle = M == 0 || T == 0;
    if (!idle) {
        if (!A || !B || !P || !dH) return fail(GEMM_ERR_INVALID_ARG, "%s: an operand is NULL", name);
        if (!aligned_to(A, 2) || !aligned_to(B, 2) || !aligned_to(dH, 2) || !aligned_to(P, 4))
            return fail(GEMM_ERR_INVALID_ARG, "%s: an operand is not aligned to its element size", name);
    }
    GatedPlan plan = gated_plan(true, !offsets, E, M, K, T, A, lda, stride_a, B, ldb);
    if (!plan.fits) return fail(GEMM_ERR_UNSUPPORTED, "%s: the operands' copies are too large", name);
    if ((st = check_workspace(name, workspace, workspace_bytes, plan.bytes, "gemm_gated_workspace")) != GEMM_OK) return st;
    if (!idle) {
        // (P and dH are read before a gradient is written, and A, for dB, before dA is)
        const Span sA(A, E, stride_a * 2, 2 * M, lda * 2, K * 2), sB(B, 1, 0, T, ldb * 2, K * 2), sO(offsets, (E + 1) * 4);
        const Span sdA(dA, E, stride_da * 2, 2 * M, ldda * 2, K * 2), sdB(dB, 1, 0, T, lddb * 2, K * 2), none(nullptr, 0);
        const Span sW(workspace, static_cast<int64_t>(plan.bytes));
        const bool in_place = dA == A && ldda == lda && (E == 1 || stride_da == stride_a);
        if ((st = check_apart(name, "dA", sdA, {dB && !in_place ? sA : none, sB, sO, sdB, sW})) != GEMM_OK) return st;
        if ((st = check_apart(name, "dB", sdB, {sA, dA ? sB : none, sO, sW})) != GEMM_OK) return st;
        if ((st = check_apart(name, "the workspace", sW, {dB ? sA : none, dA ? sB : none, sO, Span(P, 1, 0, T, ldp * 4, 2 * M * 4),
                                                          Span(dH, 1, 0, T, lddh * 2, M * 2)})) != GEMM_OK)
            return st;
    }
    DeviceState *dev = nullptr;
    if ((st = device_state(&dev, nullptr)) != GEMM_OK) return st;

    Sections ws{static_cast<uint8_t *>(workspace)};
    plan.g.x.copy &= dB != nullptr;               // (each gradient reads one of them)
    plan.g.y.copy &= dA != nullptr;
    SinkOperands o{};
    uint16_t *dP = nullptr;
    float *sum = nullptr;
    CUtensorMap *maps = nullptr;
    const float *undo = nullptr;                  // fp16: dP's factor, taken back
    const bool bf16 = type == GEMM_IN_BF16;
    if (!idle) {
        if ((st = place_operands(name, *dev, plan.g, ws, offsets, stream, o)) != GEMM_OK) return st;
        if (offsets) maps = ws.take<CUtensorMap>(size_t(E) * 2);
        dP = ws.take<uint16_t>(size_t(T) * size_t(plan.ldd));
        if (plan.floats) sum = ws.take<float>(plan.floats);
        float *room = plan.entries ? ws.take<float>(plan.entries * tn::kGatedEntry) : reinterpret_cast<float *>(dP + plan.units);
        if (!bf16) undo = room + 2;
        const tn::GatedGradParams p{P, ldp, static_cast<const uint16_t *>(dH), lddh, dP, plan.ldd, plan.units, room,
                                    plan.entries ? tn::kGatedEntry : plan.ldd / 2, offsets, static_cast<int32_t>(E),
                                    static_cast<int32_t>(T), static_cast<int32_t>(M), 0, 0, 0, false, false};
        st = act == GEMM_ACT_SILU   ? launch_gated_grad<tn::kActSilu>(name, *dev, p, bf16, stream)
             : act == GEMM_ACT_GELU ? launch_gated_grad<tn::kActGelu>(name, *dev, p, bf16, stream)
                                    : launch_gated_grad<tn::kActGeluTanh>(name, *dev, p, bf16, stream);
        if (st != GEMM_OK) return st;
    }
    GroupedCall c{name, GEMM_GROUPED_GRAD_B, type, type, E, 2 * M, K, T};
    c.offsets = offsets;
    c.stream = stream;
    const int copied = (plan.g.x.copy ? 1 : 0) | (plan.g.y.copy ? 2 : 0);
    if (dB) {
        if (!offsets && !idle) {
            st = launch_token_grad(c, *dev, plan.cut, o.x, o.ldx, o.in_x, dP, plan.ldd, 2 * M, dB, lddb, undo, sum, 0, 1);
        } else {
            tn::GroupedParams prm = sink_params(c, K, 2 * M, dB, lddb);
            prm.sink.out_scale = undo;
            st = bf16 ? launch_grad_b(c, *dev, prm, o.x, dP, o.ldx, o.stride_x, plan.ldd, o.in_x, plan.units)
                      : launch_grouped_op<tn::kGrGradBScaled>(c, *dev, prm, o.x, dP, o.ldx, o.stride_x, plan.ldd, o.in_x, plan.units);
        }
        t_rec.copied = copied;
        if (st != GEMM_OK) return st;
    }
    if (dA) {
        tn::GroupedParams prm = sink_params(c, K, T, dA, ldda);
        prm.out_stride = stride_da;
        prm.out_vec = prm.out_vec && (E == 1 || stride_da % 8 == 0);
        prm.r_extent = static_cast<int32_t>(2 * M);
        prm.sink.out_scale = undo;
        if (offsets) {
            prm.group_maps = maps;
            st = bf16 ? launch_grad_a(c, *dev, prm, dP, o.y, plan.ldd, 0, o.ldy, plan.units, o.in_y)
                      : launch_grouped_op<tn::kGrGradAScaled>(c, *dev, prm, dP, o.y, plan.ldd, 0, o.ldy, plan.units, o.in_y);
        } else {
            st = launch_grouped_op<tn::kGrGradAOne>(c, *dev, prm, dP, o.y, plan.ldd, 0, o.ldy, plan.units, o.in_y);
        }
        t_rec.copied = copied;
    }
    return st;
}

// ------------------------------------------------------------------ loss
// The gradient goes through the vocabulary in pieces of about this many bytes of
// the logits' gradients, which both products then read again, and of at least
// kLossMinPiece classes, so that the FP32 sums of the token gradient (read and written
// once a piece) stay small beside the products.  That counts for more than a piece that the L2
// keeps: measured on GB300, pieces of 64 / 128 / 256 / 512 MiB, 4096 tokens over 65536 classes of
// 4096 3798 / 3829 / 3620 / 3652 us, of 1024 1281 / 1111 / 1009 / 959, 16384 over 32768 of 2048 4482 /
// 4095 / 3974 / 3790; 256 MiB, so that a large vocabulary's logits are still not held.
constexpr int64_t kLossPieceBytes = int64_t(1) << 28, kLossMinPiece = 1024;

struct LossPlan {
    GroupedPlan g;
    int64_t pieces, piece;       // classes of a piece (the last may have fewer)
    ProductCut cut;              // of the token gradient over a piece
    size_t floats;               // ... and its parts' sums
    int64_t blocks;              // forward: 32 classes each
    size_t bytes;
    bool fits;
};

LossPlan loss_plan(bool grad, int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, const void *B, int64_t ldb)
{
    LossPlan p{};
    p.fits = true;
    if (M == 0 || N == 0) return p;
    p.g = grouped_plan(GEMM_GROUPED_PRODUCT, 1, M, K, N, A, lda, 0, B, ldb);
    p.fits = K == 0 || p.g.fits;
    size_t bytes = 0;
    auto add = [&](int64_t rows, int64_t row_bytes) {
        if (rows > (int64_t(1) << 60) / row_bytes) p.fits = false;
        else bytes += (size_t(rows) * size_t(row_bytes) + 255) & ~size_t(255);
    };
    if (!grad) {
        p.blocks = (M + 31) / 32;
        add(N, p.blocks * int64_t(sizeof(float2)));
        add(N, sizeof(float));
    } else {
        int64_t piece = kLossPieceBytes / (2 * N) / 256 * 256;
        if (piece < kLossMinPiece) piece = kLossMinPiece;
        p.pieces = (M + piece - 1) / piece;
        piece = (M + p.pieces - 1) / p.pieces;
        p.piece = (piece + 255) / 256 * 256;
        p.pieces = (M + p.piece - 1) / p.piece;
        add(N, p.piece * 2);
        add(N, sizeof(float2));
        add(1, sizeof(float));
        p.cut = token_grad_cut(N, K, p.piece);
        p.floats = token_grad_floats(p.cut, p.pieces, N, K);
        if (p.floats) add(N, p.cut.parts * K * int64_t(sizeof(float)));
    }
    p.bytes = p.g.bytes() + bytes;
    return p;
}

int64_t loss_workspace(int grad, int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, const void *B, int64_t ldb)
{
    if (M < 0 || N < 0 || K < 0 || lda < 1 || ldb < 1 || lda < K || ldb < K || !grouped_sizes_fit(1, M, K, N, lda, ldb, 0))
        return -1;
    const LossPlan p = loss_plan(grad != 0, M, N, K, A, lda, B, ldb);
    return p.fits ? static_cast<int64_t>(p.bytes) : -1;
}

gemm_status_t check_loss(const char *name, int type, int64_t M, int64_t N, int64_t K, const void *A, int64_t lda,
                         const void *B, int64_t ldb, const int64_t *targets)
{
    if (type != GEMM_IN_F16 && type != GEMM_IN_BF16)
        return fail(GEMM_ERR_INVALID_ARG, "%s: unknown or unsupported type %d (GEMM_IN_F16 or GEMM_IN_BF16)", name, type);
    if (M < 0 || N < 0 || K < 0)
        return fail(GEMM_ERR_INVALID_ARG, "%s: negative size (M=%lld N=%lld K=%lld)", name, (long long)M, (long long)N,
                    (long long)K);
    if (lda < 1 || lda < K || ldb < 1 || ldb < K)
        return fail(GEMM_ERR_INVALID_ARG, "%s: a leading dimension is below its row's length", name);
    if (!grouped_sizes_fit(1, M, K, N, lda, ldb, 0))
        return fail(GEMM_ERR_UNSUPPORTED, "%s: a size or leading dimension is too large", name);
    if (M == 0 && N > 0) return fail(GEMM_ERR_INVALID_ARG, "%s: there are no classes", name);
    if (N == 0) return GEMM_OK;
    if (!targets) return fail(GEMM_ERR_INVALID_ARG, "%s: targets is NULL", name);
    if (!aligned_to(targets, 8)) return fail(GEMM_ERR_INVALID_ARG, "%s: targets is not 8-byte aligned", name);
    if (K > 0 && (!A || !B)) return fail(GEMM_ERR_INVALID_ARG, "%s: an operand is NULL", name);
    if (K > 0 && (!aligned_to(A, 2) || !aligned_to(B, 2)))
        return fail(GEMM_ERR_INVALID_ARG, "%s: an operand is not aligned to its element size", name);
    return GEMM_OK;
}

gemm_status_t run_loss(int type, int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, const void *B, int64_t ldb,
                       const int64_t *targets, float *loss, float *lse, void *workspace, int64_t workspace_bytes,
                       cudaStream_t stream)
{
    const char *name = "gemm_tn_cross_entropy";
    gemm_status_t st = check_loss(name, type, M, N, K, A, lda, B, ldb, targets);
    if (st != GEMM_OK || N == 0) return st;
    if (!loss || !lse) return fail(GEMM_ERR_INVALID_ARG, "%s: a result is NULL", name);
    if (!aligned_to(loss, 4) || !aligned_to(lse, 4))
        return fail(GEMM_ERR_INVALID_ARG, "%s: a result is not 4-byte aligned", name);
    const LossPlan plan = loss_plan(false, M, N, K, A, lda, B, ldb);
    if (!plan.fits) return fail(GEMM_ERR_UNSUPPORTED, "%s: the workspace would be too large", name);
    if ((st = check_workspace(name, workspace, workspace_bytes, plan.bytes, "gemm_cross_entropy_workspace")) != GEMM_OK)
        return st;
    // (A and B are read before a result is written)
    const Span sT(targets, N * 8), sL(loss, N * 4), sE(lse, N * 4), sW(workspace, static_cast<int64_t>(plan.bytes));
    if ((st = check_apart(name, "the loss", sL, {sT, sE, sW})) != GEMM_OK) return st;
    if ((st = check_apart(name, "lse", sE, {sT, sW})) != GEMM_OK) return st;
    if ((st = check_apart(name, "the workspace", sW, {sT, Span(A, 1, 0, M, lda * 2, K * 2), Span(B, 1, 0, N, ldb * 2, K * 2)})) != GEMM_OK)
        return st;
    DeviceState *dev = nullptr;
    if ((st = device_state(&dev, nullptr)) != GEMM_OK) return st;

    Sections ws{static_cast<uint8_t *>(workspace)};
    SinkOperands o{};
    if (K > 0 && (st = place_operands(name, *dev, plan.g, ws, nullptr, stream, o)) != GEMM_OK) return st;
    float2 *stats = ws.take<float2>(size_t(plan.blocks) * size_t(N));
    float *z_target = ws.take<float>(size_t(N));
    GroupedCall c{name, GEMM_GROUPED_PRODUCT, type, type, 1, M, K, N};
    c.stream = stream;
    tn::GroupedParams prm = sink_params(c, M, K, nullptr, 0);
    prm.sink.targets = targets;
    prm.sink.stats = stats;
    prm.sink.z_target = z_target;
    st = launch_grouped_op<tn::kGrLossStats>(c, *dev, prm, o.x, o.y, o.ldx, o.stride_x, o.ldy, o.in_x, o.in_y);
    t_rec.copied = (plan.g.x.copy ? 1 : 0) | (plan.g.y.copy ? 2 : 0);
    if (st != GEMM_OK) return st;
    // tokens of a CTA: as many as a sector's 32 bytes of pairs at least, and no more than give every SM a CTA
    int32_t lanes = 32;
    while (lanes > 1 && (lanes / 2 >= N || (lanes > 4 && (N + lanes - 1) / lanes < dev->sms))) lanes /= 2;
    const tn::JoinParams jp{stats, z_target, targets, loss, lse, N, M, static_cast<int32_t>(plan.blocks), lanes};
    return launch_plain(name, tn::cross_entropy_join_kernel, dim3(static_cast<unsigned>((N + lanes - 1) / lanes), 1, 1),
                        tn::kJoinThreads, 0, stream, jp);
}

gemm_status_t run_loss_grad(int type, int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, const void *B, int64_t ldb,
                            const int64_t *targets, const float *lse, const float *dloss, void *dA, int64_t ldda, void *dB,
                            int64_t lddb, void *workspace, int64_t workspace_bytes, cudaStream_t stream)
{
    const char *name = "gemm_tn_cross_entropy_grad";
    gemm_status_t st = check_loss(name, type, M, N, K, A, lda, B, ldb, targets);
    if (st != GEMM_OK) return st;
    if ((dA && (ldda < 1 || ldda < K)) || (dB && (lddb < 1 || lddb < K)))
        return fail(GEMM_ERR_INVALID_ARG, "%s: a leading dimension is below its row's length", name);
    if ((dA && ldda > kMaxDim) || (dB && lddb > kMaxDim))
        return fail(GEMM_ERR_UNSUPPORTED, "%s: a leading dimension is too large", name);
    if (K == 0 || M == 0) return GEMM_OK;         // no gradient has an element
    if (N == 0) dB = nullptr;
    if (!dA && !dB) return GEMM_OK;
    if (!aligned_to(dA, 2) || !aligned_to(dB, 2))
        return fail(GEMM_ERR_INVALID_ARG, "%s: a result is not 2-byte aligned", name);
    if (N > 0) {
        if (!lse || !dloss) return fail(GEMM_ERR_INVALID_ARG, "%s: lse or dloss is NULL", name);
        if (!aligned_to(lse, 4) || !aligned_to(dloss, 4))
            return fail(GEMM_ERR_INVALID_ARG, "%s: lse or dloss is not 4-byte aligned", name);
    }
    const LossPlan plan = loss_plan(true, M, N, K, A, lda, B, ldb);
    if (!plan.fits) return fail(GEMM_ERR_UNSUPPORTED, "%s: the workspace would be too large", name);
    if ((st = check_workspace(name, workspace, workspace_bytes, plan.bytes, "gemm_cross_entropy_workspace")) != GEMM_OK)
        return st;
    if (N > 0) {
        // (a piece's classes are read before their rows of dA are written, and B for the logits before dB is)
        const Span sA(A, 1, 0, M, lda * 2, K * 2), sB(B, 1, 0, N, ldb * 2, K * 2), sT(targets, N * 8), sE(lse, N * 4), sD(dloss, N * 4);
        const Span sdA(dA, 1, 0, M, ldda * 2, K * 2), sdB(dB, 1, 0, N, lddb * 2, K * 2), none(nullptr, 0);
        const Span sW(workspace, static_cast<int64_t>(plan.bytes));
        if ((st = check_apart(name, "dA", sdA, {dA == A && ldda == lda ? none : sA, sB, sT, sE, sD, sdB, sW})) != GEMM_OK) return st;
        if ((st = check_apart(name, "dB", sdB, {sA, dA ? sB : none, sT, sE, sD, sW})) != GEMM_OK) return st;
        if ((st = check_apart(name, "the workspace", sW, {sA, sB, sT, sE, sD})) != GEMM_OK) return st;
    }
    DeviceState *dev = nullptr;
    if ((st = device_state(&dev, nullptr)) != GEMM_OK) return st;
    auto call = [&](int64_t classes) {
        GroupedCall c{name, GEMM_GROUPED_PRODUCT, type, type, 1, classes, K, N};
        c.stream = stream;
        return c;
    };
    if (N == 0) {                                 // zeros
        const GroupedCall c = call(M);
        tn::GroupedParams prm = sink_params(c, K, 0, dA, ldda);
        prm.r_extent = static_cast<int32_t>(M);
        return launch_grouped_op<tn::kGrGradAOne>(c, *dev, prm, nullptr, nullptr, 0, 0, 0, 0, 0);
    }

    Sections ws{static_cast<uint8_t *>(workspace)};
    SinkOperands o{};
    if ((st = place_operands(name, *dev, plan.g, ws, nullptr, stream, o)) != GEMM_OK) return st;
    const int copied = (plan.g.x.copy ? 1 : 0) | (plan.g.y.copy ? 2 : 0);
    const int64_t ldd = plan.piece;
    uint16_t *d = ws.take<uint16_t>(size_t(N) * size_t(ldd));
    float2 *rows = ws.take<float2>(size_t(N));
    float *scale = ws.take<float>(1);
    float *sum = plan.floats ? ws.take<float>(plan.floats) : nullptr;
    const tn::LossRowsParams rp{targets, lse, dloss, rows, scale, N, M, type == GEMM_IN_F16};
    if ((st = launch_plain(name, tn::cross_entropy_rows_kernel, dim3(1, 1, 1), tn::kRowsThreads, 0, stream, rp)) != GEMM_OK)
        return st;
    for (int64_t i = 0; i < plan.pieces; ++i) {
        const int64_t first = i * plan.piece, classes = M - first < plan.piece ? M - first : plan.piece;
        const int64_t padded = (classes + 7) / 8 * 8;      // the products read whole 16-byte units
        const GroupedCall c = call(classes);
        const uint16_t *x = static_cast<const uint16_t *>(o.x) + first * o.ldx;
        tn::GroupedParams prm = sink_params(c, padded, K, d, ldd);
        prm.sink.targets = targets;
        prm.sink.rows = rows;
        prm.sink.lse = lse;
        prm.sink.first = static_cast<int32_t>(first);
        prm.sink.classes = static_cast<int32_t>(classes);
        st = K > tn::kGrSegment * tn::kGrBlock
                 ? launch_grouped_op<tn::kGrLossGradLong>(c, *dev, prm, x, o.y, o.ldx, 0, o.ldy, o.in_x, o.in_y)
                 : launch_grouped_op<tn::kGrLossGrad>(c, *dev, prm, x, o.y, o.ldx, 0, o.ldy, o.in_x, o.in_y);
        if (st == GEMM_OK && dB)
            st = launch_token_grad(c, *dev, plan.cut, x, o.ldx, o.in_x, d, ldd, classes, dB, lddb, scale, sum, i, plan.pieces);
        if (st == GEMM_OK && dA) {
            prm = sink_params(c, K, N, static_cast<uint16_t *>(dA) + first * ldda, ldda);
            prm.r_extent = static_cast<int32_t>(classes);
            prm.sink.out_scale = scale;
            st = launch_grouped_op<tn::kGrGradAOne>(c, *dev, prm, d, o.y, ldd, 0, o.ldy, padded, o.in_y);
        }
        t_rec.copied = copied;
        if (st != GEMM_OK) return st;
    }
    return GEMM_OK;
}
