// Host side of the products grouped by expert, the 8-bit integer products and
// the row quantiser (included by tn_gemm.cu, inside its anonymous namespace).
//
// These calls keep nothing in the library: operand copies and grad_a's tensor
// maps go into a workspace that the caller passes, so calls on any streams,
// from any threads, and graphs captured from them share no buffer unless the
// caller gives them the same one.

struct GroupedCall {
    const char *name;
    int op;                       // gemm_grouped_op_t
    int type, out_type;           // operands (16-bit ones) and result
    int64_t E, M, K, T;
    const void *X;                // A, or grad_a's dC
    int64_t ldx, stride_x;
    const void *Y;                // B, or grad_b's dC
    int64_t ldy;
    const int32_t *offsets;
    void *out;
    int64_t ldo, stride_o;
    const float *scale_a, *scale_b;
    void *workspace;
    int64_t workspace_bytes;
    cudaStream_t stream;
    bool needs_offsets = false;
};

// Tiles of l x up to r rows that T rows of E experts make, at most: the counts
// are known on the device only.
int64_t grouped_tiles(int64_t l_extent, int64_t l, int64_t T, int64_t E, int64_t r)
{
    return (l_extent + l - 1) / l * (T / r + (E < T ? E : T));
}

// The 8-bit product widens both operands on the way to the tensor core, on single
// CTAs (tn_i8_kernel), for few rows per expert and where its tiles make up to one
// and a half waves of the 152 SMs; else the tokens are widened first and CTA pairs
// widen the weights (tn_i8_pair_kernel).  The rule is the workspace query's too,
// so it asks no device.  Measured on GB300, single CTAs / pairs: 1024 x 200 x 4096
// (32 tiles) 11.9 / 19.7 us, 1024 x 1024 x 1024 (136) 8.7 / 11.9, 320 x 4178 x 2560
// (198) 21.0 / 25.2, 4096 x 512 x 4096 (288) 30.3 / 24.8, 2048 x 2048 x 2048 (528)
// 31.2 / 24.0.  The host knows the mean over all experts alone.  Where it is near the
// bound and the rows go to few of them, pairs would be faster: 16 experts of 4096 x 2048
// and 2000 rows 55.1 / 48.4 spread evenly, 53.9 / 38.9 over four, 53.1 / 36.1 over one;
// 64 of 2048 x 2048 and 8000 rows 103.9 / 85.0, 102.5 / 62.5 over four.
constexpr int64_t kI8DirectRows = 128, kI8DirectTiles = 228;

bool i8_direct(int64_t M, int64_t T, int64_t E)
{
    return T <= kI8DirectRows * E || grouped_tiles(M, tn::kI8RowsL, T, E, tn::kI8Rows) <= kI8DirectTiles;
}

// An operand as `blocks` matrices of rows x inner elements, and whether it is
// copied first: when the TMA cannot address it in place -- base, row stride or
// block stride not a multiple of 16 bytes, or the sum's index contiguous and its
// extent not one (a row that ends inside a 16-byte unit is not clipped element by
// element) -- or when the blocks interleave or repeat (a block stride below a
// row's); and 8-bit tokens for many rows per expert, to be widened to f16.
struct GroupedOperand {
    const void *base;
    int64_t rows, blocks, inner, ld, stride;
    bool copy;
    int64_t copy_ld;              // elements
    bool widen;                   // 8-bit integers to f16; else the copy is of the operand's type
    size_t copy_bytes;
};

GroupedOperand grouped_operand(const void *base, int64_t rows, int64_t blocks, int64_t inner, int64_t ld,
                               int64_t stride, bool inner_is_sum, bool i8)
{
    const int64_t vec = i8 ? 16 : 8;              // elements of 16 bytes
    GroupedOperand o{base, rows, blocks, inner, ld, stride, false, 0, false, 0};
    o.copy = reinterpret_cast<uintptr_t>(base) % 16 || ld % vec || (blocks > 1 && (stride % vec || stride < ld)) ||
             (inner_is_sum && inner % vec);
    return o;
}

// Sizes the copy, if there is one; false where 63 bits do not hold its bytes.
bool grouped_copy(GroupedOperand &o, bool i8, bool widen)
{
    o.widen = widen;
    o.copy |= widen;
    if (o.copy) {
        const int64_t rows = o.rows, blocks = o.blocks, inner = o.inner;
        o.copy_ld = (inner + 63) / 64 * 64;
        if (rows * blocks > (int64_t(1) << 60) / o.copy_ld) return false;
        o.copy_bytes = size_t(rows) * size_t(blocks) * size_t(o.copy_ld) * (i8 && !widen ? 1 : 2);
        o.copy_bytes = (o.copy_bytes + 255) & ~size_t(255);
    }
    return true;
}

struct GroupedPlan {
    GroupedOperand x, y;
    size_t map_bytes;             // grad_a: two tensor maps per expert
    bool fits;                    // the bytes are a number of 63 bits
    size_t bytes() const { return x.copy_bytes + y.copy_bytes + map_bytes; }
};

bool grouped_sizes_fit(int64_t E, int64_t M, int64_t K, int64_t T, int64_t ldx, int64_t ldy, int64_t stride)
{
    return E <= tn::kGrMaxExperts && M <= kMaxDim && K <= kMaxDim && T <= kMaxDim && ldx <= kMaxDim && ldy <= kMaxDim &&
           stride <= (int64_t(1) << 38);
}

// Nothing to read: the sum, or the result, is empty.
bool grouped_idle(int64_t E, int64_t M, int64_t K, int64_t T) { return E == 0 || M == 0 || K == 0 || T == 0; }

GroupedPlan grouped_plan(int op, int64_t E, int64_t M, int64_t K, int64_t T, const void *X, int64_t ldx,
                         int64_t stride_x, const void *Y, int64_t ldy)
{
    GroupedPlan g{};
    g.fits = true;
    if (grouped_idle(E, M, K, T)) return g;
    const bool i8 = op == GEMM_GROUPED_I8;
    if (op == GEMM_GROUPED_GRAD_A) {
        g.x = grouped_operand(X, T, 1, M, ldx, 0, false, false);
        g.y = grouped_operand(Y, T, 1, K, ldy, 0, false, false);
        g.map_bytes = size_t(E) * 2 * sizeof(CUtensorMap);
    } else {
        const bool grad_b = op == GEMM_GROUPED_GRAD_B;
        g.x = grouped_operand(X, M, E, K, ldx, stride_x, !grad_b, i8);
        g.y = grouped_operand(Y, T, 1, grad_b ? M : K, ldy, 0, true, i8);
    }
    g.fits = grouped_copy(g.x, i8, false) && grouped_copy(g.y, i8, i8 && !i8_direct(M, T, E));
    return g;
}

int64_t grouped_workspace(int op, int64_t E, int64_t M, int64_t K, int64_t T, const void *X, int64_t ldx,
                          int64_t stride_x, const void *Y, int64_t ldy)
{
    if (op < GEMM_GROUPED_PRODUCT || op > GEMM_GROUPED_I8 || E < 0 || M < 0 || K < 0 || T < 0 || ldx < 0 || ldy < 0 ||
        stride_x < 0 || !grouped_sizes_fit(E, M, K, T, ldx, ldy, stride_x))
        return -1;
    const int64_t inner_x = op == GEMM_GROUPED_GRAD_A ? M : K, inner_y = op == GEMM_GROUPED_GRAD_B ? M : K;
    if (ldx < 1 || ldx < inner_x || ldy < 1 || ldy < inner_y) return -1;
    const GroupedPlan plan = grouped_plan(op, E, M, K, T, X, ldx, stride_x, Y, ldy);
    return plan.fits ? static_cast<int64_t>(plan.bytes()) : -1;
}

// Copies the operands that the plan says into the workspace, in one launch.
template <typename Src>
gemm_status_t launch_widen(const char *name, DeviceState &dev, const GroupedPlan &plan, void *x, void *y,
                           const int32_t *offsets, cudaStream_t stream)
{
    constexpr int64_t kElems = 16 / sizeof(Src);
    auto job = [](const GroupedOperand &o, void *dst) {
        tn::WidenJob<Src> j{static_cast<const Src *>(o.base), o.ld, o.stride, static_cast<uint8_t *>(dst), o.copy_ld / kElems,
                            o.widen ? 32 : 16, o.rows, o.copy ? o.rows * o.blocks : 0, o.inner, 0, 1, 0, nullptr, nullptr};
        if (o.copy)
            j.end = reinterpret_cast<const char *>(j.src + (o.blocks - 1) * o.stride + (o.rows - 1) * o.ld + o.inner);
        while (j.shift < 5 && (int64_t(1) << j.shift) < j.units) ++j.shift;
        // A short row: of 32, 16 and 8 lanes the most that leave the fewest idle in its
        // last turn.  Measured on GB300, 32 lanes -> this: 447360 rows of 40 units 143 -> 97
        // us; but 850 rows of 712 with the gradient behind them 36 -> 52 us.
        for (int t = j.shift - 1; j.units <= 64 && t >= 3; --t) {
            auto idle = [&j](int n) { return (int64_t(1) << n) - 1 - (j.units - 1) % (int64_t(1) << n); };
            if (idle(t) < idle(j.shift)) j.shift = t;
        }
        j.segs = (j.units + tn::kWidenSeg - 1) / tn::kWidenSeg;
        j.work = ((j.rows + (int64_t(32) >> j.shift) - 1) >> (5 - j.shift)) * j.segs;
        return j;
    };
    tn::WidenJob<Src> jx = job(plan.x, x);
    const tn::WidenJob<Src> jy = job(plan.y, y);
    jx.offsets = offsets;
    const int64_t warps = jx.work + jy.work, per = tn::kWidenThreads / 32;
    int64_t blocks = (warps + per - 1) / per;
    if (blocks > int64_t(dev.sms) * 32) blocks = int64_t(dev.sms) * 32;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
    cfg.blockDim = dim3(tn::kWidenThreads, 1, 1);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, tn::widen_rows_kernel<Src>, jx, jy);
    if (e != cudaSuccess) return fail(GEMM_ERR_CUDA, "%s: launch (operand copy): %s", name, cudaGetErrorString(e));
    return GEMM_OK;
}

// Clusters of this launch that fit the device at once.
int co_resident(const void *kernel, const cudaLaunchConfig_t &cfg, int fallback)
{
    int found = 0;
    if (cudaOccupancyMaxActiveClusters(&found, kernel, &cfg) != cudaSuccess || found <= 0) {
        cudaGetLastError();
        found = fallback;
    }
    return found;
}

// How many single CTAs share each tile's sum of `stages` ring stages: 1, 2, 4 or
// 8, while every tile's cluster is resident at once and each CTA has four stages at
// least; but one CTA below twelve stages, where what the join costs (1.5 us) is not
// won back.  slots: the device's co-resident clusters of 2, 4 and 8 (0 = not queried).
// Measured on GB300, whole sums -> split: 1024 x 16 x 8192 in 8 bits (8 tiles)
// 22.3 -> 10.3 us, 4096 x 16 x 4096 (32 tiles) 13.4 -> 9.7, 2048 x 16 x 1536 7.8 -> 7.5,
// 2048 x 16 x 1024 6.8 -> 7.0; token gradient of 8 experts of 8192 x 512 with 256 rows
// 28.2 -> 19.1; and with more clusters of 8 than are resident, 2048 x 16 x 4096 14.0 -> 17.6.
int grouped_split(const void *kernel, int threads, int smem, int64_t tiles, int64_t stages, int sms, int (&slots)[3])
{
    int split = 1;
    if (stages < 12) return split;
    for (int i = 0; i < 3 && stages >= 8 * split && tiles * split * 2 <= sms; ++i, split *= 2) {
        std::lock_guard<std::mutex> lock(g_mutex);
        if (slots[i] == 0) {
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = split * 2;
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(static_cast<unsigned>(sms / (split * 2) * (split * 2)), 1, 1);
            cfg.blockDim = dim3(threads, 1, 1);
            cfg.dynamicSmemBytes = smem;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            slots[i] = co_resident(kernel, cfg, 1);
        }
        if (tiles > slots[i]) break;
    }
    return split;
}

template <int kOp, int kGroup, int kRows>
gemm_status_t launch_grouped(const GroupedCall &c, DeviceState &dev, tn::GroupedParams &prm, int variant)
{
    using Cfg = tn::GroupedCfg<kGroup, kRows>;
    auto kernel = tn::tn_grouped_kernel<kOp, kGroup, kRows>;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kGroup;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.blockDim = dim3(tn::kGrThreads, 1, 1);
    cfg.dynamicSmemBytes = Cfg::kSmemBytes;
    int slots;
    {
        std::lock_guard<std::mutex> lock(g_mutex);
        int &n = dev.grouped_slots[kOp][variant];
        if (n == 0) {
            cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmemBytes);
            if (e != cudaSuccess) return fail(GEMM_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
            int found = dev.sms;
            if (kGroup == 2) {
                cfg.attrs = attr + 1;
                cfg.numAttrs = 1;
                cfg.gridDim = dim3(kGroup * (dev.sms / kGroup), 1, 1);
                found = co_resident(reinterpret_cast<const void *>(kernel), cfg, dev.sms / kGroup);
            }
            n = found;
        }
        slots = n;
    }
    const int64_t l_tiles = (int64_t(prm.l_extent) + Cfg::kTileL - 1) / Cfg::kTileL;
    const int64_t r_tiles = kOp == tn::kGrGradA ? c.E * ((c.M + kRows - 1) / kRows)
                                                : c.T / kRows + (c.E < c.T ? c.E : c.T);   // an upper bound
    if (r_tiles > (int64_t(1) << 30) / l_tiles) return fail(GEMM_ERR_UNSUPPORTED, "%s: too many output tiles", c.name);
    const int64_t tiles = r_tiles * l_tiles;
    constexpr int64_t kStageTerms = Cfg::kAtoms * tn::kGrBlock;
    if constexpr (kGroup == 1)
        prm.split = grouped_split(reinterpret_cast<const void *>(kernel), tn::kGrThreads, Cfg::kSmemBytes, tiles,
                                  (int64_t(prm.red) + kStageTerms - 1) / kStageTerms, dev.sms, dev.split_slots[kOp]);
    const int cluster = kGroup * prm.split;
    const int grid = static_cast<int>(tiles < slots ? tiles : slots) * cluster;
    attr[1].val.clusterDim.x = cluster;
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.stream = c.stream;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    t_rec = LaunchRecord{};
    t_rec.name = c.name;
    t_rec.grouped = 1;
    t_rec.cluster = cluster;
    t_rec.grid = grid;
    t_rec.slots = slots;
    t_rec.tiles = static_cast<int>(tiles);
    cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, prm);
    if (e != cudaSuccess) return fail(GEMM_ERR_CUDA, "%s: launch: %s", c.name, cudaGetErrorString(e));
    return GEMM_OK;
}

// x, y: the weights and the tokens, 8-bit integers that the TMA can address.
gemm_status_t launch_i8(const GroupedCall &c, DeviceState &dev, tn::GroupedParams &prm, const void *x, const void *y,
                        int64_t ldx, int64_t stride_x, int64_t ldy, int64_t inner_x, int64_t inner_y)
{
    gemm_status_t st;
    const uint64_t apart = c.E > 1 ? uint64_t(stride_x) : uint64_t(16);
    if (prm.red > 0) {
        if ((st = encode_map(&prm.tmap_l, CU_TENSOR_MAP_DATA_TYPE_UINT8, x, inner_x, c.M, ldx, c.E, apart, tn::kI8Block,
                             tn::kI8RowsL, "A")) != GEMM_OK)
            return st;
        for (uint32_t i = 0; i < tn::kI8Rows / 16; ++i)
            if ((st = encode_2d(&prm.tmap_r[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, y, inner_y, c.T, ldy, tn::kI8Block,
                                16 * (i + 1), "rows")) != GEMM_OK)
                return st;
    }
    auto kernel = tn::tn_i8_kernel;
    {
        std::lock_guard<std::mutex> lock(g_mutex);
        if (!dev.i8_attr) {
            cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, tn::kI8SmemBytes);
            if (e != cudaSuccess) return fail(GEMM_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
            dev.i8_attr = true;
        }
    }
    const int64_t tiles = grouped_tiles(c.M, tn::kI8RowsL, c.T, c.E, tn::kI8Rows);
    if (tiles > int64_t(1) << 30) return fail(GEMM_ERR_UNSUPPORTED, "%s: too many output tiles", c.name);
    prm.split = grouped_split(reinterpret_cast<const void *>(kernel), tn::kI8Threads, tn::kI8SmemBytes, tiles,
                              (int64_t(prm.red) + tn::kI8Block - 1) / tn::kI8Block, dev.sms, dev.split_slots[2]);
    const int grid = static_cast<int>(tiles < dev.sms ? tiles : dev.sms) * prm.split;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = prm.split;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(tn::kI8Threads, 1, 1);
    cfg.dynamicSmemBytes = tn::kI8SmemBytes;
    cfg.stream = c.stream;
    cfg.attrs = attr;
    cfg.numAttrs = prm.split > 1 ? 2 : 1;
    t_rec = LaunchRecord{};
    t_rec.name = c.name;
    t_rec.grouped = 1;
    t_rec.cluster = prm.split;
    t_rec.grid = grid;
    t_rec.slots = dev.sms;
    t_rec.tiles = static_cast<int>(tiles);
    cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, prm);
    if (e != cudaSuccess) return fail(GEMM_ERR_CUDA, "%s: launch: %s", c.name, cudaGetErrorString(e));
    return GEMM_OK;
}

// x as for launch_i8; tokens: the widened copy, ld_tokens elements a row.
template <bool kRuns>
gemm_status_t launch_i8_pair(const GroupedCall &c, DeviceState &dev, tn::GroupedParams &prm, const void *x, int64_t ldx,
                             int64_t stride_x, int64_t inner_x, const void *tokens, int64_t ld_tokens)
{
    using Cfg = tn::I8PairCfg<kRuns>;
    gemm_status_t st;
    const uint64_t apart = c.E > 1 ? uint64_t(stride_x) : uint64_t(16);
    if (prm.red > 0) {
        if ((st = encode_map(&prm.tmap_l, CU_TENSOR_MAP_DATA_TYPE_UINT8, x, inner_x, c.M, ldx, c.E, apart, tn::kI8Block,
                             128, "A")) != GEMM_OK)
            return st;
        for (uint32_t i = 0; i < tn::kIpRowsR / 16; ++i)
            if ((st = encode_2d(&prm.tmap_r[i], CU_TENSOR_MAP_DATA_TYPE_FLOAT16, tokens, ld_tokens, c.T, ld_tokens * 2,
                                tn::kGrBlock,
                                16 * (i + 1), "rows")) != GEMM_OK)
                return st;
    }
    auto kernel = tn::tn_i8_pair_kernel<kRuns>;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.blockDim = dim3(Cfg::kThreads, 1, 1);
    cfg.dynamicSmemBytes = Cfg::kSmemBytes;
    int slots;
    {
        std::lock_guard<std::mutex> lock(g_mutex);
        int &n = dev.i8_pair_slots[kRuns];
        if (n == 0) {
            cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmemBytes);
            if (e != cudaSuccess) return fail(GEMM_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
            // (with fewer registers its epilogue would wait for more than there are)
            cudaFuncAttributes fa;
            e = cudaFuncGetAttributes(&fa, kernel);
            if (e != cudaSuccess || (kRuns && fa.numRegs < tn::kIpLaunchRegs))
                return fail(GEMM_ERR_CUDA, "%s: the kernel was compiled for fewer registers than it shares out", c.name);
            cfg.attrs = attr + 1;
            cfg.numAttrs = 1;
            cfg.gridDim = dim3(2 * (dev.sms / 2), 1, 1);
            n = co_resident(reinterpret_cast<const void *>(kernel), cfg, dev.sms / 2);
        }
        slots = n;
    }
    const int64_t tiles = grouped_tiles(c.M, 256, c.T, c.E, tn::kIpRows);
    if (tiles > int64_t(1) << 30) return fail(GEMM_ERR_UNSUPPORTED, "%s: too many output tiles", c.name);
    const int grid = 2 * static_cast<int>(tiles < slots ? tiles : slots);
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.stream = c.stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    t_rec = LaunchRecord{};
    t_rec.name = c.name;
    t_rec.grouped = 1;
    t_rec.cluster = 2;
    t_rec.grid = grid;
    t_rec.slots = slots;
    t_rec.tiles = static_cast<int>(tiles);
    cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, prm);
    if (e != cudaSuccess) return fail(GEMM_ERR_CUDA, "%s: launch: %s", c.name, cudaGetErrorString(e));
    return GEMM_OK;
}

template <int kOp>
gemm_status_t launch_grouped_op(const GroupedCall &c, DeviceState &dev, tn::GroupedParams &prm,
                                const void *x, const void *y, int64_t ldx, int64_t stride_x, int64_t ldy,
                                int64_t inner_x, int64_t inner_y)
{
    // Single CTAs of 128 x 64 tiles (four times as many of them, and no pair to set
    // up) for few rows per expert, where the read of the weights is what counts, as
    // long as an expert's rows mostly fit one tile; and where their tiles make no more
    // than one wave, so that pairs leave SMs idle.  Measured on GB300, single CTAs /
    // pairs: 16 experts of 4096 x 1024 with 1 row on average 16.5 / 17.3 us, 32 rows
    // 27.6 / 28.6; 8 of 2048 x 4096 with 32 rows 26.2 / 28.2, but with 48 (some over 64)
    // 35.8 / 28.6.  By tiles: 8 of 1024 x 4096 with 512 rows in all (128) 18.1 / 20.8,
    // 5 of 200 x 5240 with 2020 (72, the sum split) 17.8 / 34.9; 4 of 2048 x 2048 with
    // 400 (160) 10.8 / 10.4, 8 of 1024 x 1024 with 1024 (192) 11.2 / 8.6.
    // The rows per expert are the mean over all, also where few experts get them; pairs
    // would then be faster: 64 experts of 2048 x 2048 and 2000 rows 85.7 / 90.4 spread
    // evenly, but 37.2 / 31.6 over 16 of them, 34.4 / 18.4 over four, 31.0 / 16.3 over one.
    const bool few = kOp != tn::kGrGradA &&
                     (c.T <= 32 * c.E || grouped_tiles(prm.l_extent, 128, c.T, c.E, 64) <= dev.sms);
    gemm_status_t st;
    if (prm.red > 0) {
        const CUtensorMapDataType type =
            prm.fmt ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
        if constexpr (kOp == tn::kGrGradA) {
            tn::GroupedMapsParams m;
            memset(&m, 0, sizeof(m));
            if ((st = encode_2d(&m.dc, type, x, inner_x, c.T, ldx * 2, 64, tn::kGrBlock, "dC")) != GEMM_OK) return st;
            if ((st = encode_2d(&m.b, type, y, inner_y, c.T, ldy * 2, 64, tn::kGrBlock, "B")) != GEMM_OK) return st;
            m.maps = const_cast<CUtensorMap *>(prm.group_maps);
            m.offsets = prm.offsets;
            m.dc_base = static_cast<const uint8_t *>(x);
            m.b_base = static_cast<const uint8_t *>(y);
            m.dc_row_bytes = ldx * 2;
            m.b_row_bytes = ldy * 2;
            m.E = prm.E;
            m.T = prm.T;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
            attr[0].val.programmaticStreamSerializationAllowed = 1;
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(static_cast<unsigned>(2 * c.E), 1, 1);
            cfg.blockDim = dim3(32, 1, 1);
            cfg.stream = c.stream;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            cudaError_t e = cudaLaunchKernelEx(&cfg, tn::grouped_maps_kernel, m);
            if (e != cudaSuccess) return fail(GEMM_ERR_CUDA, "%s: launch (tensor maps): %s", c.name, cudaGetErrorString(e));
        } else {
            const uint32_t box_l = kOp == tn::kGrGradB ? 64 : 128;
            const uint64_t apart = c.E > 1 ? uint64_t(stride_x) * 2 : uint64_t(16);
            if ((st = encode_map(&prm.tmap_l, type, x, inner_x, c.M, ldx * 2, c.E, apart, 64, box_l, "A")) != GEMM_OK)
                return st;
            for (uint32_t i = 0; i < (few ? 4 : 8); ++i)
                if ((st = encode_2d(&prm.tmap_r[i], type, y, inner_y, c.T, ldy * 2, 64, 16 * (i + 1), "rows")) != GEMM_OK)
                    return st;
        }
    }
    if constexpr (kOp != tn::kGrGradA) {
        if (few) return launch_grouped<kOp, 1, 64>(c, dev, prm, 0);
    } else {
        // Short sums are bound by what surrounds them and by the stores: tiles of two
        // halves, half as many.  Measured on GB300, 256 -> 512 rows: 32 experts of 1024 x 2048
        // and 3008 rows 51.6 -> 44.5 us; but 8 of 8192 x 4096 and 8192 rows 324 -> 340 us, of
        // 4096 x 4096 and 16384 rows 342 -> 343.  By the mean over all experts: near the bound,
        // 32 of 1024 x 2048 and 8000 rows, 41.3 -> 43.6 spread evenly, 51.1 -> 57.1 where eight
        // of them get the rows, 79.8 -> 105.6 where one does.
        if (c.M >= 512 && c.T <= 256 * c.E) return launch_grouped<kOp, 2, 512>(c, dev, prm, 2);
    }
    return launch_grouped<kOp, 2, 256>(c, dev, prm, 1);
}

gemm_status_t run_grouped(const GroupedCall &c)
{
    const char *name = c.name;
    const bool i8 = c.op == GEMM_GROUPED_I8, grad_a = c.op == GEMM_GROUPED_GRAD_A, grad_b = c.op == GEMM_GROUPED_GRAD_B;
    for (int t : {c.type, c.out_type})
        if (t != GEMM_IN_F16 && t != GEMM_IN_BF16)
            return fail(GEMM_ERR_INVALID_ARG, "%s: unknown or unsupported type %d (GEMM_IN_F16 or GEMM_IN_BF16)", name, t);
    if (c.E < 0 || c.M < 0 || c.K < 0 || c.T < 0)
        return fail(GEMM_ERR_INVALID_ARG, "%s: negative size (E=%lld M=%lld K=%lld rows=%lld)", name, (long long)c.E,
                    (long long)c.M, (long long)c.K, (long long)c.T);
    auto at_least = [](int64_t v) { return v > 1 ? v : int64_t(1); };
    const int64_t inner_x = grad_a ? c.M : c.K, inner_y = grad_b ? c.M : c.K;
    const int64_t inner_o = grad_a || grad_b ? c.K : c.M;
    if (c.ldx < at_least(inner_x) || c.ldy < at_least(inner_y) || c.ldo < at_least(inner_o))
        return fail(GEMM_ERR_INVALID_ARG, "%s: a leading dimension is below its row's length", name);
    if (c.stride_x < 0 || c.stride_o < 0) return fail(GEMM_ERR_INVALID_ARG, "%s: negative stride", name);
    if (!grouped_sizes_fit(c.E, c.M, c.K, c.T, c.ldx, c.ldy, c.stride_x > c.stride_o ? c.stride_x : c.stride_o) ||
        c.ldo > kMaxDim)
        return fail(GEMM_ERR_UNSUPPORTED, "%s: more than %d experts, or a size, leading dimension or stride too large", name,
                    tn::kGrMaxExperts);
    // the result is empty, or has no row that any expert could own
    if (c.E == 0 || inner_o == 0 || (grad_a ? c.M == 0 : c.T == 0)) return GEMM_OK;
    const int64_t red = grad_a ? c.T : (grad_b ? c.M : c.K);
    if (!c.out) return fail(GEMM_ERR_INVALID_ARG, "%s: the result is NULL", name);
    if (reinterpret_cast<uintptr_t>(c.out) % 2) return fail(GEMM_ERR_INVALID_ARG, "%s: the result is not 2-byte aligned", name);
    // the experts' matrices lie one after the other, or row by row beside each other
    if (grad_a && c.E > 1 && c.stride_o < (c.M - 1) * c.ldo + c.K &&
        (c.stride_o < c.K || c.ldo < (c.E - 1) * c.stride_o + c.K))
        return fail(GEMM_ERR_INVALID_ARG, "%s: the experts' results overlap", name);
    const uintptr_t misfit = i8 ? 0 : 1;
    if (red > 0) {
        if (!c.X || !c.Y) return fail(GEMM_ERR_INVALID_ARG, "%s: an operand is NULL", name);
        if ((reinterpret_cast<uintptr_t>(c.X) | reinterpret_cast<uintptr_t>(c.Y)) & misfit)
            return fail(GEMM_ERR_INVALID_ARG, "%s: an operand is not aligned to its element size", name);
    }
    const bool dense = i8 && !c.needs_offsets;
    if (!dense) {
        if (!c.offsets) return fail(GEMM_ERR_INVALID_ARG, "%s: offsets is NULL", name);
        if (reinterpret_cast<uintptr_t>(c.offsets) % 4)
            return fail(GEMM_ERR_INVALID_ARG, "%s: offsets is not 4-byte aligned", name);
    }
    if (i8) {
        if (!c.scale_a || !c.scale_b) return fail(GEMM_ERR_INVALID_ARG, "%s: a scale pointer is NULL", name);
        if ((reinterpret_cast<uintptr_t>(c.scale_a) | reinterpret_cast<uintptr_t>(c.scale_b)) % 4)
            return fail(GEMM_ERR_INVALID_ARG, "%s: a scale pointer is not 4-byte aligned", name);
    }
    const GroupedPlan plan = grouped_plan(c.op, c.E, c.M, c.K, c.T, c.X, c.ldx, c.stride_x, c.Y, c.ldy);
    if (!plan.fits) return fail(GEMM_ERR_UNSUPPORTED, "%s: the operands' copies are too large", name);
    if (plan.bytes() > 0) {
        if (!c.workspace || c.workspace_bytes < static_cast<int64_t>(plan.bytes()))
            return fail(GEMM_ERR_INVALID_ARG, "%s: the workspace has %lld bytes, %zu are needed (gemm_grouped_workspace)", name,
                        (long long)(c.workspace ? c.workspace_bytes : 0), plan.bytes());
        if (reinterpret_cast<uintptr_t>(c.workspace) % 256)
            return fail(GEMM_ERR_INVALID_ARG, "%s: the workspace is not 256-byte aligned", name);
    }
    DeviceState *dev = nullptr;
    gemm_status_t st = device_state(&dev, nullptr);
    if (st != GEMM_OK) return st;

    uint8_t *ws = static_cast<uint8_t *>(c.workspace);
    const void *x = c.X, *y = c.Y;
    int64_t ldx = c.ldx, stride_x = c.stride_x, ldy = c.ldy, in_x = inner_x, in_y = inner_y;
    int copied = 0;
    if (plan.x.copy) {
        x = ws;
        ws += plan.x.copy_bytes;
        ldx = in_x = plan.x.copy_ld;
        stride_x = plan.x.rows * ldx;
        copied |= 1;
    }
    if (plan.y.copy) {
        y = ws;
        ws += plan.y.copy_bytes;
        ldy = in_y = plan.y.copy_ld;
        copied |= 2;
    }
    if (copied) {
        const int32_t *per_expert = grad_a || dense ? nullptr : c.offsets;     // x is the experts' weights
        st = i8 ? launch_widen<int8_t>(name, *dev, plan, const_cast<void *>(x), const_cast<void *>(y), per_expert, c.stream)
                : launch_widen<uint16_t>(name, *dev, plan, const_cast<void *>(x), const_cast<void *>(y), per_expert, c.stream);
        if (st != GEMM_OK) return st;
    }
    tn::GroupedParams prm;
    memset(&prm, 0, sizeof(prm));
    prm.group_maps = reinterpret_cast<const CUtensorMap *>(ws);
    prm.offsets = dense ? nullptr : c.offsets;
    prm.out = static_cast<uint16_t *>(c.out);
    prm.out_ld = c.ldo;
    prm.out_stride = grad_a ? c.stride_o : 0;
    prm.E = static_cast<int32_t>(c.E);
    prm.T = static_cast<int32_t>(c.T);
    prm.l_extent = static_cast<int32_t>(inner_o);
    prm.r_extent = grad_a ? static_cast<int32_t>(c.M) : 0;
    prm.red = static_cast<int32_t>(red);
    prm.fmt = c.type == GEMM_IN_BF16 ? 1u : 0u;
    prm.out_fmt = c.out_type == GEMM_IN_BF16 ? 1u : 0u;
    prm.out_vec = reinterpret_cast<uintptr_t>(c.out) % 16 == 0 && c.ldo % 8 == 0 && (!grad_a || c.stride_o % 8 == 0);
    prm.split = 1;
    prm.scale_l = c.scale_a;
    prm.scale_r = c.scale_b;
    prm.flags = stall_flags(g_inject_stall.load());
    prm.wait_limit_ns = g_wait_limit_ns.load();
    if (i8 && plan.y.widen)
        st = red > tn::kI8Run * tn::kI8Block ? launch_i8_pair<true>(c, *dev, prm, x, ldx, stride_x, in_x, y, ldy)
                                             : launch_i8_pair<false>(c, *dev, prm, x, ldx, stride_x, in_x, y, ldy);
    else if (i8)
        st = launch_i8(c, *dev, prm, x, y, ldx, stride_x, ldy, in_x, in_y);
    else if (grad_a)
        st = launch_grouped_op<tn::kGrGradA>(c, *dev, prm, x, y, ldx, stride_x, ldy, in_x, in_y);
    else if (grad_b)
        st = launch_grouped_op<tn::kGrGradB>(c, *dev, prm, x, y, ldx, stride_x, ldy, in_x, in_y);
    else
        st = launch_grouped_op<tn::kGrProduct>(c, *dev, prm, x, y, ldx, stride_x, ldy, in_x, in_y);
    t_rec.copied = copied;
    return st;
}

// Launches the row quantiser: a warp per row up to 8 windows of 16 bytes a lane
// (4 KiB of x), unless the rows are too few to fill the SMs that way; then a
// CTA of 256, 512 or 1024 threads with up to 8 windows a thread (32, 64 and 128
// KiB); beyond that the kernel that reads x twice.
template <int kIn>
gemm_status_t launch_quant_rows(DeviceState &dev, qz::QuantRowsParams &prm, cudaStream_t stream)
{
    constexpr int64_t kElem = qz::elem_bytes(kIn), kVec = 16 / kElem;
    const bool aligned = reinterpret_cast<uintptr_t>(prm.x) % 16 == 0 && reinterpret_cast<uintptr_t>(prm.q) % kVec == 0 &&
                         (prm.rows == 1 || ((prm.ldx * kElem) % 16 == 0 && prm.ldq % kVec == 0));
    const int64_t windows = (prm.cols + kVec - 1) / kVec + (aligned ? 0 : 1);
    void (*kernel)(qz::QuantRowsParams);
    int threads = qz::kRowThreads, rows_per_cta = 1;
    // a row's codes are staged in shared memory where rows are not aligned (more
    // than it has room for: the kernel for long rows, which does not stage)
    const int64_t staging = aligned ? 0 : (windows * kVec + 4 + 15) / 16 * 16;
    const bool long_rows = windows > 1024 * 8 || staging > qz::kMaxStaging;
    prm.staging_bytes = long_rows ? 0 : static_cast<int32_t>(staging);
    if (long_rows) {
        kernel = qz::quant_long_rows_kernel<kIn>;
        threads = qz::kLongThreads;
    } else if (windows <= 32 * 2 && prm.rows > 8 * dev.sms) {
        kernel = aligned ? qz::quant_rows_kernel<kIn, 32, 2, true> : qz::quant_rows_kernel<kIn, 32, 2, false>;
        rows_per_cta = qz::kRowThreads / 32;
    } else if (windows <= 32 * 8 && prm.rows > 8 * dev.sms) {
        kernel = aligned ? qz::quant_rows_kernel<kIn, 32, 8, true> : qz::quant_rows_kernel<kIn, 32, 8, false>;
        rows_per_cta = qz::kRowThreads / 32;
    } else if (windows <= 256 * (aligned ? 4 : 5)) {      // (a row off its alignment has a window more)
        kernel = aligned ? qz::quant_rows_kernel<kIn, 256, 4, true> : qz::quant_rows_kernel<kIn, 256, 5, false>;
    } else if (windows <= 256 * 8) {
        kernel = aligned ? qz::quant_rows_kernel<kIn, 256, 8, true> : qz::quant_rows_kernel<kIn, 256, 8, false>;
    } else if (windows <= 512 * 8) {
        kernel = aligned ? qz::quant_rows_kernel<kIn, 512, 8, true> : qz::quant_rows_kernel<kIn, 512, 8, false>;
        threads = 512;
    } else {
        kernel = aligned ? qz::quant_rows_kernel<kIn, 1024, 8, true> : qz::quant_rows_kernel<kIn, 1024, 8, false>;
        threads = 1024;
    }
    int64_t grid = (prm.rows + rows_per_cta - 1) / rows_per_cta;
    if (long_rows && grid > int64_t(dev.sms) * 4) grid = int64_t(dev.sms) * 4;
    if (grid > INT32_MAX) return fail(GEMM_ERR_UNSUPPORTED, "gemm_quantize_i8_rows: too many rows");
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(rows_per_cta) * prm.staging_bytes;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    t_rec = LaunchRecord{};
    t_rec.name = "gemm_quantize_i8_rows";
    t_rec.quant = true;
    t_rec.qgrid = grid;
    t_rec.qunits = prm.rows;
    t_rec.vec = aligned;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, prm);
    if (e != cudaSuccess) return fail(GEMM_ERR_CUDA, "gemm_quantize_i8_rows: launch: %s", cudaGetErrorString(e));
    return GEMM_OK;
}

gemm_status_t run_quant_rows(const void *x, int x_type, int64_t rows, int64_t cols, int64_t ldx, int8_t *q, int64_t ldq,
                             float *scale, cudaStream_t stream)
{
    const char *name = "gemm_quantize_i8_rows";
    if (x_type < qz::kInF32 || x_type > qz::kInBF16)
        return fail(GEMM_ERR_INVALID_ARG, "%s: unknown input type %d", name, x_type);
    const int64_t esz = x_type == qz::kInF32 ? 4 : 2;
    if (rows < 0 || cols < 0) return fail(GEMM_ERR_INVALID_ARG, "%s: negative size", name);
    const int64_t cmin = cols > 1 ? cols : 1;
    if (ldx < cmin || ldq < cmin) return fail(GEMM_ERR_INVALID_ARG, "%s: ldx or ldq < max(1, cols)", name);
    if (rows == 0) return GEMM_OK;
    if (!scale) return fail(GEMM_ERR_INVALID_ARG, "%s: scale is NULL", name);
    if (reinterpret_cast<uintptr_t>(scale) % 4) return fail(GEMM_ERR_INVALID_ARG, "%s: scale is not 4-byte aligned", name);
    if (cols > 0) {
        if (!x || !q) return fail(GEMM_ERR_INVALID_ARG, "%s: x or q is NULL", name);
        if (reinterpret_cast<uintptr_t>(x) % esz)
            return fail(GEMM_ERR_INVALID_ARG, "%s: x is not aligned to its element size", name);
    }
    if (rows > (int64_t(1) << 40) / cmin) return fail(GEMM_ERR_UNSUPPORTED, "%s: more than 2^40 elements", name);
    DeviceState *dev = nullptr;
    gemm_status_t st = device_state(&dev, nullptr);
    if (st != GEMM_OK) return st;
    qz::QuantRowsParams prm{x, q, scale, ldx, ldq, rows, cols, 0};
    switch (x_type) {
    case qz::kInF32: return launch_quant_rows<qz::kInF32>(*dev, prm, stream);
    case qz::kInF16: return launch_quant_rows<qz::kInF16>(*dev, prm, stream);
    default: return launch_quant_rows<qz::kInBF16>(*dev, prm, stream);
    }
}
