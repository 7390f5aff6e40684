// How the products grouped by expert are planned and launched (included by the units
// that launch some of them, inside their anonymous namespaces).
//
// These calls keep nothing in the library: operand copies and grad_a's tensor
// maps go into a workspace that the caller passes, so calls on any streams,
// from any threads, and graphs captured from them share no buffer unless the
// caller gives them the same one.

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

// How one group's product is cut: the rows of a tile, at most, and the parts of the sum
// (more than one only where may_part says so), so that the last wave of tiles is
// nearly full.  An estimate in cycles decides: a block of 64 terms takes a CTA pair 2
// cycles a row of the tile, or the 64 bytes a cycle that its 128 + rows / 2 rows come in
// at; a tile some 2500 more; and parts are written and read again in FP32.  Measured on
// GB300, the loss's token gradient (logits again included) in one part / as the rule says: 1021
// tokens over 32003 classes of 1024 (8 tiles) 217.7 / 123.3 us in 4 (in 2 154.1, in 8 124.8), 300 over 32000
// of 2048 181.4 / 103.8; 4096 over 8192 of 4096 316.9 / 311.4 in one part of other rows (in 2
// 339.5).  Rows alone, the loss of 1021 over 32003: tiles of 256 57.2 us, as the rule says 57.1, of 192
// 63.6.  (The rule is the workspace query's too, so it asks no device: 152 SMs, a GB300's.  On another
// count results are right, and the last wave is not as full as planned.)
static_assert(kGroupedOps == tn::kGrOps, "every operation has its slots");

struct ProductCut {
    int32_t rows, parts;
};

constexpr int64_t kCutSms = 152, kSumFewRows = 64;

ProductCut cut_product(int group, int64_t rows, int64_t l_tiles, int64_t blocks, int64_t out_elems, bool may_part)
{
    const int64_t most = group == 2 ? 256 : 64, gran = 16 * group, slots = kCutSms / group;
    ProductCut best{static_cast<int32_t>(most), 1};
    if (rows <= 0 || blocks <= 0) return best;
    int64_t least = INT64_MAX;
    for (int64_t h = most; h >= most / 2; h -= gran) {
        const int64_t r_tiles = (rows + h - 1) / h, steps = (rows + gran - 1) / gran;
        const int64_t tall = (steps + r_tiles - 1) / r_tiles * gran;          // the rows are spread evenly
        const int64_t block = group == 2 ? (2 * tall > 256 + tall ? 2 * tall : 256 + tall) : 500;
        for (int64_t parts = 1; parts <= (may_part ? 16 : 1); ++parts) {
            if (parts > 1 && parts * 16 > blocks) break;
            const int64_t waves = (r_tiles * l_tiles * parts + slots - 1) / slots;
            int64_t cost = waves * ((blocks + parts - 1) / parts * block + 2500);
            if (parts > 1) cost += 8000 + parts * (out_elems / 256);
            if (cost < least) {
                least = cost;
                best = {static_cast<int32_t>(h), static_cast<int32_t>(parts)};
            }
        }
    }
    return best;
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
    cfg.blockDim = dim3(tn::GroupedWarps<kOp>::kThreads, 1, 1);
    cfg.dynamicSmemBytes = Cfg::kSmemBytes;
    int slots;
    {
        std::lock_guard<std::mutex> lock(g_mutex);
        int &n = dev.grouped_slots[kOp][variant];
        if (n == 0) {
            cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmemBytes);
            if (e != cudaSuccess) return fail(GEMM_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
            if (tn::GroupedWarps<kOp>::kSegmented && kRows > 64) {
                cudaFuncAttributes fa;
                e = cudaFuncGetAttributes(&fa, kernel);
                if (e != cudaSuccess || fa.numRegs < tn::GroupedWarps<kOp>::kRegs)
                    return fail(GEMM_ERR_CUDA, "%s: the kernel was compiled for fewer registers than it shares out", c.name);
            }
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
    constexpr int kReads = tn::grouped_reads(kOp), kSpan = kOp == tn::kGrGated ? Cfg::kTileL / 2 : Cfg::kTileL;
    const int64_t l_tiles = (int64_t(prm.l_extent) + kSpan - 1) / kSpan;
    const int64_t rows = kReads == tn::kGrGradA ? prm.r_extent : c.T;
    if (kOp >= tn::kGrGated) {
        if (kOp != tn::kGrGradBAdd)               // (there the call has cut it already)
            prm.tile_rows = prm.offsets || kRows > 256
                                ? kRows
                                : cut_product(kGroup, rows, l_tiles, (int64_t(prm.red) + 63) / 64, 0, false).rows;
    }
    const int64_t most = kOp >= tn::kGrGated ? prm.tile_rows : kRows;
    const int64_t r_tiles = kReads == tn::kGrGradA ? c.E * ((rows + most - 1) / most)
                                                : c.T / most + (c.E < c.T ? c.E : c.T);   // an upper bound
    if (r_tiles > (int64_t(1) << 30) / l_tiles) return fail(GEMM_ERR_UNSUPPORTED, "%s: too many output tiles", c.name);
    const int64_t tiles = r_tiles * l_tiles * (kOp == tn::kGrGradBAdd ? prm.parts : 1);
    constexpr int64_t kStageTerms = Cfg::kAtoms * tn::kGrBlock;
    if constexpr (kGroup == 1 && kOp != tn::kGrGradBAdd)
        prm.split = grouped_split(reinterpret_cast<const void *>(kernel), tn::GroupedWarps<kOp>::kThreads, Cfg::kSmemBytes, tiles,
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
    constexpr int kReads = tn::grouped_reads(kOp);
    // (A sum in parts has tiles enough: there the rows alone decide.)
    const bool few = kOp == tn::kGrGradBAdd ? c.T <= kSumFewRows : kReads != tn::kGrGradA &&
                     (c.T <= 32 * c.E ||
                      grouped_tiles(prm.l_extent, kOp == tn::kGrGated ? 64 : 128, c.T, c.E, 64) <= dev.sms);
    gemm_status_t st;
    if (prm.red > 0) {
        const CUtensorMapDataType type =
            prm.fmt ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
        if constexpr (kOp == tn::kGrGradAOne) {
            if ((st = encode_2d(&prm.tmap_r[0], type, x, inner_x, c.T, ldx * 2, 64, tn::kGrBlock, "dC")) != GEMM_OK) return st;
            if ((st = encode_2d(&prm.tmap_l, type, y, inner_y, c.T, ldy * 2, 64, tn::kGrBlock, "B")) != GEMM_OK) return st;
        } else if constexpr (tn::grouped_has_maps(kOp)) {
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
            const uint32_t box_l = kOp == tn::kGrGated ? 16 : kReads == tn::kGrGradB ? 64 : 128;
            const uint64_t apart = c.E > 1 ? uint64_t(stride_x) * 2 : uint64_t(16);
            const uint64_t gate_to_up = kOp == tn::kGrGated ? uint64_t(c.M) * uint64_t(ldx) * 2 : 0;
            if ((st = encode_map(&prm.tmap_l, type, x, inner_x, c.M, ldx * 2, c.E, apart, 64, box_l, "A", gate_to_up)) !=
                GEMM_OK)
                return st;
            for (uint32_t i = 0; i < (few ? 4 : 8); ++i)
                if ((st = encode_2d(&prm.tmap_r[i], type, y, inner_y, c.T, ldy * 2, 64, 16 * (i + 1), "rows")) != GEMM_OK)
                    return st;
        }
    }
    if constexpr (kReads != tn::kGrGradA) {
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
