// The calls of the products grouped by expert, of the 8-bit integer products and of
// the row quantiser (included by tn_gemm.cu, inside its anonymous namespace).

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
