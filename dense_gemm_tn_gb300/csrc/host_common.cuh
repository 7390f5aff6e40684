// What the library's translation units share on the host: per-device state, errors,
// tensor maps, the record of the last launch.  Defined in tn_gemm.cu; one unit for the
// dense, grouped and 8-bit products (tn_gemm.cu), one for the gated projections and
// the loss (layers.cu), one for the 4-bit products (w4.cu), compiled side by side.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <cstring>
#include <initializer_list>
#include <memory>
#include <mutex>
#include <unordered_map>

#include "tn_gemm.h"

namespace tn {
struct GroupedParams;
}

namespace __attribute__((visibility("hidden"))) tn_host {

constexpr int kGroupedOps = 12;                          // tn::GroupedOp
constexpr int64_t kMaxDim = (int64_t(1) << 31) - 256;   // TMA coordinates are signed 32-bit

gemm_status_t fail(gemm_status_t s, const char *fmt, ...);
void clear_error();

struct DeviceState {
    bool ready = false;
    int sms = 0, major = 0, minor = 0;
    // per kernel, indexed [kind: f16, e4m3][1: one CTA, 2: CTA pairs, 3: CTA pairs with 256 x 512 tiles,
    // 4 / 5: one CTA / CTA pairs in k-range clusters]
    bool smem_attr[2][10] = {};
    int max_clusters[2][10] = {};     // co-resident clusters of the kernel's own size (0 = not queried yet)
    // co-resident clusters of S single CTAs or S CTA pairs (kClusterReduce), by kind, CTAs per tile and S
    // (0 = not queried, -1 = none)
    int cluster_slots[2][3][5] = {};
    // Split-K partial sums of the last wave, one buffer per stream (calls on
    // one stream are ordered, so they may share it): [tickets | partials].
    struct Split {
        void *ptr = nullptr;
        size_t bytes = 0, ticket_bytes = 0;
        bool dirty = false;      // a launch may have stopped part-way (timeout): clear the tickets first
    };
    std::unordered_map<cudaStream_t, Split> split;
    // Per-CTA maxima of the quantiser, one array per stream.
    std::unordered_map<cudaStream_t, Split> quant;
    // Row copies of operands the TMA cannot address in place, one workspace
    // per stream, so calls on different streams may copy at the same time.
    std::unordered_map<cudaStream_t, Split> repack;
    // Softmax statistics: [tickets per tile row | parts], one buffer per stream.
    std::unordered_map<cudaStream_t, Split> stats;
    int quant_blocks[3] = {};         // co-resident quantiser CTAs per SM, by input type (0 = not queried)
    bool skinny_attr[2] = {};         // tn_skinny_kernel's shared-memory attribute set, by kind
    int grouped_slots[kGroupedOps][3] = {};   // co-resident tn_grouped_kernel CTAs or pairs, by operation and variant (0 = not queried)
    int split_slots[kGroupedOps][3] = {};     // co-resident clusters of 2, 4 and 8 single CTAs, by operation (8-bit: 2)
    bool few_attr[2][2] = {};         // gated_few_kernel's shared-memory attribute set, by type and token tiles
    // 4-bit products' shared-memory attribute set, by kernel (warps split the sum, warps share the
    // tokens), type, whole blocks a group, row tiles and token tiles
    bool w4_attr[2][2][2][3][9] = {};
    bool i8_attr = false;             // tn_i8_kernel's shared-memory attribute set
    int i8_pair_slots[2] = {};        // co-resident pairs of tn_i8_pair_kernel, by its kRuns (0 = not queried)
    // One lock per stream, held by a call from its first buffer lookup through
    // its last launch: a call is several launches (row copy, GEMM, reduce),
    // and two host threads' calls on one stream must not interleave them.
    std::unordered_map<cudaStream_t, std::unique_ptr<std::mutex>> stream_locks;
};

extern std::mutex g_mutex;
extern std::atomic<uint64_t> g_wait_limit_ns;
extern std::atomic<int> g_inject_stall;

// The last launch on this host thread, for gemm_debug_last_launch: the
// numbers are kept and formatted only when asked for (formatting every call
// cost host time on the path of back-to-back small GEMMs).
struct LaunchRecord {
    const char *name = nullptr;     // nullptr: nothing launched yet
    bool quant = false;
    int G = 0, wide = 0, grid = 0, clusters = 0, slots = 0;
    int tiles = 0, units = 0, tail_start = 0, tail_mode = 0, split_parts = 0, vec = 0, cluster = 0, lean = 0;
    int skinny = 0;
    int grouped = 0, copied = 0;    // a product grouped by expert (tiles: an upper bound); operands copied (1: first, 2: second)
    long long qgrid = 0, qunits = 0;
};
extern thread_local LaunchRecord t_rec;

// Current device's state, initialised on first use (caller holds no lock).
gemm_status_t device_state(DeviceState **out, int *dev_out);

// depth > 0: a 3-D map of `depth` such matrices, depth_bytes apart, with boxes
// of one matrix; with mid_bytes > 0 a 4-D map of `depth` pairs of them, a pair's
// matrices mid_bytes apart, with boxes of one pair.
gemm_status_t encode_map(CUtensorMap *map, CUtensorMapDataType type, const void *base, uint64_t inner,
                         uint64_t outer, uint64_t row_bytes, uint64_t depth, uint64_t depth_bytes,
                         uint32_t box_inner, uint32_t box_outer, const char *what, uint64_t mid_bytes = 0);
gemm_status_t encode_2d(CUtensorMap *map, CUtensorMapDataType type, const void *base, uint64_t inner,
                        uint64_t outer, uint64_t row_bytes, uint32_t box_inner, uint32_t box_outer,
                        const char *what);

// gemm_debug_inject_stall modes -> kernel flags.
uint32_t stall_flags(int mode);

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

// The grouped gradients' launches (tn_gemm.cu), for the gated projections' by expert.
gemm_status_t launch_grad_b(const GroupedCall &c, DeviceState &dev, tn::GroupedParams &prm, const void *x, const void *y,
                            int64_t ldx, int64_t stride_x, int64_t ldy, int64_t inner_x, int64_t inner_y);
gemm_status_t launch_grad_a(const GroupedCall &c, DeviceState &dev, tn::GroupedParams &prm, const void *x, const void *y,
                            int64_t ldx, int64_t stride_x, int64_t ldy, int64_t inner_x, int64_t inner_y);

// The status word of layers.cu's kernels: a unit's kernels have one of their own.
cudaError_t take_layers_status(int *value);

inline bool aligned_to(const void *p, uintptr_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

// What a call reads or writes: `blocks` matrices of rows of `width` bytes, `pitch` bytes apart, the
// matrices `stride` apart.  NULL, or no bytes: nothing.
struct Span {
    const void *base;
    int64_t blocks, stride, rows, pitch, width;

    Span(const void *p, int64_t bytes) : Span(p, 1, 0, 1, 0, bytes) {}
    Span(const void *p, int64_t blocks_, int64_t stride_, int64_t rows_, int64_t pitch_, int64_t width_)
        : base(p), blocks(blocks_), stride(stride_), rows(rows_), pitch(pitch_), width(width_)
    {
        if (!p || blocks_ < 1 || rows_ < 1 || width_ < 1) blocks = 0;
        constexpr int64_t kMost = int64_t(1) << 56;          // (no address space holds more)
        if (pitch > 0 && rows > kMost / pitch) rows = kMost / pitch;
        if (blocks > 1 && stride == rows * pitch) rows *= blocks, blocks = 1;     // one after another
    }
    uintptr_t lo() const { return reinterpret_cast<uintptr_t>(base); }
    uintptr_t hi() const { return lo() + (blocks - 1) * stride + (rows - 1) * pitch + width; }
    bool dense() const { return blocks == 1 && (rows == 1 || pitch == width); }
    Span block(int64_t i) const { return Span(static_cast<const char *>(base) + i * stride, 1, 0, rows, pitch, width); }
};

// Whether some row of x (one matrix) meets the bytes [lo, hi).
inline bool rows_meet(const Span &x, uintptr_t lo, uintptr_t hi)
{
    if (x.hi() <= lo || hi <= x.lo()) return false;
    const int64_t first = lo < x.lo() + x.width || x.pitch == 0 ? 0 : static_cast<int64_t>((lo - x.lo() - x.width) / x.pitch + 1);
    return first < x.rows && x.lo() + first * x.pitch < hi;
}

// Whether a and b share a byte.  Two sets of rows with gaps of different pitches are not told
// apart: taken as sharing none.
inline bool share_bytes(const Span &a, const Span &b)
{
    if (a.blocks == 0 || b.blocks == 0 || a.hi() <= b.lo() || b.hi() <= a.lo()) return false;
    if (a.blocks > 1 && b.blocks > 1 && a.stride == b.stride) {
        for (int64_t i = 1 - a.blocks; i < b.blocks; ++i)    // (blocks as far apart meet alike)
            if (share_bytes(a.block(0), b.block(i))) return true;
        return false;
    }
    if (a.blocks > 1 || b.blocks > 1) {
        for (int64_t i = 0; i < a.blocks; ++i)
            for (int64_t j = 0; j < b.blocks; ++j)
                if (share_bytes(a.block(i), b.block(j))) return true;
        return false;
    }
    if (a.dense()) return rows_meet(b, a.lo(), a.hi());
    if (b.dense()) return rows_meet(a, b.lo(), b.hi());
    if (a.pitch != b.pitch) return false;
    // both repeat alike, and their hulls meet: their columns do, or they lie side by side
    const int64_t off = static_cast<int64_t>((b.lo() - a.lo()) % static_cast<uintptr_t>(a.pitch));
    const int64_t from = a.lo() <= b.lo() ? off : (a.pitch - static_cast<int64_t>((a.lo() - b.lo()) % a.pitch)) % a.pitch;
    return from < a.width || from + b.width > a.pitch;
}

// Refuses a call that writes `written` where one of the others is.
inline gemm_status_t check_apart(const char *name, const char *what, const Span &written, std::initializer_list<Span> others)
{
    for (const Span &o : others)
        if (share_bytes(written, o))
            return fail(GEMM_ERR_INVALID_ARG, "%s: %s overlaps what the call reads, another result or the workspace", name, what);
    return GEMM_OK;
}

// A launch that may begin its setup before the kernel before it has ended.
template <typename... Args>
gemm_status_t launch_plain(const char *name, void (*kernel)(Args...), dim3 grid, int threads, size_t smem,
                           cudaStream_t stream, Args... args)
{
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    if (e != cudaSuccess) return fail(GEMM_ERR_CUDA, "%s: launch: %s", name, cudaGetErrorString(e));
    return GEMM_OK;
}

}  // namespace tn_host

using namespace tn_host;
