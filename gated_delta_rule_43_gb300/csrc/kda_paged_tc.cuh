// kda_paged_tc.cuh -- what the tensor-core kernels of paged attention share: waits that end, tensor
// memory, tensor maps of pages, launches behind the kernel before.
#pragma once

#include <cuda.h>
#include <string.h>

#include <mutex>

#include "kda_paged.cuh"
#include "kda_sm100.cuh"

namespace kda {
namespace paged {
namespace tc {

using namespace sm100;

constexpr float kLog2e = 1.4426950408889634f;
constexpr uint64_t kDrainNs = 100000000ull;   // limit of a wait of a CTA that has given up

constexpr int BK = 128;             // keys of a block

// A place in the row of blocks: before block k of the blocks that head h of tile `tile` (the t-th of
// sequence n) sees.  k > 0: inside an item.
struct Cut {
    int32_t tile, n, t, h, k;
};
__device__ __forceinline__ bool same_item(const Cut &a, const Cut &b) { return a.tile == b.tile && a.h == b.h; }

struct Plan {
    int32_t *tiles;           // [N + 1]: tiles of the sequences before n
    int64_t *cost;            // [tiles + 1]: that of the tiles before
    Cut *cuts;                // [ranges + 1]
    float *part;              // [2 * ranges][rows][D]: what a cut leaves, behind a range's begin, before its end
    float2 *ml;               // [2 * ranges][rows]
    int ranges, rows;         // rows: of an item, at most
    int each;                 // rows of a tile
    StatusWord *found;        // [ranges]: what each range has to report (single tokens; or null)
    int64_t most;             // tiles that there is room for
};

// What everything about tile t of a sequence follows from.
struct Tile {
    Span s;
    int row0, rows;           // of the sequence's len * group
    int first, last;          // positions of the first and last row's tokens
};
__device__ __forceinline__ Tile tile_of(const Span &s, int t, int group, int each) {
    Tile r;
    r.s = s;
    r.row0 = t * each;
    r.rows = (int)min((int64_t)each, (int64_t)s.len * group - r.row0);
    r.first = s.pos + r.row0 / group;
    r.last = s.pos + (r.row0 + r.rows - 1) / group;
    return r;
}
__device__ __forceinline__ KeyBlocks blocks_of(const Tile &t, int window, int sinks) {
    return key_blocks(max(0, t.first), t.last, window, sinks, BK);
}

// Waits of a whole warp on one barrier, which end: a try that finds nothing sleeps in hardware (3.7 us,
// measured), so tries are counted: 2.2 s.
constexpr uint32_t kTries = 600000;
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, uint32_t tries = kTries) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .u32 i;\n\t"
        "mov.u32 i, 0;\n"
        "again_%=:\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "@p bra done_%=;\n\t"
        "add.u32 i, i, 1;\n\t"
        "setp.lt.u32 q, i, %3;\n\t"
        "@q bra again_%=;\n"
        "done_%=:\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(tries)
        : "memory");
    return __all_sync(0xffffffffu, ok != 0);
}

// Those of a wait that ends only with an item: 2.2 s for every 2^18 of the blocks that the longest may have (2^18 blocks
// take the slowest kernel about half a second).
__device__ __forceinline__ uint32_t item_tries(const Cache &c) {
    return kTries * (1 + (((uint32_t)c.width << c.shift) >> 25));   // (width << shift is below 2^31)
}

// The same on up to three barriers at a time, a lane each: every wait of its own costs a warp 100 to 200
// cycles, whatever it finds.  Such tries do not sleep, so time is what is counted: 2.2 s.
__device__ __forceinline__ bool wait_warp(uint32_t bar0, uint32_t parity0, uint32_t bar1, uint32_t parity1, uint32_t bar2,
                                          uint32_t parity2) {
    const int lane = threadIdx.x & 31;
    const uint32_t bar = lane == 1 ? bar1 : lane == 2 ? bar2 : bar0, parity = lane == 1 ? parity1 : lane == 2 ? parity2 : parity0;
    uint64_t begin = 0;
    uint32_t ok = 0;
    for (uint32_t i = 0;; ++i) {
        if (!ok)
            asm volatile(
                "{\n\t.reg .pred p;\n\t"
                "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                "selp.u32 %0, 1, 0, p;\n\t}"
                : "=r"(ok)
                : "r"(bar), "r"(parity)
                : "memory");
        if (__all_sync(0xffffffffu, ok != 0)) {
            __syncwarp();   // (what one lane has seen arrive, all may use: a vote orders no memory)
            return true;
        }
        if ((i & 255u) == 0) {
            const uint64_t now = globaltimer_ns();
            if (i == 0) begin = now;
            else if (__any_sync(0xffffffffu, now - begin > 2200000000ull)) return false;
        }
    }
}

// For the others of a named barrier, from a warp that leaves its role because a wait expired: whoever stands there
// or comes there next goes on, to a wait that expires as well.
__device__ __forceinline__ void named_bar_arrive(uint32_t id, uint32_t n) {
    asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(n) : "memory");
}

// 32 lanes x 4, 8, 16 or 32 consecutive columns of tensor memory; nothing may be used before
// tmem_ld_wait
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float (&v)[4]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float (&v)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float (&v)[16]) { tmem_ld16(taddr, v); }
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float (&v)[32]) { tmem_ld32(taddr, v); }
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
        ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
          "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const float (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                 ::"r"(taddr), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// x as the compiler knows it to be the same in all lanes, so that it goes into a uniform register once, and not
// with every product that is issued: of a converged warp
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }
__device__ __forceinline__ uint64_t uniform(uint64_t d) {
    return (uint64_t)uniform((uint32_t)(d >> 32)) << 32 | uniform((uint32_t)d);
}

// A in tensor memory (lane = row, column c = K elements 2 c and 2 c + 1)
__device__ __forceinline__ void umma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                             uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d_tmem), "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Rows of a run (a page's of one head) from `row` on, channels from c on: one box of page_map.  A run past
// the last reads as zeros.
__device__ __forceinline__ void tma_load_rows(uint32_t dst, const void *tmap, int32_t c, int32_t row, int32_t run,
                                              uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(dst), "l"(tmap), "r"(c), "r"(row), "r"(run), "r"(bar)
        : "memory");
}
// Zeroes rows [begin, end) of a tile of 128 rows of BYTES bytes (in columns of at most 128 bytes, one
// behind the other); a whole warp, before the tile's products.
template <int BYTES> __device__ __forceinline__ void clear_rows(uint8_t *tile, int begin, int end) {
    constexpr int W = BYTES < 128 ? BYTES : 128, U = W / 16;   // a column's width; its 16-byte pieces
    for (int x = begin * U + (threadIdx.x & 31); x < end * U; x += 32) {
#pragma unroll
        for (int i = 0; i < BYTES / W; ++i)
            *reinterpret_cast<uint4 *>(tile + i * BK * W + x * 16) = make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async();
    __syncwarp();
}

// Rows [begin, end) of the tile of keys from key0 on that are neither in a window, the highest position below
// which is `lowest`, nor among the first tokens: their weights are zeros, but 0 times a value that is not finite
// is not.  (Whole pages of them are not loaded, but read as zeros.)
struct Unseen {
    int begin, end;
};
__device__ __forceinline__ Unseen unseen(int key0, int lowest, int sinks) {
    return Unseen{max(0, sinks - key0), min(BK, lowest + 1 - key0)};
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&x);
}
// 32 bytes, a whole sector of memory, in one store (32-byte aligned)
__device__ __forceinline__ void store32(void *to, const uint32_t *x) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                 ::"l"(to), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                 : "memory");
}
// 2^x by the special-function unit (relative error near 2^-22)
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Two at a time
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z, w;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "add.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
// the largest of three
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Programmatic launches: a kernel may be on the GPU before the one that it depends on has ended.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
template <typename... P, typename... A>
inline cudaError_t launch_after(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, A... args) {
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

// Position in a ring of barriers: stage, and the parity of its fill.
struct Ring {
    uint32_t stage = 0, phase = 0;
    __device__ __forceinline__ void step(uint32_t stages) {
        if (++stage == stages) {
            stage = 0;
            phase ^= 1;
        }
    }
};

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                   const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
inline EncodeTiledFn encode_tiled() {
    static EncodeTiledFn fn = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<EncodeTiledFn>(f);
    }();
    return fn;
}

// Pages [P, Hk, page size, D] of bf16 or e4m3 as runs of rows, `page_runs` from one page's to the next's, in
// boxes of up to 128 rows of a run x 128 bytes (64 for e4m3 heads of up to 64), swizzled as the products want them.
// Heads of 32 stand in the boxes of heads of 64: what a box has beyond a row reads as zeros.
constexpr int in_tile(int D) { return D < 64 ? 64 : D; }   // a head's channels in shared and tensor memory
inline int box_rows(const Cache &c) { return c.shift >= 7 ? 128 : 1 << c.shift; }
__host__ __device__ inline int page_runs(const Cache &c, int D) { return (int)((c.stride / D) >> c.shift); }
inline cudaError_t page_map(CUtensorMap *m, const Cache &c, const void *pages, int D, bool e4m3) {
    EncodeTiledFn enc = encode_tiled();
    if (!enc) return cudaErrorNotSupported;
    const cuuint64_t row = D * (e4m3 ? 1 : 2);
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)1 << c.shift,
                                (cuuint64_t)(c.P - 1) * page_runs(c, D) + c.Hk};
    const cuuint64_t strides[2] = {row, row << c.shift};
    const cuuint32_t box[3] = {(cuuint32_t)(e4m3 ? in_tile(D) : 64), (cuuint32_t)box_rows(c), 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    const CUresult r = enc(m, e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                           const_cast<void *>(pages), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           e4m3 && D <= 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Single tokens.  An item is a sequence, a key/value head and up to `each` query heads; costs follow from the
// lengths, so each CTA finds its own range.
namespace one {

constexpr int kItemCost = 1;        // an item's queries and outputs, in tiles
constexpr int kUncut = 2;           // tiles of an item that is not cut

// The place `x` of a row of items whose costs follow from the lengths; the caller's thread holds sequences
// [n0, n1), which begin at `before`.
__device__ __forceinline__ Cut cut_at(const Cache &c, int64_t x, int n0, int n1, int64_t before, int groups, int window,
                                      int sinks) {
    Cut cut{0, n0, 0, 0, 0};
    for (int n = n0; n < n1; ++n) {
        const Span s = span_of(c, n);
        if (s.len == 0) continue;
        const int count = key_blocks(max(0, s.pos), s.pos, window, sinks, BK).count, each = kItemCost + count;
        const int64_t cost = (int64_t)groups * c.Hk * each, rest = x - before;
        before += cost;
        if (rest >= cost) continue;
        const int item = (int)(rest / each);
        cut.k = (int)(rest - (int64_t)item * each) - kItemCost;
        if (cut.k < 1 || count <= kUncut) cut.k = 0;   // to the item's begin
        cut.n = n;
        cut.t = item / c.Hk;
        cut.h = item - cut.t * c.Hk;
        cut.tile = cut.n * groups + cut.t;
        return cut;
    }
    return cut;
}

// Eight warps add up the costs of all sequences, and whoever holds the two ends of this CTA's range writes them
// down: cuts[0], cuts[1].  All threads, 256 at least; sums: of eight warps.
__device__ __forceinline__ void own_range(const Cache &c, int ranges, int groups, int window, int sinks, int64_t *sums,
                                          Cut *cuts, StatusWord *st) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int per = (c.N + 255) / 256, n0 = min(c.N, tid * per), n1 = min(c.N, n0 + per);
    int64_t mine = 0, upto = 0;
    if (tid < 256) {
        for (int n = n0; n < n1; ++n) {
            const Span s = span_of(c, n);
            if (s.len) mine += (int64_t)groups * c.Hk * (kItemCost + key_blocks(max(0, s.pos), s.pos, window, sinks, BK).count);
        }
        upto = mine;
#pragma unroll
        for (int i = 1; i < 32; i <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, upto, i);
            if (lane >= i) upto += x;
        }
        if (lane == 31) sums[warp] = upto;
    }
    __syncthreads();
    if (blockIdx.x == 0) check_spans(c, st);
    int64_t total = 0;
    for (int w = 0; w < 8; ++w) {
        if (w < warp) upto += sums[w];
        total += sums[w];
    }
    const int64_t share = max((total + ranges - 1) / ranges, (int64_t)(kItemCost + 1));
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
        const int64_t x = (int64_t)(blockIdx.x + i) * share;
        if (x >= total) {
            if (tid == 0) cuts[i] = Cut{c.N * groups, c.N, 0, 0, 0};
        } else if (tid < 256 && x >= upto - mine && x < upto) {
            cuts[i] = cut_at(c, x, n0, n1, upto - mine, groups, window, sinks);
        }
    }
    __syncthreads();
}

}  // namespace one

// Joins what the cuts inside items have left, behind the kernel that left it.
cudaError_t launch_join(bool f32, int D, const Cache &c, const Plan &p, void *o, int group, StatusWord *st, cudaStream_t s);

}  // namespace tc
}  // namespace paged
}  // namespace kda
