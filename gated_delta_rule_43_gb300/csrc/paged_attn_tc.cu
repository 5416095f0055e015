// paged_attn_tc.cu -- attention of a chunk of new tokens over paged keys and values on the sm_103a
// tensor cores (bf16 operands, fp32 accumulation).
//
//   S = Q K^T;   m_i the running maximum of a row;   P = 2^(f S - f m), f = scale log2(e)
//   O = sum over blocks of P V,   l = sum of P,   o = O / l
// The query heads that share a key/value head are rows beside each other (row = token * group + head), so
// that a block of keys is read once for all of them: an item is 256 such rows of one sequence and
// key/value head, in two tiles of 128, and goes through the blocks of 128 keys that it sees.  4 D flops a
// row and key against 4 D bytes a key: with 256 rows a block takes 2048 cycles of products and 64 KB.
//
// The running maximum only moves when it would grow by more than 2^8: until then P is up to 256 times
// larger than it could be, which neither bf16 nor the fp32 sums mind, and O is not rescaled.
// P is rounded to bf16 for its product (a product takes two operands of one type; P in two parts would cost a second product),
// l is the sum before that: 2.1e-3 of relative L2 against 64 bits, of which rounding the outputs is 1.7e-3.
//
// The work.  A plan lists the tiles of all sequences, with the blocks that each sees, heads inside tiles, in
// one row and cuts it into equal ranges, one an SM, wherever that falls: with few rows against a
// long context the SMs share the keys of one item.  What a cut leaves on both sides is kept in the
// workspace (O, m, l in fp32) and joined by a second kernel.
//
// One CTA an SM:
//   warps 0-3, 4-7   the rows of the two tiles, a thread each: scores out of tensor memory, P into it, over
//                    the scores
//   warp 8           issues the products (and zeroes values that may be anything: in slots behind a sequence's
//                    end and before the windows)
//   warp 9           loads keys and values, page by page
//   warp 10          goes through the range's items for everyone
//   warps 12-15      an item's edges: its queries, into the place of the last one's after the last scores, and
//                    its outputs, while the next item's first weights are formed (done by the rows' own warps,
//                    an item cost 10k cycles beside its blocks)
//   warps 16-19      (e4m3 pages) make the operands out of the bytes that warp 9 loads: scale * e4m3 is a
//                    bf16 exactly, so the products are those of a bf16 cache
// Products of one tile run while the other's scores become weights: P0 V, Q0 K', P1 V, Q1 K', ...
//
// What bounds it: the chain scores -> weights -> product of each tile, two of which share one tensor pipe.  With D =
// 128 a block takes 3.3k to 3.5k cycles, 2063 of them products (54 % of the tensor pipe's time; the
// special-function unit is at 27 %).  8192 tokens, 32 heads on 8 of 128, bf16: 451 to 463 us, 1.19 to 1.22 PFLOP/s; 512
// tokens behind 65000: 410 to 458 us, 1.20 to 1.33; 16 chunks with prefixes from e4m3 pages 0.94 to 0.97, the making of
// operands beside it (51 % of all issue slots).  D = 64: 0.85 (the rows' own time), with a window of 1024 0.44.  Many
// sequences of few new tokens cost as if they had 128 rows each: 256 of 4 tokens behind 512 to 8192 take 726 us from bf16
// pages (6.3 TB/s), 1148 from e4m3 (2.1).
//
// A row's thread holds 128 scores in 168 registers (144 beside e4m3 pages) and spills: 176 bytes for heads of 128, 96 of
// 64, 60 of 32; from e4m3 pages 380, 276, 252.
#include "kda_paged_tc.cuh"

namespace kda {
namespace paged {
namespace tc {

constexpr int kRows = 256;          // rows of an item
template <bool E4M3> constexpr int kThreads = E4M3 ? 640 : 512;
constexpr int kRowWarps = 8, kMmaWarp = 8, kLoadWarp = 9, kItemWarp = 10, kEdgeWarp = 12, kMakeWarp = 16;
constexpr int kItemCost = 3;        // an item's queries and outputs, in blocks
constexpr int kUncut = 6;           // blocks of an item that is not cut
// Blocks in one sum: the tensor cores cut off what does not fit beside a large one, 7e-7 of it a block (262144 tokens in
// one sum lost 1.4e-3, 4 M 2.4e-2), so a range's share of an item is gone through in links of up to 256 blocks (1.7e-4),
// which are joined in fp32.  They also bound how long anyone waits for an item.
constexpr int kSum = 256;
constexpr int kRing = 4;            // items known ahead
constexpr float kGrow = 8.f;        // log2 of what the maximum may grow before O is rescaled

constexpr int kPlanThreads = 1024;

// Inclusive sums over a block's threads; returns the total.
__device__ __forceinline__ int64_t warp_scan(int64_t x) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    return x;
}
__device__ __forceinline__ int64_t block_scan(int64_t &x, int64_t *warps) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    x = warp_scan(x);
    __syncthreads();
    if (lane == 31) warps[warp] = x;
    __syncthreads();
    const int64_t upto = warp_scan(warps[lane]);
    if (warp > 0) x += __shfl_sync(0xffffffffu, upto, warp - 1);
    return __shfl_sync(0xffffffffu, upto, 31);
}
static_assert(kPlanThreads == 1024, "a warp scans the warps");

// The last n in [0, count) with a[n] <= x
template <typename T> __device__ __forceinline__ int last_at_most(const T *a, int count, T x) {
    int lo = 0, hi = count;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (a[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

// (What is searched stands in shared memory where it fits: from global memory, the searches' chains of reads
// made the plan take 8 us.)
constexpr int kNearSeqs = 2048, kNearTiles = 4096;
__global__ void __launch_bounds__(kPlanThreads)
paged_plan_kernel(Cache c, Plan p, int group, int window, int sinks, StatusWord *st) {
    __shared__ int64_t warps[kPlanThreads / 32];
    __shared__ int64_t near_cost[kNearTiles + 1];
    __shared__ int32_t near_tiles[kNearSeqs + 1];
    let_next_start();
    const int tid = threadIdx.x;
    if (tid == 0) *st = StatusWord{0, 0, 0};
    __syncthreads();
    int32_t *first = c.N <= kNearSeqs ? near_tiles : p.tiles;
    int64_t tiles = 0, rows = 0;
    for (int n0 = 0; n0 < c.N; n0 += kPlanThreads) {
        const int n = n0 + tid;
        int64_t x = 0, len = 0;
        if (n < c.N) {
            const int ctx = c.kv_lens[n], begin = c.cu[n], end = c.cu[n + 1];
            if (lens_ok(c, n, begin, end, ctx)) len = end - begin;
            else report(st, KDA_ERR_SEQLENS, n, 61);
            x = (len * group + kRows - 1) / kRows;
        }
        const int64_t mine = x, some = block_scan(x, warps);
        if (n < c.N && tiles + x < ((int64_t)1 << 31)) first[n] = p.tiles[n] = (int)(tiles + x - mine);
        rows += block_scan(len, warps);
        tiles += some;
    }
    // sequences that overlap (of a cu_seqlens that is not ascending, which has been reported): their
    // work would have no bound
    if (rows > c.T || tiles > p.most) tiles = 0;
    if (tid == 0) p.tiles[c.N] = (int)tiles;
    __syncthreads();
    int64_t *cost = tiles <= kNearTiles ? near_cost : p.cost;
    int64_t total = 0;
    for (int64_t i0 = 0; i0 < tiles; i0 += kPlanThreads) {
        const int64_t i = i0 + tid;
        int64_t x = 0;
        if (i < tiles) {
            int n = last_at_most(first, c.N, (int)i);
            const Tile t = tile_of(span_of(c, n), (int)i - first[n], group, kRows);
            x = (int64_t)c.Hk * (kItemCost + blocks_of(t, window, sinks).count);
        }
        const int64_t mine = x, some = block_scan(x, warps);
        if (i < tiles) cost[i] = total + x - mine;
        total += some;
    }
    if (tid == 0) cost[tiles] = total;
    __syncthreads();
    // ranges of at least an item of one block
    const int64_t share = max((total + p.ranges - 1) / p.ranges, (int64_t)kItemCost + 1);
    for (int i = tid; i <= p.ranges; i += kPlanThreads) {
        const int64_t x = min((int64_t)i * share, total);
        Cut cut{(int)tiles, c.N, 0, 0, 0};
        if (x < total) {
            cut.tile = last_at_most(cost, (int)tiles, x);
            const int64_t rest = x - cost[cut.tile];
            const int each = (int)((cost[cut.tile + 1] - cost[cut.tile]) / c.Hk), count = each - kItemCost;
            cut.h = (int)(rest / each);
            cut.k = (int)(rest - (int64_t)cut.h * each) - kItemCost;
            bool next = false;   // to the item's nearer end
            if (count <= kUncut) next = 2 * cut.k > count;
            else if (cut.k > count - 2) next = true;
            if (cut.k < 2 || next || count <= kUncut) cut.k = 0;
            if (next && ++cut.h == c.Hk) {
                cut.h = 0;
                ++cut.tile;
            }
            if (cut.tile < tiles) {
                cut.n = last_at_most(first, c.N, cut.tile);
                cut.t = cut.tile - first[cut.n];
            } else {
                cut.n = c.N;
            }
        }
        p.cuts[i] = cut;
    }
}

// What the roles need of an item.
struct alignas(16) Item {
    int n;                    // -1: no more
    int h, row0, rows;
    int tok0, pos0;           // the sequence's first new token: its row of q, its position
    int k0, k1;               // of the list of blocks
    int k1a;                  // ... for the first tile, whose rows stand earlier
    int sinks, from;          // the list (KeyBlocks)
    int first, last;          // positions of the first and last token
    int ctx;
    int slot;                 // of Plan.part, or -1: the whole item
    int chain;                // bit 0: links of it came before, bit 1: more come
    // Of Plan.part, where the links before leave what they have: the item's own slot, or that of the range's last
    // item, which is still to come.
    int aside;
    __device__ __forceinline__ int block(int k) const { return k < sinks ? k : from + k - sinks; }
    __device__ __forceinline__ int end(int tile) const {
        return tile == 0 ? k1a : rows > 128 ? k1 : k0;
    }
};

template <int D, bool E4M3> struct Map {
    static constexpr uint32_t kTile = 128 * D * 2;           // of keys, values or a tile's queries
    static constexpr uint32_t kRawTile = E4M3 ? 128 * D : 0; // of keys or values as they lie in e4m3 pages
    static constexpr int kStages = D == 64 ? 8 : E4M3 ? 4 : 5, kRaws = E4M3 ? D == 64 ? 4 : 2 : 0;
    static constexpr uint32_t kQ = 0, kKV = 2 * kTile, kRaw = kKV + kStages * kTile;
    static constexpr uint32_t kItems = kRaw + kRaws * kRawTile;
    static constexpr uint32_t kTops = kItems + kRing * (uint32_t)sizeof(Item);   // [2 tiles][maximum, sum][128 rows]
    static constexpr uint32_t kBar = kTops + 2048;
    // barriers
    static constexpr int kFull = 0, kFree = kStages, kQFull = 2 * kStages, kQFree = kQFull + 2, kSReady = kQFree + 2,
                         kPReady = kSReady + 2 /* [2 parts][2 tiles] */, kODone = kPReady + 4, kOFree = kODone + 2, kEnds = kOFree + 2, kEndsFree = kEnds + 2, kItemFull = kEndsFree + 2,
                         kItemFree = kItemFull + kRing, kDrain = kItemFree + kRing, kRawFull = kDrain + 1, kRawFree = kRawFull + kRaws,
                         kBars = kRawFree + kRaws;
    static constexpr uint32_t kSlot = kBar + kBars * 8, kBytes = kSlot + 16;
    static_assert(sizeof(Item) % 8 == 0 && kBytes <= 232448 && kItems % 1024 == 0, "layout");
};

// Bits 0 .. x of a word (none below 0)
__device__ __forceinline__ uint32_t bits_upto(int x) { return x < 0 ? 0u : 0xffffffffu >> (31 - min(x, 31)); }

template <int DIM, bool E4M3>
__global__ void __launch_bounds__(kThreads<E4M3>, 1)
paged_attn_kernel(Cache c, Plan p, const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                  const __nv_bfloat16 *__restrict__ q, int64_t q_stride, __nv_bfloat16 *__restrict__ o, int group,
                  float scale, int window, int sinks, int left_out, StatusWord *st) {
    extern __shared__ __align__(1024) uint8_t sm[];
    constexpr int D = in_tile(DIM);   // (channels beyond DIM are products' columns that nobody reads)
    using M = Map<D, E4M3>;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    let_next_start();
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + M::kBar);
    Item *items = reinterpret_cast<Item *>(sm + M::kItems);
    uint32_t *tslot = reinterpret_cast<uint32_t *>(sm + M::kSlot);
    const uint32_t base = smem_u32(sm), bars = base + M::kBar;
    if (base & 1023u) {   // the operand images need their alignment
        wait_for_previous();
        if (tid == 0) report(st, KDA_ERR_CUDA, 0, 70);
        return;
    }
    if (tid == 0) {
        for (int i = 0; i < M::kStages; ++i) {
            mbar_init(&bar[M::kFull + i], E4M3 ? 4 : 1);
            mbar_init(&bar[M::kFree + i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar[M::kQFull + i], 4);
            mbar_init(&bar[M::kQFree + i], 1);
            mbar_init(&bar[M::kOFree + i], 4);
            mbar_init(&bar[M::kEnds + i], 4);
            mbar_init(&bar[M::kEndsFree + i], 4);
            mbar_init(&bar[M::kSReady + i], 1);
            mbar_init(&bar[M::kPReady + i], 4);
            mbar_init(&bar[M::kPReady + 2 + i], 4);
            mbar_init(&bar[M::kODone + i], 1);
        }
        for (int i = 0; i < kRing; ++i) {
            mbar_init(&bar[M::kItemFull + i], 1);
            mbar_init(&bar[M::kItemFree + i], kRowWarps + (E4M3 ? 10 : 6));
        }
        for (int i = 0; i < M::kRaws; ++i) {
            mbar_init(&bar[M::kRawFull + i], 1);
            mbar_init(&bar[M::kRawFree + i], 4);
        }
        mbar_init(&bar[M::kDrain], 1);
        fence_mbar_init();
    }
    constexpr uint32_t kCols = 512;
    if (warp == kMmaWarp) {
        tmem_alloc(tslot, kCols);
        tmem_relinquish();
        tc_fence_before();
    }
    if (warp == kLoadWarp && lane == 0) {
        tma_prefetch_map(&tk);
        tma_prefetch_map(&tv);
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;
    wait_for_previous();
    bool ok = true;
    auto wait = [&](int which, uint32_t parity) {
        ok = ok && wait_warp(bars + 8 * which, parity);
        return ok;
    };
    // Each role goes through the items for itself; role(item) returns with ok false when a wait expired.
    auto each_item = [&](auto role) {
        Ring at;
        while (wait(M::kItemFull + at.stage, at.phase)) {
            const Item &it = items[at.stage];   // (read where it is used: registers are few)
            if (it.n < 0) break;
            role(it);
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[M::kItemFree + at.stage]);
            at.step(kRing);
            if (!ok) break;
        }
    };
    Ring kv;            // fills of the ring of keys and values (keys, values, keys, ...)
    uint32_t loads = 0; // (load warp) fills issued

    // Registers for the rows' threads from the others: launched with 512 x 128 = 65536, then 256 x 168 +
    // 256 x 88, the same; for e4m3 pages 640 x 96 = 61440, then 256 x 144 + 384 x 64, the same.
    if (warp < kRowWarps) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(E4M3 ? 144 : 168));
        const int tile = warp >> 2, quarter = warp & 3;
        const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
        const uint32_t tS = tmem + 128 * tile + lanes, tO = tmem + 256 + D * tile + lanes;
        const float f = scale * kLog2e;
        // P goes to its product in two parts, so that the first runs while the second is formed
        auto part_done = [&](int part) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[M::kPReady + 2 * part + tile]);
            __syncwarp();
        };
        uint32_t s_phase = 0;
        uint32_t ends = 0;   // parity of items with anything for this tile
        each_item([&](const Item &it) {
            const int r = 128 * tile + 32 * quarter + lane;
            const bool live = r - lane < it.rows, mine = r < it.rows;   // (of a whole warp; this row)
            const int pos = it.pos0 + (it.row0 + min(r, it.rows - 1)) / group;
            const int pos_lo = __shfl_sync(0xffffffffu, pos, 0), pos_hi = __shfl_sync(0xffffffffu, pos, 31);
            const int lowest = window > 0 ? max(max(pos, 0) - window, -1) : -1;   // keys above it are in the window
            const int end = it.end(tile), begin = it.k0;
            float m = -INFINITY, l = 0.f;   // m: of the scores as they come
            for (int k = begin; k < end; ++k) {
                if (!wait(M::kSReady + tile, s_phase)) return;
                s_phase ^= 1;
                tc_fence_after();
                if (live) {
                    const int key0 = it.block(k) * BK;
                    float s[4][32];
#pragma unroll
                    for (int b = 0; b < 4; ++b) tmem_ld32(tS + 32 * b, s[b]);
                    tmem_ld_wait();
                    // keys that one of the warp's rows does not see: -inf where it is this one
                    if (key0 + BK - 1 > pos_lo || (window > 0 && key0 <= max(pos_hi, 0) - window && key0 + BK - 1 >= sinks)) {
                        // (bits of a word at a time: compared key by key, a masked block took 2000 cycles more than others, and
                        // its code cost those 200)
                        const int upto = pos - key0, above = lowest - key0, first = sinks - key0;
#pragma unroll
                        for (int b = 0; b < 4; ++b) {
                            const uint32_t see = bits_upto(upto - 32 * b) & (~bits_upto(above - 32 * b) | bits_upto(first - 1 - 32 * b));
#pragma unroll
                            for (int j = 0; j < 32; ++j) s[b][j] = see & (1u << j) ? s[b][j] : -INFINITY;
                        }
                    }
                    float t[4];
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        t[b] = s[b][0];
#pragma unroll
                        for (int j = 0; j < 32; j += 2) t[b] = max3(t[b], s[b][j], s[b][j + 1]);
                    }
                    const float top = max3(fmaxf(t[0], t[1]), t[2], t[3]);
                    if (k == begin) {
                        m = top;
                    } else if (__any_sync(0xffffffffu, mine && top > m && !((top - m) * f <= kGrow))) {
                        const float grown = fmaxf(m, top);
                        const float keep = m == grown ? 1.f : ex2((m - grown) * f);
                        m = grown;
                        l *= keep;
#pragma unroll 1
                        for (int j = 0; j < DIM; j += 8) {
                            float x[8];
                            tmem_ld(tO + j, x);
                            tmem_ld_wait();
#pragma unroll
                            for (int i = 0; i < 8; ++i) x[i] *= keep;
                            tmem_st8(tO + j, x);
                        }
                    }
                    const float ref = m == -INFINITY ? 0.f : -m * f;
                    const float2 f2 = make_float2(f, f), ref2 = make_float2(ref, ref);
                    float2 sum = make_float2(0.f, 0.f), sum1 = sum;
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        uint32_t w[16];
#pragma unroll
                        for (int j = 0; j < 32; j += 2) {
                            float2 x = fma2(make_float2(s[b][j], s[b][j + 1]), f2, ref2);
                            x.x = ex2(x.x);
                            x.y = ex2(x.y);
                            if (j & 2) sum1 = add2(sum1, x);
                            else sum = add2(sum, x);
                            w[j / 2] = pack2(x.x, x.y);
                        }
                        tmem_st16(tS + 16 * b, w);
                        if (b == 1) {
                            tmem_st_wait();
                            part_done(0);
                        }
                    }
                    sum = add2(sum, sum1);
                    l += sum.x + sum.y;
                    tmem_st_wait();
                } else {
                    part_done(0);
                }
                part_done(1);
            }
            if (end == begin) return;
            // the row's maximum and sum, for those who store its outputs (and have taken the last item's)
            if (!wait(M::kEndsFree + tile, ends ^ 1)) return;
            ends ^= 1;
            float *tops = reinterpret_cast<float *>(sm + M::kTops) + 256 * tile + 32 * quarter + lane;
            tops[0] = m == -INFINITY ? 0.f : m * f;
            tops[128] = l;
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[M::kEnds + tile]);
            __syncwarp();
        });
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(E4M3 ? 64 : 88));
        if (warp == kMmaWarp) {
            uint32_t q_phase[2] = {0, 0}, p_phase[2] = {0, 0}, o_phase[2] = {0, 0};
            constexpr uint32_t id_s = idesc_bf16(128, BK, false, false), id_o = idesc_bf16(128, D, false, true);
            const uint64_t dq0 = uniform(sdesc_sw128(base + M::kQ, 16, 1024)), dk0 = sdesc_sw128(base + M::kKV, 16, 1024),
                           dv0 = sdesc_sw128(base + M::kKV, BK * 128, 1024);
            const uint32_t t0 = uniform(tmem);
            auto scores = [&](int tile, uint64_t dk) {   // S = Q K^T
#pragma unroll
                for (int s = 0; s < DIM / 16; ++s)
                    umma_bf16(t0 + 128 * tile, desc_add(dq0, tile * M::kTile + (s >> 2) * 16384 + (s & 3) * 32),
                              desc_add(dk, (s >> 2) * 16384 + (s & 3) * 32), id_s, s > 0);
            };
            auto keys_at = [&](uint32_t stage) { return uniform(desc_add(dk0, stage * M::kTile)); };
            each_item([&](const Item &it) {
                const int n0 = it.end(0) - it.k0, n1 = it.end(1) - it.k0, blocks = it.k1 - it.k0, ctx = it.ctx;
                if (blocks == 0) return;
                const int lowest = window > 0 ? max(max(0, it.first) - window, -1) : -1;   // keys above it are in someone's window
                Ring key = kv;
                if (!wait(M::kFull + key.stage, key.phase)) return;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if ((i ? n1 : n0) == 0) continue;
                    if (!wait(M::kQFull + i, q_phase[i])) return;
                    q_phase[i] ^= 1;
                    tc_fence_after();
                    const uint64_t dk = keys_at(key.stage);
                    if (elect_one()) {
                        scores(i, dk);
                        umma_commit(&bar[M::kSReady + i]);
                        if ((i ? n1 : n0) == 1) umma_commit(&bar[M::kQFree + i]);
                    }
                    __syncwarp();
                }
                if (elect_one()) umma_commit(&bar[M::kFree + key.stage]);
                __syncwarp();
                for (int j = 0; j < blocks; ++j) {
                    Ring val = key;
                    val.step(M::kStages);
                    key = val;
                    key.step(M::kStages);
                    const bool more = j + 1 < blocks;
                    const uint32_t val_bar = bars + 8 * (M::kFull + val.stage), key_bar = bars + 8 * (M::kFull + key.stage);
                    // (bf16) values that may be anything: behind the sequence's end, which is in the list's last block,
                    // and before the windows
                    const int key0 = it.block(it.k0 + j) * BK;
                    const bool tail = ctx - key0 < BK && (ctx & ((1 << c.shift) - 1)) != 0;
                    const Unseen gap = unseen(key0, lowest, sinks);
                    bool there = false;   // the block's values, the next block's keys
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int n = i ? n1 : n0;
                        if (j >= n) continue;
                        const uint32_t p_bar = bars + 8 * (M::kPReady + i);
                        ok = there ? wait_warp(p_bar, p_phase[i])
                                   : wait_warp(p_bar, p_phase[i], val_bar, val.phase, more ? key_bar : val_bar,
                                               more ? key.phase : val.phase);
                        if (!ok) return;
                        p_phase[i] ^= 1;
                        if (!E4M3 && !there) {
                            if (tail) clear_rows<2 * D>(sm + M::kKV + val.stage * M::kTile, ctx - key0, BK);
                            if (gap.begin < gap.end) clear_rows<2 * D>(sm + M::kKV + val.stage * M::kTile, gap.begin, gap.end);
                        }
                        there = true;
                        tc_fence_after();
                        const uint64_t dv = uniform(desc_add(dv0, val.stage * M::kTile)), dk = keys_at(key.stage);
                        const uint32_t onto = uniform((uint32_t)(j > 0));
                        if (j == 0) {   // the last item's outputs have been read
                            if (!wait(M::kOFree + i, o_phase[i] ^ 1)) return;
                            o_phase[i] ^= 1;
                            tc_fence_after();
                        }
                        if (elect_one()) {
#pragma unroll
                            for (int s = 0; s < BK / 16; ++s)
                                if (s < BK / 32)
                                    umma_bf16_ts(t0 + 256 + D * i, t0 + 128 * i + 8 * s, desc_add(dv, s * 2048), id_o,
                                                 s > 0 ? 1u : onto);
                        }
                        __syncwarp();
                        if (!wait(M::kPReady + 2 + i, p_phase[i] ^ 1)) return;
                        tc_fence_after();
                        if (elect_one()) {
#pragma unroll
                            for (int s = 0; s < BK / 16; ++s)
                                if (s >= BK / 32)
                                    umma_bf16_ts(t0 + 256 + D * i, t0 + 128 * i + 8 * s, desc_add(dv, s * 2048), id_o, 1u);
                            if (j + 1 == n) {
                                umma_commit(&bar[M::kODone + i]);
                            } else {
                                scores(i, dk);
                                umma_commit(&bar[M::kSReady + i]);
                                if (j + 2 == n) umma_commit(&bar[M::kQFree + i]);
                            }
                        }
                        __syncwarp();
                    }
                    if (elect_one()) {
                        umma_commit(&bar[M::kFree + val.stage]);
                        if (j + 1 < blocks) umma_commit(&bar[M::kFree + key.stage]);
                    }
                    __syncwarp();
                }
                kv = key;
            });
        } else if (warp == kLoadWarp) {
            const int rows = min(BK, 1 << c.shift), boxes = BK / rows, runs = page_runs(c, DIM);
            const int none = (c.P - 1) * runs + c.Hk;   // past the last run: zeros
            each_item([&](const Item &it) {
                // the page that holds the rows of this lane's box in block k; -1: a row that nobody sees
                auto page_of = [&](int k) {
                    if (k >= it.k1 || lane >= boxes) return -1;
                    const int key = it.block(k) * BK + lane * rows;
                    const bool seen = key <= it.last && (window <= 0 || key < sinks ||
                                                         key + rows > max(0, it.first) - window + 1);
                    return seen ? c.table[(int64_t)it.n * c.width + (key >> c.shift)] : c.P;
                };
                int next = page_of(it.k0);
                for (int k = it.k0; k < it.k1; ++k) {
                    int page = next;
                    next = page_of(k + 1);
                    const int key = it.block(k) * BK + lane * rows;
                    if (lane < boxes && (page < 0 || page > c.P || (page == c.P && key <= it.last &&
                        (window <= 0 || key < sinks || key + rows > max(0, it.first) - window + 1)))) {
                        report(st, KDA_ERR_INVALID_ARG, it.n, 71);
                        page = c.P;
                    }
#pragma unroll 1
                    for (int v = 0; v < 2; ++v) {
                        // (e4m3 pages go through a ring of their own)
                        const uint32_t full = E4M3 ? M::kRawFull : M::kFull, free = E4M3 ? M::kRawFree : M::kFree;
                        if (!wait(free + kv.stage, kv.phase ^ 1)) return;
                        const bool left = loads == 0 && left_out == (int)blockIdx.x;
                        if (lane == 0 && !left) mbar_arrive_expect_tx(&bar[full + kv.stage], E4M3 ? M::kRawTile : M::kTile);
                        __syncwarp();
                        if (lane < boxes && !left) {
                            const int row = key & ((1 << c.shift) - 1), run = page == c.P ? none : page * runs + it.h;
                            const uint32_t to = base + (E4M3 ? M::kRaw + kv.stage * M::kRawTile : M::kKV + kv.stage * M::kTile) +
                                                lane * rows * (E4M3 ? D : 128);
#pragma unroll
                            for (int x = 0; x < (E4M3 ? 1 : D / 64); ++x)
                                tma_load_rows(to + x * 16384, v ? &tv : &tk, 64 * x, row, run, bars + 8 * (full + kv.stage));
                        }
                        __syncwarp();
                        kv.step(E4M3 ? M::kRaws : M::kStages);
                        ++loads;
                    }
                }
            });
        } else if (warp == kItemWarp) {
            Ring at;
            Cut from = p.cuts[blockIdx.x];
            const Cut to = p.cuts[blockIdx.x + 1];
            const int tiles = p.tiles[c.N];
            Span s{0, 0, 0};
            int known = -1, begin = from.k;   // the first link's first block
            while (true) {
                const bool more = from.tile < tiles && (from.tile < to.tile || (from.tile == to.tile &&
                                                        (from.h < to.h || (from.h == to.h && from.k < to.k))));
                Item it;
                it.n = -1;
                it.chain = 0;
                if (more) {
                    if (known != from.n) {
                        s = span_of(c, from.n);
                        known = from.n;
                    }
                    const Tile t = tile_of(s, from.t, group, kRows);
                    const KeyBlocks kb = blocks_of(t, window, sinks);
                    it.n = from.n;
                    it.h = from.h;
                    it.row0 = t.row0;
                    it.rows = t.rows;
                    it.tok0 = s.begin;
                    it.pos0 = s.pos;
                    it.k0 = from.k;
                    const int k1 = same_item(from, to) ? min(to.k, kb.count) : kb.count;   // of the last link
                    it.k1 = min(k1, it.k0 + kSum);
                    it.chain = (it.k0 > begin ? 1 : 0) + (it.k1 < k1 ? 2 : 0);
                    const int last = t.s.pos + (t.row0 + min(t.rows, 128) - 1) / group;
                    it.k1a = last < 0 ? it.k0 : max(it.k0, min(it.k1, kb.sinks + last / BK + 1 - kb.from));
                    it.sinks = kb.sinks;
                    it.from = kb.from;
                    it.first = t.first;
                    it.last = t.last;
                    it.ctx = s.pos + s.len;
                    it.slot = begin > 0 ? 2 * (int)blockIdx.x : k1 < kb.count ? 2 * (int)blockIdx.x + 1 : -1;
                    it.aside = 2 * (int)blockIdx.x + (begin > 0 ? 0 : 1);
                }
                if (!wait(M::kItemFree + at.stage, at.phase ^ 1)) break;
                if (lane == 0) {
                    items[at.stage] = it;
                    mbar_arrive(&bar[M::kItemFull + at.stage]);
                }
                __syncwarp();
                if (!more) break;
                at.step(kRing);
                if (it.chain & 2) {
                    from.k = it.k1;
                    continue;
                }
                from.k = begin = 0;
                if (++from.h == c.Hk) {
                    from.h = 0;
                    ++from.tile;
                    ++from.t;
                    if (from.tile < tiles) {
                        // the next sequence with tiles, 32 a step
                        while (p.tiles[from.n + 1] <= from.tile) {
                            const int n = from.n + 1 + lane;
                            const uint32_t past = __ballot_sync(0xffffffffu, n < c.N && p.tiles[n + 1] <= from.tile);
                            from.n += 1 + __popc(past);
                            from.n = min(from.n, c.N - 1);
                            from.t = 0;
                        }
                    }
                }
            }
        } else if (warp >= kEdgeWarp && warp < kMakeWarp) {
            const int quarter = warp - kEdgeWarp;
            const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
            const float *tops = reinterpret_cast<const float *>(sm + M::kTops) + 32 * quarter + lane;
            uint32_t q_phase = 3, o_phase = 0;   // a bit a tile
            // The queries of this warp's rows: a row's address by its lane, its 16-byte pieces side by side;
            // both tiles' on their way before the first is waited for
            auto load_queries = [&](const Ring &at) {
                if (!wait(M::kItemFull + at.stage, at.phase)) return;
                const Item &it = items[at.stage];
                if (it.n < 0) return;
#pragma unroll 1
                for (int tile = 0; tile < 2; ++tile) {
                    if (it.end(tile) == it.k0) continue;
                    if (!wait(M::kQFree + tile, (q_phase >> tile) & 1)) return;
                    q_phase ^= 1u << tile;
                    const int row = 128 * tile + 32 * quarter;
                    if (row < it.rows) {
                        const int mine = it.row0 + min(row + lane, it.rows - 1), token = mine / group;
                        const int64_t from = (int64_t)(it.tok0 + token) * q_stride + (int64_t)(it.h * group + mine - token * group) * DIM;
                        constexpr int U = DIM / 8;   // pieces of a row
#pragma unroll 4
                        for (int i = 0; i < U; ++i) {
                            const int r = (32 * i + lane) / U, x = lane % U;
                            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                                             base + M::kQ + tile * M::kTile + sw128_offset(32 * quarter + r, 8 * x, 128)),
                                         "l"(q + __shfl_sync(0xffffffffu, from, r) + 8 * x)
                                         : "memory");
                        }
                    }
                    asm volatile("cp.async.commit_group;" ::: "memory");
                }
                const bool two = it.end(1) > it.k0;
#pragma unroll 1
                for (int tile = 0; tile < 2; ++tile) {
                    if (it.end(tile) == it.k0) continue;
                    if (tile == 0 && two) asm volatile("cp.async.wait_group 1;" ::: "memory");
                    else asm volatile("cp.async.wait_group 0;" ::: "memory");
                    fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar[M::kQFull + tile]);
                    __syncwarp();
                }
            };
            Ring at_next;
            load_queries(at_next);
            each_item([&](const Item &it) {
                at_next.step(kRing);
                load_queries(at_next);
                float m[2], l[2];
#pragma unroll
                for (int tile = 0; tile < 2; ++tile) {
                    m[tile] = l[tile] = 0.f;
                    if (it.end(tile) == it.k0) continue;
                    if (!wait(M::kEnds + tile, (o_phase >> tile) & 1)) return;
                    m[tile] = tops[256 * tile];
                    l[tile] = tops[256 * tile + 128];
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar[M::kEndsFree + tile]);
                    __syncwarp();
                }
#pragma unroll 1
                for (int tile = 0; tile < 2; ++tile) {
                    const bool any = it.end(tile) > it.k0;
                    if (any) {
                        if (!wait(M::kODone + tile, (o_phase >> tile) & 1)) return;
                        o_phase ^= 1u << tile;
                        tc_fence_after();
                    }
                    const int r = 128 * tile + 32 * quarter + lane;
                    const bool live = r - lane < it.rows, mine = r < it.rows;   // (of a whole warp; this row)
                    const float sum = tile ? l[1] : l[0];
                    const uint32_t tO = tmem + 256 + D * tile + lanes;
                    if (live) {
                        // with what the links before have left, in units of the larger maximum; to `aside` if more is to
                        // come or to be joined
                        const int64_t at = (int64_t)it.aside * p.rows + r;
                        const bool stored = it.slot >= 0 || (it.chain & 2);
                        float2 was = make_float2(0.f, 0.f);
                        if (mine && (it.chain & 1)) was = p.ml[at];
                        const float own = tile ? m[1] : m[0], top = was.y == 0.f ? own : sum == 0.f ? was.x : fmaxf(was.x, own);
                        const float a = sum != 0.f ? ex2(own - top) : 0.f, by = was.y != 0.f ? ex2(was.x - top) : 0.f;
                        const float total = a * sum + by * was.y, inv = total != 0.f ? 1.f / total : 0.f;   // (no visible key: zeros)
                        if (mine && stored) p.ml[at] = make_float2(top, total);
                        const int token = (it.row0 + min(r, it.rows - 1)) / group, head = it.h * group + (it.row0 + r) - token * group;
                        __nv_bfloat16 *to = o + ((int64_t)(it.tok0 + token) * c.Hk * group + head) * DIM;
                        const bool wide = ((uintptr_t)to & 31) == 0;
#pragma unroll 1
                        for (int j = 0; j < DIM; j += 16) {
                            float x[16];
                            if (any) {
                                tmem_ld(tO + j, x);
                                tmem_ld_wait();
                            }
                            if (by != 0.f) {
#pragma unroll
                                for (int i = 0; i < 16; i += 4) {
                                    const float4 y = *reinterpret_cast<const float4 *>(p.part + at * DIM + j + i);
                                    x[i] = (a != 0.f ? a * x[i] : 0.f) + by * y.x;
                                    x[i + 1] = (a != 0.f ? a * x[i + 1] : 0.f) + by * y.y;
                                    x[i + 2] = (a != 0.f ? a * x[i + 2] : 0.f) + by * y.z;
                                    x[i + 3] = (a != 0.f ? a * x[i + 3] : 0.f) + by * y.w;
                                }
                            }
                            uint32_t v[16];
                            if (stored) {
#pragma unroll
                                for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(x[i]);
                                if (mine) {
                                    store32(p.part + at * DIM + j, v);
                                    store32(p.part + at * DIM + j + 8, v + 8);
                                }
                            } else {
#pragma unroll
                                for (int i = 0; i < 16; i += 2) v[i / 2] = inv != 0.f ? pack2(x[i] * inv, x[i + 1] * inv) : 0u;
                                if (mine && wide) {
                                    store32(to + j, v);
                                } else if (mine) {
                                    *reinterpret_cast<uint4 *>(to + j) = make_uint4(v[0], v[1], v[2], v[3]);
                                    *reinterpret_cast<uint4 *>(to + j + 8) = make_uint4(v[4], v[5], v[6], v[7]);
                                }
                            }
                            __syncwarp();
                        }
                    }
                    if (any) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&bar[M::kOFree + tile]);
                        __syncwarp();
                    }
                }
            });
        } else if (E4M3 && warp >= kMakeWarp) {
            // this thread's row of a block: its page, then (a block later) its scales, ahead of their use
            const int row = tid - 32 * kMakeWarp;
            Ring raw;
            each_item([&](const Item &it) {
                const int lowest = window > 0 ? max(0, it.first) - window : -1;   // keys above it are in someone's window
                auto slot_of = [&](int k, int &page) {   // of the block's row, with a page to look up
                    const int key = it.block(k) * BK + row;
                    page = -1;
                    if (k < it.k1 && key <= it.last && (key > lowest || key < sinks))
                        page = c.table[(int64_t)it.n * c.width + (key >> c.shift)];
                };
                auto scales_of = [&](int k, int page, float &ks, float &vs) {
                    ks = vs = 0.f;   // (what nobody sees, and a page outside the pool, count as zeros)
                    if (page >= 0 && page < c.P) {
                        const int key = it.block(k) * BK + row;
                        const int64_t at = page * c.scale_stride + ((int64_t)it.h << c.shift) + (key & ((1 << c.shift) - 1));
                        ks = c.ks[at];
                        vs = c.vs[at];
                    }
                };
                int page, next_page;
                float ks, vs;
                slot_of(it.k0, page);
                slot_of(it.k0 + 1, next_page);
                scales_of(it.k0, page, ks, vs);
                for (int k = it.k0; k < it.k1; ++k) {
                    const bool seen = page >= 0 && page < c.P;
                    const float now[2] = {ks, vs};
                    page = next_page;
                    slot_of(k + 2, next_page);
                    scales_of(k + 1, page, ks, vs);
#pragma unroll
                    for (int v = 0; v < 2; ++v) {
                        if (!wait(M::kRawFull + raw.stage, raw.phase)) return;
                        if (!wait(M::kFree + kv.stage, kv.phase ^ 1)) return;
                        const uint8_t *from = sm + M::kRaw + raw.stage * M::kRawTile + row * D;
                        uint8_t *to = sm + M::kKV + kv.stage * M::kTile;
                        const float s = now[v];
#pragma unroll 4
                        for (int x = 0; x < DIM / 16; ++x) {
                            // 16 bytes (their places swizzled by the load) become 16 bf16
                            const int place = D == 128 ? x ^ (row & 7) : x ^ ((row >> 1) & 3);
                            const uint4 in = *reinterpret_cast<const uint4 *>(from + 16 * place);
                            const uint32_t word[4] = {seen ? in.x : 0u, seen ? in.y : 0u, seen ? in.z : 0u, seen ? in.w : 0u};
                            uint32_t out[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
                                    (__nv_fp8x2_storage_t)(word[i / 2] >> (16 * (i & 1))), __NV_E4M3);
                                const float2 y = __half22float2(__half2(h));
                                out[i] = pack2(y.x * s, y.y * s);
                            }
                            *reinterpret_cast<uint4 *>(to + sw128_offset(row, 16 * x, BK)) =
                                make_uint4(out[0], out[1], out[2], out[3]);
                            *reinterpret_cast<uint4 *>(to + sw128_offset(row, 16 * x + 8, BK)) =
                                make_uint4(out[4], out[5], out[6], out[7]);
                        }
                        fence_proxy_async();
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(&bar[M::kFull + kv.stage]);
                            mbar_arrive(&bar[M::kRawFree + raw.stage]);
                        }
                        __syncwarp();
                        raw.step(M::kRaws);
                        kv.step(M::kStages);
                    }
                }
            });
        }
    }
    if (!ok && lane == 0) report(st, KDA_ERR_TIMEOUT, blockIdx.x, 72 + warp);
    if (__syncthreads_or(!ok)) {
        // an expired wait: what is in flight ends (each wait bounded again) before the tensor memory is
        // released and the CTA leaves
        asm volatile("cp.async.wait_all;" ::: "memory");
        tmem_st_wait();
        tc_fence_before();
        if (warp == kMmaWarp) {
            tc_fence_after();
            if (elect_one()) umma_commit(&bar[M::kDrain]);
            __syncwarp();
            mbar_wait(&bar[M::kDrain], 0, kDrainNs);
        }
        if (warp == kLoadWarp) {   // (only each stage's last load can be in flight)
            constexpr uint32_t stages = E4M3 ? M::kRaws : M::kStages, full = E4M3 ? M::kRawFull : M::kFull;
            for (uint32_t x = loads >= stages ? loads - stages : 0; x < loads; ++x)
                mbar_wait(&bar[full + x % stages], (x / stages) & 1, kDrainNs);
        }
        __syncthreads();
    }
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, kCols);
    }
}

// What the cuts inside one item have left, put together: a CTA for 32 rows of the item that the cut is
// the first inside of.
constexpr int kJoinThreads = 512;
template <typename TO, int D>
__global__ void __launch_bounds__(kJoinThreads)
paged_join_kernel(Cache c, Plan p, TO *__restrict__ o, int group, StatusWord *st) {
    constexpr int V = D / 32;
    const int cut = blockIdx.x + 1, lane = threadIdx.x & 31;
    wait_for_previous();
    if (p.found && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < 32) {   // the first of what was found
        StatusWord first{0, 0, 0};
        for (int i0 = 0; i0 < p.ranges && first.code == 0; i0 += 32) {
            StatusWord x{0, 0, 0};
            if (i0 + lane < p.ranges) x = p.found[i0 + lane];
            const uint32_t some = __ballot_sync(0xffffffffu, x.code != 0);
            if (some == 0) continue;
            const int l = __ffs(some) - 1;
            first.code = __shfl_sync(0xffffffffu, x.code, l);
            first.site = __shfl_sync(0xffffffffu, x.site, l);
            first.info = __shfl_sync(0xffffffffu, x.info, l);
        }
        if (lane == 0) *st = first;
    }
    if (cut >= p.ranges) return;
    const Cut here = p.cuts[cut];
    if (here.k == 0) return;
    const Cut before = p.cuts[cut - 1];
    if (same_item(here, before) && before.k > 0) return;
    const Tile t = tile_of(span_of(c, here.n), here.t, group, p.each);
    int last = cut;   // the last cut inside the item
    while (last < p.ranges && p.cuts[last + 1].k > 0 && same_item(p.cuts[last + 1], here)) ++last;
    // A row a warp, a piece a lane: what the pieces count for at once, then their sums, four on their way.
    // (One after the other, 19 pieces took 30 us.)
    const int pieces = last - cut + 2;
    for (int r = blockIdx.y * 32 + (threadIdx.x >> 5); r < min(t.rows, (int)blockIdx.y * 32 + 32); r += kJoinThreads / 32) {
        auto place = [&](int i) { return (int64_t)(i == 0 ? 2 * cut - 1 : 2 * (cut - 1 + i)) * p.rows + r; };
        float top = -INFINITY;
        for (int i0 = 0; i0 < pieces; i0 += 32) {
            float2 b = make_float2(0.f, 0.f);
            if (i0 + lane < pieces) b = p.ml[place(i0 + lane)];
            float x = b.y != 0.f ? b.x : -INFINITY;
#pragma unroll
            for (int i = 16; i > 0; i >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, i));
            top = fmaxf(top, x);
        }
        float l = 0.f, x[V];
#pragma unroll
        for (int j = 0; j < V; ++j) x[j] = 0.f;
        for (int i0 = 0; i0 < pieces; i0 += 32) {
            float2 b = make_float2(0.f, 0.f);
            if (i0 + lane < pieces) b = p.ml[place(i0 + lane)];
            const float mine = b.y != 0.f ? ex2(b.x - top) : 0.f;   // (0: its sums may be anything)
            l += warp_sum(mine * b.y);
#pragma unroll 4
            for (int i = 0; i < min(32, pieces - i0); ++i) {
                const float e = __shfl_sync(0xffffffffu, mine, i);
                const float *from = p.part + place(i0 + i) * D + lane * V;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float y = from[j];
                    x[j] += e != 0.f ? e * y : 0.f;
                }
            }
        }
        const float inv = l != 0.f ? 1.f / l : 0.f;
        const int at = t.row0 + r, token = at / group;
        TO *to = o + ((int64_t)(t.s.begin + token) * c.Hk * group + here.h * group + at - token * group) * D + lane * V;
        if constexpr (sizeof(TO) == 2 && V > 1) {
#pragma unroll
            for (int j = 0; j < V; j += 2) *reinterpret_cast<uint32_t *>(to + j) = pack2(x[j] * inv, x[j + 1] * inv);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) to[j] = from_f<TO>(x[j] * inv);
        }
    }
}

template <typename TO>
static cudaError_t join(int D, const Cache &c, const Plan &p, void *o, int group, StatusWord *st, cudaStream_t s) {
    const dim3 grid(p.ranges > 1 ? p.ranges - 1 : 1, (p.rows + 31) / 32);
    return launch_after(D == 128 ? paged_join_kernel<TO, 128> : D == 64 ? paged_join_kernel<TO, 64> : paged_join_kernel<TO, 32>,
                        grid, dim3(kJoinThreads), 0, s, c, p, (TO *)o, group, st);
}
cudaError_t launch_join(bool f32, int D, const Cache &c, const Plan &p, void *o, int group, StatusWord *st, cudaStream_t s) {
    return f32 ? join<float>(D, c, p, o, group, st, s) : join<__nv_bfloat16>(D, c, p, o, group, st, s);
}

struct Layout {
    int64_t most;
    int ranges, rows;
    size_t tiles, cost, cuts, ml, part, total;
};
static Layout layout_of(const Cache &c, int group, int D, int sms) {
    Layout L;
    const int64_t rows = (int64_t)c.T * group;
    L.most = rows / kRows + c.N;
    L.rows = (int)(rows < kRows ? rows : kRows);
    L.ranges = sms;
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    L.tiles = kHeaderBytes;
    L.cost = L.tiles + up(sizeof(int32_t) * ((size_t)c.N + 1));
    L.cuts = L.cost + up(sizeof(int64_t) * ((size_t)L.most + 1));
    L.ml = L.cuts + up(sizeof(Cut) * ((size_t)L.ranges + 1));
    L.part = L.ml + up(sizeof(float2) * 2 * L.ranges * L.rows);
    L.total = L.part + sizeof(float) * 2 * L.ranges * L.rows * D;
    return L;
}

// Shared memory above 48 KB, once per kernel and device.
template <int D, bool E4M3> static cudaError_t allow_smem() {
    static std::mutex mutex;
    static bool done[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(mutex);
    if (dev >= 0 && dev < 64 && done[dev]) return cudaSuccess;
    e = cudaFuncSetAttribute(paged_attn_kernel<D, E4M3>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)Map<in_tile(D), E4M3>::kBytes);
    if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev] = true;
    return e;
}

template <int D, bool E4M3>
static cudaError_t launch(const Cache &c, const void *q, int64_t qs, void *o, int group, float scale, int window,
                          int sinks, uint8_t *ws, int sms, int left_out, cudaStream_t s) {
    const Layout L = layout_of(c, group, D, sms);
    const Plan p{(int32_t *)(ws + L.tiles), (int64_t *)(ws + L.cost), (Cut *)(ws + L.cuts), (float *)(ws + L.part),
                 (float2 *)(ws + L.ml), L.ranges, L.rows, kRows, nullptr, L.most};
    StatusWord *st = (StatusWord *)ws;
    CUtensorMap tk, tv;
    cudaError_t e = page_map(&tk, c, c.k, D, E4M3);
    if (e == cudaSuccess) e = page_map(&tv, c, c.v, D, E4M3);
    if (e == cudaSuccess) e = allow_smem<D, E4M3>();
    if (e != cudaSuccess) return e;
    paged_plan_kernel<<<1, kPlanThreads, 0, s>>>(c, p, group, window, sinks, st);
    e = cudaGetLastError();
    if (e == cudaSuccess)
        e = launch_after(paged_attn_kernel<D, E4M3>, dim3(L.ranges), dim3(kThreads<E4M3>),
                         Map<in_tile(D), E4M3>::kBytes, s, c, p, tk, tv,
                         (const __nv_bfloat16 *)q, qs, (__nv_bfloat16 *)o, group, scale, window, sinks, left_out, st);
    return e == cudaSuccess ? launch_join(false, D, c, p, o, group, st, s) : e;
}

}  // namespace tc
}  // namespace paged

size_t paged_tc_bytes(const paged::Cache &c, int group, int D, int sms) {
    return paged::tc::layout_of(c, group, D, sms).total;
}

cudaError_t launch_paged_tc(bool e4m3, int D, const paged::Cache &c, const void *q, int64_t qs, void *o, int group,
                            float scale, int window, int sinks, void *ws, int sms, int left_out, cudaStream_t s) {
    using paged::tc::launch;
    uint8_t *w = (uint8_t *)ws;
    const auto run = e4m3 ? (D == 128 ? launch<128, true> : D == 64 ? launch<64, true> : launch<32, true>)
                          : (D == 128 ? launch<128, false> : D == 64 ? launch<64, false> : launch<32, false>);
    return run(c, q, qs, o, group, scale, window, sinks, w, sms, left_out, s);
}

}  // namespace kda
