// paged_decode_tc.cu -- attention of one new token a sequence over paged keys and values on the sm_103a
// tensor cores.
//
//   S^T = K Q^T,  P = 2^(f S - f m),  O^T = V^T P^T     (formulas: paged_attn_tc.cu)
// Memory-bound: each key and value is read once for up to 16 query heads that share it (more are further items: 64
// heads on one read it four times).  These are few, so
// keys and channels are the products' 128 rows and the heads their columns: a tile of 128 keys goes from
// its pages into shared memory and is an operand as it lies there, in bf16 or in e4m3.
//
// e4m3 pages meet e4m3 queries and weights, of which there are two each: x = hi + lo / 16, hi = e4m3(x), lo =
// e4m3(16 (x - hi)), in columns of their own.  Together they hold the 8 bits of a bf16, down to 2^-21 of
// the largest (rows of queries are scaled by a power of two, weights so that their largest is 2^7 to 2^8), so the
// keys' and values' bytes need no conversion: nothing but the products touches them.  A key's scale
// multiplies its scores, a value's is part of its weight.
//
// bf16 pages meet weights that are rounded to bf16 once; their sum is of those before the rounding.
//
// A piece of up to 4 tiles is gone through twice, keys, then values: all its scores stand in tensor memory
// before the first weight is formed, so its maximum is known and nothing that the tensor cores add up
// is rescaled.  Pieces are joined in registers, a thread a channel.  Loads and products take the keys of
// a piece before the values of the one before, so that weights are formed while keys arrive (in pieces of
// 8, one after the other, with the scales looked up by those who form the weights, 256 sequences of e4m3
// took 671 us).
//
// The work is cut as for chunks (kda_paged_tc.cuh): an item is a sequence, a key/value head and up to `each`
// query heads; each CTA finds its own range (a scan over the lengths, 1 us) instead of waiting for a
// plan.  What cuts inside items leave is joined by paged_join_kernel.
//
// 256 sequences of 512 to 8192 tokens, 32 heads on 8 of 128: 359 to 374 us from e4m3 pages, 6.3 to 6.6 TB/s; 660 us
// from bf16, 6.9 TB/s.  64 heads 436 us, 128 heads 680 (e4m3; the weights' instructions), 256 heads 1313 (1385 from bf16: read
// twice), heads of 64 311.
//
//   warps 0-3, 4-7   every other piece's scores -> weights, and its outputs; what the two have of an item
//                    meets at its end
//   warp 8   products (and zeroes values that may be anything: in slots behind a sequence's end and before
//            the window)
//   warp 9   loads of keys and values   warp 10  goes through the items, and loads their queries
//   warp 11  scales of e4m3 pages
#include "kda_paged_tc.cuh"

namespace kda {
namespace paged {
namespace tc {
namespace one {

constexpr int kThreads = 384;
constexpr int kRowWarps = 8, kMmaWarp = 8, kLoadWarp = 9, kItemWarp = 10;   // (the last: scales)
constexpr int kTiles = 4;           // of a piece
constexpr int kRing = 4;            // items known ahead

struct alignas(16) Item {
    int n;                    // -1: no more
    int h, row0, rows;        // query heads row0 .. of the group
    int pos, ctx;
    int k0, k1, sinks, from;  // tiles [k0, k1) of the list (KeyBlocks)
    int slot;                 // of Plan.part, or -1: the whole item
    int pad;
    __device__ __forceinline__ int tile(int k) const { return k < sinks ? k : from + k - sinks; }
};
// Pieces of an item's tiles, and where piece u begins: the first few have a tile more than the others.  (tiles * u /
// count would pass 32 bits from 92681 tiles on.)
__device__ __forceinline__ int pieces(int tiles) { return (tiles + kTiles - 1) / kTiles; }
__device__ __forceinline__ int piece_at(int tiles, int count, int u) { return u * (tiles / count) + min(u, tiles % count); }

template <int D, int NR, bool E4M3> struct Map {
    static constexpr int kCols = E4M3 ? 2 * NR : NR;         // columns in use: heads; (e4m3) their second parts
    static constexpr int N = kCols < 16 ? 16 : kCols;        // of a product
    static constexpr uint32_t kTile = 128 * D * (E4M3 ? 1 : 2);
    static constexpr uint32_t kQBytes = 4096, kPTile = N * (E4M3 ? 128 : 256);
    static constexpr uint32_t kScaleBytes = E4M3 ? 2 * kTiles * 512 : 0;   // of a piece: keys', then values'
    static constexpr uint32_t kMeet = NR * 512;              // outputs of warps 4-7 at an item's end
    static constexpr uint32_t kQ = 0, kP = 2 * kQBytes, kScales = kP + 2 * kTiles * kPTile,
                              kOther = kScales + 2 * kScaleBytes, kKV = (kOther + 2 * kMeet + 1023) / 1024 * 1024;
    static constexpr uint32_t kSmall = 5120;                 // what stands behind the ring
    static constexpr int kFit = (232448 - kKV - kSmall) / kTile, kStages = kFit > 16 ? 16 : kFit;
    static constexpr uint32_t kItems = kKV + kStages * kTile;
    static constexpr uint32_t kQf = kItems + kRing * sizeof(Item);     // [2][16]: a query row's factor
    static constexpr uint32_t kRed = kQf + 128;                        // [2 groups][2][4][32]: warps' maxima
    static constexpr uint32_t kSums = kRed + 2048;                     // [2][8][16]: warps' sums
    static constexpr uint32_t kTops = kSums + 1024;                    // [2][16]: maxima of warps 4-7
    static constexpr uint32_t kBar = kTops + 128;
    static constexpr int kFull = 0, kFree = kStages, kQFull = 2 * kStages, kQFree = kQFull + 2, kSReady = kQFree + 2,
                         kPReady = kSReady + 2, kODone = kPReady + 2, kItemFull = kODone + 2,
                         kItemFree = kItemFull + kRing, kDrain = kItemFree + kRing, kScFull = kDrain + 1, kScFree = kScFull + 2,
                         kBars = kScFree + 2;
    static constexpr uint32_t kFound = kBar + kBars * 8, kCuts = kFound + 16, kScan = kCuts + 48, kSlot = kScan + 80,
                              kBytes = kSlot + 16;
    static_assert(kStages >= 4 && kKV % 1024 == 0 && kPTile % 1024 == 0 && kBytes <= 232448 && kBytes - kItems <= kSmall && kFound % 8 == 0 &&
                      N * (E4M3 ? 128 : 2 * D) <= kQBytes && sizeof(Cut) <= 24,
                  "layout");
};

__device__ __forceinline__ void umma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                        uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Instruction descriptor of kind::f8f6f4 with e4m3 A and B and an fp32 accumulator.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N, bool a_mn_major) {
    return (1u << 4) | ((a_mn_major ? 1u : 0u) << 15) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// Largest of a warp, by an order of the bits as integers (a NaN is above all)
__device__ __forceinline__ float warp_top(float x) {
    int i = __float_as_int(x);
    i ^= (i >> 31) & 0x7fffffff;
    i = __reduce_max_sync(0xffffffffu, i);
    return __int_as_float(i ^ ((i >> 31) & 0x7fffffff));
}
// x[0], x[1] as two e4m3 each: hi in the low, lo in the high half; hi + lo / 16 is x but for 2^-8 of it
__device__ __forceinline__ uint32_t split_e4m3(float a, float b) {
    const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const float2 back = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(hi, __NV_E4M3)));
    const __nv_fp8x2_storage_t lo =
        __nv_cvt_float2_to_fp8x2(make_float2(16.f * (a - back.x), 16.f * (b - back.y)), __NV_SATFINITE, __NV_E4M3);
    return (uint32_t)hi | (uint32_t)lo << 16;
}

template <int DIM, int NR, bool E4M3>
__global__ void __launch_bounds__(kThreads, 1)
paged_decode_kernel(Cache c, Plan p, const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                    const __nv_bfloat16 *__restrict__ q, int64_t q_stride, __nv_bfloat16 *__restrict__ o, int group,
                    float scale, int window, int sinks, int left_out) {
    extern __shared__ __align__(1024) uint8_t sm[];
    constexpr int D = in_tile(DIM);   // (channels beyond DIM are products' rows that nobody reads)
    using M = Map<D, NR, E4M3>;
    constexpr int N = M::N, C = M::kCols;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    let_next_start();
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + M::kBar);
    Item *items = reinterpret_cast<Item *>(sm + M::kItems);
    StatusWord *st = reinterpret_cast<StatusWord *>(sm + M::kFound);
    Cut *cuts = reinterpret_cast<Cut *>(sm + M::kCuts);
    int64_t *sums = reinterpret_cast<int64_t *>(sm + M::kScan);
    uint32_t *tslot = reinterpret_cast<uint32_t *>(sm + M::kSlot);
    const uint32_t base = smem_u32(sm), bars = base + M::kBar;
    if (base & 1023u) {   // the operand images need their alignment; nothing is left to be joined
        if (tid == 0) p.found[blockIdx.x] = StatusWord{KDA_ERR_CUDA, 90, 0};
        if (tid < 2 && (tid == 0 || blockIdx.x + 1 == p.ranges)) p.cuts[blockIdx.x + tid] = Cut{0, 0, 0, 0, 0};
        return;
    }
    const int groups = (group + NR - 1) / NR;
    if (tid == 0) {
        *st = StatusWord{0, 0, 0};
        tslot[1] = 0;
        for (int i = 0; i < M::kStages; ++i) {
            mbar_init(&bar[M::kFull + i], 1);
            mbar_init(&bar[M::kFree + i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar[M::kQFull + i], 1);
            mbar_init(&bar[M::kQFree + i], 1 + kRowWarps);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar[M::kSReady + i], 1);
            mbar_init(&bar[M::kPReady + i], 4);
            mbar_init(&bar[M::kODone + i], 1);
            mbar_init(&bar[M::kScFull + i], 32);
            mbar_init(&bar[M::kScFree + i], 4);
        }
        for (int i = 0; i < kRing; ++i) {
            mbar_init(&bar[M::kItemFull + i], 1);
            mbar_init(&bar[M::kItemFree + i], kRowWarps + (E4M3 ? 3 : 2));
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
    own_range(c, p.ranges, groups, window, sinks, sums, cuts, st);
    tc_fence_after();
    const uint32_t tmem = *tslot;
    if (tid < 2 && (tid == 0 || blockIdx.x + 1 == p.ranges)) p.cuts[blockIdx.x + tid] = cuts[tid];
    const uint32_t tO = tmem + 2 * kTiles * N;   // behind two pieces' scores
    volatile int *failed = reinterpret_cast<volatile int *>(tslot + 1);
    bool ok = true;
    auto wait = [&](int which, uint32_t parity) {
        ok = ok && wait_warp(bars + 8 * which, parity);
        return ok;
    };
    auto wait_item = [&](int which, uint32_t parity) {
        ok = ok && wait_warp(bars + 8 * which, parity, item_tries(c));
        return ok;
    };
    auto each_item = [&](auto role) {
        Ring at;
        while (wait_item(M::kItemFull + at.stage, at.phase)) {
            const Item &it = items[at.stage];   // (read where it is used: registers are few)
            if (it.n < 0) break;
            role(it);
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[M::kItemFree + at.stage]);
            at.step(kRing);
            if (!ok) break;
        }
    };
    Ring kv;            // fills of the ring of tiles (a piece's keys, its values, ...)
    Ring qs;            // of the two places of queries
    Ring ps;            // of those of a piece's scores, scales, weights and outputs
    uint32_t loads = 0; // (load warp) fills issued

    if (warp < kRowWarps) {
        const int side = warp >> 2, quarter = warp & 3, key_at = tid & 127;
        const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
        const float f = scale * kLog2e;
        uint32_t turn = 0, ends = 0;   // of the maxima's places; of those where the two sides meet
        // Named barriers, which have no limit of their own: nobody waits there for a warp that has given up.
        auto meet = [&](uint32_t id, uint32_t n) {
            if (__any_sync(0xffffffffu, *failed != 0)) ok = false;
            else named_bar_sync(id, n);
            return ok;
        };
        each_item([&](const Item &it) {
            float run_m[NR], run_l[NR], run_o[NR];
#pragma unroll
            for (int g = 0; g < NR; ++g) {
                run_m[g] = -INFINITY;
                run_l[g] = run_o[g] = 0.f;
            }
            const int tiles = it.k1 - it.k0, count = pieces(tiles);
            const int pos = it.pos, lowest = window > 0 ? pos - window : -1;   // keys above it are in the window
            // (heads four at a time: a branch a head leaves the chains of instructions one behind the
            // other, 8.5k cycles a piece where the memory takes 5.8k)
            const int rows = it.rows;
            const float *qf = reinterpret_cast<const float *>(sm + M::kQf) + 16 * qs.stage;
            if (tiles > 0 && !wait(M::kQFull + qs.stage, qs.phase)) return;
            for (int u = 0; u < count; ++u) {
                if (ps.stage != side) {   // the other side's piece
                    ps.step(2);
                    continue;
                }
                const int first = it.k0 + piece_at(tiles, count, u), many = it.k0 + piece_at(tiles, count, u + 1) - first;
                // whether this thread's key of each tile is visible; (e4m3) its scales
                uint32_t seen = 0;
#pragma unroll
                for (int t = 0; t < kTiles; ++t) {
                    const int key = it.tile(first + t) * BK + key_at;
                    seen |= (uint32_t)(t < many && key <= pos && (key > lowest || key < sinks)) << t;
                }
                if (E4M3 && !wait(M::kScFull + ps.stage, ps.phase)) return;
                const float *sc = reinterpret_cast<const float *>(sm + M::kScales + ps.stage * M::kScaleBytes) + key_at;
                auto key_scale = [&](int t) { return sc[128 * t]; };
                // (a value's scale by its exponent, which sets what weights are measured in, and what it is over
                // that: 1 for a power of two)
                auto value_log = [&](int t) { return (float)((int)(__float_as_uint(sc[128 * (kTiles + t)]) >> 23) - 127); };
                auto value_rest = [&](int t) {
                    return __uint_as_float((__float_as_uint(sc[128 * (kTiles + t)]) & 0x7fffffu) | 0x3f800000u);
                };
                if (!wait(M::kSReady + ps.stage, ps.phase)) return;
                tc_fence_after();
                // The scores in units of log 2, -inf where the key is not visible, and the piece's maxima: m
                // of the scores; (e4m3) m2 of the weights with the values' scales
                const uint32_t tS = tmem + lanes + ps.stage * kTiles * N;
                // Up to 4 heads: all tiles at once, held from there on.  More: tile by tile in loops that stay
                // loops, read again for the weights.  (Straight-line code for 8 heads and 4 tiles misses the
                // instruction cache: 14k cycles a piece.)
                constexpr bool kAll = NR <= 4;
                constexpr int kUnroll = kAll ? kTiles : 1, kHeld = kAll ? kTiles : 1;
                float x[kHeld][NR], m[NR], m2[NR];
                auto scores = [&](const float(&y)[C], int t, float(&x)[NR]) {
                    const bool see = (seen >> t) & 1;
                    const float ks = E4M3 ? key_scale(t) : f;
#pragma unroll
                    for (int g = 0; g < NR; ++g)
                        x[g] = !see ? -INFINITY : E4M3 ? (y[g] + 0.0625f * y[(E4M3 ? NR : 0) + g]) * (ks * qf[g]) : y[g] * ks;
                };
#pragma unroll
                for (int g = 0; g < NR; ++g) m[g] = m2[g] = -INFINITY;
                auto highest = [&](const float(&z)[NR], int t) {
                    const float ev = E4M3 ? value_log(t) : 0.f;
#pragma unroll
                    for (int g = 0; g < NR; ++g) {
                        m[g] = fmaxf(m[g], z[g]);
                        if (E4M3) m2[g] = fmaxf(m2[g], z[g] + ev);
                    }
                };
                if constexpr (kAll) {   // (a tile behind the piece's last is read, but nothing of it is seen)
                    float y[kTiles][C];
#pragma unroll
                    for (int t = 0; t < kTiles; ++t) tmem_ld(tS + t * N, y[t]);
                    tmem_ld_wait();
#pragma unroll
                    for (int t = 0; t < kTiles; ++t) {
                        scores(y[t], t, x[kHeld > 1 ? t : 0]);
                        highest(x[kHeld > 1 ? t : 0], t);
                    }
                } else {
#pragma unroll 1
                    for (int t = 0; t < many; ++t) {
                        float y[C];
                        tmem_ld(tS + t * N, y);
                        tmem_ld_wait();
                        scores(y, t, x[0]);
                        highest(x[0], t);
                    }
                }
                float *place = reinterpret_cast<float *>(sm + M::kRed) + 256 * side + 128 * (turn & 1);
                ++turn;
#pragma unroll
                for (int g0 = 0; g0 < NR; g0 += 4) {
                    if (g0 >= rows) break;
                    float a[4], b[4];
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        a[g] = warp_top(m[g0 + g]);
                        if (E4M3) b[g] = warp_top(m2[g0 + g]);
                    }
                    if (lane == 0) {
                        *reinterpret_cast<float4 *>(place + 32 * quarter + g0) = make_float4(a[0], a[1], a[2], a[3]);
                        if (E4M3) *reinterpret_cast<float4 *>(place + 32 * quarter + 16 + g0) = make_float4(b[0], b[1], b[2], b[3]);
                    }
                }
                if (!meet(1 + side, 128)) return;
                float l[NR];
#pragma unroll
                for (int g0 = 0; g0 < NR; g0 += 4) {
                    if (g0 >= rows) break;
#pragma unroll
                    for (int e = 0; e < (E4M3 ? 2 : 1); ++e) {
                        float4 w[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const float4 *>(place + 32 * i + 16 * e + g0);
                        float *to = e ? &m2[g0] : &m[g0];
                        to[0] = fmaxf(fmaxf(w[0].x, w[1].x), fmaxf(w[2].x, w[3].x));
                        to[1] = fmaxf(fmaxf(w[0].y, w[1].y), fmaxf(w[2].y, w[3].y));
                        to[2] = fmaxf(fmaxf(w[0].z, w[1].z), fmaxf(w[2].z, w[3].z));
                        to[3] = fmaxf(fmaxf(w[0].w, w[1].w), fmaxf(w[2].w, w[3].w));
                    }
#pragma unroll
                    for (int g = g0; g < g0 + 4; ++g) l[g] = 0.f;
                }
                // The weights, as the products' columns
                const int last = kAll ? kTiles : many;
#pragma unroll kUnroll
                for (int t = 0; t < last; ++t) {
                    if constexpr (!kAll) {
                        float y[C];
                        tmem_ld(tS + t * N, y);
                        tmem_ld_wait();
                        scores(y, t, x[0]);
                    }
                    const float(&z)[NR] = x[kHeld > 1 ? t : 0];
                    const float ev = E4M3 ? value_log(t) : 0.f, rest = E4M3 ? value_rest(t) : 1.f;
                    uint8_t *to = sm + M::kP + (ps.stage * kTiles + t) * M::kPTile;
#pragma unroll
                    for (int g0 = 0; g0 < NR; g0 += 4) {
                        if (g0 >= rows) break;
                        float p[4];
#pragma unroll
                        for (int g = 0; g < 4; ++g) {
                            p[g] = ex2(z[g0 + g] - (m[g0 + g] == -INFINITY ? 0.f : m[g0 + g]));
                            l[g0 + g] += p[g];
                        }
                        // (neighbouring lanes, that is keys, exchange what they have of these heads, so that each
                        // stores a head's four bytes, or two bf16, in one)
                        if constexpr (E4M3) {
                            float v[4];
#pragma unroll
                            for (int g = 0; g < 4; ++g)
                                v[g] = rest * ex2(z[g0 + g] + ev - (m2[g0 + g] == -INFINITY ? 0.f : m2[g0 + g] - 7.f));
                            const uint32_t w[2] = {split_e4m3(v[0], v[1]), split_e4m3(v[2], v[3])};
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                uint32_t y = __byte_perm(w[0], w[1], i ? 0x7632 : 0x5410);
                                y = __byte_perm(y, __shfl_xor_sync(0xffffffffu, y, 1), lane & 1 ? 0x3715 : 0x6240);
                                y = __byte_perm(y, __shfl_xor_sync(0xffffffffu, y, 2), lane & 2 ? 0x3276 : 0x5410);
                                const int row = i * NR + g0 + (lane & 3);
                                *reinterpret_cast<uint32_t *>(to + row * 128 + (((key_at >> 4) ^ (row & 7)) << 4) + (key_at & 12)) = y;
                            }
                        } else {
#pragma unroll
                            for (int g = 0; g < 4; g += 2) {
                                uint32_t y = pack2(p[g], p[g + 1]);
                                y = __byte_perm(y, __shfl_xor_sync(0xffffffffu, y, 1), lane & 1 ? 0x3276 : 0x5410);
                                *reinterpret_cast<uint32_t *>(to + sw128_offset(g0 + g + (lane & 1), key_at & ~1, 16)) = y;
                            }
                        }
                    }
                }
                fence_proxy_async();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&bar[M::kPReady + ps.stage]);
                    if (E4M3) mbar_arrive(&bar[M::kScFree + ps.stage]);
                }
                __syncwarp();
                // what the piece's outputs count for, and, once its product is done, these
                float keep[NR], add[NR];
#pragma unroll
                for (int g0 = 0; g0 < NR; g0 += 4) {
#pragma unroll
                    for (int g = g0; g < g0 + 4; ++g) keep[g] = add[g] = 0.f;
                    if (g0 >= rows) continue;
#pragma unroll
                    for (int g = g0; g < g0 + 4; ++g) {
                        const float top = fmaxf(run_m[g], m[g]), ref = top == -INFINITY ? 0.f : top;
                        const float b = ex2(m[g] - ref);
                        keep[g] = ex2(run_m[g] - ref);
                        add[g] = E4M3 ? ex2(m2[g] - 7.f - ref) : b;
                        run_l[g] = run_l[g] * keep[g] + l[g] * b;
                        run_m[g] = top;
                    }
                }
                if (!wait(M::kODone + side, ps.phase)) return;
                tc_fence_after();
                float y[C];
                tmem_ld(tO + side * N + lanes, y);
                tmem_ld_wait();
                tc_fence_before();
#pragma unroll
                for (int g = 0; g < NR; ++g)
                    run_o[g] = run_o[g] * keep[g] + (E4M3 ? y[g] + 0.0625f * y[(E4M3 ? NR : 0) + g] : y[g]) * add[g];
                ps.step(2);
            }
            if (tiles > 0) {
                if (lane == 0) mbar_arrive(&bar[M::kQFree + qs.stage]);
                __syncwarp();
                qs.step(2);
            }
            // The item's end: warps 4-7 leave what they have, warps 0-3 put it together.  (Two places: one
            // may be written while the other is still read.)
            const uint32_t end = ends & 1;
            ++ends;
            float *sums = reinterpret_cast<float *>(sm + M::kSums) + 128 * end, *tops = reinterpret_cast<float *>(sm + M::kTops) + 16 * end;
            float *other = reinterpret_cast<float *>(sm + M::kOther + end * M::kMeet);
#pragma unroll
            for (int g0 = 0; g0 < NR; g0 += 4) {
                if (g0 >= rows) break;
                float a[4];
#pragma unroll
                for (int g = 0; g < 4; ++g) a[g] = warp_sum(run_l[g0 + g]);
                if (lane == 0) *reinterpret_cast<float4 *>(sums + 16 * warp + g0) = make_float4(a[0], a[1], a[2], a[3]);
                if (side == 1) {
                    if (key_at == 0)
                        *reinterpret_cast<float4 *>(tops + g0) = make_float4(run_m[g0], run_m[g0 + 1], run_m[g0 + 2], run_m[g0 + 3]);
#pragma unroll
                    for (int g = g0; g < g0 + 4; ++g) other[128 * g + key_at] = run_o[g];
                }
            }
            if (!meet(3, 256)) return;
            if (side == 1) return;
            const int d = D == 128 ? tid : 16 * warp + lane;   // (64 rows of a product stand in 16 lanes of each warp)
            const bool there = D == 128 || (lane < 16 && d < DIM);
#pragma unroll
            for (int g = 0; g < NR; ++g) {
                if (g >= rows) break;
                const float m1 = tops[g], top = fmaxf(run_m[g], m1), ref = top == -INFINITY ? 0.f : top;
                const float a = ex2(run_m[g] - ref), b = ex2(m1 - ref);
                const float l = a * (sums[g] + sums[16 + g] + sums[32 + g] + sums[48 + g]) +
                                b * (sums[64 + g] + sums[80 + g] + sums[96 + g] + sums[112 + g]);
                const float x = a * run_o[g] + b * other[128 * g + tid];
                if (it.slot >= 0) {
                    const int64_t at = (int64_t)it.slot * p.rows + g;
                    if (tid == 0) p.ml[at] = make_float2(ref, l);
                    if (there) p.part[at * DIM + d] = x;
                } else if (there) {
                    o[((int64_t)it.n * c.Hk * group + it.h * group + it.row0 + g) * DIM + d] =
                        __float2bfloat16_rn(l != 0.f ? x / l : 0.f);
                }
            }
        });
        if (!ok) {   // (whoever stands at a barrier goes on; whoever comes to one later sees why not to)
            if (lane == 0) *failed = 1;
            __threadfence_block();
            __syncwarp();
            named_bar_arrive(1 + side, 128);
            named_bar_arrive(3, 256);
        }
    } else if (warp == kMmaWarp) {
        constexpr uint32_t id_s = E4M3 ? idesc_e4m3(128, N, false) : idesc_bf16(128, N, false, false);
        constexpr uint32_t id_o = E4M3 ? idesc_e4m3(D, N, true) : idesc_bf16(D, N, true, false);
        // keys: rows of 128 bytes (64 for e4m3 heads of 64), channels along them; values the other way round
        constexpr bool narrow = E4M3 && D == 64;
        const uint64_t dk0 = narrow ? sdesc_sw64(base + M::kKV, 16, 512) : sdesc_sw128(base + M::kKV, 16, 1024);
        const uint64_t dv0 = narrow ? sdesc_sw64(base + M::kKV, 16, 512) : sdesc_sw128(base + M::kKV, BK * 128, 1024);
        const uint64_t dq0 = sdesc_sw128(base + M::kQ, 16, 1024), dp0 = sdesc_sw128(base + M::kP, 16, 1024);
        // the piece whose values are still to come: its tiles, and what the last lacks (0: nothing); (with a
        // window) its first tile's place in the list, and the list
        int owed = 0, owed_left = 0, owed_first = 0, owed_sinks = 0, owed_from = 0, owed_lowest = -1;
        Ring os;   // its place
        auto values = [&] {
            if (owed == 0) return;
            if (!wait(M::kPReady + os.stage, os.phase)) return;
            for (int t = 0; t < owed; ++t) {
                if (!wait(M::kFull + kv.stage, kv.phase)) return;
                if (owed_left && t + 1 == owed) clear_rows<D * (E4M3 ? 1 : 2)>(sm + M::kKV + kv.stage * M::kTile, owed_left, BK);
                if (owed_lowest >= 0) {
                    const int k = owed_first + t;
                    const Unseen gap = unseen((k < owed_sinks ? k : owed_from + k - owed_sinks) * BK, owed_lowest, sinks);
                    if (gap.begin < gap.end)
                        clear_rows<D * (E4M3 ? 1 : 2)>(sm + M::kKV + kv.stage * M::kTile, gap.begin, gap.end);
                }
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t dv = desc_add(dv0, kv.stage * M::kTile), dp = desc_add(dp0, (os.stage * kTiles + t) * M::kPTile);
                    if constexpr (E4M3) {
#pragma unroll
                        for (int s = 0; s < BK / 32; ++s)
                            umma_f8(tO + os.stage * N, desc_add(dv, s * 32 * D), desc_add(dp, s * 32), id_o, t > 0 || s > 0);
                    } else {
#pragma unroll
                        for (int s = 0; s < BK / 16; ++s)
                            umma_bf16(tO + os.stage * N, desc_add(dv, s * 2048), desc_add(dp, (s >> 2) * 2048 + (s & 3) * 32), id_o,
                                      t > 0 || s > 0);
                    }
                    umma_commit(&bar[M::kFree + kv.stage]);
                    if (t + 1 == owed) umma_commit(&bar[M::kODone + os.stage]);
                }
                __syncwarp();
                kv.step(M::kStages);
            }
            owed = 0;
            os.step(2);
        };
        each_item([&](const Item &it) {
            const int tiles = it.k1 - it.k0, count = pieces(tiles);
            if (tiles == 0) {   // (nothing may be owed over items that have none: the ring of items is short)
                values();
                return;
            }
            if (!wait(M::kQFull + qs.stage, qs.phase)) return;
            for (int u = 0; u < count; ++u) {
                const int first = it.k0 + piece_at(tiles, count, u), many = it.k0 + piece_at(tiles, count, u + 1) - first;
                for (int t = 0; t < many; ++t) {
                    if (!wait(M::kFull + kv.stage, kv.phase)) return;
                    tc_fence_after();
                    if (elect_one()) {
                        const uint64_t dk = desc_add(dk0, kv.stage * M::kTile), dq = desc_add(dq0, qs.stage * M::kQBytes);
                        const uint32_t to = tmem + (ps.stage * kTiles + t) * N;
                        if constexpr (E4M3) {
#pragma unroll
                            for (int s = 0; s < DIM / 32; ++s)
                                umma_f8(to, desc_add(dk, s * 32), desc_add(dq, s * 32), id_s, s > 0);
                        } else {
#pragma unroll
                            for (int s = 0; s < DIM / 16; ++s)
                                umma_bf16(to, desc_add(dk, (s >> 2) * 16384 + (s & 3) * 32),
                                          desc_add(dq, (s >> 2) * 2048 + (s & 3) * 32), id_s, s > 0);
                        }
                        umma_commit(&bar[M::kFree + kv.stage]);
                        if (t + 1 == many) {
                            umma_commit(&bar[M::kSReady + ps.stage]);
                            if (u + 1 == count) umma_commit(&bar[M::kQFree + qs.stage]);
                        }
                    }
                    __syncwarp();
                    kv.step(M::kStages);
                }
                ps.step(2);
                values();
                if (!ok) return;
                owed = many;
                owed_first = first;
                owed_sinks = it.sinks;
                owed_from = it.from;
                owed_lowest = window > 0 ? it.pos - window : -1;   // (keys above it are in the window)
                const int left = it.ctx - it.tile(first + many - 1) * BK;   // (below BK only in an item's last tile)
                owed_left = left < BK && (it.ctx & ((1 << c.shift) - 1)) != 0 ? left : 0;
            }
            qs.step(2);
        });
        if (ok) values();
    } else if (warp == kLoadWarp) {
        // Lane 8 t + b has to do with box b of a piece's tile t: its page is looked up a piece ahead, and the
        // loop over tiles is short (with every lane holding a box of all tiles, unrolled, a tile took the warp
        // 800 cycles, more than the memory).
        const int rows = min(BK, 1 << c.shift), boxes = BK / rows, runs = page_runs(c, DIM);
        const int none = (c.P - 1) * runs + c.Hk;   // past the last run: zeros
        const int my_tile = lane >> 3, box = lane & 7;
        int owed = 0, owed_run = 0, owed_row = 0;   // the piece whose values are still to be loaded
        auto load = [&](const void *map, int many, int run, int row) {
#pragma unroll 1
            for (int t = 0; t < many; ++t) {
                if (!wait(M::kFree + kv.stage, kv.phase ^ 1)) return;
                const bool left = loads == 0 && left_out == (int)blockIdx.x;
                if (lane == 0 && !left) mbar_arrive_expect_tx(&bar[M::kFull + kv.stage], M::kTile);
                __syncwarp();
                if (t == my_tile && box < boxes && !left) {
                    const uint32_t to = base + M::kKV + kv.stage * M::kTile + box * rows * (E4M3 ? D : 128);
#pragma unroll
                    for (int x = 0; x < (E4M3 ? 1 : D / 64); ++x)
                        tma_load_rows(to + x * 16384, map, 64 * x, row, run, bars + 8 * (M::kFull + kv.stage));
                }
                __syncwarp();
                kv.step(M::kStages);
                ++loads;
            }
        };
        each_item([&](const Item &it) {
            const int tiles = it.k1 - it.k0, count = pieces(tiles), pos = it.pos, n = it.n, h = it.h;
            int page = -1;
            bool seen = false;   // by the token; else no page is needed
            auto key_of = [&](int u) { return it.tile(it.k0 + piece_at(tiles, count, u) + my_tile) * BK + box * rows; };
            auto look_up = [&](int u) {
                const int many = piece_at(tiles, count, u + 1) - piece_at(tiles, count, u), key = key_of(u);
                seen = my_tile < many && box < boxes && key <= pos && (window <= 0 || key < sinks || key + rows > pos - window + 1);
                if (seen) page = c.table[(int64_t)n * c.width + (key >> c.shift)];
            };
            if (tiles > 0) look_up(0);
            // (a turn more, for the values of the last piece where the next item has none)
            for (int u = 0; u < count || (tiles == 0 && owed); ++u) {
                int run = none, row = 0, many = 0;
                if (u < count) {
                    many = piece_at(tiles, count, u + 1) - piece_at(tiles, count, u);
                    row = key_of(u) & ((1 << c.shift) - 1);
                    if (seen) {
                        if (page >= 0 && page < c.P) run = page * runs + h;
                        else report(st, KDA_ERR_INVALID_ARG, n, 91);
                    }
                    if (u + 1 < count) look_up(u + 1);
                    load(&tk, many, run, row);
                }
                if (ok && owed) load(&tv, owed, owed_run, owed_row);
                if (!ok) return;
                owed = many;
                owed_run = run;
                owed_row = row;
            }
        });
        if (ok && owed) load(&tv, owed, owed_run, owed_row);
    } else if (warp == kItemWarp) {
        Ring at;
        Cut from = cuts[0];
        const Cut to = cuts[1];
        while (true) {
            Span s{0, 0, 0};
            while (from.n < c.N && (from.tile < to.tile || (from.tile == to.tile && (from.h < to.h || (from.h == to.h && from.k < to.k))))) {
                s = span_of(c, from.n);
                if (s.len) break;
                ++from.n;   // (a sequence that does not fit)
                from.t = from.h = from.k = 0;
                from.tile = from.n * groups;
            }
            Item it{};
            it.n = -1;
            const bool more = s.len > 0;
            if (more) {
                const Tile t = tile_of(s, from.t, group, NR);
                const KeyBlocks kb = key_blocks(max(0, s.pos), s.pos, window, sinks, BK);
                it.n = from.n;
                it.h = from.h;
                it.row0 = t.row0;
                it.rows = t.rows;
                it.pos = s.pos;
                it.ctx = s.pos + 1;
                it.k0 = from.k;
                it.k1 = same_item(from, to) ? min(to.k, kb.count) : kb.count;
                it.sinks = kb.sinks;
                it.from = kb.from;
                it.slot = it.k0 > 0 ? 2 * (int)blockIdx.x : it.k1 < kb.count ? 2 * (int)blockIdx.x + 1 : -1;
            }
            if (!wait_item(M::kItemFree + at.stage, at.phase ^ 1)) break;
            if (lane == 0) {
                items[at.stage] = it;
                mbar_arrive(&bar[M::kItemFull + at.stage]);
            }
            __syncwarp();
            if (!more) break;
            at.step(kRing);
            from.k = 0;
            if (++from.h == c.Hk) {
                from.h = 0;
                ++from.tile;
                if (++from.t == groups) {
                    from.t = 0;
                    ++from.n;
                }
            }
            if (it.k1 == it.k0) continue;
            // its queries
            const __nv_bfloat16 *x0 = q + (int64_t)it.n * q_stride + (int64_t)(it.h * group + it.row0) * DIM;
            uint8_t *place = sm + M::kQ + qs.stage * M::kQBytes;
            float *qf = reinterpret_cast<float *>(sm + M::kQf) + 16 * qs.stage;
            if (!wait_item(M::kQFree + qs.stage, qs.phase ^ 1)) break;
            if constexpr (E4M3) {
                constexpr int V = D / 32;   // channels a lane (heads of 32: the last 16 lanes have zeros)
#pragma unroll 4
                for (int g = 0; g < it.rows; ++g) {
                    float x[V], top = 0.f;
#pragma unroll
                    for (int j = 0; j < V; j += 2) {
                        __nv_bfloat162 y = __floats2bfloat162_rn(0.f, 0.f);
                        if (D == DIM || lane * V < DIM) y = *reinterpret_cast<const __nv_bfloat162 *>(x0 + g * DIM + lane * V + j);
                        x[j] = __low2float(y);
                        x[j + 1] = __high2float(y);
                        top = fmaxf(top, fmaxf(fabsf(x[j]), fabsf(x[j + 1])));
                    }
                    top = warp_top(top);
                    // (a row that is not finite has no scale: its factor is NaN, and so is what it gives)
                    const bool fine = __all_sync(0xffffffffu, x[0] - x[0] == 0.f && x[1] - x[1] == 0.f &&
                                                                  x[V - 1] - x[V - 1] == 0.f && x[V - 2] - x[V - 2] == 0.f);
                    const int e = fine && top > 0.f ? scale_exponent(top) : 0;
                    const float inv = two_to(-e);
                    uint32_t hi = 0, lo = 0;
#pragma unroll
                    for (int j = 0; j < V; j += 2) {
                        const uint32_t w = split_e4m3(x[j] * inv, x[j + 1] * inv);
                        hi |= (w & 0xffffu) << (8 * j);
                        lo |= (w >> 16) << (8 * j);
                    }
                    const uint32_t to = lane * V;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int row = i * NR + g;
                        uint8_t *y = place + row * 128 + (((to >> 4) ^ (row & 7)) << 4) + (to & 15);
                        if constexpr (V == 4) *reinterpret_cast<uint32_t *>(y) = i ? lo : hi;
                        else *reinterpret_cast<uint16_t *>(y) = (uint16_t)(i ? lo : hi);
                    }
                    if (lane == 0) qf[g] = fine ? two_to(e) * scale * kLog2e : __int_as_float(0x7fffffff);
                }
            } else {
                constexpr int U = DIM / 8;
                for (int x = lane; x < it.rows * U; x += 32)
                    *reinterpret_cast<uint4 *>(place + sw128_offset(x / U, 8 * (x % U), 16)) =
                        *reinterpret_cast<const uint4 *>(x0 + x * 8);
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[M::kQFull + qs.stage]);
            __syncwarp();
            qs.step(2);
        }
    } else if (E4M3) {
        // a piece's scales: four keys' a lane and tile, their pages looked up a piece ahead
        each_item([&](const Item &it) {
            const int tiles = it.k1 - it.k0, count = pieces(tiles), pos = it.pos;
            int page[kTiles];
            auto look_up = [&](int u) {
                const int first = it.k0 + piece_at(tiles, count, u), many = it.k0 + piece_at(tiles, count, u + 1) - first;
#pragma unroll
                for (int t = 0; t < kTiles; ++t) {
                    const int key = it.tile(first + t) * BK + 4 * lane;
                    page[t] = -1;
                    if (t < many && key <= pos && (window <= 0 || key < sinks || key + 4 > pos - window + 1))
                        page[t] = c.table[(int64_t)it.n * c.width + (key >> c.shift)];
                }
            };
            if (tiles > 0) look_up(0);
            for (int u = 0; u < count; ++u) {
                const int first = it.k0 + piece_at(tiles, count, u), many = it.k0 + piece_at(tiles, count, u + 1) - first;
                int64_t at[kTiles];
                uint32_t there = 0;
#pragma unroll
                for (int t = 0; t < kTiles; ++t) {
                    const bool fine = page[t] >= 0 && page[t] < c.P;   // (else zeros)
                    there |= (uint32_t)fine << t;
                    at[t] = fine ? page[t] * c.scale_stride + ((int64_t)it.h << c.shift) +
                                       ((it.tile(first + t) * BK + 4 * lane) & ((1 << c.shift) - 1))
                                 : 0;
                }
                if (u + 1 < count) look_up(u + 1);
                if (!wait(M::kScFree + ps.stage, ps.phase ^ 1)) return;
                const uint32_t place = base + M::kScales + ps.stage * M::kScaleBytes + 16 * lane;
#pragma unroll
                for (int t = 0; t < kTiles; ++t) {
                    if (t >= many) break;
                    const uint32_t bytes = (there >> t) & 1 ? 16 : 0;
#pragma unroll
                    for (int v = 0; v < 2; ++v)
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(place + 512 * (v * kTiles + t)),
                                     "l"((v ? c.vs : c.ks) + at[t]), "r"(bytes)
                                     : "memory");
                }
                asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bars + 8 * (M::kScFull + ps.stage))
                             : "memory");
                ps.step(2);
            }
        });
        asm volatile("cp.async.wait_all;" ::: "memory");
    }
    if (!ok && lane == 0) report(st, KDA_ERR_TIMEOUT, blockIdx.x, 92 + warp);
    if (__syncthreads_or(!ok)) {
        // an expired wait: what is in flight ends (each wait bounded again) before the tensor memory is
        // released and the CTA leaves
        asm volatile("cp.async.wait_all;" ::: "memory");
        tc_fence_before();
        if (warp == kMmaWarp) {
            tc_fence_after();
            if (elect_one()) umma_commit(&bar[M::kDrain]);
            __syncwarp();
            mbar_wait(&bar[M::kDrain], 0, kDrainNs);
        }
        if (warp == kLoadWarp)   // (only each stage's last load can be in flight)
            for (uint32_t x = loads >= (uint32_t)M::kStages ? loads - M::kStages : 0; x < loads; ++x)
                mbar_wait(&bar[M::kFull + x % M::kStages], (x / M::kStages) & 1, kDrainNs);
        __syncthreads();
    }
    if (tid == 0) p.found[blockIdx.x] = *st;
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, kCols);
    }
}

struct Layout {
    int ranges, rows, each;
    size_t cuts, found, ml, part, total;
};
static Layout layout_of(int group, int D, int sms) {
    Layout L;
    L.each = group <= 4 ? 4 : group <= 8 ? 8 : 16;
    L.rows = group < L.each ? group : L.each;
    L.ranges = sms;
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    L.cuts = kHeaderBytes;
    L.found = L.cuts + up(sizeof(Cut) * ((size_t)L.ranges + 1));
    L.ml = L.found + up(sizeof(StatusWord) * L.ranges);
    L.part = L.ml + up(sizeof(float2) * 2 * L.ranges * L.rows);
    L.total = L.part + sizeof(float) * 2 * L.ranges * L.rows * D;
    return L;
}

// Shared memory above 48 KB, once per kernel and device.
template <int D, int NR, bool E4M3> static cudaError_t allow_smem() {
    static std::mutex mutex;
    static bool done[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(mutex);
    if (dev >= 0 && dev < 64 && done[dev]) return cudaSuccess;
    e = cudaFuncSetAttribute(paged_decode_kernel<D, NR, E4M3>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)Map<in_tile(D), NR, E4M3>::kBytes);
    if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev] = true;
    return e;
}

template <int D, int NR, bool E4M3>
static cudaError_t launch(const Cache &c, const void *q, int64_t qs, void *o, int group, float scale, int window,
                          int sinks, uint8_t *ws, int sms, int left_out, cudaStream_t s) {
    const Layout L = layout_of(group, D, sms);
    const Plan p{nullptr, nullptr, (Cut *)(ws + L.cuts), (float *)(ws + L.part), (float2 *)(ws + L.ml), L.ranges, L.rows,
                 L.each, (StatusWord *)(ws + L.found), 0};
    CUtensorMap tk, tv;
    cudaError_t e = page_map(&tk, c, c.k, D, E4M3);
    if (e == cudaSuccess) e = page_map(&tv, c, c.v, D, E4M3);
    if (e == cudaSuccess) e = allow_smem<D, NR, E4M3>();
    if (e != cudaSuccess) return e;
    paged_decode_kernel<D, NR, E4M3><<<L.ranges, kThreads, Map<in_tile(D), NR, E4M3>::kBytes, s>>>(
        c, p, tk, tv, (const __nv_bfloat16 *)q, qs, (__nv_bfloat16 *)o, group, scale, window, sinks, left_out);
    e = cudaGetLastError();
    return e == cudaSuccess ? launch_join(false, D, c, p, o, group, (StatusWord *)ws, s) : e;
}

}  // namespace one
}  // namespace tc
}  // namespace paged

size_t paged_decode_bytes(int group, int D, int sms) { return paged::tc::one::layout_of(group, D, sms).total; }

cudaError_t launch_paged_decode(bool e4m3, int D, const paged::Cache &c, const void *q, int64_t qs, void *o, int group,
                                float scale, int window, int sinks, void *ws, int sms, int left_out, cudaStream_t s) {
    using paged::tc::one::launch;
    uint8_t *w = (uint8_t *)ws;
#define KDA_ONE(D_, NR_, E_) \
    if (D == D_ && group <= (NR_ == 16 ? 0x7fffffff : NR_) && e4m3 == E_) \
        return launch<D_, NR_, E_>(c, q, qs, o, group, scale, window, sinks, w, sms, left_out, s);
#define KDA_ONES(D_, E_) KDA_ONE(D_, 4, E_) KDA_ONE(D_, 8, E_) KDA_ONE(D_, 16, E_)
    KDA_ONES(32, false) KDA_ONES(64, false) KDA_ONES(128, false) KDA_ONES(32, true) KDA_ONES(64, true) KDA_ONES(128, true)
#undef KDA_ONES
#undef KDA_ONE
    return cudaErrorInvalidValue;
}

}  // namespace kda
