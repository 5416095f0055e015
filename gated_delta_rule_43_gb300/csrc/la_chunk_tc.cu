// la_chunk_tc.cu -- linear attention with one decay per head on the sm_103a tensor cores
// (bf16 operands, fp32 accumulation), 128-token chunks, dk and dv up to 128.
//
// Inside a chunk that starts from state S, with G_t = g_1 + ... + g_t and C tokens:
//   P  = (Q K^T) * exp(G_t - G_s) for s <= t, else 0
//   O  = P V + exp(G_t) Q S
//   S' = exp(G_C) S + K~^T V,     K~_s = exp(g_{s+1} + ... + g_C) k_s
// Four products of 128 x 128 x 128 a chunk: 131 kflop a token and head against 1 KB of q, k,
// v and o, so that a walk at the memory's rate keeps the tensor cores 40% busy.
//
// Roundings.  q, k, v are bf16 as they come.  P and the copy of S that meets the queries are
// rounded to bf16, like the output they go into.  The state that is carried on is not: K~ is
// the sum of two bf16 (hi + lo, 2^-17 of its value), their products with V add up in fp32,
// and S stays in fp32 registers for the whole walk; each chunk's contribution starts from
// zero in tensor memory, so that the tensor cores' own accumulation is never longer than a
// chunk.
//
// exp(G_t - G_s) is never a quotient of far-apart numbers: with R the value of G at the end
// of the 32-token block of s, it is exp(G_t - R) exp(R - G_s), two factors of at most one,
// for the blocks before that of t, and is formed token by token inside t's own block.
//
// One CTA an SM walks its range (see kda_la.cuh), every role for itself through the same
// items and chunks:
//   warps 0-3    rows of P (tensor memory, as the A operand of P V), rows of O (through
//                shared memory, over the image of S, in one bulk store: rows stored straight
//                from registers cost 2k cycles a chunk and held up everyone's shared memory)
//   warps 4-11   K~ (over K and Q, whose products are done by then), and the state: thread
//                (row, half) holds its columns of S
//   warp 12      issues the products          warp 13   loads q, k, v (two stages)
//   warp 14      the chunk's decays, one chunk ahead
// 96 KB a stage and the 32 KB image of S fill the SM's shared memory.
#include <cuda.h>

#include <mutex>

#include "kda_la.cuh"
#include "kda_sm100.cuh"

namespace kda {
namespace la {
namespace tc {

using namespace sm100;

constexpr int C = kChunk;
constexpr int kThreads = 512;
constexpr int kRowWarps = 4, kStateWarps = 8;
constexpr int kMmaWarp = 12, kLoadWarp = 13, kGateWarp = 14;
constexpr uint64_t kWaitNs = 1000000000ull;

// What one chunk's decays give, for one stage.
struct Gates {
    float G[C];        // prefix sums times log2(e)
    float w[C];        // exp(g_{s+1} + ... + g_C)
    float cf[96];      // exp(R - G_s); the last block needs none
};

enum Bar {
    kFull = 0,      // [2] a stage's tiles have landed
    kGate = 2,      // [2] a stage's decays are there
    kGateFree = 4,  // [2] ... and have been used
    kKvDone = 6,    // [2] K~^T V, and with it every product that reads the stage
    kPvDone = 8,    // [2] P V
    kQkDone = 10,   // Q K^T
    kQsDone = 11,   // Q S
    kPReady = 12,   // P is in tensor memory
    kKtReady = 13,  // K~ is in shared memory
    kSReady = 14,   // the image of S is
    kOFree = 15,    // the accumulators of O have been read
    kSFree = 16,    // the outputs that lay over the image of S have left
    kDrain = 17,
    kBars = 18
};

template <int DKP, int DVP> struct Map {
    static constexpr uint32_t kQ = 0, kK = DKP * 256, kV = 2 * DKP * 256;   // within a stage
    static constexpr uint32_t kStage = kV + DVP * 256;
    static constexpr uint32_t kS = 2 * kStage;                 // S image, [DKP rows][DVP]
    static constexpr uint32_t kGates = kS + C * DVP * 2;       // ... or a chunk's outputs, [C][DVP]
    static constexpr uint32_t kTot = kGates + 2 * sizeof(Gates);   // decay of the chunk, [2]
    static constexpr uint32_t kBar = kTot + 8;
    static constexpr uint32_t kBytes = kBar + kBars * 8 + 8;
    static_assert(kBar % 8 == 0 && kS % 1024 == 0 && kStage % 1024 == 0 && kBytes <= 232448, "layout");
};

__device__ __forceinline__ void umma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc,
                                             uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d_tmem), "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// 16 consecutive columns of the warp's 32 lanes
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
        ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
          "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]),
          "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// shared -> global through a tensor map (full boxes; what lies outside the tensor is dropped)
__device__ __forceinline__ void tma_store_3d(const void *tmap, const void *src, int32_t c0,
                                             int32_t c1, int32_t c2) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];"
                 ::"l"(tmap), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(src))
                 : "memory");
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&x);
}
__device__ __forceinline__ float2 unpack2(uint32_t u) {
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u));
}

// 2^x by the special-function unit (relative error near 2^-22)
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
constexpr float kLog2e = 1.4426950408889634f;

// The parts of w x: x two bf16, hi the product rounded to bf16, lo the rounded rest.
__device__ __forceinline__ void split2(uint32_t x, float w, uint32_t &hi, uint32_t &lo) {
    const float a0 = w * __uint_as_float(x << 16), a1 = w * __uint_as_float(x & 0xffff0000u);
    hi = pack2(a0, a1);
    lo = pack2(a0 - __uint_as_float(hi << 16), a1 - __uint_as_float(hi & 0xffff0000u));
}

// Waits that end: after kWaitNs, or when another role of the CTA has given up.
struct Waits {
    uint64_t *bar;
    volatile int *abort;
    __device__ __forceinline__ bool operator()(int which, uint32_t parity) const {
        if (mbar_try_wait(&bar[which], parity)) return true;
        const uint64_t t0 = globaltimer_ns();
        for (uint32_t i = 1;; ++i) {
            if (mbar_try_wait(&bar[which], parity)) return true;
            if ((i & 63u) == 0 && (*abort || globaltimer_ns() - t0 > kWaitNs)) return false;
        }
    }
};

// OUT: outputs and final states of the CTA's range.  Else what the end of the range leaves at
// the cut behind it (only K~^T V; no queries).
template <int DKP, int DVP, bool OUT>
__global__ void __launch_bounds__(kThreads, 1)
la_chunk_tc_kernel(Plan p, const __grid_constant__ CUtensorMap tq,
                   const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                   const __grid_constant__ CUtensorMap to,
                   const float *__restrict__ g, int g_per_token, const float *h0, float *hT,
                   __nv_bfloat16 *__restrict__ o, int dk, int dv, float *__restrict__ bnd,
                   float *__restrict__ bnd_log, StatusWord *st) {
    extern __shared__ __align__(1024) uint8_t sm[];
    using M = Map<DKP, DVP>;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int range = blockIdx.x;
    if (OUT ? p.cuts[range].x >= p.cuts[range + 1].x : !p.cuts[range + 1].inner) return;
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + M::kBar);
    uint32_t *tslot = reinterpret_cast<uint32_t *>(sm + M::kBar + kBars * 8);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + M::kBar + kBars * 8 + 4);
    Gates *gates = reinterpret_cast<Gates *>(sm + M::kGates);
    float *tot = reinterpret_cast<float *>(sm + M::kTot);
    const uint32_t base = smem_u32(sm);
    if (base & 1023u) {   // the operand images need their alignment
        if (tid == 0) report(st, KDA_ERR_CUDA, 0, 40);
        return;
    }
    if (tid == 0) {
        for (int b = 0; b < 2; ++b) {
            mbar_init(&bar[kFull + b], 1);
            mbar_init(&bar[kGate + b], 1);
            mbar_init(&bar[kGateFree + b], kStateWarps + (OUT ? kRowWarps : 0));
            mbar_init(&bar[kKvDone + b], 1);
            mbar_init(&bar[kPvDone + b], 1);
        }
        mbar_init(&bar[kQkDone], 1);
        mbar_init(&bar[kQsDone], 1);
        mbar_init(&bar[kPReady], kRowWarps);
        mbar_init(&bar[kKtReady], kStateWarps);
        mbar_init(&bar[kSReady], kStateWarps);
        mbar_init(&bar[kOFree], kRowWarps);
        mbar_init(&bar[kSFree], 1);
        mbar_init(&bar[kDrain], 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    constexpr uint32_t kCols = OUT ? 512 : 128;
    if (warp == kMmaWarp) {
        tmem_alloc(tslot, kCols);
        tmem_relinquish();
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;
    // scores (then P), Q S, P V, K~^T V
    const uint32_t tA = tmem, tQS = tmem + 128, tPV = tmem + 256, tKV = OUT ? tmem + 384 : tmem;
    const Waits wait{bar, abort_flag};
    const int64_t dkdv = (int64_t)dk * dv;
    const int group = p.H / p.Hk;
    uint32_t gi = 0;    // chunks so far: stage gi & 1, phase parities
    bool ok = true;
    uint32_t loaded = 0, landed = 0;   // (load warp)

    Item it;
    Walk walk(p, range);
    bool more = OUT ? walk.next(it) : before_cut(p, range + 1, it);
    for (; more && ok; more = OUT && walk.next(it)) {
        const int h = it.h;
        const int chunks = it.c1 - it.c0;

        if (warp < kRowWarps) {
            if (!OUT) continue;
            const int t = tid;   // this thread's row of the chunk
            const uint32_t lanes = (uint32_t)(32 * warp) << 16;
            for (int c = 0; c < chunks; ++c, ++gi) {
                const uint32_t b = gi & 1, ph = (gi >> 1) & 1;
                const int64_t t0 = it.t0 + (int64_t)c * C;
                ok = __all_sync(0xffffffffu, wait(kGate + b, ph) && wait(kQkDone, gi & 1));
                float eG = 0.f;
                if (ok) {
                    tc_fence_after();
                    const Gates &G = gates[b];
                    const float Gt = G.G[t];
                    eG = ex2(Gt);
                    // (loops that stay loops: the roles' code shares one instruction cache)
#pragma unroll 1
                    for (int cb = 0; cb < 4; ++cb) {
                        uint32_t pk[16];
                        if (cb <= warp) {
                            float a[32];
                            tmem_ld32(tA + lanes + 32 * cb, a);
                            tmem_ld_wait();
                            if (cb < warp) {
                                const float rf = ex2(Gt - G.G[32 * cb + 31]);
#pragma unroll
                                for (int j = 0; j < 32; j += 4) {
                                    const float4 f = *reinterpret_cast<const float4 *>(&G.cf[32 * cb + j]);
                                    pk[j / 2] = pack2(a[j] * (rf * f.x), a[j + 1] * (rf * f.y));
                                    pk[j / 2 + 1] = pack2(a[j + 2] * (rf * f.z), a[j + 3] * (rf * f.w));
                                }
                            } else {
#pragma unroll
                                for (int j = 0; j < 32; j += 4) {
                                    const float4 f = *reinterpret_cast<const float4 *>(&G.G[32 * cb + j]);
                                    pk[j / 2] = pack2(j <= lane ? a[j] * ex2(Gt - f.x) : 0.f,
                                                      j + 1 <= lane ? a[j + 1] * ex2(Gt - f.y) : 0.f);
                                    pk[j / 2 + 1] = pack2(j + 2 <= lane ? a[j + 2] * ex2(Gt - f.z) : 0.f,
                                                          j + 3 <= lane ? a[j + 3] * ex2(Gt - f.w) : 0.f);
                                }
                            }
                        } else {
#pragma unroll
                            for (int j = 0; j < 16; ++j) pk[j] = 0;
                        }
                        // (columns of scores that this warp has read)
                        tmem_st16(tA + lanes + 16 * cb, pk);
                    }
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&bar[kPReady]);
                        mbar_arrive(&bar[kGateFree + b]);
                    }
                    ok = __all_sync(0xffffffffu, wait(kPvDone + b, ph));
                }
                // these warps stop together: the barriers below have no time limit
                ok = bar_and(2, 32 * kRowWarps, ok);
                if (!ok) break;
                tc_fence_after();
                // the outputs over the image of S, which Q S was the last to read
#pragma unroll 1
                for (int cb = 0; cb < DVP / 32; ++cb) {
                    float x[32], y[32];
                    tmem_ld32(tQS + lanes + 32 * cb, x);
                    tmem_ld32(tPV + lanes + 32 * cb, y);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 32; j += 8) {
                        uint4 u;
                        u.x = pack2(eG * x[j] + y[j], eG * x[j + 1] + y[j + 1]);
                        u.y = pack2(eG * x[j + 2] + y[j + 2], eG * x[j + 3] + y[j + 3]);
                        u.z = pack2(eG * x[j + 4] + y[j + 4], eG * x[j + 5] + y[j + 5]);
                        u.w = pack2(eG * x[j + 6] + y[j + 6], eG * x[j + 7] + y[j + 7]);
                        *reinterpret_cast<uint4 *>(sm + M::kS + sw128_offset(t, 32 * cb + j, C)) = u;
                    }
                }
                tc_fence_before();
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[kOFree]);
                named_bar_sync(1, 32 * kRowWarps);
                const int len = (int)min((int64_t)C, it.t1 - t0);
                if (len == C) {
                    if (tid == 0) {
#pragma unroll
                        for (int x = 0; x < DVP / 64; ++x)
                            tma_store_3d(&to, sm + M::kS + x * 16384, 64 * x, h, (int32_t)t0);
                        bulk_commit();
                        bulk_wait_read_all();
                    }
                } else {   // rows past the segment belong to others
                    const int per = dv / 8;
                    for (int x = tid; x < len * per; x += 32 * kRowWarps) {
                        const int r = x / per, j = 8 * (x - r * per);
                        *reinterpret_cast<uint4 *>(o + ((t0 + r) * p.H + h) * (int64_t)dv + j) =
                            *reinterpret_cast<const uint4 *>(sm + M::kS + sw128_offset(r, j, C));
                    }
                    named_bar_sync(1, 32 * kRowWarps);
                }
                if (tid == 0) mbar_arrive(&bar[kSFree]);
            }
        } else if (warp < kRowWarps + kStateWarps) {
            constexpr int NC = DVP / 2;
            const int bt = tid - 32 * kRowWarps;
            const int half = bt >> 7, r = bt & 127;           // token row and half of its channels
            const int i = 32 * (warp & 3) + lane;             // state row, columns j0 ..
            const int j0 = NC * ((warp - kRowWarps) >> 2);
            const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
            const bool mine = i < dk && j0 < dv;
            const int64_t at = (int64_t)i * dv + j0;
            float S[NC];
            const float *start = OUT ? start_state(p, it, range, h0, bnd, dkdv) : nullptr;
#pragma unroll
            for (int j = 0; j < NC; j += 4) {
                const float4 x = start && mine ? *reinterpret_cast<const float4 *>(start + at + j)
                                               : make_float4(0.f, 0.f, 0.f, 0.f);
                S[j] = x.x; S[j + 1] = x.y; S[j + 2] = x.z; S[j + 3] = x.w;
            }
            // the image of S for chunk number `gn`, once the outputs of the one before have left
            auto put_image = [&](uint32_t gn) {
                const bool free = gn == 0 || wait(kSFree, (gn - 1) & 1);
                if (!__all_sync(0xffffffffu, free)) return false;
                if (i < DKP) {
#pragma unroll
                    for (int j = 0; j < NC; j += 8) {
                        uint4 u;
                        u.x = pack2(S[j], S[j + 1]);
                        u.y = pack2(S[j + 2], S[j + 3]);
                        u.z = pack2(S[j + 4], S[j + 5]);
                        u.w = pack2(S[j + 6], S[j + 7]);
                        *reinterpret_cast<uint4 *>(sm + M::kS + sw128_offset(i, j0 + j, DKP)) = u;
                    }
                }
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[kSReady]);
                return true;
            };
            if (OUT) ok = put_image(gi);
            for (int c = 0; c < chunks && ok; ++c, ++gi) {
                const uint32_t b = gi & 1, ph = (gi >> 1) & 1;
                const int len = (int)min((int64_t)C, it.t1 - it.t0 - (int64_t)c * C);
                uint8_t *stage = sm + b * M::kStage;
                // K and Q are read by Q K^T and Q S; after these K~ takes their place
                ok = wait(kGate + b, ph) && wait(kFull + b, ph) && (!OUT || wait(kQsDone, gi & 1));
                if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                const float w = gates[b].w[r];
                const float decay = tot[b];
                constexpr int UK = DKP / 16, UV = DVP / 16;   // 16-byte pieces of a thread
#pragma unroll 1
                for (int u = 0; u < UK; u += 4) {   // four in flight
                    uint4 x[4];
#pragma unroll
                    for (int m = 0; m < 4; ++m)
                        x[m] = *reinterpret_cast<const uint4 *>(
                            stage + M::kK + sw128_offset(r, 8 * (half * UK + u + m), C));
#pragma unroll
                    for (int m = 0; m < 4; ++m) {
                        uint4 hi = make_uint4(0, 0, 0, 0), lo = hi;
                        if (r < len) {
                            split2(x[m].x, w, hi.x, lo.x);
                            split2(x[m].y, w, hi.y, lo.y);
                            split2(x[m].z, w, hi.z, lo.z);
                            split2(x[m].w, w, hi.w, lo.w);
                        }
                        const uint32_t off = sw128_offset(r, 8 * (half * UK + u + m), C);
                        *reinterpret_cast<uint4 *>(stage + M::kK + off) = hi;
                        *reinterpret_cast<uint4 *>(stage + M::kQ + off) = lo;
                    }
                }
                if (r >= len) {   // rows of other sequences must not meet the zeros of P and K~
#pragma unroll 1
                    for (int u = 0; u < UV; ++u)
                        *reinterpret_cast<uint4 *>(stage + M::kV +
                                                   sw128_offset(r, 8 * (half * UV + u), C)) =
                            make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&bar[kKtReady]);
                    mbar_arrive(&bar[kGateFree + b]);
                }
                ok = wait(kKvDone + b, ph);
                if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                tc_fence_after();
#pragma unroll
                for (int jb = 0; jb < NC; jb += 32) {
                    float x[32];
                    tmem_ld32(tKV + lanes + j0 + jb, x);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 32; ++j) S[jb + j] = decay * S[jb + j] + x[j];
                }
                tc_fence_before();
                if (OUT && c + 1 < chunks) ok = put_image(gi + 1);
            }
            float *dst = OUT ? (it.c1 == it.nc && hT ? hT + ((int64_t)it.n * p.H + h) * dkdv
                                                     : nullptr)
                             : bnd + cut_state(range + 1) * dkdv;
            if (ok && dst && mine) {
#pragma unroll
                for (int j = 0; j < NC; j += 4)
                    *reinterpret_cast<float4 *>(dst + at + j) =
                        make_float4(S[j], S[j + 1], S[j + 2], S[j + 3]);
            }
        } else if (warp == kMmaWarp) {
            const uint32_t id_kk = idesc_bf16(128, 128, false, false);   // Q K^T
            const uint32_t id_km = idesc_bf16(128, DVP, false, true);    // Q S, P V
            const uint32_t id_mm = idesc_bf16(128, DVP, true, true);     // K~^T V
            for (int c = 0; c < chunks; ++c, ++gi) {
                const uint32_t b = gi & 1, ph = (gi >> 1) & 1;
                const int len = (int)min((int64_t)C, it.t1 - it.t0 - (int64_t)c * C);
                const uint32_t stage = base + b * M::kStage;
                const uint64_t dq = sdesc_sw128(stage + M::kQ, 16, 1024);
                const uint64_t dkk = sdesc_sw128(stage + M::kK, 16, 1024);
                // token-major tiles as operands whose K dimension is the token
                const uint64_t dkt = sdesc_sw128(stage + M::kK, C * 128, 1024);
                const uint64_t dlo = sdesc_sw128(stage + M::kQ, C * 128, 1024);
                const uint64_t dvt = sdesc_sw128(stage + M::kV, C * 128, 1024);
                const uint64_t ds = sdesc_sw128(base + M::kS, DKP * 128, 1024);
                if (OUT) {
                    ok = wait(kFull + b, ph) &&
                         (gi == 0 || wait(kPvDone + (b ^ 1), ((gi - 1) >> 1) & 1));
                    if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int s = 0; s < DKP / 16; ++s)
                            umma_bf16(tA, desc_add(dq, (s >> 2) * 16384 + (s & 3) * 32),
                                      desc_add(dkk, (s >> 2) * 16384 + (s & 3) * 32), id_kk, s > 0);
                        umma_commit(&bar[kQkDone]);
                    }
                    __syncwarp();
                    ok = wait(kSReady, gi & 1) && (gi == 0 || wait(kOFree, (gi - 1) & 1));
                    if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int s = 0; s < DKP / 16; ++s)
                            umma_bf16(tQS, desc_add(dq, (s >> 2) * 16384 + (s & 3) * 32),
                                      desc_add(ds, s * 2048), id_km, s > 0);
                        umma_commit(&bar[kQsDone]);
                    }
                    __syncwarp();
                    // (the rows of V past the segment are cleared together with K~)
                    ok = wait(kPReady, gi & 1) && (len == C || wait(kKtReady, gi & 1));
                    if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int s = 0; s < C / 16; ++s)
                            umma_bf16_ts(tPV, tA + 8 * s, desc_add(dvt, s * 2048), id_km, s > 0);
                        umma_commit(&bar[kPvDone + b]);
                    }
                    __syncwarp();
                }
                ok = wait(kKtReady, gi & 1);
                if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int s = 0; s < C / 16; ++s)
                        umma_bf16(tKV, desc_add(dkt, s * 2048), desc_add(dvt, s * 2048), id_mm, s > 0);
#pragma unroll
                    for (int s = 0; s < C / 16; ++s)
                        umma_bf16(tKV, desc_add(dlo, s * 2048), desc_add(dvt, s * 2048), id_mm, 1);
                    umma_commit(&bar[kKvDone + b]);
                }
                __syncwarp();
            }
        } else if (warp == kLoadWarp) {
            const int hk = h / group;
            for (int c = 0; c < chunks; ++c, ++gi) {
                const uint32_t b = gi & 1;
                if (gi >= 2) {
                    ok = wait(kKvDone + b, ((gi - 2) >> 1) & 1);
                    if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                }
                if (lane == 0) {
                    uint8_t *stage = sm + b * M::kStage;
                    uint64_t *full = &bar[kFull + b];
                    const int32_t t0 = (int32_t)(it.t0 + (int64_t)c * C);
                    mbar_arrive_expect_tx(full, M::kStage - (OUT ? 0 : M::kK));
#pragma unroll
                    for (int x = 0; x < DKP / 64; ++x) {
                        if (OUT) tma_load_3d(stage + M::kQ + x * 16384, &tq, 64 * x, hk, t0, full);
                        tma_load_3d(stage + M::kK + x * 16384, &tk, 64 * x, hk, t0, full);
                    }
#pragma unroll
                    for (int x = 0; x < DVP / 64; ++x)
                        tma_load_3d(stage + M::kV + x * 16384, &tv, 64 * x, h, t0, full);
                }
                loaded = gi + 1;
                __syncwarp();
            }
        } else if (warp == kGateWarp) {
            float log_sum = 0.f;
            for (int c = 0; c < chunks; ++c, ++gi) {
                const uint32_t b = gi & 1;
                const int64_t t0 = it.t0 + (int64_t)c * C;
                const int len = (int)min((int64_t)C, it.t1 - t0);
                float x[4], pre[4], suf[4];
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const int s = 4 * lane + m;
                    x[m] = s < len ? (g_per_token ? g[(t0 + s) * p.H + h] : g[h]) : 0.f;
                }
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    if (!log_decay_ok(x[m]))
                        report(st, KDA_ERR_DECAY_RANGE,
                               g_per_token ? (t0 + 4 * lane + m) * p.H + h : h, 30);
                    const float y = x[m] < kLogZero ? kLogZero : x[m];
                    pre[m] = m ? pre[m - 1] + y : y;
                }
                const float all = x[0] + x[1] + x[2] + x[3];
                float up = pre[3], down = all;   // inclusive scans over the lanes
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const float a = __shfl_up_sync(0xffffffffu, up, d);
                    const float e = __shfl_down_sync(0xffffffffu, down, d);
                    if (lane >= d) up += a;
                    if (lane + d < 32) down += e;
                }
                float before = __shfl_up_sync(0xffffffffu, up, 1);
                float after = __shfl_down_sync(0xffffffffu, down, 1);
                if (lane == 0) before = 0.f;
                if (lane == 31) after = 0.f;
                suf[3] = after;
#pragma unroll
                for (int m = 2; m >= 0; --m) suf[m] = suf[m + 1] + x[m + 1];
#pragma unroll
                for (int m = 0; m < 4; ++m) pre[m] = (pre[m] + before) * kLog2e;
                const float R = __shfl_sync(0xffffffffu, pre[3], lane | 7);   // end of the block
                const float total = __shfl_sync(0xffffffffu, down, 0);
                log_sum += total;
                if (gi >= 2) {
                    ok = wait(kGateFree + b, ((gi - 2) >> 1) & 1);
                    if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                }
                Gates &G = gates[b];
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const int s = 4 * lane + m;
                    G.G[s] = pre[m];
                    G.w[s] = expf(suf[m]);
                    if (s < 96) G.cf[s] = ex2(R - pre[m]);
                }
                if (lane == 0) tot[b] = expf(total);
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[kGate + b]);
            }
            if (!OUT && ok && lane == 0) bnd_log[cut_state(range + 1)] = log_sum;
        }
        if (!ok) {
            *abort_flag = 1;
            if (lane == 0) report(st, KDA_ERR_TIMEOUT, range, 41 + warp);
        }
    }
    __syncthreads();
    if (*abort_flag) {
        // an expired wait: what is in flight ends (each wait bounded again) before the tensor
        // memory is released and the CTA leaves
        if (warp == kMmaWarp) {
            tc_fence_after();
            if (elect_one()) umma_commit(&bar[kDrain]);
            __syncwarp();
            mbar_wait(&bar[kDrain], 0, kWaitNs);
        }
        if (warp == kLoadWarp) {
            landed = loaded >= 2 ? loaded - 2 : 0;
            for (; landed < loaded; ++landed)
                mbar_wait(&bar[kFull + (landed & 1)], (landed >> 1) & 1, kWaitNs);
        }
        __syncthreads();
    }
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, kCols);
    }
}

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                   const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                   const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
static EncodeTiledFn encode_tiled() {
    static EncodeTiledFn fn = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000,
                                             cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<EncodeTiledFn>(f);
    }();
    return fn;
}

// [T, heads, D] bf16, tokens `stride` elements apart, in boxes of 128 tokens x 1 head x 64
// channels with the 128-byte swizzle; what lies outside (channels of 32-wide heads, tokens
// past the last) reads as zeros.
static cudaError_t tensor_map(CUtensorMap *m, const void *x, int64_t T, int heads, int D,
                              int64_t stride) {
    EncodeTiledFn enc = encode_tiled();
    if (!enc) return cudaErrorNotSupported;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)T};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)stride * 2};
    const cuuint32_t box[3] = {64, 1, C};
    const cuuint32_t estr[3] = {1, 1, 1};
    const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(x), dims,
                           strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Shared memory above 48 KB, once per kernel and device.
template <int DKP, int DVP, bool OUT> static cudaError_t allow_smem(int dev) {
    static std::mutex mutex;
    static bool done[64] = {};
    std::lock_guard<std::mutex> lock(mutex);
    if (dev >= 0 && dev < 64 && done[dev]) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(la_chunk_tc_kernel<DKP, DVP, OUT>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)Map<DKP, DVP>::kBytes);
    if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev] = true;
    return e;
}

template <int DKP, int DVP, bool OUT>
static cudaError_t launch(const Plan &p, const CUtensorMap (&m)[4], const float *g, int gpt,
                          const float *h0, float *hT, void *o, int dk, int dv, float *bnd,
                          float *bnd_log, StatusWord *st, cudaStream_t s) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = allow_smem<DKP, DVP, OUT>(dev);
    if (e != cudaSuccess) return e;
    la_chunk_tc_kernel<DKP, DVP, OUT>
        <<<OUT ? p.ranges : p.ranges - 1, kThreads, Map<DKP, DVP>::kBytes, s>>>(
            p, m[0], m[1], m[2], m[3], g, gpt, h0, hT, (__nv_bfloat16 *)o, dk, dv, bnd, bnd_log, st);
    return cudaGetLastError();
}

}  // namespace tc
}  // namespace la

cudaError_t la_tensor_maps(CUtensorMap (&m)[4], const void *q, const void *k, const void *v,
                           const void *o, int64_t T, int H, int Hk, int dk, int dv, int64_t qs, int64_t ks,
                           int64_t vs) {
    cudaError_t e = la::tc::tensor_map(&m[0], q, T, Hk, dk, qs);
    if (e == cudaSuccess) e = la::tc::tensor_map(&m[1], k, T, Hk, dk, ks);
    if (e == cudaSuccess) e = la::tc::tensor_map(&m[2], v, T, H, dv, vs);
    if (e == cudaSuccess) e = la::tc::tensor_map(&m[3], o, T, H, dv, (int64_t)H * dv);
    return e;
}

cudaError_t launch_la_tc(bool out, const la::Plan &p, const CUtensorMap (&m)[4], const float *g,
                         int gpt, const float *h0, float *hT, void *o, int dk, int dv, float *bnd,
                         float *bnd_log, StatusWord *st, cudaStream_t s) {
#define KDA_LA(DK_, DV_)                                                                          \
    if ((dk <= 64) == (DK_ == 64) && (dv <= 64) == (DV_ == 64))                                   \
        return out ? la::tc::launch<DK_, DV_, true>(p, m, g, gpt, h0, hT, o, dk, dv, bnd, bnd_log, \
                                                    st, s)                                        \
                   : la::tc::launch<DK_, DV_, false>(p, m, g, gpt, h0, hT, o, dk, dv, bnd, bnd_log, \
                                                     st, s);
    KDA_LA(64, 64) KDA_LA(64, 128) KDA_LA(128, 64) KDA_LA(128, 128)
#undef KDA_LA
    return cudaErrorInvalidValue;
}

}  // namespace kda
