// la_chunk_tc.cu -- linear attention with one decay per head on the sm_103a tensor cores
// (bf16 operands, fp32 accumulation), 128-token chunks, dk and dv up to 128.
//
// Inside a chunk that starts from state S, with G_t = g_1 + ... + g_t and C tokens:
//   P  = (Q K^T) * exp(G_t - G_s) for s <= t, else 0
//   O  = P V + exp(G_t) Q S
//   S' = exp(G_C) S + K~^T V,     K~_s = exp(g_{s+1} + ... + g_C) k_s
// Five products of 128 x 128 x 128 a chunk (K~ counts twice): 164 kflop a token and head
// against 1 KB of q, k, v and o, half of what the tensor cores do in the time that the memory
// takes.
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
// for the blocks before that of t, and is formed token by token inside t's own block.  A reset (-inf)
// counts as -104 in G, so behind many of them its last bit is larger: 1e-4 of the outputs at a reset
// every two tokens (emulated), against 2e-3 of their rounding to bf16.
//
// One CTA an SM walks its range (see kda_la.cuh), every role for itself through the same
// items and chunks:
//   warps 0-3    rows of P (tensor memory, as the A operand of P V) and of O
//   warps 4-11   K~^T (read transposed, weighted and split into tensor memory as the A operand
//                of K~^T V) and the state: thread (row, half) holds its columns of S
//   warp 12      issues the products          warp 13   loads q, k, v (two stages)
//   warp 14      the chunk's decays, one chunk ahead
//   warp 15      stores O and final states by bulk copies of whole tiles (1.6k cycles a chunk; done
//                by plain stores they hold up everyone's shared memory meanwhile)
// Two stages of q, k and v (32 KB each, each free as soon as its own readers are done) and the
// 32 KB image of S fill the SM's shared memory; scores / P, O, K~^T V and K~^T (hi, lo) fill
// its tensor memory.  Loops stay loops: the roles' code shares one instruction cache
// (unrolled, a chunk took 13k cycles), and what a role keeps in registers stays near its 128 (the
// compiler reports 60 bytes of spills a thread in the output kernels of 128 value columns; local memory
// is shared by 512 threads in 28 KB of L1, and with the items' walk in it a call took 20% longer).
//
// What bounds it.  Outputs take 4.5k cycles a chunk: 2.6k of products on the tensor cores, among
// dependent steps of 0.2 to 1.2k (scores -> P -> outputs; K~^T V -> S -> its image -> Q S).
// Reading and writing the tiles alone takes 3.9k where four heads share queries and keys and
// 6.0k where none do (6.2 TB/s), less what the first pass left in L2.  The first pass (K~^T V
// only) takes 2.9k, its tiles at 6.4 TB/s.  Measured: 36k packed tokens of 32 heads on 8
// query/key heads 203 us, 65536 tokens of 16 heads 277 us (first pass 100), 8192 tokens of 32 heads
// 86 us (first pass 29, of which 6 before the first product).
#include <cuda.h>
#include <string.h>

#include <mutex>

#include "kda_la.cuh"
#include "kda_sm100.cuh"

namespace kda {
namespace la {
namespace tc {

using namespace sm100;

constexpr int C = kTcChunk;
constexpr int kThreads = 512;
constexpr int kRowWarps = 4, kStateWarps = 8;
constexpr int kMmaWarp = 12, kLoadWarp = 13, kGateWarp = 14, kStoreWarp = 15;
constexpr uint64_t kHandedNs = 1000000000ull;   // limit of the wait for a state that is handed on
constexpr uint64_t kDrainNs = 100000000ull;     // ... for what a CTA that gives up has in flight

// What one chunk's decays give, for one stage.
struct Gates {
    float G[C];        // prefix sums times log2(e)
    // w_s = exp(g_{s+1} + ... + g_C) as the sum of two bf16, in pairs of tokens: hi, lo
    uint2 w[C / 2];
    float cf[96];      // exp(R - G_s); the last block needs none
};

enum Bar {
    kFullQ = 0,      // [2] a stage's q has landed
    kFullK = 2,      // [2] k (or a start state, over both)
    kFullV = 4,      // [2] v
    kFreeQ = 6,      // [2] q has been read, and half of a final state that took its place has left
    kFreeK = 8,      // [2] k (or a start state) has been read
    kFreeV = 10,     // [2] v has, and the outputs that took its place have left
    kGate = 12,      // [2] a chunk's decays are there
    kGateFree = 14,  // [2] ... and have been used
    kKtReady = 16,   // [2] K~^T is in tensor memory, a half of each 64 tokens at a time (without
                     //     outputs: whole, two buffers)
    kKvDone = 18,    // [2] K~^T V of a half, of both (of a buffer)
    kQkDone = 20,    // Q K^T
    kQsDone = 21,    // Q S
    kPvDone = 22,    // P V
    kPReady = 23,    // P and the decayed Q S are in tensor memory
    kSReady = 24,    // the image of S is in shared memory
    kOFree = 25,     // [2] the accumulator of O has been read: the outputs are in shared memory
    kEndReady = 27,  // an item's final state is in shared memory
    kEndFree = 28,   // ... and has left the place of the image of S
    kStartRead = 29, // [2] a start state has been read out of its stage
    kBars = 31
};

// Two stages of q, k and v, the image of S ([DKP rows][DVP]), the decays.  A start state (fp32, in
// 32-column blocks of 128-byte rows) takes the place of q and k, a final state that of the
// image of S and of q.  A chunk's outputs are laid out for their store over its v, which is read
// last and needed last (over q, they held up the load of the next but one: 5.0k cycles a chunk).
template <int DKP, int DVP> struct Map {
    static constexpr uint32_t kQ = 0, kK = DKP * 256, kQK = 2 * DKP * 256;   // within a stage
    static constexpr uint32_t kV = 2 * kQK, kVBytes = DVP * 256;
    static constexpr uint32_t kS = kV + 2 * kVBytes;
    static constexpr uint32_t kGates = kS + DKP * DVP * 2;
    static constexpr uint32_t kTot = kGates + 2 * sizeof(Gates);   // decay of the chunk, [2]; at first the TMEM slot
    static constexpr uint32_t kBar = kTot + 8;
    static constexpr uint32_t kBytes = kBar + kBars * 8;
    static_assert(kBar % 8 == 0 && kS % 1024 == 0 && kQK % 1024 == 0 && kV % 1024 == 0 &&
                      kBytes <= 232448 && DKP * DVP * 4 <= kQK && DKP * DVP * 2 <= kK,
                  "layout");
};

// A in tensor memory (lane = row, column c = K elements 2 c and 2 c + 1)
__device__ __forceinline__ void umma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc,
                                             uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d_tmem), "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
#define KDA_R16(r)                                                                              \
    "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),     \
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
// the warp's 32 lanes, 16 consecutive columns: thread = lane
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
        ::"r"(taddr), KDA_R16(r)
        : "memory");
}
// 16 lanes, 8 consecutive columns: register 2 i + j of thread t is lane t / 4 + 8 j, column
// 4 i + t % 4
__device__ __forceinline__ void tmem_st_16x8(uint32_t taddr, const uint32_t (&r)[4]) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1,%2,%3,%4};"
                 ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
                 : "memory");
}
#undef KDA_R16
__device__ __forceinline__ void tmem_st_wait() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// Four 8 x 8 blocks of 16-bit values, transposed: thread t gets row t / 4, columns 2 (t % 4)
// and the next, of each
__device__ __forceinline__ void ldmatrix_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
// shared -> global through a tensor map (full boxes; what lies outside the tensor is dropped)
__device__ __forceinline__ void tma_store_3d(const void *tmap, uint32_t src, int32_t c0, int32_t c1,
                                             int32_t c2) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];"
                 ::"l"(tmap), "r"(c0), "r"(c1), "r"(c2), "r"(src)
                 : "memory");
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&x);
}
// two products in one instruction
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "mul.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
// 2^x by the special-function unit (relative error near 2^-22)
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
constexpr float kLog2e = 1.4426950408889634f;

// x: two bf16 of successive tokens, w their weights (hi, lo); hi + lo = w x but for 2^-17 of it:
// x w.hi less its own rounding is a bf16 exactly, so the second line loses nothing, and the
// third rounds what is 2^-8 of the product.
__device__ __forceinline__ void split2(uint32_t x, uint2 w, uint32_t &hi, uint32_t &lo) {
    const __nv_bfloat162 v = *reinterpret_cast<const __nv_bfloat162 *>(&x);
    const __nv_bfloat162 wh = *reinterpret_cast<const __nv_bfloat162 *>(&w.x);
    const __nv_bfloat162 wl = *reinterpret_cast<const __nv_bfloat162 *>(&w.y);
    const __nv_bfloat162 h = __hmul2(v, wh);
    const __nv_bfloat162 rest = __hfma2(v, wh, __hneg2(h));
    const __nv_bfloat162 l = __hfma2(v, wl, rest);
    hi = *reinterpret_cast<const uint32_t *>(&h);
    lo = *reinterpret_cast<const uint32_t *>(&l);
}

// Waits that end, after two seconds or a little more: what is behind the wait for a state that is
// handed on gives up after it.
struct Waits {
    uint32_t bar;   // shared-memory address of the first barrier
    // A whole warp on one barrier: its tries sleep in hardware (3.7 us, measured where nothing
    // arrives), so they are counted: 2.2 s.  Small code, for there are many of them.
    __device__ __forceinline__ bool warp(int which, uint32_t parity) const {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t.reg .u32 i;\n\t"
            "mov.u32 i, 0;\n"
            "again_%=:\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "@p bra done_%=;\n\t"
            "add.u32 i, i, 1;\n\t"
            "setp.lt.u32 q, i, 600000;\n\t"
            "@q bra again_%=;\n"
            "done_%=:\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar + 8 * which), "r"(parity)
            : "memory");
        return __all_sync(0xffffffffu, ok != 0);
    }
    // Several at a time, a lane each: beside the products' reads of shared memory each look at a
    // barrier takes 200 cycles, so they are not taken in turn.  Such tries do not sleep (70 to 100
    // ns each), so time is what is counted: t counts tries in its lowest 8 bits, every 256th looks
    // at the clock, and the first look stands in the bits above.  (In all waits this is too much code
    // for the instruction cache: packed prompts 8% slower.)
    __device__ __forceinline__ bool lanes(int which, uint32_t parity) const {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t.reg .u32 t, now;\n\t"
            "mov.u32 t, 0;\n"
            "again_%=:\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "@p bra done_%=;\n\t"
            "add.u32 t, t, 1;\n\t"
            "and.b32 now, t, 255;\n\t"
            "setp.ne.u32 q, now, 0;\n\t"
            "@q bra again_%=;\n\t"
            "mov.u32 now, %%globaltimer_lo;\n\t"
            "setp.eq.u32 q, t, 256;\n\t"
            "@q and.b32 t, now, 0xffffff00;\n\t"
            "sub.u32 now, now, t;\n\t"
            "setp.lt.u32 q, now, 2000000000;\n\t"
            "@q bra again_%=;\n"
            "done_%=:\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar + 8 * which), "r"(parity)
            : "memory");
        return __all_sync(0xffffffffu, ok != 0);
    }
    __device__ __forceinline__ bool warp(int w0, uint32_t p0, int w1, uint32_t p1) const {
        const bool one = threadIdx.x & 1;
        return lanes(one ? w1 : w0, one ? p1 : p0);
    }
    __device__ __forceinline__ bool warp(int w0, uint32_t p0, int w1, uint32_t p1, int w2, uint32_t p2,
                                         int w3, uint32_t p3) const {
        const bool one = threadIdx.x & 1, two = threadIdx.x & 2;
        const int wa = two ? w2 : w0, wb = two ? w3 : w1;
        const uint32_t pa = two ? p2 : p0, pb = two ? p3 : p1;
        return lanes(one ? wb : wa, one ? pb : pa);
    }
};

// OUT: outputs and final states of the CTA's range.  Else what the end of the range leaves at
// the cut behind it (only K~^T V; no queries): from its last chunk to its first, so that the
// chunks which the output pass reads first are the ones that L2 still holds, with weights that
// reach to the cut, so that nothing is decayed on the way.
template <int DKP, int DVP, bool OUT>
__global__ void __launch_bounds__(kThreads, 1)
la_chunk_tc_kernel(Plan p, const __grid_constant__ CUtensorMap tq,
                   const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                   const __grid_constant__ CUtensorMap to, const __grid_constant__ CUtensorMap to8,
                   const __grid_constant__ CUtensorMap th0,
                   const __grid_constant__ CUtensorMap thT, const __grid_constant__ CUtensorMap tbnd,
                   const float *__restrict__ g, int g_per_token, int has_h0, int has_hT,
                   __nv_bfloat16 *__restrict__ o, int dk, int dv, float *__restrict__ bnd,
                   float *__restrict__ bnd_log, StatusWord *st) {
    extern __shared__ __align__(1024) uint8_t sm[];
    using M = Map<DKP, DVP>;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    let_next_start();
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + M::kBar);
    Gates *gates = reinterpret_cast<Gates *>(sm + M::kGates);
    float *tot = reinterpret_cast<float *>(sm + M::kTot);
    uint32_t *tslot = reinterpret_cast<uint32_t *>(sm + M::kTot);
    const uint32_t base = smem_u32(sm);
    if (base & 1023u) {   // the operand images need their alignment
        wait_for_previous();
        if (tid == 0) report(st, KDA_ERR_CUDA, 0, 40);
        return;
    }
    if (tid == 0) {
        for (int b = 0; b < 2; ++b) {
            mbar_init(&bar[kFullQ + b], 1);
            mbar_init(&bar[kFullK + b], 1);
            mbar_init(&bar[kFullV + b], 1);
            mbar_init(&bar[kFreeQ + b], 1);
            mbar_init(&bar[kFreeK + b], 1);
            mbar_init(&bar[kFreeV + b], 1);
            mbar_init(&bar[kGate + b], 1);
            mbar_init(&bar[kGateFree + b], kStateWarps + (OUT ? kRowWarps : 0));
            mbar_init(&bar[kKtReady + b], kStateWarps);
            mbar_init(&bar[kKvDone + b], 1);
            mbar_init(&bar[kStartRead + b], kStateWarps);
            mbar_init(&bar[kOFree + b], kRowWarps);
        }
        mbar_init(&bar[kQkDone], 1);
        mbar_init(&bar[kQsDone], 1);
        mbar_init(&bar[kPvDone], 1);
        mbar_init(&bar[kPReady], kRowWarps);
        mbar_init(&bar[kSReady], kStateWarps);
        mbar_init(&bar[kEndReady], kStateWarps);
        mbar_init(&bar[kEndFree], 1);
        fence_mbar_init();
    }
    constexpr uint32_t kCols = 512;
    if (warp == kMmaWarp) {
        tmem_alloc(tslot, kCols);
        tmem_relinquish();
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;
    // (so far nothing that another kernel has written)
    wait_for_previous();
    int place = blockIdx.x;
    if (OUT && p.flags) {   // in the order in which the CTAs begin: a range may wait for the one before
        if (tid == 0) place = atomicAdd(&p.flags[p.ranges * p.lanes], 1);
        __syncthreads();   // (all have read the slot)
        if (tid == 0) *tslot = place;
        __syncthreads();
        place = *tslot;
    }
    __syncthreads();   // the slot has been read by all: from here on its place is a chunk's decay
    const int range = place / p.lanes, side = place % p.lanes;
    const bool work = OUT ? p.cuts[range].x < p.cuts[range + 1].x
                          : p.cuts[range + 1].inner != 0 && !p.cuts[range + 1].handed;
    // K~^T (hi, lo) and K~^T V; then, of a second chunk's, or scores (then P) and O
    const uint32_t tHi = tmem, tLo = tmem + 64, tKV = tmem + 128;
    constexpr uint32_t kOther = 256;
    const uint32_t tA = tmem + 256, tO = tmem + 384;
    const Waits wait{smem_u32(bar)};
    const int64_t dkdv = (int64_t)dk * dv;
    uint32_t gi = 0;    // chunks so far: stages of v, and parities of what happens once a chunk
    uint32_t si = 0;    // stages of q and k so far (chunks and start states)
    bool ok = true;
    uint32_t issued_q = 0, issued_k = 0, issued_v = 0;   // (load warp)
    uint32_t start_in = 0, starts_read = 0;              // ... a bit a stage: holds a start state; parity of those
    uint32_t ends_before = 0;                            // (store and state warps) final states so far

    // Each role goes through the range's items for itself: role(item, its start, whether it has a
    // state to store at its end, which is a final state or one to hand on).
    auto each_item = [&](auto role) {
        if (!work) return;
        Item it;
        if (OUT) {
            Items items(p, range, side);
            while (ok && items.next(p, range, side, it))
                role(it, start_state(p, it, range, side, has_h0),
                     it.part == Item::kHead || (has_hT && it.c1 == it.nc));
        } else if (before_cut(p, range + 1, side, it)) {
            role(it, Start{}, false);
        }
    };
    constexpr int NC = DVP / 2;

    if (warp < kRowWarps) {
        if (OUT) each_item([&](const Item &it, const Start &start, bool ends) {
            const int chunks = it.c1 - it.c0;
            const int t = tid;   // this thread's row of the chunk
            const uint32_t lanes = (uint32_t)(32 * warp) << 16;
            for (int c = 0; c < chunks; ++c, ++gi) {
                const uint32_t b = gi & 1, ph = (gi >> 1) & 1;
                ok = wait.warp(kGate + b, ph);
                if (!ok) break;
                // All that depends on the decays alone while the scores are formed: the factors of
                // t's own block and, for the blocks before, exp(G_t - R).
                const Gates &G = gates[b];
                const float Gt = G.G[t];
                const float e = ex2(Gt);
                float r[3], own[32];
#pragma unroll
                for (int cb = 0; cb < 3; ++cb) r[cb] = ex2(Gt - G.G[32 * cb + 31]);
#pragma unroll
                for (int j = 0; j < 32; j += 4) {
                    const float4 f = *reinterpret_cast<const float4 *>(&G.G[32 * warp + j]);
                    own[j] = ex2(Gt - f.x);
                    own[j + 1] = ex2(Gt - f.y);
                    own[j + 2] = ex2(Gt - f.z);
                    own[j + 3] = ex2(Gt - f.w);
                }
                ok = wait.warp(kQkDone, gi & 1);
                if (!ok) break;
                tc_fence_after();
                // P, over scores that this warp has read: its own block first, kept until its
                // columns are free, then the blocks before.
                uint32_t mine[16];
                {
                    float a[32];
                    tmem_ld32(tA + lanes + 32 * warp, a);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 32; j += 2)   // (a score past t may be anything)
                        mine[j / 2] = pack2(j <= lane ? a[j] * own[j] : 0.f, j < lane ? a[j + 1] * own[j + 1] : 0.f);
                }
#pragma unroll 1
                for (int cb = 0; cb < warp; ++cb) {
                    const float rb = cb == 0 ? r[0] : cb == 1 ? r[1] : r[2];
                    const float2 rf = make_float2(rb, rb);
                    float a[32];
                    float4 f[8];
                    tmem_ld32(tA + lanes + 32 * cb, a);
#pragma unroll
                    for (int j = 0; j < 8; ++j) f[j] = *reinterpret_cast<const float4 *>(&G.cf[32 * cb + 4 * j]);
                    tmem_ld_wait();
                    uint32_t pk[16];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float2 x = mul2(make_float2(a[4 * j], a[4 * j + 1]), mul2(rf, make_float2(f[j].x, f[j].y)));
                        const float2 y = mul2(make_float2(a[4 * j + 2], a[4 * j + 3]), mul2(rf, make_float2(f[j].z, f[j].w)));
                        pk[2 * j] = pack2(x.x, x.y);
                        pk[2 * j + 1] = pack2(y.x, y.y);
                    }
                    tmem_st16(tA + lanes + 16 * cb, pk);
                }
                tmem_st16(tA + lanes + 16 * warp, mine);
#pragma unroll
                for (int j = 0; j < 16; ++j) mine[j] = 0;
#pragma unroll 1
                for (int cb = warp + 1; cb < 4; ++cb) tmem_st16(tA + lanes + 16 * cb, mine);
                ok = wait.warp(kQsDone, gi & 1);
                if (!ok) break;
                tc_fence_after();   // P V adds to exp(G_t) Q S
                const float2 eG = make_float2(e, e);
#pragma unroll 1
                for (int j0 = 0; j0 < DVP; j0 += 64) {
                    float x[2][32];
                    tmem_ld32(tO + lanes + j0, x[0]);
                    tmem_ld32(tO + lanes + j0 + 32, x[1]);
                    tmem_ld_wait();
#pragma unroll
                    for (int m = 0; m < 4; ++m) {
                        uint32_t y[16];
#pragma unroll
                        for (int j = 0; j < 16; j += 2) {
                            const float2 z = mul2(eG, make_float2(x[m / 2][16 * (m & 1) + j], x[m / 2][16 * (m & 1) + j + 1]));
                            y[j] = __float_as_uint(z.x);
                            y[j + 1] = __float_as_uint(z.y);
                        }
                        tmem_st16(tO + lanes + j0 + 16 * m, y);
                    }
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&bar[kPReady]);
                    mbar_arrive(&bar[kGateFree + b]);
                }
                ok = wait.warp(kPvDone, gi & 1);
                if (!ok) break;
                tc_fence_after();
                // the outputs, for the store warp
                uint8_t *so = sm + M::kV + b * M::kVBytes;
#pragma unroll 1
                for (int cb = 0; cb < DVP / 32; cb += 2) {
                    float x[2][32];
                    tmem_ld32(tO + lanes + 32 * cb, x[0]);
                    tmem_ld32(tO + lanes + 32 * cb + 32, x[1]);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 64; j += 8) {
                        const float *y = &x[j / 32][j % 32];
                        uint4 u;
                        u.x = pack2(y[0], y[1]);
                        u.y = pack2(y[2], y[3]);
                        u.z = pack2(y[4], y[5]);
                        u.w = pack2(y[6], y[7]);
                        *reinterpret_cast<uint4 *>(so + sw128_offset(t, 32 * cb + j, C)) = u;
                    }
                }
                tc_fence_before();
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[kOFree + b]);
            }
        });
    } else if (warp < kRowWarps + kStateWarps) {
        // state row i, columns j0 .. of half the columns
        const int quarter = warp & 3, half = ((warp - kRowWarps) >> 2) & 1;
        const int i = 32 * quarter + lane;                // state row, columns j0 ..
        const int j0 = NC * half;
        const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
        const bool mine = i < dk && j0 < dv;
        float S[NC];
#pragma unroll
        for (int j = 0; j < NC; ++j) S[j] = 0.f;
        bool image_taken = false;   // the image's place holds a final state
        // S as the final state of an item, for the store warp: over the image of S (first half of
        // the columns) and the last chunk's q, in 32-column blocks of 128-byte rows
        auto put_end = [&] {
            if (!wait.warp(kQsDone, (gi - 1) & 1)) return false;
            if (mine) {
                uint8_t *at = sm + (half ? ((si - 1) & 1) * M::kQK + M::kQ : M::kS);
#pragma unroll
                for (int j = 0; j < NC; j += 4)
                    *reinterpret_cast<float4 *>(at + (j / 32) * dk * 128 + i * 128 + ((((j % 32) / 4) ^ (i & 7)) << 4)) =
                        make_float4(S[j], S[j + 1], S[j + 2], S[j + 3]);
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[kEndReady]);
            __syncwarp();
            return true;
        };
        // S <- decay S + the product, from tensor memory
        auto add_product = [&](uint32_t other, float decay) {
#pragma unroll
            for (int jb = 0; jb < NC; jb += 32) {
                float x[32];
                tmem_ld32(tKV + other + lanes + j0 + jb, x);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 32; ++j) S[jb + j] = decay * S[jb + j] + x[j];
            }
        };
        each_item([&](const Item &it, const Start &start, bool ends) {
            const int chunks = it.c1 - it.c0;
            const uint32_t first_si = si;   // the start states' stages
            si += start.steps;
            // Round c ends chunk c (adds its product to S) and makes K~^T and the image of S for
            // chunk c + 1: the first half of K~^T while the second half's product still runs, the
            // image last.  (Without outputs, in two buffers: K~^T first.)
            float decay = 0.f, decay_next = 0.f;   // of chunk c, c + 1
            auto read_start = [&] {
#pragma unroll
                for (int j = 0; j < NC; ++j) S[j] = 0.f;
#pragma unroll 1
                for (int s = 0; s < start.steps; ++s) {
                    const uint32_t fs = first_si + s, fb = fs & 1;
                    ok = wait.warp(kFullK + fb, (fs >> 1) & 1);
                    if (!ok) return;
                    if (mine) {
                        const float e = s ? expf(bnd_log[start.index(s)]) : 0.f;
#pragma unroll
                        for (int j = 0; j < NC; j += 4) {
                            const int col = j0 + j;
                            const float4 x = *reinterpret_cast<const float4 *>(
                                sm + fb * M::kQK + (col / 32) * dk * 128 + i * 128 + ((((col % 32) / 4) ^ (i & 7)) << 4));
                            S[j] = e * S[j] + x.x;
                            S[j + 1] = e * S[j + 1] + x.y;
                            S[j + 2] = e * S[j + 2] + x.z;
                            S[j + 3] = e * S[j + 3] + x.w;
                        }
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar[kStartRead + fb]);
                    __syncwarp();
                }
            };
            // (a start of several states: they come through the stages before the first chunk)
            if (OUT && start.steps > 1) {
                read_start();
                if (!ok) return;
            }
            // (gi and si here: of chunk c + 1)
#pragma unroll 1
            for (int c = -1; c < chunks; ++c) {
                const uint32_t b = gi & 1, ph = (gi >> 1) & 1, sb = si & 1;
                const bool next = c + 1 < chunks;
                const int at_chunk = OUT ? c + 1 : chunks - 2 - c;
                const int len = next ? min(C, it.t1 - it.t0 - at_chunk * C) : C;
                if (next) {
                    const bool half_done = OUT && c >= 0;   // (K~^T of chunk c: its first half)
                    ok = wait.warp(kGate + b, ph, kFullK + sb, (si >> 1) & 1,
                                   half_done ? kKvDone : kGate + b, half_done ? (gi - 1) & 1 : ph,
                                   len < C ? kFullV + b : kGate + b, ph);
                    if (!ok) break;
                    tc_fence_after();
                    decay_next = OUT ? tot[b] : 1.f;
                }
#pragma unroll 1
                for (int u = 0; u < 2; ++u) {
                    if (next) {
                        // channels of this warp's quarter, tokens of its half, 32 x 32 a turn: all of a
                        // turn's reads first (they take 300 cycles beside the products')
                        if (32 * quarter < DKP) {
                            const int first = 64 * half + 32 * u;
                            uint32_t x[2][2][4];
                            uint2 w[2][2];
#pragma unroll
                            for (int m = 0; m < 2; ++m) {
#pragma unroll
                                for (int cg = 0; cg < 2; ++cg)
                                    ldmatrix_t(base + sb * M::kQK + M::kK +
                                                   sw128_offset(first + 16 * m + (lane >> 4) * 8 + (lane & 7),
                                                                32 * quarter + 16 * cg + ((lane >> 3) & 1) * 8, C),
                                               x[m][cg]);
                                w[m][0] = gates[b].w[first / 2 + 8 * m + (lane & 3)];
                                w[m][1] = gates[b].w[first / 2 + 8 * m + (lane & 3) + 4];
                            }
                            const uint32_t to_col = lanes + first / 2 + (OUT ? 0 : b * kOther);
#pragma unroll
                            for (int m = 0; m < 2; ++m) {
                                const int at = first + 16 * m + 2 * (lane & 3);   // and + 1, + 8, + 9
                                uint32_t m0 = ~0u, m1 = ~0u;
                                if (len < C) {   // tokens past the sequence count as zeros
                                    m0 = (at < len ? 0xffffu : 0u) | (at + 1 < len ? 0xffff0000u : 0u);
                                    m1 = (at + 8 < len ? 0xffffu : 0u) | (at + 9 < len ? 0xffff0000u : 0u);
                                }
#pragma unroll
                                for (int cg = 0; cg < 2; ++cg) {
                                    uint32_t hi[4], lo[4];
                                    split2(x[m][cg][0] & m0, w[m][0], hi[0], lo[0]);
                                    split2(x[m][cg][1] & m0, w[m][0], hi[1], lo[1]);
                                    split2(x[m][cg][2] & m1, w[m][1], hi[2], lo[2]);
                                    split2(x[m][cg][3] & m1, w[m][1], hi[3], lo[3]);
                                    tmem_st_16x8(tHi + to_col + ((uint32_t)cg << 20) + 8 * m, hi);
                                    tmem_st_16x8(tLo + to_col + ((uint32_t)cg << 20) + 8 * m, lo);
                                }
                            }
                        }
                        if (u == 0 && len < C) {   // their rows of V must not meet the zeros of P and K~
                            constexpr int U = DVP / 8;   // 16-byte pieces of a row
#pragma unroll 1
                            for (int x = len * U + (tid - 32 * kRowWarps); x < C * U; x += 32 * kStateWarps)
                                *reinterpret_cast<uint4 *>(sm + M::kV + b * M::kVBytes + sw128_offset(x / U, 8 * (x % U), C)) =
                                    make_uint4(0, 0, 0, 0);
                            fence_proxy_async();
                        }
                    }
                    if (OUT ? u == 0 && c >= 0 : false) {
                        ok = wait.warp(kKvDone + 1, (gi - 1) & 1);
                        if (!ok) break;
                        tc_fence_after();
                        add_product(0, decay);
                    }
                    if (next) {
                        if (32 * quarter < DKP) tmem_st_wait();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) {
                            if (OUT || u) mbar_arrive(&bar[kKtReady + (OUT ? u : b)]);
                            if (u) mbar_arrive(&bar[kGateFree + b]);
                        }
                        __syncwarp();
                    }
                    if (OUT && u == 0 && c < 0) {
                        if (start.steps <= 1) read_start();
                        if (ok && image_taken) ok = wait.warp(kEndFree, (ends_before - 1) & 1);
                        if (!ok) break;
                        image_taken = false;
                    }
                    if (OUT && u == 0 && next) {   // Q S of the chunk before has read the old image
                        ok = gi == 0 || wait.warp(kQsDone, (gi - 1) & 1);
                        if (!ok) break;
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
                        __syncwarp();
                    }
                }
                if (!ok) break;
                if (!OUT && c >= 0) {
                    ok = wait.warp(kKvDone + (b ^ 1), ((gi - 1) >> 1) & 1);
                    if (!ok) break;
                    tc_fence_after();
                    add_product((b ^ 1) * kOther, decay);
                    tc_fence_before();
                }
                decay = decay_next;
                if (next) {
                    ++gi;
                    ++si;
                }
            }
            if (ends && ok) {
                ok = put_end();
                image_taken = true;
                ++ends_before;
            }
            if (!OUT && ok && mine) {
                float *row = bnd + cut_state(p, range + 1, side) * dkdv + (int64_t)i * dv + j0;
#pragma unroll
                for (int j = 0; j < NC; j += 4)
                    *reinterpret_cast<float4 *>(row + j) = make_float4(S[j], S[j + 1], S[j + 2], S[j + 3]);
            }
        });
    } else if (warp == kMmaWarp) {
        each_item([&](const Item &it, const Start &start, bool ends) {
            const int chunks = it.c1 - it.c0;
            si += start.steps;
            const uint32_t id_kk = idesc_bf16(128, 128, false, false);   // Q K^T
            const uint32_t id_km = idesc_bf16(128, DVP, false, true);    // the others: B is V or S
            for (int c = 0; c < chunks; ++c, ++gi, ++si) {
                const uint32_t b = gi & 1, ph = (gi >> 1) & 1, sb = si & 1;
                const uint32_t qk = base + sb * M::kQK;
                const uint64_t dq = sdesc_sw128(qk + M::kQ, 16, 1024);
                const uint64_t dkk = sdesc_sw128(qk + M::kK, 16, 1024);
                // token-major V and channel-major S: the K dimension is the row
                const uint64_t dvt = sdesc_sw128(base + M::kV + b * M::kVBytes, C * 128, 1024);
                const uint64_t ds = sdesc_sw128(base + M::kS, DKP * 128, 1024);
                if (OUT) {
                    // A start of several states has been through both stages before this chunk:
                    // K~^T says that this is over, and that a parity names one phase again.
                    if (c == 0 && start.steps > 1) ok = wait.warp(kKtReady, gi & 1);
                    // P of the chunk before lies over the scores
                    const uint32_t landed = (si >> 1) & 1;
                    ok = ok && wait.warp(kFullK + sb, landed, kFullQ + sb, landed) &&
                         (gi == 0 || wait.warp(kPvDone, (gi - 1) & 1));
                    if (!ok) break;
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll 2
                        for (int s = 0; s < DKP / 16; ++s)
                            umma_bf16(tA, desc_add(dq, (s >> 2) * 16384 + (s & 3) * 32),
                                      desc_add(dkk, (s >> 2) * 16384 + (s & 3) * 32), id_kk, s > 0);
                        umma_commit(&bar[kQkDone]);
                    }
                    __syncwarp();
                    ok = wait.warp(kSReady, gi & 1, gi ? kOFree + (b ^ 1) : kSReady, gi ? ((gi - 1) >> 1) & 1 : gi & 1);
                    if (!ok) break;
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll 2
                        for (int s = 0; s < DKP / 16; ++s)
                            umma_bf16(tO, desc_add(dq, (s >> 2) * 16384 + (s & 3) * 32),
                                      desc_add(ds, s * 2048), id_km, s > 0);
                        umma_commit(&bar[kQsDone]);
                        if (!(ends && c + 1 == chunks)) umma_commit(&bar[kFreeQ + sb]);
                    }
                    __syncwarp();
                }
                const uint32_t other = OUT ? 0 : b * kOther;
#pragma unroll 1
                for (int u = 0; u < 2 && ok; ++u) {   // half of each 64 tokens
                    if (OUT || u == 0) {
                        ok = wait.warp(kKtReady + (OUT ? u : b), OUT ? gi & 1 : ph, kFullV + b, ph);
                        if (!ok) break;
                        tc_fence_after();
                    }
                    if (elect_one()) {
                        if (u) umma_commit(&bar[kFreeK + sb]);   // (Q K^T so far)
#pragma unroll 2
                        for (int j = 0; j < 4; ++j) {
                            const int s = 4 * (j >> 1) + 2 * u + (j & 1);
                            umma_bf16_ts(tKV + other, tHi + other + 8 * s, desc_add(dvt, s * 2048), id_km, u + j > 0);
                        }
#pragma unroll 2
                        for (int j = 0; j < 4; ++j) {
                            const int s = 4 * (j >> 1) + 2 * u + (j & 1);
                            umma_bf16_ts(tKV + other, tLo + other + 8 * s, desc_add(dvt, s * 2048), id_km, 1);
                        }
                        if (OUT || u) umma_commit(&bar[kKvDone + (OUT ? u : b)]);
                        if (!OUT && u) umma_commit(&bar[kFreeV + b]);
                    }
                    __syncwarp();
                }
                if (!ok) break;
                if (OUT) {
                    ok = wait.warp(kPReady, gi & 1);
                    if (!ok) break;
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll 2
                        for (int s = 0; s < C / 16; ++s)
                            umma_bf16_ts(tO, tA + 8 * s, desc_add(dvt, s * 2048), id_km, 1);
                        umma_commit(&bar[kPvDone]);
                    }
                    __syncwarp();
                }
            }
        });
        // nothing arrives at this CTA's barriers after it has left
        if (ok && gi) ok = wait.warp(kFreeV + ((gi - 1) & 1), ((gi - 1) >> 1) & 1);
    } else if (warp == kLoadWarp) {
        // (the states at the cuts were written by plain stores)
        if (OUT) asm volatile("fence.proxy.async.global;" ::: "memory");
        each_item([&](const Item &it, const Start &start, bool ends) {
            const int h = it.h, chunks = it.c1 - it.c0;
            const uint32_t first_si = si;   // the start states' stages
            si += start.steps;
            const int hk = h / (p.H / p.Hk);
            // a stage that holds a start state is free when that has been read
            auto behind_start = [&](uint32_t sb) {
                if (!(start_in >> sb & 1)) return true;
                const bool read = wait.warp(kStartRead + sb, (starts_read >> sb) & 1);
                starts_read ^= 1u << sb;
                start_in ^= 1u << sb;
                if (lane == 0) {
                    mbar_arrive(&bar[kFreeK + sb]);
                    mbar_arrive(&bar[kFreeQ + sb]);
                }
                __syncwarp();
                return read;
            };
            for (int s = 0; s < start.steps; ++s) {
                const uint32_t fs = first_si + s, sb = fs & 1, before = ((fs - 2) >> 1) & 1;
                ok = behind_start(sb);
                if (ok && fs >= 2) ok = wait.warp(kFreeK + sb, before, kFreeQ + sb, before);
                if (!ok) return;
                if (it.part == Item::kTail) {   // handed on by the range before
                    bool there = lane != 0;
                    const uint64_t t0 = globaltimer_ns();
                    for (uint32_t i = 1; !there; ++i) {
                        uint32_t flag;
                        asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(flag) : "l"(p.flags + start.index(s)) : "memory");
                        there = flag != 0;
                        if ((i & 63u) == 0 && globaltimer_ns() - t0 > kHandedNs) break;
                    }
                    ok = __all_sync(0xffffffffu, there);
                    if (!ok) return;
                    asm volatile("fence.proxy.async.global;" ::: "memory");
                }
                if (lane == 0) {
                    uint64_t *full = &bar[kFullK + sb];
                    mbar_arrive(&bar[kFullQ + sb]);
                    mbar_arrive_expect_tx(full, (uint32_t)dkdv * 4);
#pragma unroll 1
                    for (int x = 0; x < dv / 32; ++x)
                        tma_load_3d(sm + sb * M::kQK + x * dk * 128, start.in_bnd(s) ? &tbnd : &th0, 32 * x,
                                    0, start.index(s), full);
                }
                issued_k = fs + 1;
                start_in |= 1u << sb;
                __syncwarp();
            }
            for (int c = 0; c < chunks; ++c, ++gi, ++si) {
                const uint32_t b = gi & 1, sb = si & 1, before = ((si - 2) >> 1) & 1;
                const int32_t t0 = it.t0 + (OUT ? c : chunks - 1 - c) * C;
                uint8_t *qk = sm + sb * M::kQK;
                ok = behind_start(sb);
                if (ok && si >= 2) ok = wait.warp(kFreeK + sb, before);
                if (!ok) break;
                if (lane == 0 && !(gi == 0 && range * p.lanes + side == p.left_out)) {
                    uint64_t *full = &bar[kFullK + sb];
                    mbar_arrive_expect_tx(full, M::kK);
#pragma unroll
                    for (int x = 0; x < DKP / 64; ++x)
                        tma_load_3d(qk + M::kK + x * 16384, &tk, 64 * x, hk, t0, full);
                }
                issued_k = si + 1;
                __syncwarp();
                if (OUT) {
                    if (si >= 2) ok = wait.warp(kFreeQ + sb, before);
                    if (!ok) break;
                    if (lane == 0) {
                        uint64_t *full = &bar[kFullQ + sb];
                        mbar_arrive_expect_tx(full, M::kK);
#pragma unroll
                        for (int x = 0; x < DKP / 64; ++x)
                            tma_load_3d(qk + M::kQ + x * 16384, &tq, 64 * x, hk, t0, full);
                    }
                    issued_q = si + 1;
                    __syncwarp();
                }
                if (gi >= 2) ok = wait.warp(kFreeV + b, ((gi - 2) >> 1) & 1);
                if (!ok) break;
                if (lane == 0) {
                    uint64_t *full = &bar[kFullV + b];
                    mbar_arrive_expect_tx(full, M::kVBytes);
#pragma unroll
                    for (int x = 0; x < DVP / 64; ++x)
                        tma_load_3d(sm + M::kV + b * M::kVBytes + x * 16384, &tv, 64 * x, h, t0, full);
                }
                issued_v = gi + 1;
                __syncwarp();
            }
        });
    } else if (warp == kGateWarp) {
        each_item([&](const Item &it, const Start &start, bool ends) {
            const int h = it.h, chunks = it.c1 - it.c0;
            float log_sum = 0.f;
            for (int c = 0; c < chunks; ++c, ++gi, ++si) {
                const uint32_t b = gi & 1;
                const int64_t t0 = it.t0 + (OUT ? c : chunks - 1 - c) * C;
                const int len = (int)min((int64_t)C, it.t1 - t0);
                float x[4], pre[4], suf[4];
                int bad = -1;
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const int s = 4 * lane + m;
                    x[m] = s < len ? (g_per_token ? g[(t0 + s) * p.H + h] : g[h]) : 0.f;
                }
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    if (!log_decay_ok(x[m])) bad = m;
                    const float y = x[m] < kLogZero ? kLogZero : x[m];
                    pre[m] = m ? pre[m - 1] + y : y;
                }
                if (bad >= 0)
                    report(st, KDA_ERR_DECAY_RANGE, g_per_token ? (t0 + 4 * lane + bad) * p.H + h : h, 30);
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
                suf[3] = OUT ? after : after + log_sum;
#pragma unroll
                for (int m = 2; m >= 0; --m) suf[m] = suf[m + 1] + x[m + 1];
#pragma unroll
                for (int m = 0; m < 4; ++m) pre[m] = (pre[m] + before) * kLog2e;
                const float R = __shfl_sync(0xffffffffu, pre[3], lane | 7);   // end of the block
                const float total = __shfl_sync(0xffffffffu, down, 0);
                log_sum += total;
                if (gi >= 2) ok = wait.warp(kGateFree + b, ((gi - 2) >> 1) & 1);
                if (!ok) break;
                Gates &G = gates[b];
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const int s = 4 * lane + m;
                    G.G[s] = pre[m];
                    if (s < 96) G.cf[s] = ex2(R - pre[m]);
                }
#pragma unroll
                for (int m = 0; m < 4; m += 2) {
                    const float w0 = expf(suf[m]), w1 = expf(suf[m + 1]);
                    const uint32_t hi = pack2(w0, w1);
                    G.w[2 * lane + m / 2] = make_uint2(hi, pack2(w0 - __uint_as_float(hi << 16),
                                                                 w1 - __uint_as_float(hi & 0xffff0000u)));
                }
                if (OUT && lane == 0) tot[b] = expf(total);
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[kGate + b]);
            }
            if (!OUT && ok && lane == 0) bnd_log[cut_state(p, range + 1, side)] = log_sum;
        });
    } else if (OUT && warp == kStoreWarp) {
        each_item([&](const Item &it, const Start &start, bool ends) {
            const int h = it.h, chunks = it.c1 - it.c0;
            si += start.steps;
            for (int c = 0; c < chunks; ++c, ++gi, ++si) {
                const uint32_t b = gi & 1, sb = si & 1;
                const int64_t t0 = it.t0 + c * C;
                const int len = (int)min((int64_t)C, it.t1 - t0);
                const uint32_t so = M::kV + b * M::kVBytes;
                if (ends && c + 1 == chunks) {
                    // the final state, which is there before the outputs are, and first the half
                    // whose place the next item's queries wait for
                    ok = wait.warp(kEndReady, ends_before & 1);
                    if (!ok) break;
                    ++ends_before;
                    if (lane == 0) {
                        constexpr int kHalf = DVP / 64;   // blocks of a half
                        const void *map = it.part == Item::kHead ? &tbnd : &thT;
                        const int index = it.part == Item::kHead ? (int)cut_state(p, range + 1, side) : it.n * p.H + h;
#pragma unroll 1
                        for (int x = kHalf; x < 2 * kHalf; ++x)
                            if (32 * x < dv)
                                tma_store_3d(map, base + sb * M::kQK + M::kQ + (x - kHalf) * dk * 128, 32 * x, 0,
                                             index);
                        bulk_commit();
#pragma unroll 1
                        for (int x = 0; x < kHalf; ++x)
                            tma_store_3d(map, base + M::kS + x * dk * 128, 32 * x, 0, index);
                        bulk_commit();
                        asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
                        mbar_arrive(&bar[kFreeQ + sb]);
                        bulk_wait_read_all();
                        mbar_arrive(&bar[kEndFree]);
                    }
                    __syncwarp();
                }
                ok = wait.warp(kOFree + b, (gi >> 1) & 1);
                if (!ok) break;
                if (len == C) {
                    if (lane == 0) {
#pragma unroll
                        for (int x = 0; x < DVP / 64; ++x)
                            tma_store_3d(&to, base + so + x * 16384, 64 * x, h, (int32_t)t0);
                        bulk_commit();
                        bulk_wait_read_all();
                    }
                } else {   // rows past the sequence belong to others: eight at a time, then single
                    const int eights = len & ~7, per = dv / 8;   // per: 16-byte pieces of a row
                    if (lane == 0) {
#pragma unroll 1
                        for (int r = 0; r < eights; r += 8)
#pragma unroll
                            for (int x = 0; x < DVP / 64; ++x)
                                tma_store_3d(&to8, base + so + x * 16384 + r * 128, 64 * x, h, (int32_t)t0 + r);
                        bulk_commit();
                    }
#pragma unroll 1
                    for (int x = eights * per + lane; x < len * per; x += 32) {
                        const int r = x / per, j = 8 * (x - r * per);
                        *reinterpret_cast<uint4 *>(o + ((t0 + r) * p.H + h) * (int64_t)dv + j) =
                            *reinterpret_cast<const uint4 *>(sm + so + sw128_offset(r, j, C));
                    }
                    if (lane == 0) bulk_wait_read_all();
                    fence_proxy_async();   // before v of a later chunk takes the place
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[kFreeV + b]);
                if (it.part == Item::kHead && c + 1 == chunks && lane == 0) {
                    // the state is written, not only read: hand it on
                    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
                    asm volatile("fence.proxy.async.global;" ::: "memory");
                    __threadfence();
                    asm volatile("st.release.gpu.global.u32 [%0], %1;"
                                 ::"l"(p.flags + cut_state(p, range + 1, side)), "r"(1u)
                                 : "memory");
                }
                __syncwarp();
            }
        });
    }
    if (!ok) {
        if (lane == 0) report(st, KDA_ERR_TIMEOUT, blockIdx.x, 41 + warp);
    }
    if (__syncthreads_or(!ok)) {
        // an expired wait: what is in flight ends (each wait bounded again) before the tensor
        // memory is released and the CTA leaves
        tmem_st_wait();
        tc_fence_before();
        if (warp == kMmaWarp) {
            tc_fence_after();   // (on a barrier whose role has stopped, at whichever phase it is)
            const uint32_t phase = mbar_try_wait(&bar[kEndFree], 0) ? 1 : 0;
            __syncwarp();
            if (elect_one()) umma_commit(&bar[kEndFree]);
            __syncwarp();
            mbar_wait(&bar[kEndFree], phase, kDrainNs);
        }
        if (warp == kLoadWarp) {   // (only each stage's last load can be in flight)
            for (uint32_t x = issued_q >= 2 ? issued_q - 2 : 0; x < issued_q; ++x)
                mbar_wait(&bar[kFullQ + (x & 1)], (x >> 1) & 1, kDrainNs);
            for (uint32_t x = issued_k >= 2 ? issued_k - 2 : 0; x < issued_k; ++x)
                mbar_wait(&bar[kFullK + (x & 1)], (x >> 1) & 1, kDrainNs);
            for (uint32_t x = issued_v >= 2 ? issued_v - 2 : 0; x < issued_v; ++x)
                mbar_wait(&bar[kFullV + (x & 1)], (x >> 1) & 1, kDrainNs);
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

static cudaError_t encode(CUtensorMap *m, CUtensorMapDataType type, const void *x,
                          const cuuint64_t (&dims)[3], const cuuint64_t (&strides)[2],
                          const cuuint32_t (&box)[3]) {
    EncodeTiledFn enc = encode_tiled();
    if (!enc) return cudaErrorNotSupported;
    const cuuint32_t estr[3] = {1, 1, 1};
    const CUresult r = enc(m, type, 3, const_cast<void *>(x), dims, strides, box, estr,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// [T, heads, D] bf16, tokens `stride` elements apart, in boxes of `rows` tokens x 1 head x 64
// channels with the 128-byte swizzle; what lies outside (channels of 32-wide heads, tokens
// past the last) reads as zeros.
static cudaError_t tensor_map(CUtensorMap *m, const void *x, int64_t T, int heads, int D,
                              int64_t stride, int rows = C) {
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, x,
                  {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)T},
                  {(cuuint64_t)D * 2, (cuuint64_t)stride * 2}, {64, 1, (cuuint32_t)rows});
}

// [states, dk, dv] fp32 in boxes of one state's rows x 32 columns
static cudaError_t state_map(CUtensorMap *m, const float *x, int64_t states, int dk, int dv) {
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, x,
                  {(cuuint64_t)dv, (cuuint64_t)dk, (cuuint64_t)states},
                  {(cuuint64_t)dv * 4, (cuuint64_t)dk * dv * 4}, {32, (cuuint32_t)dk, 1});
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
static cudaError_t launch(const Plan &p, const CUtensorMap (&m)[8], const float *g, int gpt,
                          int has_h0, int has_hT, void *o, int dk, int dv, float *bnd,
                          float *bnd_log, StatusWord *st, cudaStream_t s) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = allow_smem<DKP, DVP, OUT>(dev);
    if (e != cudaSuccess) return e;
    return launch_after(la_chunk_tc_kernel<DKP, DVP, OUT>, dim3((OUT ? p.ranges : p.ranges - 1) * p.lanes),
                        dim3(kThreads), Map<DKP, DVP>::kBytes, s, p, m[0], m[1], m[2], m[3], m[4], m[5],
                        m[6], m[7], g, gpt, has_h0, has_hT, (__nv_bfloat16 *)o, dk, dv, bnd, bnd_log, st);
}

}  // namespace tc
}  // namespace la

// The maps of one call: q, k, v, o and, where they are used, the initial and the final states
// and those at the cuts.
cudaError_t la_tensor_maps(CUtensorMap (&m)[8], const void *q, const void *k, const void *v,
                           const void *o, const float *h0, const float *hT, const float *bnd,
                           const la::Plan &p, int64_t T, int dk, int dv, int64_t qs, int64_t ks,
                           int64_t vs) {
    memset(&m[5], 0, 3 * sizeof m[5]);
    const int64_t nh = (int64_t)p.N * p.H;
    cudaError_t e = la::tc::tensor_map(&m[0], q, T, p.Hk, dk, qs);
    if (e == cudaSuccess) e = la::tc::tensor_map(&m[1], k, T, p.Hk, dk, ks);
    if (e == cudaSuccess) e = la::tc::tensor_map(&m[2], v, T, p.H, dv, vs);
    if (e == cudaSuccess) e = la::tc::tensor_map(&m[3], o, T, p.H, dv, (int64_t)p.H * dv);
    if (e == cudaSuccess) e = la::tc::tensor_map(&m[4], o, T, p.H, dv, (int64_t)p.H * dv, 8);
    if (e == cudaSuccess && h0) e = la::tc::state_map(&m[5], h0, nh, dk, dv);
    if (e == cudaSuccess && hT) e = la::tc::state_map(&m[6], hT, nh, dk, dv);
    if (e == cudaSuccess && bnd) e = la::tc::state_map(&m[7], bnd, 2 * (int64_t)p.ranges * p.lanes, dk, dv);
    return e;
}

cudaError_t launch_la_tc(bool out, const la::Plan &p, const CUtensorMap (&m)[8], const float *g,
                         int gpt, int has_h0, int has_hT, void *o, int dk, int dv, float *bnd,
                         float *bnd_log, StatusWord *st, cudaStream_t s) {
#define KDA_LA(DK_, DV_)                                                                          \
    if ((dk <= 64) == (DK_ == 64) && (dv <= 64) == (DV_ == 64))                                   \
        return out ? la::tc::launch<DK_, DV_, true>(p, m, g, gpt, has_h0, has_hT, o, dk, dv, bnd, bnd_log, \
                                                    st, s)                                        \
                   : la::tc::launch<DK_, DV_, false>(p, m, g, gpt, has_h0, has_hT, o, dk, dv, bnd, bnd_log, \
                                                     st, s);
    KDA_LA(64, 64) KDA_LA(64, 128) KDA_LA(128, 64) KDA_LA(128, 128)
#undef KDA_LA
    return cudaErrorInvalidValue;
}

}  // namespace kda
