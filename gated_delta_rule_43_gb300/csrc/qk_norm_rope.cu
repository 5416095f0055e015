// qk_norm_rope.cu -- per-head norm of queries and keys and their position rotation, one pass.
//
// Memory-bound: every value is read once and written once, nothing else is large.  A group
// of D / 16 lanes owns one head of one token; a lane holds two 16-byte vectors (bf16; twice
// as many in fp32) of eight channels each, laid out so that rotation never leaves the lane:
//   half layout        channels 8 j .. 8 j + 7 and rot / 2 + 8 j .. of the rotated part
//   interleaved        channels 16 j .. 16 j + 15
//   past the rotated part, channels rot + 16 j' .. (no rotation)
// so a norm is a few shuffles deep and rotation needs none.  A CTA takes the heads (or a part of
// them) of a few tokens: first each thread works out one angle's cosine and sine, which the
// heads of a token share, into shared memory; then each warp goes through rows, the loads of several
// rows in flight.  8192 tokens of 32 + 32 heads of 128 (268 MB): 50.0 us, 5.4 TB/s; a plain copy of
// as much takes 43.  In fp32 83 us, 6.4 TB/s, a copy 79.  With weights and rotated in neighbouring pairs
// (half of each head) 65 and 120 us: every row reads its weights again.  (Three CTAs an SM: with two 58 us, with four, in 64 registers, 63; two
// tokens a CTA 52.)
//
// The rotation's angle is a whole number of turns plus a fraction, and only the fraction
// counts.  The rate in turns per position is held as a 64-bit binary fraction, so position *
// rate modulo one turn is one integer product, exact but for the rate's own last bit
// (2^-64 turns a position); a product in fp32 would be off by 0.06 rad at position 10^6.
// The fraction itself is formed in integers too: 24 bits of inv_freq times 128 of 1 / (2 pi), as in
// Payne and Hanek's reduction (1983).
#include "kda_common.cuh"

namespace kda {
namespace qk {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kTokens = 4;   // of a CTA, at most: kThreads angles of 64 pairs

struct Side {
    const void *x;
    void *y;
    const float *w;
    int64_t xs, ys;
    int heads;
    float scale;
};

// Eight channels as they lie in memory, and as fp32 in pairs
template <typename T> struct Raw;
template <> struct Raw<__nv_bfloat16> {
    uint4 u;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { u = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void get(float2 (&x)[4]) const {
        const __nv_bfloat162 *b = reinterpret_cast<const __nv_bfloat162 *>(&u);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = __bfloat1622float2(b[i]);
    }
};
template <> struct Raw<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p) {
        a = reinterpret_cast<const float4 *>(p)[0];
        b = reinterpret_cast<const float4 *>(p)[1];
    }
    __device__ __forceinline__ void get(float2 (&x)[4]) const {
        x[0] = make_float2(a.x, a.y); x[1] = make_float2(a.z, a.w);
        x[2] = make_float2(b.x, b.y); x[3] = make_float2(b.z, b.w);
    }
};
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float2 (&x)[4]) {
    uint4 u;
    __nv_bfloat162 *b = reinterpret_cast<__nv_bfloat162 *>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = __floats2bfloat162_rn(x[i].x, x[i].y);
    *reinterpret_cast<uint4 *>(p) = u;
}
__device__ __forceinline__ void store8(float *p, const float2 (&x)[4]) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(x[0].x, x[0].y, x[1].x, x[1].y);
    reinterpret_cast<float4 *>(p)[1] = make_float4(x[2].x, x[2].y, x[3].x, x[3].y);
}

// Two products, two products and sums in one instruction: with single ones the arithmetic
// takes as long as the memory
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "mul.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 z, x, y, z;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}

// f turns of 2 pi radians, in units of 2^-64 turn, modulo one turn, rounded down in magnitude.
__device__ __forceinline__ uint64_t turn_fraction(float f) {
    constexpr uint64_t hi = 0x28be60db9391054aull, lo = 0x7f09d5f47d4d3770ull;   // 2^128 / (2 pi)
    const uint32_t b = __float_as_uint(f);
    const int ex = (b >> 23) & 255;
    const uint64_t m = (b & 0x7fffffu) | (ex ? 0x800000u : 0u);   // |f| = m 2^e
    const int e = (ex ? ex : 1) - 150, s = 64 - e;                // product >> s
    const uint64_t p0 = m * lo, c = __umul64hi(m, lo), p1 = m * hi + c;
    const uint64_t p2 = __umul64hi(m, hi) + (p1 < c ? 1u : 0u);
    uint64_t r = 0;
    if (s > 0 && s < 64) r = (p0 >> s) | (p1 << (64 - s));
    if (s == 64) r = p1;
    if (s > 64 && s < 128) r = (p1 >> (s - 64)) | (p2 << (128 - s));
    if (s >= 128 && s < 192) r = p2 >> (s - 128);
    return (b >> 31) ? 0u - r : r;
}

// CTA x: tokens [t0, t0 + tokens) of group x / parts, heads [h0, h1) of part x % parts.
// Rows in flight: as many bytes in either type
template <typename T> constexpr int ahead() { return sizeof(T) == 2 ? 4 : 2; }

template <int D, typename T>
__global__ void __launch_bounds__(kThreads, 3)
qk_norm_rope_kernel(Side q, Side k, int64_t T_tot, int tokens, int parts, int norm, float eps,
                    const int32_t *__restrict__ positions, const float *__restrict__ inv_freq,
                    int rot, int interleaved, float rope_scale) {
    constexpr int LPR = D / 16;      // lanes per head
    constexpr int RPW = 32 / LPR;    // heads a warp holds at a time
    constexpr int kAhead = ahead<T>();
    __shared__ __align__(16) float s_cos[kTokens][D / 2], s_sin[kTokens][D / 2];
    const int64_t t0 = (int64_t)(blockIdx.x / parts) * tokens;
    const int part = blockIdx.x % parts;
    const int here = (int)min((int64_t)tokens, T_tot - t0), pairs = rot / 2;
    const int lane = threadIdx.x & 31, j = lane % LPR, row = lane / LPR;
    const bool turned = 16 * j < rot;
    const int c0 = turned ? (interleaved ? 16 * j : 8 * j) : 16 * j;
    const int c1 = turned ? (interleaved ? c0 + 8 : rot / 2 + c0) : c0 + 8;
    const int all = q.heads + k.heads;
    const int h0 = (int)((int64_t)all * part / parts), h1 = (int)((int64_t)all * (part + 1) / parts);
    const int rows = here * (h1 - h0);
    // (the first turn's rows are on their way while the angles are worked out)
    Raw<T> xa[kAhead], xb[kAhead];
    T *dst[kAhead];
    int tok[kAhead];   // -1: none
    bool is_k[kAhead];
    auto fetch = [&](int m, int r) {
        tok[m] = -1;
        dst[m] = nullptr;
        is_k[m] = false;
        xa[m] = Raw<T>{};
        xb[m] = Raw<T>{};
        if (r < rows) {
            int h = r, token = 0;   // (at most kTokens)
#pragma unroll
            for (int i = 1; i < kTokens; ++i) {
                const bool past = h >= h1 - h0;
                h -= past ? h1 - h0 : 0;
                token += past;
            }
            h += h0;
            tok[m] = token;
            is_k[m] = h >= q.heads;
            const Side &s = is_k[m] ? k : q;
            const int64_t t = t0 + token, hh = is_k[m] ? h - q.heads : h;
            const T *src = (const T *)s.x + t * s.xs + hh * D;
            dst[m] = (T *)s.y + t * s.ys + hh * D;
            xa[m].load(src + c0);
            xb[m].load(src + c1);
        }
    };
    constexpr int kTurn = kWarps * RPW * kAhead;
    int r0 = (threadIdx.x >> 5) * RPW * kAhead;
#pragma unroll
    for (int m = 0; m < kAhead; ++m) fetch(m, r0 + m * RPW + row);
    for (int x = threadIdx.x; x < here * pairs; x += kThreads) {
        const int t = x / pairs, i = x - t * pairs;
        // position * turns modulo 2^64: the angle's fraction of a turn, in [-1/2, 1/2)
        const int64_t pos = positions[t0 + t];
        const int64_t f = (int64_t)((uint64_t)pos * turn_fraction(inv_freq[i]));
        float c, sn;
        sincospif((float)(int32_t)(f >> 32) * 4.656612873077393e-10f, &sn, &c);   // 2^-31
        s_cos[t][i] = c * rope_scale;
        s_sin[t][i] = sn * rope_scale;
    }
    __syncthreads();
    for (; r0 < rows; r0 += kTurn) {
#pragma unroll
        for (int m = 0; m < kAhead; ++m) {
            float2 a[4], b[4];
            xa[m].get(a);
            xb[m].get(b);
            const int t = tok[m];
            const bool of_k = is_k[m];
            T *const to = dst[m];
            const float *w = of_k ? k.w : q.w;
            float factor = of_k ? k.scale : q.scale;   // rotation is linear: first the factors
            if (norm != KDA_NORM_NONE) {
                float2 sums = make_float2(0.f, 0.f);
#pragma unroll
                for (int i = 0; i < 4; ++i) sums = fma2(a[i], a[i], fma2(b[i], b[i], sums));
                float sum = sums.x + sums.y;
#pragma unroll
                for (int d = LPR / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                factor *= rsqrtf((norm == KDA_NORM_RMS ? sum * (1.f / D) : sum) + eps);
            }
            if (t < 0) continue;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                a[i] = mul2(a[i], make_float2(factor, factor));
                b[i] = mul2(b[i], make_float2(factor, factor));
            }
            if (w) {
                Raw<float> wa, wb;
                wa.load(w + c0);
                wb.load(w + c1);
                float2 fa[4], fb[4];
                wa.get(fa);
                wb.get(fb);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    a[i] = mul2(a[i], fa[i]);
                    b[i] = mul2(b[i], fb[i]);
                }
            }
            if (turned) {
                Raw<float> rc, rs;
                rc.load(&s_cos[t][8 * j]);
                rs.load(&s_sin[t][8 * j]);
                float2 cs[4], sn[4];
                rc.get(cs);
                rs.get(sn);
                if (interleaved) {
                    auto turn = [](float2 &x, float c, float s) {
                        x = make_float2(x.x * c - x.y * s, x.y * c + x.x * s);
                    };
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        turn(a[2 * i], cs[i].x, sn[i].x);
                        turn(a[2 * i + 1], cs[i].y, sn[i].y);
                        turn(b[2 * i], cs[2 + i].x, sn[2 + i].x);
                        turn(b[2 * i + 1], cs[2 + i].y, sn[2 + i].y);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 x = a[i], y = b[i];
                        a[i] = fma2(x, cs[i], mul2(y, make_float2(-sn[i].x, -sn[i].y)));
                        b[i] = fma2(y, cs[i], mul2(x, sn[i]));
                    }
                }
            }
            store8(to + c0, a);
            store8(to + c1, b);
        }
#pragma unroll
        for (int m = 0; m < kAhead; ++m) fetch(m, r0 + kTurn + m * RPW + row);
    }
}

template <int D, typename T>
static cudaError_t launch_dims(const Side &q, const Side &k, int64_t T_tot, int norm, float eps,
                               const int32_t *pos, const float *inv_freq, int rot, int interleaved,
                               float rope_scale, int sms, cudaStream_t s) {
    constexpr int kRows = kWarps * (32 / (D / 16)) * ahead<T>();   // of a CTA's turn
    // Several tokens a CTA while that leaves four CTAs an SM, and a token's heads over several
    // CTAs (each works out the token's angles again) while there are fewer than two.
    int tokens = kTokens;
    while (tokens > 1 && (T_tot + tokens - 1) / tokens < 4LL * sms) tokens >>= 1;
    const int64_t groups = (T_tot + tokens - 1) / tokens, all = q.heads + k.heads;
    const int64_t most = (all * tokens + kRows - 1) / kRows;
    int64_t parts = (2LL * sms + groups - 1) / groups;
    parts = parts > most ? most : parts;
    if (groups * parts > 0x7fffffffLL) return cudaErrorInvalidValue;
    qk_norm_rope_kernel<D, T><<<(unsigned)(groups * parts), kThreads, 0, s>>>(
        q, k, T_tot, tokens, (int)parts, norm, eps, pos, inv_freq, rot, interleaved, rope_scale);
    return cudaGetLastError();
}

}  // namespace qk

cudaError_t launch_qk(int dtype, int D, const void *q, const void *k, void *qo, void *ko,
                      int64_t T_tot, int Hq, int Hk, int64_t qs, int64_t ks, int64_t qos,
                      int64_t kos, const float *qw, const float *kw, int norm, float eps,
                      float q_scale, float k_scale, const int32_t *pos, const float *inv_freq,
                      int rot, int interleaved, float rope_scale, int sms, cudaStream_t s) {
    const qk::Side a{q, qo, qw, qs, qos, Hq, q_scale}, b{k, ko, kw, ks, kos, Hk, k_scale};
#define KDA_QK(D_)                                                                               \
    if (D == D_)                                                                                 \
        return dtype == KDA_BF16                                                                 \
                   ? qk::launch_dims<D_, __nv_bfloat16>(a, b, T_tot, norm, eps, pos, inv_freq, rot, \
                                                        interleaved, rope_scale, sms, s)         \
                   : qk::launch_dims<D_, float>(a, b, T_tot, norm, eps, pos, inv_freq, rot,       \
                                                interleaved, rope_scale, sms, s);
    KDA_QK(32) KDA_QK(64) KDA_QK(128)
#undef KDA_QK
    return cudaErrorInvalidValue;
}

}  // namespace kda
