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
// rows in flight.
//
// The rotation's angle is a whole number of turns plus a fraction, and only the fraction
// counts.  The rate in turns per position is held as a 64-bit binary fraction, so position *
// rate modulo one turn is one integer product, exact but for the rate's own last bit
// (2^-64 turns a position); a product in fp32 would be off by 0.06 rad at position 10^6.
// The fraction itself is formed in integers too: 24 bits of inv_freq times 128 of 1 / (2 pi).
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

// Eight channels as they lie in memory, and as fp32
template <typename T> struct Raw;
template <> struct Raw<__nv_bfloat16> {
    uint4 u;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { u = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        const __nv_bfloat162 *b = reinterpret_cast<const __nv_bfloat162 *>(&u);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __bfloat1622float2(b[i]);
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
};
template <> struct Raw<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p) {
        a = reinterpret_cast<const float4 *>(p)[0];
        b = reinterpret_cast<const float4 *>(p)[1];
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
};
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&x)[8]) {
    uint4 u;
    __nv_bfloat162 *b = reinterpret_cast<__nv_bfloat162 *>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    *reinterpret_cast<uint4 *>(p) = u;
}
__device__ __forceinline__ void store8(float *p, const float (&x)[8]) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
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
    const int lane = threadIdx.x & 31, j = lane % LPR, row = lane / LPR;
    const bool turned = 16 * j < rot;
    const int c0 = turned ? (interleaved ? 16 * j : 8 * j) : 16 * j;
    const int c1 = turned ? (interleaved ? c0 + 8 : rot / 2 + c0) : c0 + 8;
    const int all = q.heads + k.heads;
    const int h0 = (int)((int64_t)all * part / parts), h1 = (int)((int64_t)all * (part + 1) / parts);
    const int rows = here * (h1 - h0);
    for (int r0 = (threadIdx.x >> 5) * RPW * kAhead; r0 < rows; r0 += kWarps * RPW * kAhead) {
        Raw<T> xa[kAhead], xb[kAhead];
        T *dst[kAhead];
        int tok[kAhead];
        bool is_k[kAhead];
#pragma unroll
        for (int m = 0; m < kAhead; ++m) {
            const int r = r0 + m * RPW + row;
            tok[m] = -1;
            dst[m] = nullptr;
            is_k[m] = false;
            xa[m] = Raw<T>{};
            xb[m] = Raw<T>{};
            if (r < rows) {
                tok[m] = r / (h1 - h0);
                const int h = h0 + r - tok[m] * (h1 - h0);
                is_k[m] = h >= q.heads;
                const Side &s = is_k[m] ? k : q;
                const int64_t t = t0 + tok[m], hh = is_k[m] ? h - q.heads : h;
                const T *src = (const T *)s.x + t * s.xs + hh * D;
                dst[m] = (T *)s.y + t * s.ys + hh * D;
                xa[m].load(src + c0);
                xb[m].load(src + c1);
            }
        }
#pragma unroll
        for (int m = 0; m < kAhead; ++m) {
            float a[8], b[8];
            xa[m].get(a);
            xb[m].get(b);
            const float *w = is_k[m] ? k.w : q.w;
            float scale = is_k[m] ? k.scale : q.scale;
            if (norm != KDA_NORM_NONE) {
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) sum += a[i] * a[i] + b[i] * b[i];
#pragma unroll
                for (int d = LPR / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                const float n = rsqrtf((norm == KDA_NORM_RMS ? sum * (1.f / D) : sum) + eps);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    a[i] *= n;
                    b[i] *= n;
                }
            }
            if (tok[m] < 0) continue;
            if (w) {
                Raw<float> wa, wb;
                wa.load(w + c0);
                wb.load(w + c1);
                float fa[8], fb[8];
                wa.get(fa);
                wb.get(fb);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    a[i] *= fa[i];
                    b[i] *= fb[i];
                }
            }
            if (turned) {
                Raw<float> rc, rs;
                rc.load(&s_cos[tok[m]][8 * j]);
                rs.load(&s_sin[tok[m]][8 * j]);
                float cs[8], sn[8];
                rc.get(cs);
                rs.get(sn);
                if (interleaved) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float x0 = a[2 * i], y0 = a[2 * i + 1], x1 = b[2 * i], y1 = b[2 * i + 1];
                        a[2 * i] = x0 * cs[i] - y0 * sn[i];
                        a[2 * i + 1] = y0 * cs[i] + x0 * sn[i];
                        b[2 * i] = x1 * cs[4 + i] - y1 * sn[4 + i];
                        b[2 * i + 1] = y1 * cs[4 + i] + x1 * sn[4 + i];
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float x = a[i], y = b[i];
                        a[i] = x * cs[i] - y * sn[i];
                        b[i] = y * cs[i] + x * sn[i];
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                a[i] *= scale;
                b[i] *= scale;
            }
            store8(dst[m] + c0, a);
            store8(dst[m] + c1, b);
        }
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
