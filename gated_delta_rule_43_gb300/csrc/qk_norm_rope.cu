// qk_norm_rope.cu -- per-head norm of queries and keys and their position rotation, one pass.
//
// Memory-bound: every value is read once and written once, nothing else is large.  A group
// of D / 16 lanes owns one head of one token; a lane holds two 16-byte vectors (bf16; twice
// as many in fp32) of eight channels each, laid out so that rotation never leaves the lane:
//   half layout        channels 8 j .. 8 j + 7 and rot / 2 + 8 j .. of the rotated part
//   interleaved        channels 16 j .. 16 j + 15
//   past the rotated part, channels rot + 16 j' .. (no rotation)
// so a norm is two shuffles-and-adds deep and there is no shared memory.  A warp keeps to
// one token while it goes through that token's heads: the eight cosines and sines of a lane
// are worked out once a token.
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

struct Side {
    const void *x;
    void *y;
    const float *w;
    int64_t xs, ys;
    int heads;
    float scale;
};

__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&x)[8]) {
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    const __nv_bfloat162 *b = reinterpret_cast<const __nv_bfloat162 *>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __bfloat1622float2(b[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}
__device__ __forceinline__ void load8(const float *p, float (&x)[8]) {
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
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

// A warp takes (token, part of its heads) units; `parts` units share a token.
template <int D, typename T>
__global__ void __launch_bounds__(kThreads)
qk_norm_rope_kernel(Side q, Side k, int64_t units, int parts, int norm, float eps,
                    const int32_t *__restrict__ positions, const float *__restrict__ inv_freq,
                    int rot, int interleaved, float rope_scale) {
    constexpr int LPR = D / 16;      // lanes per head
    constexpr int RPW = 32 / LPR;    // heads a warp holds at a time
    const int lane = threadIdx.x & 31, j = lane % LPR, row = lane / LPR;
    const bool turned = 16 * j < rot;
    const int c0 = turned ? (interleaved ? 16 * j : 8 * j) : 16 * j;
    const int c1 = turned ? (interleaved ? c0 + 8 : rot / 2 + c0) : c0 + 8;
    // turns per position of this lane's eight pairs, as fractions of 2^64
    uint64_t rate[8];
    if (turned) {
#pragma unroll
        for (int i = 0; i < 8; ++i) rate[i] = turn_fraction(inv_freq[8 * j + i]);
    }
    const int all = q.heads + k.heads;
    for (int64_t u = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); u < units;
         u += (int64_t)gridDim.x * kWarps) {
        const int64_t t = u / parts;
        const int part = (int)(u - t * parts);
        float cs[8], sn[8];
        if (turned) {
            const int64_t pos = positions[t];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                // the product modulo 2^64 is the angle's fraction of a turn in [-1/2, 1/2)
                const int64_t f = (int64_t)((uint64_t)pos * rate[i]);
                sincospif((float)(int32_t)(f >> 32) * 4.656612873077393e-10f, &sn[i], &cs[i]);   // 2^-31
                cs[i] *= rope_scale;
                sn[i] *= rope_scale;
            }
        }
        for (int h = part * RPW + row; h - row < all; h += parts * RPW) {
            const bool here = h < all;
            const bool is_k = h >= q.heads;
            const Side &s = is_k ? k : q;
            const int hh = is_k ? h - q.heads : h;
            float a[8], b[8];
            if (here) {
                const T *x = (const T *)s.x + t * s.xs + (int64_t)hh * D;
                load8(x + c0, a);
                load8(x + c1, b);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) a[i] = b[i] = 0.f;
            }
            if (norm != KDA_NORM_NONE) {
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) sum += a[i] * a[i] + b[i] * b[i];
#pragma unroll
                for (int d = LPR / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                const float r = rsqrtf((norm == KDA_NORM_RMS ? sum * (1.f / D) : sum) + eps);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    a[i] *= r;
                    b[i] *= r;
                }
            }
            if (!here) continue;
            if (s.w) {
                float wa[8], wb[8];
                load8(s.w + c0, wa);
                load8(s.w + c1, wb);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    a[i] *= wa[i];
                    b[i] *= wb[i];
                }
            }
            if (turned) {
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
                a[i] *= s.scale;
                b[i] *= s.scale;
            }
            T *y = (T *)s.y + t * s.ys + (int64_t)hh * D;
            store8(y + c0, a);
            store8(y + c1, b);
        }
    }
}

template <int D, typename T>
static cudaError_t launch_dims(const Side &q, const Side &k, int64_t T_tot, int norm, float eps,
                               const int32_t *pos, const float *inv_freq, int rot, int interleaved,
                               float rope_scale, int sms, cudaStream_t s) {
    constexpr int RPW = 32 / (D / 16);
    // a token's heads go to one warp, unless there are too few tokens to fill the SMs
    const int64_t most = (q.heads + k.heads + RPW - 1) / RPW;
    int64_t parts = (8LL * kWarps * sms + T_tot - 1) / T_tot;
    parts = parts < 1 ? 1 : parts > most ? most : parts;
    const int64_t units = T_tot * parts, blocks = (units + kWarps - 1) / kWarps;
    const int64_t cap = 8LL * sms;
    qk_norm_rope_kernel<D, T><<<(unsigned)(blocks < cap ? blocks : cap), kThreads, 0, s>>>(
        q, k, units, (int)parts, norm, eps, pos, inv_freq, rot, interleaved, rope_scale);
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
