// paged_attn_simt.cu -- attention over a paged cache on the CUDA cores, in fp32: single-precision
// storage and heads of 32.
//
//   o_i = sum_j w_ij v_j / sum_j w_ij,   w_ij = exp(scale q_i k_j - m_i),   m_i the largest exponent
// One pass over the keys with the running maximum and sum.  The query heads that share a key/value head
// are rows beside each other (row = token * group + head), so that keys are read once for all of
// them.  A CTA takes 32 rows and goes through blocks of 32 keys staged in shared memory as fp32; four
// threads share a row.  Where there are few rows, `splits` CTAs share their keys and a second kernel
// joins what they found.
#include "kda_paged.cuh"

namespace kda {
namespace paged {
namespace simt {

constexpr int BR = 32, BK = 32, kThreads = 128;
constexpr float kLog2e = 1.4426950408889634f;

// Rows [first, first + rows) of sequence n's len * group.
struct Tile {
    int n, first, rows;
    Span s;
};
// The `tile`-th tile of 32 rows in the batch; a whole warp.  False past the last.
__device__ __forceinline__ bool find_tile(const Cache &c, int tile, int group, Tile &r) {
    const int lane = threadIdx.x & 31;
    int64_t before = 0;
    for (int n0 = 0; n0 < c.N; n0 += 32) {
        Span s{0, 0, 0};
        if (n0 + lane < c.N) s = span_of(c, n0 + lane);
        const int64_t rows = (int64_t)s.len * group;
        const int64_t mine = (rows + BR - 1) / BR;
        int64_t sum = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += x;
        }
        const uint32_t m = __ballot_sync(0xffffffffu, before + sum > tile);
        if (m) {
            const int l = __ffs(m) - 1;
            r.n = n0 + l;
            r.s.begin = __shfl_sync(0xffffffffu, s.begin, l);
            r.s.len = __shfl_sync(0xffffffffu, s.len, l);
            r.s.pos = __shfl_sync(0xffffffffu, s.pos, l);
            const int64_t t = tile - before - __shfl_sync(0xffffffffu, sum - mine, l);
            r.first = (int)(t * BR);
            r.rows = (int)min((int64_t)BR, __shfl_sync(0xffffffffu, rows, l) - t * BR);
            return true;
        }
        before += __shfl_sync(0xffffffffu, sum, 31);
    }
    return false;
}

template <int D> struct Shared {
    float q[BR][D + 4];
    float k[BK][D + 4];
    float v[BK][D + 4];
    float p[BR][BK + 4];
    Tile tile;
    int there;
};

template <typename TQ, typename TC, int D>
__global__ void __launch_bounds__(kThreads)
paged_simt_kernel(Cache c, const TQ *__restrict__ q, int64_t q_stride, TQ *__restrict__ o, int group, float scale,
                  int window, int sinks, int splits, float *__restrict__ part, StatusWord *st) {
    extern __shared__ __align__(16) uint8_t raw[];
    Shared<D> &sm = *reinterpret_cast<Shared<D> *>(raw);
    const int tid = threadIdx.x, H = c.Hk * group;
    const int tile = blockIdx.x / c.Hk, h = blockIdx.x % c.Hk, split = blockIdx.y;
    if (blockIdx.x == 0 && split == 0) check_spans(c, st);
    if (tid < 32) {
        Tile t;
        const bool there = find_tile(c, tile, group, t);
        if (tid == 0) {
            sm.there = there;
            if (there) sm.tile = t;
        }
    }
    __syncthreads();
    if (!sm.there) return;
    const Tile t = sm.tile;
    for (int x = tid; x < BR * D; x += kThreads) {
        const int r = x / D, d = x % D;
        float y = 0.f;
        if (r < t.rows) {
            const int at = t.first + r;
            y = to_f(q[(int64_t)(t.s.begin + at / group) * q_stride + (int64_t)(h * group + at % group) * D + d]);
        }
        sm.q[r][d] = y;
    }
    const int r = tid / 4, quarter = tid % 4;
    const int pos = t.s.pos + (t.first + r) / group;
    const int lowest = window > 0 ? max(max(pos, 0) - window, -1) : -1;   // keys above it are in the window
    const KeyBlocks kb = key_blocks(max(0, t.s.pos + t.first / group), t.s.pos + (t.first + t.rows - 1) / group, window,
                                    sinks, BK);
    const int b0 = (int)((int64_t)kb.count * split / splits), b1 = (int)((int64_t)kb.count * (split + 1) / splits);
    float m = -INFINITY, l = 0.f, acc[D / 4];
#pragma unroll
    for (int j = 0; j < D / 4; ++j) acc[j] = 0.f;
    const float f = scale * kLog2e;
    const int ctx = t.s.pos + t.s.len;
    for (int b = b0; b < b1; ++b) {
        const int key0 = kb.block(b) * BK;
        __syncthreads();
        for (int x = tid; x < BK * D / 4; x += kThreads) {
            const int j = x / (D / 4), d = x % (D / 4) * 4, key = key0 + j;
            float4 kx = make_float4(0.f, 0.f, 0.f, 0.f), vx = kx;
            if (key < ctx) {
                const int page = c.table[(int64_t)t.n * c.width + (key >> c.shift)];
                const bool seen = window <= 0 || key < sinks || key > max(0, t.s.pos + t.first / group) - window;
                if (page >= 0 && page < c.P) {
                    const int64_t at = ((int64_t)h << c.shift) + (key & ((1 << c.shift) - 1));
                    const TC *ka = (const TC *)c.k + page * c.stride + at * D + d;
                    const TC *va = (const TC *)c.v + page * c.stride + at * D + d;
                    float sk = 1.f, sv = 1.f;
                    if (sizeof(TC) == 1) {
                        sk = c.ks[page * c.scale_stride + at];
                        sv = c.vs[page * c.scale_stride + at];
                    }
                    if (seen) {   // (what nobody sees may be anything)
                        kx = make_float4(stored_to_f(ka[0]) * sk, stored_to_f(ka[1]) * sk, stored_to_f(ka[2]) * sk,
                                         stored_to_f(ka[3]) * sk);
                        vx = make_float4(stored_to_f(va[0]) * sv, stored_to_f(va[1]) * sv, stored_to_f(va[2]) * sv,
                                         stored_to_f(va[3]) * sv);
                    }
                } else if (seen) {
                    report(st, KDA_ERR_INVALID_ARG, t.n, 64);
                }
            }
            *reinterpret_cast<float4 *>(&sm.k[j][d]) = kx;
            *reinterpret_cast<float4 *>(&sm.v[j][d]) = vx;
        }
        __syncthreads();
        float s[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) s[j] = 0.f;
#pragma unroll 4
        for (int d = 0; d < D; d += 4) {
            const float4 x = *reinterpret_cast<const float4 *>(&sm.q[r][d]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float4 y = *reinterpret_cast<const float4 *>(&sm.k[quarter + 4 * j][d]);
                s[j] += x.x * y.x + x.y * y.y + x.z * y.z + x.w * y.w;
            }
        }
        float top = m;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int key = key0 + quarter + 4 * j;
            s[j] = key <= pos && (key > lowest || key < sinks) ? s[j] * f : -INFINITY;
            top = fmaxf(top, s[j]);
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const float ref = top == -INFINITY ? 0.f : top;
        const float keep = exp2f(m - ref);
        m = top;
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float p = exp2f(s[j] - ref);
            sum += p;
            sm.p[r][quarter + 4 * j] = p;
        }
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        l = l * keep + sum;
        __syncwarp();
#pragma unroll
        for (int j = 0; j < D / 4; ++j) acc[j] *= keep;
#pragma unroll 4
        for (int j = 0; j < BK; ++j) {
            const float p = sm.p[r][j];
#pragma unroll
            for (int d = 0; d < D / 16; ++d) {
                const float4 y = *reinterpret_cast<const float4 *>(&sm.v[j][16 * d + 4 * quarter]);
                acc[4 * d] += p * y.x;
                acc[4 * d + 1] += p * y.y;
                acc[4 * d + 2] += p * y.z;
                acc[4 * d + 3] += p * y.w;
            }
        }
    }
    if (r >= t.rows) return;
    if (splits > 1) {   // [tile, head][split][row]: D sums, the maximum, the sum of weights
        float *to = part + (((int64_t)blockIdx.x * splits + split) * BR + r) * (D + 4);
#pragma unroll
        for (int d = 0; d < D / 16; ++d)
            *reinterpret_cast<float4 *>(to + 16 * d + 4 * quarter) =
                make_float4(acc[4 * d], acc[4 * d + 1], acc[4 * d + 2], acc[4 * d + 3]);
        if (quarter == 0) {
            to[D] = m;
            to[D + 1] = l;
        }
        return;
    }
    const float inv = l != 0.f ? 1.f / l : 0.f;   // (no visible key: zeros)
    const int at = t.first + r;
    TQ *to = o + ((int64_t)(t.s.begin + at / group) * H + h * group + at % group) * D;
#pragma unroll
    for (int d = 0; d < D / 16; ++d)
#pragma unroll
        for (int j = 0; j < 4; ++j) to[16 * d + 4 * quarter + j] = from_f<TQ>(l != 0.f ? acc[4 * d + j] * inv : 0.f);
}

template <typename TQ, int D>
__global__ void __launch_bounds__(kThreads)
paged_simt_join(Cache c, TQ *__restrict__ o, int group, int splits, const float *__restrict__ part) {
    __shared__ Tile tile;
    __shared__ int there;
    const int tid = threadIdx.x, h = blockIdx.x % c.Hk, H = c.Hk * group;
    if (tid < 32) {
        Tile t;
        const bool found = find_tile(c, blockIdx.x / c.Hk, group, t);
        if (tid == 0) {
            there = found;
            if (found) tile = t;
        }
    }
    __syncthreads();
    if (!there) return;
    for (int x = tid; x < tile.rows * D; x += kThreads) {
        const int r = x / D, d = x % D;
        const float *from = part + ((int64_t)blockIdx.x * splits * BR + r) * (D + 4);
        const int64_t step = (int64_t)BR * (D + 4);
        float top = -INFINITY;
        for (int s = 0; s < splits; ++s) top = fmaxf(top, from[s * step + D]);
        float sum = 0.f, l = 0.f;
        for (int s = 0; s < splits; ++s) {
            const float w = from[s * step + D + 1];
            if (w == 0.f) continue;
            const float e = exp2f(from[s * step + D] - top);
            l += e * w;
            sum += e * from[s * step + d];
        }
        const int at = tile.first + r;
        o[((int64_t)(tile.s.begin + at / group) * H + h * group + at % group) * D + d] =
            from_f<TQ>(l != 0.f ? sum / l : 0.f);
    }
}

// Tiles that a batch can have at most.
static int64_t tiles_of(const Cache &c, int group) {
    return c.cu ? (int64_t)c.T * group / BR + c.N : c.N * (int64_t)((group + BR - 1) / BR);
}
// CTAs that share a tile's keys: enough for two a multiprocessor, each with 256 keys or more.
static int splits_of(const Cache &c, int group, int sms) {
    const int64_t ctas = tiles_of(c, group) * c.Hk;
    if (ctas == 0) return 1;
    int64_t s = (2 * sms + ctas - 1) / ctas;
    const int64_t most = (((int64_t)c.width << c.shift) + 255) / 256;
    s = s < most ? s : most;
    return (int)(s < 1 ? 1 : s > 64 ? 64 : s);
}

template <typename TQ, typename TC, int D>
static cudaError_t launch(const Cache &c, const void *q, int64_t qs, void *o, int group, float scale, int window,
                          int sinks, int splits, float *part, StatusWord *st, cudaStream_t s) {
    const int64_t ctas = tiles_of(c, group) * c.Hk;
    if (ctas > 0x7fffffff) return cudaErrorInvalidValue;
    const cudaError_t e = cudaFuncSetAttribute(paged_simt_kernel<TQ, TC, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)sizeof(Shared<D>));
    if (e != cudaSuccess) return e;
    paged_simt_kernel<TQ, TC, D><<<dim3((unsigned)ctas, splits), kThreads, sizeof(Shared<D>), s>>>(
        c, (const TQ *)q, qs, (TQ *)o, group, scale, window, sinks, splits, part, st);
    if (splits > 1) paged_simt_join<TQ, D><<<(unsigned)ctas, kThreads, 0, s>>>(c, (TQ *)o, group, splits, part);
    return cudaGetLastError();
}

}  // namespace simt
}  // namespace paged

size_t paged_simt_bytes(const paged::Cache &c, int group, int D, int sms) {
    const int splits = paged::simt::splits_of(c, group, sms);
    if (splits == 1) return 0;
    return (size_t)paged::simt::tiles_of(c, group) * c.Hk * splits * paged::simt::BR * (D + 4) * sizeof(float);
}

cudaError_t launch_paged_simt(int dtype, int cache_dtype, int D, const paged::Cache &c, const void *q, int64_t qs,
                              void *o, int group, float scale, int window, int sinks, float *part, int sms,
                              StatusWord *st, cudaStream_t s) {
    const int splits = paged::simt::splits_of(c, group, sms);
#define KDA_PAGED(TQ_, TC_, D_)                                                                                   \
    if (D == D_)                                                                                                  \
        return paged::simt::launch<TQ_, TC_, D_>(c, q, qs, o, group, scale, window, sinks, splits, part, st, s);
#define KDA_PAGED_D(TQ_, TC_) KDA_PAGED(TQ_, TC_, 32) KDA_PAGED(TQ_, TC_, 64) KDA_PAGED(TQ_, TC_, 128)
    if (dtype == KDA_F32) {
        if (cache_dtype == KDA_E4M3) { KDA_PAGED_D(float, __nv_fp8_e4m3) }
        else { KDA_PAGED_D(float, float) }
    } else {
        if (cache_dtype == KDA_E4M3) { KDA_PAGED_D(__nv_bfloat16, __nv_fp8_e4m3) }
        else { KDA_PAGED_D(__nv_bfloat16, __nv_bfloat16) }
    }
#undef KDA_PAGED_D
#undef KDA_PAGED
    return cudaErrorInvalidValue;
}

}  // namespace kda
