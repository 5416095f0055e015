// paged_cache.cu -- new keys and values into the pages of a cache, and back.
//
//   write: row x of D values   ->  x, or e4m3(x / s) and s = 2^e, e least with max|x| / s <= 448
//   read:  the row             ->  x, or s * e4m3
// Memory-bound: each row is read once and written once.  A row is spread over D * size / 16 lanes, 16
// bytes each (of the wider side).  A CTA takes 8, 4 or (few tokens) one token: its first warp looks their places up
// while the others' first rows are on their way, then all warps go through the tokens' rows, kRows
// loads ahead of the stores.  Tokens a CTA, 8 heads of 128: 36864 e4m3 tokens read back take 78, 47, 43, 44 us with 1,
// 4, 8, 16 (5.3 TB/s of the 6.8 of a copy; 69 with a look-up for every warp of eight rows); 8192 written to e4m3
// 24, 17, 18, 21.  Beside memory it is instructions that count: with two integer divisions a row and
// conversions one by one the same took 73 and 25.  With nothing of it in L2: 8192 tokens written to bf16 or e4m3 18 us, fp32 to
// fp32 29, to e4m3 31; 65536 to e4m3 92, to bf16 90 (6.0 TB/s); 36864 read from bf16 51, e4m3 to fp32 66, fp32 96.
#include "kda_paged.cuh"

namespace kda {
namespace paged {

constexpr int kThreads = 256, kRows = 4, kMost = 8;

// Where a token's rows lie: page -1: nowhere (not of this call: -2).
struct Place {
    int page, slot;
};
// Of tokens t0 .. t0 + count - 1 into `places`; the CTA's first warp.
__device__ __forceinline__ void find_places(const Cache &c, int t0, int count, Place *places, StatusWord *st, int site) {
    const int lane = threadIdx.x & 31;
    int n = c.cu ? sequence_of(c, t0) : t0 + lane;
    const int t = t0 + lane;
    if (lane < count) {
        Place x{-2, 0};
        if (c.cu && n >= 0)
            while (n + 1 < c.N && c.cu[n + 1] <= t) ++n;
        if (n >= 0 && n < c.N) {
            const Span s = span_of(c, n);
            const int pos = s.pos + (t - s.begin);
            if (t >= s.begin && t < s.begin + s.len) {
                x.page = -1;
                if (pos >= 0) {
                    const int page = c.table[(int64_t)n * c.width + (pos >> c.shift)];
                    if (page >= 0 && page < c.P) x.page = page;
                    else report(st, KDA_ERR_INVALID_ARG, n, site);
                    x.slot = pos & ((1 << c.shift) - 1);
                }
            }
        }
        places[lane] = x;
    }
}

template <typename T, int V> struct alignas(sizeof(T) * V) Vec { T x[V]; };

// r / (2 * Hk) for the rows of up to 8 tokens: magic = ceil(2^32 / (2 Hk)) is exact there while
// 8 (2 Hk)^2 < 2^32; 0 (one token a CTA) gives 0.
__device__ __forceinline__ int token_of(int r, uint32_t magic) { return (int)__umulhi((uint32_t)r, magic); }

// 16 bytes as fp32, and fp32 into 16 bytes
__device__ __forceinline__ void unpack(const Vec<float, 4> &x, float (&y)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = x.x[j];
}
__device__ __forceinline__ void unpack(const Vec<__nv_bfloat16, 8> &x, float (&y)[8]) {
    const uint32_t *w = reinterpret_cast<const uint32_t *>(&x);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        y[2 * j] = __uint_as_float(w[j] << 16);
        y[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
}
__device__ __forceinline__ void pack(const float (&x)[4], Vec<float, 4> &y) {
#pragma unroll
    for (int j = 0; j < 4; ++j) y.x[j] = x[j];
}
__device__ __forceinline__ void pack(const float (&x)[8], Vec<__nv_bfloat16, 8> &y) {
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        const __nv_bfloat162 z = __floats2bfloat162_rn(x[j], x[j + 1]);
        y.x[j] = z.x;
        y.x[j + 1] = z.y;
    }
}
// V e4m3, two an instruction
template <int V> __device__ __forceinline__ void to_e4m3(const float (&x)[V], float by, Vec<__nv_fp8_e4m3, V> &y) {
    __nv_fp8x2_storage_t *to = reinterpret_cast<__nv_fp8x2_storage_t *>(&y);
#pragma unroll
    for (int j = 0; j < V; j += 2)
        to[j / 2] = __nv_cvt_float2_to_fp8x2(make_float2(x[j] * by, x[j + 1] * by), __NV_SATFINITE, __NV_E4M3);
}
template <int V> __device__ __forceinline__ void from_e4m3(const Vec<__nv_fp8_e4m3, V> &x, float by, float (&y)[V]) {
    const __nv_fp8x2_storage_t *from = reinterpret_cast<const __nv_fp8x2_storage_t *>(&x);
#pragma unroll
    for (int j = 0; j < V; j += 2) {
        const float2 z = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(from[j / 2], __NV_E4M3)));
        y[j] = z.x * by;
        y[j + 1] = z.y * by;
    }
}

template <typename TX, typename TC, int D>
__global__ void __launch_bounds__(kThreads)
kv_write_kernel(Cache c, const TX *__restrict__ k, const TX *__restrict__ v, int64_t ks, int64_t vs, int each,
                uint32_t magic, StatusWord *st) {
    constexpr int V = 16 / sizeof(TX), L = D / V, R = kThreads / L;   // values a lane; lanes a row; rows at a time
    __shared__ Place places[kMost];
    if (blockIdx.x == 0) check_spans(c, st);
    const int t0 = blockIdx.x * each, count = min(each, c.T - t0), rows = count * 2 * c.Hk;
    const int sub = threadIdx.x / L, lane = threadIdx.x % L * V;
    Vec<TX, V> x[kRows];
    auto load = [&](int r0) {   // a token's keys of all heads, then its values, then the next token's
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int r = r0 + i * R + sub, t = token_of(r, magic), row = r - t * 2 * c.Hk;
            if (r < rows)
                x[i] = *reinterpret_cast<const Vec<TX, V> *>(
                    (row < c.Hk ? k + (t0 + t) * ks + (int64_t)row * D : v + (t0 + t) * vs + (int64_t)(row - c.Hk) * D) + lane);
        }
    };
    load(0);
    if (threadIdx.x < 32) find_places(c, t0, count, places, st, 62);
    __syncthreads();
    for (int r0 = 0; r0 < rows; r0 += kRows * R) {
        if (r0) load(r0);
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int r = r0 + i * R + sub, t = token_of(min(r, rows - 1), magic), row = r - t * 2 * c.Hk;
            const bool key = row < c.Hk;
            const Place to = places[t];
            const int64_t at = ((int64_t)(key ? row : row - c.Hk) << c.shift) + to.slot;
            Vec<TC, V> y;
            if constexpr (sizeof(TC) == 1) {
                float z[V], top = 0.f;
                unpack(x[i], z);
#pragma unroll
                for (int j = 0; j < V; ++j) top = fmaxf(top, fabsf(z[j]));
#pragma unroll
                for (int o = L / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                if (__any_sync(0xffffffffu, top > 3.4028234e38f)) {   // (infinities are stored as 448 s)
                    top = 0.f;
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        const float a = fabsf(z[j]);
                        top = fmaxf(top, a <= 3.4028234e38f ? a : 0.f);
                    }
#pragma unroll
                    for (int o = L / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                }
                const int e = top > 0.f ? scale_exponent(top) : 0;
                to_e4m3(z, two_to(-e), y);
                if (r < rows && to.page >= 0 && lane == 0) (key ? c.ks : c.vs)[to.page * c.scale_stride + at] = two_to(e);
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j) y.x[j] = x[i].x[j];
            }
            if (r < rows && to.page >= 0)
                *reinterpret_cast<Vec<TC, V> *>((TC *)(key ? c.k : c.v) + to.page * c.stride + at * D + lane) = y;
        }
    }
}

template <typename TX, typename TC, int D>
__global__ void __launch_bounds__(kThreads)
kv_read_kernel(Cache c, TX *__restrict__ k, TX *__restrict__ v, int each, uint32_t magic, StatusWord *st) {
    constexpr int V = 16 / sizeof(TX), L = D / V, R = kThreads / L;
    __shared__ Place places[kMost];
    if (blockIdx.x == 0) check_spans(c, st);
    const int t0 = blockIdx.x * each, count = min(each, c.T - t0), rows = count * 2 * c.Hk;
    const int sub = threadIdx.x / L, lane = threadIdx.x % L * V;
    if (threadIdx.x < 32) find_places(c, t0, count, places, st, 63);
    __syncthreads();
    for (int r0 = 0; r0 < rows; r0 += kRows * R) {
        Vec<TC, V> x[kRows];
        float scale[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int r = r0 + i * R + sub, t = token_of(min(r, rows - 1), magic), row = r - t * 2 * c.Hk;
            const bool key = row < c.Hk;
            const Place from = places[t];
            const int64_t at = ((int64_t)(key ? row : row - c.Hk) << c.shift) + from.slot;
            if (r < rows && from.page >= 0) {
                x[i] = *reinterpret_cast<const Vec<TC, V> *>((const TC *)(key ? c.k : c.v) + from.page * c.stride + at * D + lane);
                scale[i] = sizeof(TC) == 1 ? (key ? c.ks : c.vs)[from.page * c.scale_stride + at] : 1.f;
            }
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int r = r0 + i * R + sub, t = token_of(min(r, rows - 1), magic), row = r - t * 2 * c.Hk;
            const int page = places[t].page;
            if (r >= rows || page < -1) continue;
            Vec<TX, V> y;
            float z[V];
            if constexpr (sizeof(TC) == 1) from_e4m3(x[i], scale[i], z);
            else unpack(x[i], z);
            if (page < 0) {
#pragma unroll
                for (int j = 0; j < V; ++j) z[j] = 0.f;
            }
            pack(z, y);
            *reinterpret_cast<Vec<TX, V> *>((row < c.Hk ? k + ((int64_t)(t0 + t) * c.Hk + row) * D
                                                        : v + ((int64_t)(t0 + t) * c.Hk + row - c.Hk) * D) + lane) = y;
        }
    }
}

template <typename TX, typename TC, int D>
static cudaError_t launch(bool write, const Cache &c, void *k, void *v, int64_t ks, int64_t vs, StatusWord *st,
                          cudaStream_t s) {
    const int d = 2 * c.Hk;
    const int each = d >= 16384 || c.T < 2048 ? 1 : c.T < 16384 ? 4 : kMost;
    const uint32_t magic = each > 1 ? (uint32_t)((((uint64_t)1 << 32) + d - 1) / d) : 0u;
    const unsigned ctas = (unsigned)(((int64_t)c.T + each - 1) / each);
    if (write)
        kv_write_kernel<TX, TC, D><<<ctas, kThreads, 0, s>>>(c, (const TX *)k, (const TX *)v, ks, vs, each, magic, st);
    else
        kv_read_kernel<TX, TC, D><<<ctas, kThreads, 0, s>>>(c, (TX *)k, (TX *)v, each, magic, st);
    return cudaGetLastError();
}

template <typename TX, typename TC>
static cudaError_t launch_d(bool write, int D, const Cache &c, void *k, void *v, int64_t ks, int64_t vs, StatusWord *st,
                            cudaStream_t s) {
    if (D == 32) return launch<TX, TC, 32>(write, c, k, v, ks, vs, st, s);
    if (D == 64) return launch<TX, TC, 64>(write, c, k, v, ks, vs, st, s);
    return launch<TX, TC, 128>(write, c, k, v, ks, vs, st, s);
}

}  // namespace paged

// write: k, v [T, Hk, D] with token strides; else read, packed outputs
cudaError_t launch_kv_cache(bool write, int dtype, int cache_dtype, int D, const paged::Cache &c, void *k, void *v,
                            int64_t ks, int64_t vs, StatusWord *st, cudaStream_t s) {
    using paged::launch_d;
    const bool e4m3 = cache_dtype == KDA_E4M3;
    if (dtype == KDA_F32)
        return e4m3 ? launch_d<float, __nv_fp8_e4m3>(write, D, c, k, v, ks, vs, st, s)
                    : launch_d<float, float>(write, D, c, k, v, ks, vs, st, s);
    return e4m3 ? launch_d<__nv_bfloat16, __nv_fp8_e4m3>(write, D, c, k, v, ks, vs, st, s)
                : launch_d<__nv_bfloat16, __nv_bfloat16>(write, D, c, k, v, ks, vs, st, s);
}

}  // namespace kda
