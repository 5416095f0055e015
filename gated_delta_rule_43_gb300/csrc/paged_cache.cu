// paged_cache.cu -- new keys and values into the pages of a cache, and back.
//
//   write: row x of D values   ->  x, or e4m3(x / s) and s = 2^e, e least with max|x| / s <= 448
//   read:  the row             ->  x, or s * e4m3
// Memory-bound: each row is read once and written once.  A row is spread over D * size / 16 lanes, 16
// bytes each (of the wider side); a warp looks its token's place up once and moves kRows rows for
// each group of lanes, all loads before the first store.
#include "kda_paged.cuh"

namespace kda {
namespace paged {

constexpr int kThreads = 128, kRows = 4;

template <typename T, int V> struct alignas(sizeof(T) * V) Vec { T x[V]; };

template <typename TX, typename TC, int D>
__global__ void __launch_bounds__(kThreads)
kv_write_kernel(Cache c, const TX *__restrict__ k, const TX *__restrict__ v, int64_t ks, int64_t vs,
                int parts, StatusWord *st) {
    constexpr int V = 16 / sizeof(TX), L = D / V, R = 32 / L;   // values a lane; lanes a row; rows at a time
    if (blockIdx.x == 0) check_spans(c, st);
    const int lane = threadIdx.x & 31;
    const int64_t unit = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int64_t t = unit / parts;
    if (t >= c.T) return;
    const int part = (int)(unit - t * parts);
    // this lane's rows: keys of all heads, then values
    Vec<TX, V> x[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int row = (part * kRows + i) * R + lane / L;
        if (row < 2 * c.Hk)
            x[i] = *reinterpret_cast<const Vec<TX, V> *>(
                (row < c.Hk ? k + t * ks + (int64_t)row * D : v + t * vs + (int64_t)(row - c.Hk) * D) + lane % L * V);
    }
    const int n = c.cu ? sequence_of(c, (int)t) : (int)t;
    if (n < 0) return;
    const Span s = span_of(c, n);
    if (t < s.begin || t >= s.begin + s.len) return;
    const int pos = s.pos + (int)(t - s.begin);
    if (pos < 0) return;
    const int page = c.table[(int64_t)n * c.width + (pos >> c.shift)], slot = pos & ((1 << c.shift) - 1);
    if (page < 0 || page >= c.P) {
        if (lane == 0) report(st, KDA_ERR_INVALID_ARG, n, 62);
        return;
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int row = (part * kRows + i) * R + lane / L;
        const bool key = row < c.Hk;
        const int64_t at = ((int64_t)(key ? row : row - c.Hk) << c.shift) + slot;
        TC *to = (TC *)(key ? c.k : c.v) + page * c.stride + at * D + lane % L * V;
        Vec<TC, V> y;
        if constexpr (sizeof(TC) == 1) {
            float top = 0.f;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float a = fabsf(to_f(x[i].x[j]));
                top = fmaxf(top, a <= 3.4028234e38f ? a : 0.f);   // (infinities are stored as 448 s)
            }
#pragma unroll
            for (int o = L / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            const int e = top > 0.f ? scale_exponent(top) : 0;
            const float inv = two_to(-e);
#pragma unroll
            for (int j = 0; j < V; ++j) y.x[j] = TC(to_f(x[i].x[j]) * inv);
            if (row < 2 * c.Hk && lane % L == 0) (key ? c.ks : c.vs)[page * c.scale_stride + at] = two_to(e);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) y.x[j] = x[i].x[j];
        }
        if (row < 2 * c.Hk) *reinterpret_cast<Vec<TC, V> *>(to) = y;
    }
}

template <typename TX, typename TC, int D>
__global__ void __launch_bounds__(kThreads)
kv_read_kernel(Cache c, TX *__restrict__ k, TX *__restrict__ v, int parts, StatusWord *st) {
    constexpr int V = 16 / sizeof(TX), L = D / V, R = 32 / L;
    if (blockIdx.x == 0) check_spans(c, st);
    const int lane = threadIdx.x & 31;
    const int64_t unit = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int64_t t = unit / parts;
    if (t >= c.T) return;
    const int part = (int)(unit - t * parts);
    const int n = c.cu ? sequence_of(c, (int)t) : (int)t;
    if (n < 0) return;
    const Span s = span_of(c, n);
    if (t < s.begin || t >= s.begin + s.len) return;
    const int pos = s.pos + (int)(t - s.begin);
    int page = -1, slot = 0;
    if (pos >= 0) {
        page = c.table[(int64_t)n * c.width + (pos >> c.shift)];
        slot = pos & ((1 << c.shift) - 1);
        if (page < 0 || page >= c.P) {
            if (lane == 0) report(st, KDA_ERR_INVALID_ARG, n, 63);
            page = -1;
        }
    }
    Vec<TC, V> x[kRows];
    float scale[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int row = (part * kRows + i) * R + lane / L;
        const bool key = row < c.Hk;
        const int64_t at = ((int64_t)(key ? row : row - c.Hk) << c.shift) + slot;
        if (row < 2 * c.Hk && page >= 0) {
            x[i] = *reinterpret_cast<const Vec<TC, V> *>((const TC *)(key ? c.k : c.v) + page * c.stride + at * D +
                                                         lane % L * V);
            scale[i] = sizeof(TC) == 1 ? (key ? c.ks : c.vs)[page * c.scale_stride + at] : 1.f;
        }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int row = (part * kRows + i) * R + lane / L;
        if (row >= 2 * c.Hk) continue;
        Vec<TX, V> y;
#pragma unroll
        for (int j = 0; j < V; ++j)
            y.x[j] = from_f<TX>(page < 0 ? 0.f
                                         : sizeof(TC) == 1 ? stored_to_f(x[i].x[j]) * scale[i] : stored_to_f(x[i].x[j]));
        *reinterpret_cast<Vec<TX, V> *>((row < c.Hk ? k + (t * c.Hk + row) * D : v + (t * c.Hk + row - c.Hk) * D) +
                                        lane % L * V) = y;
    }
}

template <typename TX, typename TC, int D>
static cudaError_t launch(bool write, const Cache &c, void *k, void *v, int64_t ks, int64_t vs, StatusWord *st,
                          cudaStream_t s) {
    constexpr int R = 32 / (D * (int)sizeof(TX) / 16) * kRows;   // rows a warp
    const int parts = (2 * c.Hk + R - 1) / R;
    const int64_t units = (int64_t)c.T * parts;
    const int64_t ctas = (units + kThreads / 32 - 1) / (kThreads / 32);
    if (ctas > 0x7fffffff) return cudaErrorInvalidValue;
    if (write)
        kv_write_kernel<TX, TC, D><<<(unsigned)ctas, kThreads, 0, s>>>(c, (const TX *)k, (const TX *)v, ks, vs, parts, st);
    else
        kv_read_kernel<TX, TC, D><<<(unsigned)ctas, kThreads, 0, s>>>(c, (TX *)k, (TX *)v, parts, st);
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
