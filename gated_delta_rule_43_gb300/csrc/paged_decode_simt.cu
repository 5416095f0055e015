// paged_decode_simt.cu -- attention of one new token a sequence over paged keys and values in single precision,
// on the CUDA cores.
//
//   o = sum_j w_j v_j / sum_j w_j,   w_j = 2^(s_j - m),   s_j = scale log2(e) q k_j
// Memory-bound: each key and value is read once for up to NR query heads that share it (NR = 8, 4 from e4m3 pages:
// more are further items, which read it again), 16 bytes a lane, so a
// row of D values takes L = D / V lanes and a warp's load G = 32 / L rows.  Each lane multiplies its V channels of
// U rows with those of the NR queries, and the U * NR sums over the L lanes of a row are put together by halves: a
// lane passes on the half that is its neighbour's, so that each ends up with U * NR / L scores of its own, one
// shuffle a score (five, added up one by one).  Maxima move only when they would grow by more than 2^8; sums
// are fp32.
//
// The work is cut as for the tensor cores (paged_decode_tc.cu), into two ranges an SM.  A CTA's eight
// warps take every eighth unit of 32 keys, each with its own maxima, and meet at an item's end.  64 sequences of
// 512 to 8192 tokens, 32 heads on 8 of 128, fp32: 391 to 399 us, 5.7 to 5.8 TB/s (four heads an item spill 108 bytes; from
// e4m3 pages 351); 4 of 300 to 20000, 8 heads of 64: 40 us.
#include "kda_paged_tc.cuh"

namespace kda {
namespace paged {
namespace tc {
namespace one {
namespace simt {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kUnit = 32;           // keys

template <typename TC, int D, int NR> struct Shape {
    static constexpr int V = 16 / sizeof(TC), L = D / V, G = 32 / L;      // values a lane; lanes a row; rows a load
    static constexpr int U = V == 4 ? (NR == 8 ? 4 : 8) : 2;   // loads of a step
    static constexpr int M = U * NR;                                      // scores of a row of lanes
    static constexpr int m = M > L ? M / L : 1, DUP = L > M ? L / M : 1;  // ... of a lane; lanes that share one
    static constexpr int MG = m < NR ? m : NR;                            // heads that a lane has scores of
    static constexpr int kSame = DUP * (NR / MG);                         // from here on, lane bits leave them the same
    static constexpr int kStep = U * G;                                   // keys
    static_assert(kUnit % kStep == 0 && (m % NR == 0 || NR % m == 0), "shape");
};

// 16 bytes as fp32
__device__ __forceinline__ void widen(const uint4 &x, float (&y)[4]) {
    y[0] = __uint_as_float(x.x);
    y[1] = __uint_as_float(x.y);
    y[2] = __uint_as_float(x.z);
    y[3] = __uint_as_float(x.w);
}
__device__ __forceinline__ void widen(const uint4 &x, float (&y)[16]) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 z = __half22float2(__half2(
            __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i / 2] >> (16 * (i & 1))), __NV_E4M3)));
        y[2 * i] = z.x;
        y[2 * i + 1] = z.y;
    }
}

template <typename TC, int D, int NR>
__global__ void __launch_bounds__(kThreads, 2)
paged_decode_simt_kernel(Cache c, Plan p, const float *__restrict__ q, int64_t q_stride, float *__restrict__ o, int group,
                         float scale, int window, int sinks) {
    using S = Shape<TC, D, NR>;
    constexpr int V = S::V, L = S::L, G = S::G, U = S::U, M = S::M, m = S::m, MG = S::MG;
    __shared__ __align__(16) float sq[NR][D];
    __shared__ __align__(16) float red[kWarps][NR][D];
    __shared__ float2 ends[kWarps][NR];
    __shared__ Cut cuts[2];
    __shared__ int64_t sums[kWarps];
    __shared__ StatusWord found;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, sub = lane % L, r = lane / L;
    let_next_start();
    const int groups = (group + NR - 1) / NR;
    if (tid == 0) found = StatusWord{0, 0, 0};
    own_range(c, p.ranges, groups, window, sinks, sums, cuts, &found);
    if (tid < 2 && (tid == 0 || blockIdx.x + 1 == p.ranges)) p.cuts[blockIdx.x + tid] = cuts[tid];
    Cut from = cuts[0];
    const Cut to = cuts[1];
    const float f = scale * kLog2e;
    const int mask = (1 << c.shift) - 1;
    while (true) {
        Span s{0, 0, 0};
        while (from.n < c.N && (from.tile < to.tile || (from.tile == to.tile && (from.h < to.h || (from.h == to.h && from.k < to.k))))) {
            s = span_of(c, from.n);
            if (s.len) break;
            ++from.n;   // (a sequence that does not fit)
            from.t = from.h = from.k = 0;
            from.tile = from.n * groups;
        }
        if (s.len == 0) break;
        const int n = from.n, h = from.h, pos = s.pos, row0 = from.t * NR, rows = min(NR, group - row0);
        const KeyBlocks kb = key_blocks(max(0, pos), pos, window, sinks, BK);
        const int k0 = from.k, k1 = same_item(from, to) ? min(to.k, kb.count) : kb.count;
        const int lowest = window > 0 ? pos - window : -1;   // keys above it are in the window
        __syncthreads();   // (the last item's sums have been read)
        for (int x = tid; x < NR * D; x += kThreads)
            sq[x / D][x % D] = x < rows * D ? q[(int64_t)n * q_stride + (int64_t)(h * group + row0) * D + x] * f : 0.f;
        __syncthreads();

        float top[MG], l[MG], acc[NR][V];
#pragma unroll
        for (int i = 0; i < MG; ++i) {
            top[i] = -INFINITY;
            l[i] = 0.f;
        }
#pragma unroll
        for (int g = 0; g < NR; ++g)
#pragma unroll
            for (int v = 0; v < V; ++v) acc[g][v] = 0.f;
        const int units = (k1 - k0) * (BK / kUnit);
        auto key_of = [&](int x) { return kb.block(k0 + x / (BK / kUnit)) * BK + x % (BK / kUnit) * kUnit; };
        // the page of this lane's half (16 keys) of a unit, or -1: nothing of it is visible
        auto page_of = [&](int x) {
            if (x >= units) return -1;
            const int half = key_of(x) + (lane & 16);
            const bool seen = half <= pos && (half + 15 > lowest || half < sinks);
            if (!seen) return -1;
            const int page = c.table[(int64_t)n * c.width + (half >> c.shift)];
            if (page >= 0 && page < c.P) return page;
            report(&found, KDA_ERR_INVALID_ARG, n, 95);
            return -1;   // (zeros)
        };
        int next = page_of(warp);
        for (int x = warp; x < units; x += kWarps) {
            const int page = next, key0 = key_of(x), key = key0 + lane;
            next = page_of(x + kWarps);
            const bool seen = key <= pos && (key > lowest || key < sinks);
            const uint32_t vis = __ballot_sync(0xffffffffu, seen), load = __ballot_sync(0xffffffffu, seen && page >= 0);
            float ks = 0.f, vs = 0.f;
            if (sizeof(TC) == 1 && seen && page >= 0) {
                const int64_t at = page * c.scale_stride + ((int64_t)h << c.shift) + (key & mask);
                ks = c.ks[at];
                vs = c.vs[at];
            }
            // where the unit's two halves lie
            int64_t half[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int y = max(0, __shfl_sync(0xffffffffu, page, 16 * i));
                half[i] = y * c.stride + (((int64_t)h << c.shift) + ((key0 + 16 * i) & mask)) * D + r * D + sub * V;
            }
#pragma unroll 1
            for (int k = 0; k < kUnit; k += S::kStep) {
                if ((vis >> k & (uint32_t)((1ull << S::kStep) - 1)) == 0) continue;
                uint4 kx[U], vx[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    kx[u] = vx[u] = make_uint4(0, 0, 0, 0);
                    const int at = k + u * G;
                    if (load >> (at + r) & 1) {
                        const int64_t y = (at & 16 ? half[1] : half[0]) + (at & 15) * D;
                        kx[u] = __ldg(reinterpret_cast<const uint4 *>((const TC *)c.k + y));
                        vx[u] = __ldg(reinterpret_cast<const uint4 *>((const TC *)c.v + y));
                    }
                }
                float y[M];   // [row u][head g]
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float kf[V];
                    widen(kx[u], kf);
#pragma unroll
                    for (int g = 0; g < NR; ++g) {
                        float z = 0.f;
#pragma unroll
                        for (int v = 0; v < V; v += 4) {
                            const float4 w = *reinterpret_cast<const float4 *>(&sq[g][sub * V + v]);
                            z = fmaf(w.x, kf[v], z);
                            z = fmaf(w.y, kf[v + 1], z);
                            z = fmaf(w.z, kf[v + 2], z);
                            z = fmaf(w.w, kf[v + 3], z);
                        }
                        y[u * NR + g] = z;
                    }
                }
                // over the lanes of a row: lane `sub` ends up with sums (sub / DUP) * m ..
#pragma unroll
                for (int i = 1; L >> i; ++i) {
                    const int off = L >> i, count = M >> i;   // sums that are left
                    if (count > 0) {
                        const bool upper = lane & off;
#pragma unroll
                        for (int j = 0; j < count; ++j) {
                            const float mine = upper ? y[j + count] : y[j], other = upper ? y[j] : y[j + count];
                            y[j] = mine + __shfl_xor_sync(0xffffffffu, other, off);
                        }
                    } else {
                        y[0] += __shfl_xor_sync(0xffffffffu, y[0], off);
                    }
                }
                const int j0 = sub / S::DUP * m;
                float high[MG];
#pragma unroll
                for (int i = 0; i < MG; ++i) high[i] = -INFINITY;
#pragma unroll
                for (int i = 0; i < m; ++i) {
                    const int at = k + (j0 + i) / NR * G + r;
                    if (sizeof(TC) == 1) y[i] *= __shfl_sync(0xffffffffu, ks, at);
                    y[i] = vis >> at & 1 ? y[i] : -INFINITY;
                    high[i % MG] = fmaxf(high[i % MG], y[i]);
                }
                bool grown = false;
#pragma unroll
                for (int i = 0; i < MG; ++i) {
#pragma unroll
                    for (int off = S::kSame; off < 32; off *= 2) high[i] = fmaxf(high[i], __shfl_xor_sync(0xffffffffu, high[i], off));
                    grown |= high[i] > top[i] && !(high[i] - top[i] <= 8.f);
                }
                if (__any_sync(0xffffffffu, grown)) {
                    float keep[MG];
#pragma unroll
                    for (int i = 0; i < MG; ++i) {
                        const float t = fmaxf(top[i], high[i]);
                        keep[i] = t == top[i] ? 1.f : ex2(top[i] - t);
                        top[i] = t;
                        l[i] *= keep[i];
                    }
#pragma unroll
                    for (int g = 0; g < NR; ++g) {
                        const float z = __shfl_sync(0xffffffffu, keep[g % MG], g / MG * S::DUP);
#pragma unroll
                        for (int v = 0; v < V; ++v) acc[g][v] *= z;
                    }
                }
#pragma unroll
                for (int i = 0; i < m; ++i) {
                    y[i] = ex2(y[i] - (top[i % MG] == -INFINITY ? 0.f : top[i % MG]));
                    l[i % MG] += y[i];
                    if (sizeof(TC) == 1) y[i] *= __shfl_sync(0xffffffffu, vs, k + (j0 + i) / NR * G + r);
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float vf[V];
                    widen(vx[u], vf);
#pragma unroll
                    for (int g = 0; g < NR; ++g) {
                        const int j = u * NR + g;
                        const float w = __shfl_sync(0xffffffffu, y[j % m], j / m * S::DUP, L);
#pragma unroll
                        for (int v = 0; v < V; ++v) acc[g][v] = fmaf(w, vf[v], acc[g][v]);
                    }
                }
            }
        }
        // The item's end: a warp's sums, then those of all warps
#pragma unroll
        for (int i = 0; i < MG; ++i) {
#pragma unroll
            for (int off = S::kSame; off < 32; off *= 2) l[i] += __shfl_xor_sync(0xffffffffu, l[i], off);
            if (r == 0 && sub < S::kSame && sub % S::DUP == 0) ends[warp][sub / S::DUP * MG + i] = make_float2(top[i], l[i]);
        }
#pragma unroll
        for (int g = 0; g < NR; ++g) {
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int off = L; off < 32; off *= 2) acc[g][v] += __shfl_xor_sync(0xffffffffu, acc[g][v], off);
            if (r == 0)
#pragma unroll
                for (int v = 0; v < V; v += 4)
                    *reinterpret_cast<float4 *>(&red[warp][g][sub * V + v]) =
                        make_float4(acc[g][v], acc[g][v + 1], acc[g][v + 2], acc[g][v + 3]);
        }
        __syncthreads();
        const int slot = k0 > 0 ? 2 * (int)blockIdx.x : k1 < kb.count ? 2 * (int)blockIdx.x + 1 : -1;
        for (int x = tid; x < rows * D; x += kThreads) {
            const int g = x / D, d = x % D;
            float high = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) high = fmaxf(high, ends[w][g].x);
            const float ref = high == -INFINITY ? 0.f : high;
            float sum = 0.f, z = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float2 e = ends[w][g];
                const float by = e.y != 0.f ? ex2(e.x - ref) : 0.f;
                sum += by * e.y;
                z += by * red[w][g][d];
            }
            if (slot >= 0) {
                const int64_t at = (int64_t)slot * p.rows + g;
                if (d == 0) p.ml[at] = make_float2(ref, sum);
                p.part[at * D + d] = z;
            } else {
                o[((int64_t)n * c.Hk * group + h * group + row0) * D + x] = sum != 0.f ? z / sum : 0.f;
            }
        }
        from.k = 0;
        if (++from.h == c.Hk) {
            from.h = 0;
            ++from.tile;
            if (++from.t == groups) {
                from.t = 0;
                ++from.n;
            }
        }
    }
    __syncthreads();
    if (tid == 0) p.found[blockIdx.x] = found;
}

struct Layout {
    int ranges, rows, each;
    size_t cuts, found, ml, part, total;
};
static Layout layout_of(bool e4m3, int group, int D, int sms) {
    Layout L;
    L.each = group == 1 ? 1 : group <= 4 || e4m3 ? 4 : 8;
    L.rows = group < L.each ? group : L.each;
    L.ranges = 2 * sms;
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    L.cuts = kHeaderBytes;
    L.found = L.cuts + up(sizeof(Cut) * ((size_t)L.ranges + 1));
    L.ml = L.found + up(sizeof(StatusWord) * L.ranges);
    L.part = L.ml + up(sizeof(float2) * 2 * L.ranges * L.rows);
    L.total = L.part + sizeof(float) * 2 * L.ranges * L.rows * D;
    return L;
}

template <typename TC, int D, int NR>
static cudaError_t launch(const Layout &L, const Cache &c, const void *q, int64_t qs, void *o, int group, float scale,
                          int window, int sinks, uint8_t *ws, cudaStream_t s) {
    const Plan p{nullptr, nullptr, (Cut *)(ws + L.cuts), (float *)(ws + L.part), (float2 *)(ws + L.ml), L.ranges, L.rows,
                 L.each, (StatusWord *)(ws + L.found), 0};
    paged_decode_simt_kernel<TC, D, NR>
        <<<L.ranges, kThreads, 0, s>>>(c, p, (const float *)q, qs, (float *)o, group, scale, window, sinks);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? launch_join(true, D, c, p, o, group, (StatusWord *)ws, s) : e;
}

}  // namespace simt
}  // namespace one
}  // namespace tc
}  // namespace paged

size_t paged_decode_simt_bytes(bool e4m3, int group, int D, int sms) {
    return paged::tc::one::simt::layout_of(e4m3, group, D, sms).total;
}

cudaError_t launch_paged_decode_simt(bool e4m3, int D, const paged::Cache &c, const void *q, int64_t qs, void *o, int group,
                                     float scale, int window, int sinks, void *ws, int sms, cudaStream_t s) {
    using paged::tc::one::simt::launch;
    const auto L = paged::tc::one::simt::layout_of(e4m3, group, D, sms);
#define KDA_ONE(T_, E_, D_, NR_) \
    if (e4m3 == E_ && D == D_ && L.each == NR_) return launch<T_, D_, NR_>(L, c, q, qs, o, group, scale, window, sinks, (uint8_t *)ws, s);
#define KDA_ONES(D_)                                                                                       \
    KDA_ONE(float, false, D_, 1) KDA_ONE(float, false, D_, 4) KDA_ONE(float, false, D_, 8)                 \
    KDA_ONE(__nv_fp8_e4m3, true, D_, 1) KDA_ONE(__nv_fp8_e4m3, true, D_, 4)
    KDA_ONES(32) KDA_ONES(64) KDA_ONES(128)
#undef KDA_ONES
#undef KDA_ONE
    return cudaErrorInvalidValue;
}

}  // namespace kda
