// paged_attn_simt.cu -- attention of a chunk of new tokens over a paged cache in single precision, on the CUDA cores;
// and any attention over a pool without pages.
//
//   o_i = sum_j w_ij v_j / sum_j w_ij,   w_ij = exp(scale q_i k_j - m_i),   m_i the largest exponent
// One pass over the keys with the running maximum and sum.  The query heads that share a key/value head
// are rows beside each other (row = token * group + head), so that keys are read once for all of
// them.  A CTA takes 64 rows and goes through blocks of 32 keys staged in shared memory as fp32; a thread has 4
// rows and 4 keys of the scores, and of the outputs 4 rows and every eighth four channels, so that it multiplies 8 to 13 times
// for every 16 bytes that it reads from there.  Where there are few rows, `splits` CTAs share their keys and a
// second kernel joins what they found.  4096 new tokens, 8 heads on 2 of 128: 0.98 to 1.0 ms (0.97 from e4m3 pages), 35 TFLOP/s of the 74 that fp32
// multiply-adds reach; the stores that stage a block and the reads of it are what the rest goes to.
#include "kda_paged.cuh"

namespace kda {
namespace paged {
namespace simt {

constexpr int BR = 64, BK = 32, kThreads = 128;
// Blocks in one sum (8192 keys): a longer one leaves out what is small beside it (behind 1 M tokens 9e-5 on average, 3.7e-4 at
// most; 65536 8e-6; with 1024 blocks a sum 2.7e-5 behind 1 M), so sums go to the outputs' place, in fp32 as they are, and begin again.  (Sums of weights have 32 times fewer terms.)  Then 8e-6
// behind 1 M.
constexpr int kSum = 256;
constexpr float kLog2e = 1.4426950408889634f;

// Rows [first, first + rows) of sequence n's len * group.
struct Tile {
    int n, first, rows;
    Span s;
};
// The `tile`-th tile of 64 rows in the batch; a whole warp.  False past the last.
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

// Where a key lies: -1: nowhere, or nobody sees it (zeros).
struct Place {
    int64_t at;
    float ks, vs;
};
struct Found {
    Tile tile;
    int there;
    int64_t rows[kThreads / 32 - 1];   // of all sequences, added up by three warps
};
// The `tile`-th tile for a whole block.  False past the last, and where the sequences have more rows than there
// are (of a cu_seqlens that goes back, which has been reported): none is gone through then.
__device__ __forceinline__ bool find(const Cache &c, int tile, int group, Found &found) {
    const int tid = threadIdx.x;
    if (tid < 32) {
        Tile t;
        const bool there = find_tile(c, tile, group, t);
        if (tid == 0) {
            found.there = there;
            if (there) found.tile = t;
        }
    } else {
        int64_t rows = 0;
        for (int n = tid - 32; n < c.N; n += kThreads - 32) rows += span_of(c, n).len;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) rows += __shfl_xor_sync(0xffffffffu, rows, o);
        if (tid % 32 == 0) found.rows[tid / 32 - 1] = rows;
    }
    __syncthreads();
    return found.there && found.rows[0] + found.rows[1] + found.rows[2] <= c.T;
}
static_assert(kThreads == 128, "three warps beside the first");
template <int D> struct Shared {   // (D = 128: 76800 bytes, three CTAs an SM)
    float q[BR][D + 4];
    float k[BK][D + 4];
    float v[BK][D];
    union {
        float p[BR][BK + 4];
        Found found;   // (before the first weights)
    };
    Place places[BK];
};

// V stored values as fp32, times s
__device__ __forceinline__ void widen(const uint4 &x, float s, float (&y)[4], float) {
    y[0] = __uint_as_float(x.x);
    y[1] = __uint_as_float(x.y);
    y[2] = __uint_as_float(x.z);
    y[3] = __uint_as_float(x.w);
}
__device__ __forceinline__ void widen(const uint4 &x, float s, float (&y)[16], __nv_fp8_e4m3) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 z = __half22float2(__half2(
            __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i / 2] >> (16 * (i & 1))), __NV_E4M3)));
        y[2 * i] = z.x * s;
        y[2 * i + 1] = z.y * s;
    }
}

template <typename TC, int D>
__global__ void __launch_bounds__(kThreads, D == 128 ? 3 : D == 32 && sizeof(TC) == 1 ? 5 : 4)
paged_simt_kernel(Cache c, const float *__restrict__ q, int64_t q_stride, float *__restrict__ o, int group, float scale,
                  int window, int sinks, int splits, float *__restrict__ part, StatusWord *st) {
    constexpr int V = 16 / sizeof(TC), R = 4, C = D / 32;   // values a load; rows a thread; channels of it, in fours
    extern __shared__ __align__(16) uint8_t raw[];
    Shared<D> &sm = *reinterpret_cast<Shared<D> *>(raw);
    const int tid = threadIdx.x, H = c.Hk * group;
    const int tile = (gridDim.x - 1 - blockIdx.x) / c.Hk, h = (gridDim.x - 1 - blockIdx.x) % c.Hk, split = blockIdx.y;
    if (blockIdx.x == 0 && split == 0) check_spans(c, st);
    if (!find(c, tile, group, sm.found)) return;
    const Tile t = sm.found.tile;
    const float f = scale * kLog2e;
    for (int x = tid; x < BR * D; x += kThreads) {
        const int r = x / D, d = x % D;
        float y = 0.f;
        if (r < t.rows) {
            const int at = t.first + r;
            y = q[(int64_t)(t.s.begin + at / group) * q_stride + (int64_t)(h * group + at % group) * D + d] * f;
        }
        sm.q[r][d] = y;
    }
    // this thread's rows r0 + 16 i, keys k0 + 8 j of a block, channels 4 k0 + 32 j
    const int r0 = tid / 8, k0 = tid % 8;
    const int first = max(0, t.s.pos + t.first / group);    // the earliest token's position
    const KeyBlocks kb = key_blocks(first, t.s.pos + (t.first + t.rows - 1) / group, window, sinks, BK);
    const int b0 = (int)((int64_t)kb.count * split / splits), b1 = (int)((int64_t)kb.count * (split + 1) / splits);
    const int ctx = t.s.pos + t.s.len;
    int pos[R], lowest[R];   // keys above lowest are in the row's window
    float m[R], l[R], acc[R][C][4];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        pos[i] = t.s.pos + (t.first + min(r0 + 16 * i, t.rows - 1)) / group;
        lowest[i] = window > 0 ? max(max(pos[i], 0) - window, -1) : -1;
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int j = 0; j < C; ++j) acc[i][j][0] = acc[i][j][1] = acc[i][j][2] = acc[i][j][3] = 0.f;
    }
    // A row's outputs: o, or [tile, head][split][row] of `part`: D sums, the maximum, the sum of weights
    auto place = [&](int r) {
        const int at = t.first + r;
        return splits > 1 ? part + (((int64_t)blockIdx.x * splits + split) * BR + r) * (D + 4)
                          : o + ((int64_t)(t.s.begin + at / group) * H + h * group + at % group) * D;
    };
    // Adds what stands in the outputs' place to the sums (a thread's own elements); its maximum stands behind the
    // row's queries
    auto take = [&](int i) {
        const float was = sm.q[r0 + 16 * i][D], by = was == -INFINITY ? 0.f : exp2f(was - m[i]);
        if (by == 0.f || r0 + 16 * i >= t.rows) return;
        const float *from = place(r0 + 16 * i);
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const float4 y = *reinterpret_cast<const float4 *>(from + 32 * j + 4 * k0);
            acc[i][j][0] = fmaf(by, y.x, acc[i][j][0]);
            acc[i][j][1] = fmaf(by, y.y, acc[i][j][1]);
            acc[i][j][2] = fmaf(by, y.z, acc[i][j][2]);
            acc[i][j][3] = fmaf(by, y.w, acc[i][j][3]);
        }
    };
    auto look_up = [&](int b) {   // the place of block b's key tid
        const int key = kb.block(b) * BK + tid;
        Place y{-1, 0.f, 0.f};
        const bool seen = key < ctx && (window <= 0 || key < sinks || key > first - window);   // (what nobody sees may be anything)
        if (seen) {
            const int page = c.table[(int64_t)t.n * c.width + (key >> c.shift)];
            if (page >= 0 && page < c.P) {
                const int64_t at = ((int64_t)h << c.shift) + (key & ((1 << c.shift) - 1));
                y.at = page * c.stride + at * D;
                if (sizeof(TC) == 1) {
                    y.ks = c.ks[page * c.scale_stride + at];
                    y.vs = c.vs[page * c.scale_stride + at];
                }
            } else {
                report(st, KDA_ERR_INVALID_ARG, t.n, 64);
            }
        }
        return y;
    };
    if (tid < BK && b0 < b1) sm.places[tid] = look_up(b0);
    __syncthreads();
    for (int b = b0; b < b1;) {
        const int stop = min(b1, b + kSum);
        if (b > b0) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                if (b - b0 > kSum) take(i);
                __syncwarp();   // (a warp's rows are its own)
                if (k0 == 0) sm.q[r0 + 16 * i][D] = m[i];
                float *to = place(r0 + 16 * i);
#pragma unroll
                for (int j = 0; j < C; ++j) {
                    if (r0 + 16 * i < t.rows)
                        *reinterpret_cast<float4 *>(to + 32 * j + 4 * k0) = make_float4(acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]);
                    acc[i][j][0] = acc[i][j][1] = acc[i][j][2] = acc[i][j][3] = 0.f;
                }
            }
        }
        for (; b < stop; ++b) {
            const int key0 = kb.block(b) * BK;
#pragma unroll 4
            for (int x = tid; x < BK * D / V; x += kThreads) {
                const int j = x / (D / V), d = x % (D / V) * V;
                const Place y = sm.places[j];
                uint4 kx = make_uint4(0, 0, 0, 0), vx = kx;
                if (y.at >= 0) {
                    kx = __ldg(reinterpret_cast<const uint4 *>((const TC *)c.k + y.at + d));
                    vx = __ldg(reinterpret_cast<const uint4 *>((const TC *)c.v + y.at + d));
                }
                float kf[V], vf[V];
                widen(kx, y.ks, kf, TC());
                widen(vx, y.vs, vf, TC());
#pragma unroll
                for (int i = 0; i < V; i += 4) {
                    *reinterpret_cast<float4 *>(&sm.k[j][d + i]) = make_float4(kf[i], kf[i + 1], kf[i + 2], kf[i + 3]);
                    *reinterpret_cast<float4 *>(&sm.v[j][d + i]) = make_float4(vf[i], vf[i + 1], vf[i + 2], vf[i + 3]);
                }
            }
            __syncthreads();
            Place next{-1, 0.f, 0.f};   // (on its way while the scores are formed)
            if (tid < BK && b + 1 < b1) next = look_up(b + 1);
            float s[R][4];
#pragma unroll
            for (int i = 0; i < R; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
#pragma unroll 4
            for (int d = 0; d < D; d += 4) {
                float4 x[R];
#pragma unroll
                for (int i = 0; i < R; ++i) x[i] = *reinterpret_cast<const float4 *>(&sm.q[r0 + 16 * i][d]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float4 y = *reinterpret_cast<const float4 *>(&sm.k[k0 + 8 * j][d]);
#pragma unroll
                    for (int i = 0; i < R; ++i)
                        s[i][j] = fmaf(x[i].x, y.x, fmaf(x[i].y, y.y, fmaf(x[i].z, y.z, fmaf(x[i].w, y.w, s[i][j]))));
                }
            }
#pragma unroll
            for (int i = 0; i < R; ++i) {
                float top = m[i];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int key = key0 + k0 + 8 * j;
                    s[i][j] = key <= pos[i] && (key > lowest[i] || key < sinks) ? s[i][j] : -INFINITY;
                    top = fmaxf(top, s[i][j]);
                }
#pragma unroll
                for (int x = 1; x < 8; x *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
                const float ref = top == -INFINITY ? 0.f : top;
                const float keep = exp2f(m[i] - ref);
                m[i] = top;
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float p = exp2f(s[i][j] - ref);
                    sum += p;
                    sm.p[r0 + 16 * i][k0 + 8 * j] = p;
                }
                l[i] = l[i] * keep + sum;   // (of this thread's keys: joined at the end)
#pragma unroll
                for (int j = 0; j < C; ++j)
#pragma unroll
                    for (int x = 0; x < 4; ++x) acc[i][j][x] *= keep;
            }
            __syncwarp();   // (a warp's rows are its own)
#pragma unroll 4
            for (int k = 0; k < BK; k += 4) {
                float4 p[R];
#pragma unroll
                for (int i = 0; i < R; ++i) p[i] = *reinterpret_cast<const float4 *>(&sm.p[r0 + 16 * i][k]);
#pragma unroll
                for (int x = 0; x < 4; ++x)
#pragma unroll
                    for (int j = 0; j < C; ++j) {
                        const float4 y = *reinterpret_cast<const float4 *>(&sm.v[k + x][4 * k0 + 32 * j]);
#pragma unroll
                        for (int i = 0; i < R; ++i) {
                            const float w = x == 0 ? p[i].x : x == 1 ? p[i].y : x == 2 ? p[i].z : p[i].w;
                            acc[i][j][0] = fmaf(w, y.x, acc[i][j][0]);
                            acc[i][j][1] = fmaf(w, y.y, acc[i][j][1]);
                            acc[i][j][2] = fmaf(w, y.z, acc[i][j][2]);
                            acc[i][j][3] = fmaf(w, y.w, acc[i][j][3]);
                        }
                    }
            }
            if (tid < BK) sm.places[tid] = next;
            __syncthreads();
        }
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
        if (b1 - b0 > kSum) take(i);
#pragma unroll
        for (int x = 1; x < 8; x *= 2) l[i] += __shfl_xor_sync(0xffffffffu, l[i], x);
        const int r = r0 + 16 * i;
        if (r >= t.rows) continue;
        float *to = place(r);
        if (splits > 1) {
#pragma unroll
            for (int j = 0; j < C; ++j)
                *reinterpret_cast<float4 *>(to + 32 * j + 4 * k0) = make_float4(acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]);
            if (k0 == 0) {
                to[D] = m[i];
                to[D + 1] = l[i];
            }
            continue;
        }
        const float inv = l[i] != 0.f ? 1.f / l[i] : 0.f;   // (no visible key: zeros)
#pragma unroll
        for (int j = 0; j < C; ++j)
#pragma unroll
            for (int x = 0; x < 4; ++x) to[32 * j + 4 * k0 + x] = l[i] != 0.f ? acc[i][j][x] * inv : 0.f;
    }
}

// A row a warp, a split a lane: what the splits count for at once, then their sums, four on their way.  (An
// element a thread, one split after the other, 40 of them took 400 us; four rows a warp 25 us longer than one.)
template <int D>
__global__ void __launch_bounds__(kThreads)
paged_simt_join(Cache c, float *__restrict__ o, int group, int splits, const float *__restrict__ part) {
    constexpr int V = D / 32;
    __shared__ Found found;
    const int tid = threadIdx.x, lane = tid & 31, h = (gridDim.x - 1 - blockIdx.x) % c.Hk, H = c.Hk * group;
    if (!find(c, (gridDim.x - 1 - blockIdx.x) / c.Hk, group, found)) return;
    const Tile t = found.tile;
    for (int r = blockIdx.y * (kThreads / 32) + tid / 32; r < t.rows; r += gridDim.y * (kThreads / 32)) {
        const float *from = part + ((int64_t)blockIdx.x * splits * BR + r) * (D + 4);
        const int64_t step = (int64_t)BR * (D + 4);
        float top = -INFINITY;
        for (int s = lane; s < splits; s += 32)
            if (from[s * step + D + 1] != 0.f) top = fmaxf(top, from[s * step + D]);
#pragma unroll
        for (int x = 16; x > 0; x /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
        float l = 0.f, sum[V];
#pragma unroll
        for (int j = 0; j < V; ++j) sum[j] = 0.f;
        for (int s0 = 0; s0 < splits; s0 += 32) {
            float mine = 0.f;   // (0: its sums may be anything)
            if (s0 + lane < splits) {
                const float w = from[(s0 + lane) * step + D + 1];
                if (w != 0.f) mine = exp2f(from[(s0 + lane) * step + D] - top);
                l += mine * w;
            }
#pragma unroll 4
            for (int s = s0; s < min(splits, s0 + 32); ++s) {
                const float e = __shfl_sync(0xffffffffu, mine, s - s0);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float y = from[s * step + lane * V + j];
                    sum[j] += e != 0.f ? e * y : 0.f;
                }
            }
        }
#pragma unroll
        for (int x = 16; x > 0; x /= 2) l += __shfl_xor_sync(0xffffffffu, l, x);
        const int at = t.first + r;
        float *to = o + ((int64_t)(t.s.begin + at / group) * H + h * group + at % group) * D + lane * V;
#pragma unroll
        for (int j = 0; j < V; ++j) to[j] = l != 0.f ? sum[j] / l : 0.f;
    }
}

// Over a pool without pages: every page is outside it, so that what tokens see counts as zeros and is reported.
// `pieces`: 16-byte pieces of a row.
__global__ void __launch_bounds__(kThreads)
paged_none_kernel(Cache c, uint4 *__restrict__ o, int group, int pieces, StatusWord *st) {
    __shared__ Found found;
    const int tile = blockIdx.x / c.Hk, h = blockIdx.x % c.Hk, H = c.Hk * group;
    if (blockIdx.x == 0) check_spans(c, st);
    if (!find(c, tile, group, found)) return;
    const Tile t = found.tile;
    if (threadIdx.x == 0 && t.s.pos + (t.first + t.rows - 1) / group >= 0) report(st, KDA_ERR_INVALID_ARG, t.n, 64);
    for (int x = threadIdx.x; x < t.rows * pieces; x += kThreads) {
        const int at = t.first + x / pieces;
        o[((int64_t)(t.s.begin + at / group) * H + h * group + at % group) * pieces + x % pieces] = make_uint4(0, 0, 0, 0);
    }
}

// Tiles that a batch can have at most.
static int64_t tiles_of(const Cache &c, int group) {
    return c.cu ? (int64_t)c.T * group / BR + c.N : c.N * (int64_t)((group + BR - 1) / BR);
}
// CTAs that share a tile's keys: enough for four a multiprocessor, each with 128 keys or more.  (Three are there
// at once with D = 128, four or five with less.  With 2, 3, 4, 6 a multiprocessor 4096 new tokens, 8 heads on 2 of 128,
// took 1231, 1234, 997, 1008 us; 2048 tokens 331, 331, 350, 335; of 64: 195, 196, 160, 176.)
static int splits_of(const Cache &c, int group, int sms) {
    const int64_t ctas = tiles_of(c, group) * c.Hk;
    if (ctas == 0) return 1;
    int64_t s = (4 * sms + ctas - 1) / ctas;
    const int64_t most = (((int64_t)c.width << c.shift) + 127) / 128;
    s = s < most ? s : most;
    return (int)(s < 1 ? 1 : s > 64 ? 64 : s);
}

template <typename TC, int D>
static cudaError_t launch(const Cache &c, const void *q, int64_t qs, void *o, int group, float scale, int window,
                          int sinks, int splits, float *part, StatusWord *st, cudaStream_t s) {
    const int64_t ctas = tiles_of(c, group) * c.Hk;
    if (ctas > 0x7fffffff) return cudaErrorInvalidValue;
    const cudaError_t e = cudaFuncSetAttribute(paged_simt_kernel<TC, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)sizeof(Shared<D>));
    if (e != cudaSuccess) return e;
    paged_simt_kernel<TC, D><<<dim3((unsigned)ctas, splits), kThreads, sizeof(Shared<D>), s>>>(
        c, (const float *)q, qs, (float *)o, group, scale, window, sinks, splits, part, st);
    if (splits > 1)
        paged_simt_join<D><<<dim3((unsigned)ctas, BR * 32 / kThreads), kThreads, 0, s>>>(c, (float *)o, group, splits, part);
    return cudaGetLastError();
}

}  // namespace simt
}  // namespace paged

size_t paged_simt_bytes(const paged::Cache &c, int group, int D, int sms) {
    const int splits = paged::simt::splits_of(c, group, sms);
    if (splits == 1) return 0;
    return (size_t)paged::simt::tiles_of(c, group) * c.Hk * splits * paged::simt::BR * (D + 4) * sizeof(float);
}

cudaError_t launch_paged_simt(int cache_dtype, int D, const paged::Cache &c, const void *q, int64_t qs, void *o, int group,
                              float scale, int window, int sinks, float *part, int sms, StatusWord *st, cudaStream_t s) {
    const int splits = paged::simt::splits_of(c, group, sms);
#define KDA_PAGED(TC_, D_) \
    if (D == D_) return paged::simt::launch<TC_, D_>(c, q, qs, o, group, scale, window, sinks, splits, part, st, s);
#define KDA_PAGED_D(TC_) KDA_PAGED(TC_, 32) KDA_PAGED(TC_, 64) KDA_PAGED(TC_, 128)
    if (cache_dtype == KDA_E4M3) { KDA_PAGED_D(__nv_fp8_e4m3) }
    else { KDA_PAGED_D(float) }
#undef KDA_PAGED_D
#undef KDA_PAGED
    return cudaErrorInvalidValue;
}

cudaError_t launch_paged_none(int64_t row_bytes, const paged::Cache &c, void *o, int group, StatusWord *st, cudaStream_t s) {
    const int64_t ctas = paged::simt::tiles_of(c, group) * c.Hk;
    if (ctas > 0x7fffffff) return cudaErrorInvalidValue;
    paged::simt::paged_none_kernel<<<(unsigned)ctas, paged::simt::kThreads, 0, s>>>(c, (uint4 *)o, group, (int)(row_bytes / 16), st);
    return cudaGetLastError();
}

}  // namespace kda
