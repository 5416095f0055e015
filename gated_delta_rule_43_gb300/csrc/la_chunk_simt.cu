// la_chunk_simt.cu -- linear attention with one decay per head, chunked, in fp32 on the CUDA
// cores; the plan and the boundary scan of kda_la_chunk_fwd.
//
// With G_t = g_1 + ... + g_t inside a chunk that starts from state S:
//   O  = [(Q K^T) * D] V + exp(G_t) Q S,   D_ts = exp(G_t - G_s) for t >= s, else 0
//   S' = exp(G_C) S + (K * exp(g_{s+1} + ... + g_C))^T V
// The state product's weights come from suffix sums, not from differences of prefix sums:
// a suffix sum keeps its relative precision next to the chunk's end, where the weights
// matter, however fast the earlier tokens decay.  The scores do need differences, and behind a few
// resets G is in the thousands: it is kept as the sum of two fp32 (each addition with its rounding,
// Knuth's two-sum), so that D is as exact behind resets as without any (outputs 3e-8 off by it; with
// plain prefix sums 2e-5 at a reset every four tokens).
// Bound by fp32 arithmetic fed from shared memory, and in small calls by the steps before each
// other: three sequences of 1000, 37 and 513 tokens, 4 heads of 64 x 128, 45 us (plan 7, first
// pass 9, scan 6, outputs 24).
#include "kda_la.cuh"

namespace kda {
namespace la {

// ------------------------------------------------------------------------- plan
// CTA 0: validates cu_seqlens (see plan_chunks_kernel), counts chunks and places the cuts.
// The others: final states of sequences without tokens (S_out not NULL).
constexpr int kPlanThreads = 256, kPlanSeqs = 1024;

// The largest n with off[n] * H <= x, for x < off[N] * H: entry n spans x.
__device__ __forceinline__ int owner(const int32_t *off, int N, int H, int64_t x) {
    int lo = 0, hi = N - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if ((int64_t)off[mid] * H <= x) lo = mid; else hi = mid - 1;
    }
    return lo;
}

__device__ Cut place(const int32_t *off, int N, int H, int64_t total, int64_t x) {
    Cut r{};
    r.x = x;
    r.n = N;
    if (x >= total) {
        r.x = total;
        return r;
    }
    r.n = owner(off, N, H, x);
    r.nc = off[r.n + 1] - off[r.n];
    const int64_t nc = r.nc, rest = x - (int64_t)off[r.n] * H;
    r.h = (int)(rest / nc);
    r.c = (int)(rest - r.h * nc);
    r.inner = r.c > 0;
    return r;
}

// Ranges a unit of nc chunks is worth when there are SMs to spare
__device__ __forceinline__ int pieces(int nc, int split, int chunk) {
    const int length = chunk == kTcChunk ? max(2, (int)(0.5f * sqrtf((float)nc))) : 2;
    return nc == 0 ? 0 : !split || nc < 2 * length ? 1 : nc / length;
}

__global__ void __launch_bounds__(kPlanThreads)
la_plan_kernel(const int32_t *__restrict__ cu, int N, int64_t T_tot, int32_t *off,
               int32_t *piece_off, int32_t *cost_off, int unit_cost, int chunk,
               int uncut, Cut *cuts, int ranges, int split, uint32_t *flags, int n_flags,
               StatusWord *st, const float *h0, float *S_out, int all_heads, int H,
               int64_t dkdv4) {   // H: heads of a lane
    let_next_start();
    if (blockIdx.x != 0) {
        for (int64_t nh = blockIdx.x - 1; nh < (int64_t)N * all_heads; nh += gridDim.x - 1) {
            const int n = (int)(nh / all_heads);
            const int64_t b = cu[n], e = cu[n + 1];
            if (b < e && b >= 0 && e <= T_tot) continue;
            float4 *dst = reinterpret_cast<float4 *>(S_out) + nh * dkdv4;
            const float4 *src = h0 ? reinterpret_cast<const float4 *>(h0) + nh * dkdv4 : nullptr;
            for (int64_t i = threadIdx.x; i < dkdv4; i += blockDim.x)
                dst[i] = src ? src[i] : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        return;
    }
    __shared__ Cut s_cut[kMaxRanges + 1];
    // The prefix sums are searched again and again: in shared memory where they fit.
    __shared__ int32_t s_sum[3][kPlanSeqs + 1];
    const bool fits = N <= kPlanSeqs;
    int32_t *const chunks = fits ? s_sum[0] : off;
    int32_t *const parts = fits ? s_sum[1] : piece_off;
    int32_t *const costs = fits ? s_sum[2] : cost_off;
    constexpr int NW = kPlanThreads / 32;
    __shared__ int3 s_warp[NW];
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    if (tid == 0) {
        st->code = 0u;
        st->site = 0u;
        st->info = 0ull;
    }
    __syncthreads();
    for (int i = tid; i < n_flags; i += kPlanThreads) flags[i] = 0;
    if (tid == 0 && (cu[0] != 0 || (int64_t)cu[N] != T_tot)) report(st, KDA_ERR_SEQLENS, N, 1);
    int3 carry = make_int3(0, 0, 0);   // chunks, pieces, costs
    auto add = [](int3 &x, const int3 &y) {   // (sums that do not fit are not used, see below)
        x.x = (int)((uint32_t)x.x + (uint32_t)y.x);
        x.y = (int)((uint32_t)x.y + (uint32_t)y.y);
        x.z = (int)((uint32_t)x.z + (uint32_t)y.z);
    };
    bool bad = false;
    for (int base = 0; base < N; base += kPlanThreads) {
        const int n = base + tid;
        int3 own = make_int3(0, 0, 0);
        if (n < N) {
            const int64_t b = cu[n], e = cu[n + 1];
            if (b < 0 || e < b || e > T_tot) {
                report(st, KDA_ERR_SEQLENS, n, 2);
                bad = true;
            } else {
                own.x = (int)((e - b + chunk - 1) / chunk);
            }
            own.y = pieces(own.x, split, chunk);
            own.z = own.x ? own.x + unit_cost : 0;
        }
        int3 x = own;   // inclusive warp scan
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int3 y = make_int3(__shfl_up_sync(0xffffffffu, x.x, o),
                                     __shfl_up_sync(0xffffffffu, x.y, o),
                                     __shfl_up_sync(0xffffffffu, x.z, o));
            if (lane >= o) add(x, y);
        }
        if (lane == 31) s_warp[wid] = x;
        __syncthreads();
        int3 before = carry;
        for (int w = 0; w < NW; ++w) {
            if (w < wid) add(before, s_warp[w]);
            add(carry, s_warp[w]);
        }
        if (n < N) {
            off[n] = chunks[n] = before.x + x.x - own.x;
            parts[n] = before.y + x.y - own.y;
            costs[n] = before.z + x.z - own.z;
        }
        __syncthreads();
    }
    if (tid == 0) {
        off[N] = chunks[N] = carry.x;
        parts[N] = carry.y;
        costs[N] = carry.z;
    }
    // Where an offending sequence lets the others overlap, what they add up to has no bound by the
    // call's sizes (nor have the sums): then none is gone through.
    if (__syncthreads_or(bad)) {
        __shared__ unsigned long long s_tokens;
        if (tid == 0) s_tokens = 0;
        __syncthreads();
        unsigned long long tokens = 0;
        for (int n = tid; n < N; n += kPlanThreads) {
            const int64_t b = cu[n], e = cu[n + 1];
            if (b >= 0 && e >= b && e <= T_tot) tokens += e - b;
        }
        atomicAdd(&s_tokens, tokens);
        __syncthreads();
        if (s_tokens > (unsigned long long)T_tot) carry = make_int3(0, 0, 0);
    }
    const int64_t total = (int64_t)carry.x * H, fine = (int64_t)carry.y * H;
    const int64_t cost = (int64_t)carry.z * H;
    // SMs to spare: every unit gets its own range, a long one several.  Else equal parts
    // (without a first pass nothing can be cut: the units are dealt out whole).
    const bool spare = fine <= ranges && total < (int64_t)ranges * uncut;
    for (int i = tid; i <= ranges; i += kPlanThreads) {
        Cut r;
        if (spare) {
            int64_t x = total;
            if (i < fine) {
                const int n = owner(parts, N, H, i);
                const int nc = chunks[n + 1] - chunks[n], m = parts[n + 1] - parts[n];
                const int rest = i - parts[n] * H;
                x = (int64_t)chunks[n] * H + (int64_t)(rest / m) * nc + (int64_t)(rest % m) * nc / m;
            }
            r = place(chunks, N, H, total, x);
        } else {
            const int64_t y = (int64_t)i * cost / ranges;
            int64_t x = total;
            if (y < cost) {
                const int n = owner(costs, N, H, y);
                const int64_t nc = chunks[n + 1] - chunks[n], m = nc + unit_cost;
                const int64_t rest = y - (int64_t)costs[n] * H, c = rest % m - unit_cost;
                x = (int64_t)chunks[n] * H + rest / m * nc + (c > 0 ? c : 0);
            }
            r = place(chunks, N, H, total, x);
            if (r.inner) {
                if (!split || r.nc <= uncut)
                    r = place(chunks, N, H, total, r.x + (2 * r.c >= r.nc ? r.nc - r.c : -r.c));
            }
        }
        if (r.nc) {
            r.begin = cu[r.n];
            r.stop = cu[r.n + 1];
        }
        s_cut[i] = r;
    }
    __syncthreads();
    for (int i = tid; i <= ranges; i += kPlanThreads) {
        Cut r = s_cut[i];
        if (r.inner) {
            for (int j = i - 1; j > 0 && s_cut[j].inner && s_cut[j].n == r.n && s_cut[j].h == r.h; --j)
                ++r.before;
            for (int j = i + 1; j < ranges && s_cut[j].inner && s_cut[j].n == r.n && s_cut[j].h == r.h; ++j)
                ++r.inner;
            r.handed = n_flags > 0 && r.inner == 1 && r.before == 0 &&
                       r.c <= s_cut[i + 1].x - r.x - (r.nc - r.c);
        }
        cuts[i] = r;
    }
}

// ------------------------------------------------------------------------- scan
// Along the cuts of each unit, from its initial state: S <- exp(bnd_log) S + bnd, where bnd
// holds what the tokens since the cut before leave and then the state.  One thread per four
// state values; the loads of kAhead cuts are in flight at a time.
constexpr int kScanThreads = 256, kAhead = 8;
__global__ void __launch_bounds__(kScanThreads)
la_scan_kernel(Plan p, const float *__restrict__ h0, float *__restrict__ bnd,
               const float *__restrict__ bnd_log, int64_t dkdv4) {
    wait_for_previous();
    let_next_start();
    const int first = blockIdx.y / p.lanes + 1, lane = blockIdx.y % p.lanes;
    const Cut f = p.cuts[first];
    if (!f.inner || f.before || f.handed) return;   // a unit's chain starts at its first cut
    const int64_t i = (int64_t)blockIdx.x * kScanThreads + threadIdx.x;
    if (i >= dkdv4) return;
    const int last = first + f.inner - 1;
    float4 S = h0 ? reinterpret_cast<const float4 *>(h0)[((int64_t)f.n * p.H + f.h * p.lanes + lane) * dkdv4 + i]
                  : make_float4(0.f, 0.f, 0.f, 0.f);
    float4 *at = reinterpret_cast<float4 *>(bnd) + i;
    if (p.in_place) at[initial_copy(p, first - 1, lane) * dkdv4] = S;
    for (int b = first; b <= last; b += kAhead) {
        float4 add[kAhead];
        float a[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (b + j <= last) {
                add[j] = at[cut_state(p, b + j, lane) * dkdv4];
                a[j] = bnd_log[cut_state(p, b + j, lane)];
            }
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (b + j <= last) {
                const float e = expf(a[j]);
                S.x = e * S.x + add[j].x;
                S.y = e * S.y + add[j].y;
                S.z = e * S.z + add[j].z;
                S.w = e * S.w + add[j].w;
                at[cut_state(p, b + j, lane) * dkdv4] = S;
            }
    }
}

// ----------------------------------------------------------------------- chunks
constexpr int kThreads = 256;
constexpr int C = kSimtChunk;   // one warp scans its decays

template <int DK, int DVB> struct Smem {
    static constexpr int LK = DK + 4;   // padded rows: 16-byte reads of 8 rows miss no bank twice
    float q[C][LK], k[C][LK];
    float v[C][DVB];
    float S[DK][DVB];
    float p[C][C + 4];
    float G[C], Glo[C], eG[C], w[C];    // prefix sums (two parts), their exponentials, weights to the end
    float total, total_log;             // the chunk's decay and its log
};

__device__ __forceinline__ void fma4(float (&acc)[4], float a, const float4 &b) {
    acc[0] += a * b.x;
    acc[1] += a * b.y;
    acc[2] += a * b.z;
    acc[3] += a * b.w;
}

// hi + lo += x + y, the rounding of the larger parts' sum kept in the smaller one
__device__ __forceinline__ void add2(float &hi, float &lo, float x, float y) {
    const float sum = __fadd_rn(hi, x), of_x = __fsub_rn(sum, hi);
    lo = __fadd_rn(__fadd_rn(lo, y), __fadd_rn(__fsub_rn(hi, __fsub_rn(sum, of_x)), __fsub_rn(x, of_x)));
    hi = sum;
}

// OUT: outputs and final states of the CTA's range.  Else what the end of the range leaves at
// the cut behind it.  The column blocks of a range are CTAs of their own.  The next chunk's
// tokens are on their way in registers while a chunk is worked on.
template <int DK, int DV, int DVB, bool OUT>
__global__ void __launch_bounds__(kThreads)
la_chunk_simt_kernel(Plan p, const float *__restrict__ q, const float *__restrict__ k,
                     const float *__restrict__ v, int64_t qs, int64_t ks, int64_t vs,
                     const float *__restrict__ g, int g_per_token, const float *h0,
                     float *hT, float *__restrict__ o, float *__restrict__ bnd,
                     float *__restrict__ bnd_log, StatusWord *st) {
    extern __shared__ __align__(16) uint8_t raw[];
    using Sm = Smem<DK, DVB>;
    Sm &sm = *reinterpret_cast<Sm *>(raw);
    constexpr int NB = DV / DVB;
    constexpr int TC = DVB / 4;              // threads across the columns, four each
    constexpr int TR = kThreads / TC;        // thread rows
    constexpr int SR = DK / TR;              // state rows per thread
    constexpr int OR = C / TR > 0 ? C / TR : 1;   // output rows per thread
    constexpr int LQ = C * DK / 4 / kThreads, LV = (C * DVB / 4 + kThreads - 1) / kThreads;
    static_assert(DK % TR == 0 && SR >= 1 && C % OR == 0 && C * DK / 4 % kThreads == 0 && LQ >= 1, "shape");
    const int tid = threadIdx.x;
    const int c4 = (tid % TC) * 4, rg = tid / TC;
    const int64_t dkdv = (int64_t)DK * DV;
    const int blk = blockIdx.x % NB, range = blockIdx.x / NB;
    const int j0 = blk * DVB;
    Item it;
    Walk walk(p, range, 0);   // (one lane)
    bool more = OUT ? walk.next(p, it) : before_cut(p, range + 1, 0, it);

    for (; more; more = OUT && walk.next(p, it)) {
        const int h = it.h;
        const int hk = h / (p.H / p.Hk);
        const int64_t nh = ((int64_t)it.n * p.H + h) * dkdv;
        const Start from = OUT ? start_state(p, it, range, 0, h0 != nullptr) : Start{};
        const float *start = from.steps ? (from.in_bnd(0) ? bnd : h0) + from.index(0) * dkdv : nullptr;
        // rows past the sequence are zeros whatever memory holds there
        float4 nq[LQ], nk[LQ], nv[LV];
        float ng = 0.f;
        auto fetch = [&](int64_t t0) {
            const int len = (int)min((int64_t)C, it.t1 - t0);
#pragma unroll
            for (int m = 0; m < LQ; ++m) {
                const int x = tid + m * kThreads, r = x / (DK / 4), c = 4 * (x % (DK / 4));
                const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
                const bool in = r < len;
                if (OUT) nq[m] = in ? *reinterpret_cast<const float4 *>(q + (t0 + r) * qs + (int64_t)hk * DK + c) : zero;
                nk[m] = in ? *reinterpret_cast<const float4 *>(k + (t0 + r) * ks + (int64_t)hk * DK + c) : zero;
            }
#pragma unroll
            for (int m = 0; m < LV; ++m) {
                const int x = tid + m * kThreads, r = x / (DVB / 4), c = 4 * (x % (DVB / 4));
                nv[m] = r < len ? *reinterpret_cast<const float4 *>(v + (t0 + r) * vs + (int64_t)h * DV + j0 + c)
                                : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            ng = 0.f;
            if (tid < len) ng = g_per_token ? g[(t0 + tid) * p.H + h] : g[h];
        };
        fetch(it.t0);
        float S[SR][4];
#pragma unroll
        for (int r = 0; r < SR; ++r) {
            const float4 x = start ? *reinterpret_cast<const float4 *>(
                                         start + (int64_t)(rg * SR + r) * DV + j0 + c4)
                                   : make_float4(0.f, 0.f, 0.f, 0.f);
            S[r][0] = x.x; S[r][1] = x.y; S[r][2] = x.z; S[r][3] = x.w;
        }
        float log_sum = 0.f;
        for (int64_t t0 = it.t0; t0 < it.t1; t0 += C) {
            const int len = (int)min((int64_t)C, it.t1 - t0);
#pragma unroll
            for (int m = 0; m < LQ; ++m) {
                const int x = tid + m * kThreads, r = x / (DK / 4), c = 4 * (x % (DK / 4));
                if (OUT) *reinterpret_cast<float4 *>(&sm.q[r][c]) = nq[m];
                *reinterpret_cast<float4 *>(&sm.k[r][c]) = nk[m];
            }
#pragma unroll
            for (int m = 0; m < LV; ++m) {
                const int x = tid + m * kThreads, r = x / (DVB / 4), c = 4 * (x % (DVB / 4));
                if (r < C) *reinterpret_cast<float4 *>(&sm.v[r][c]) = nv[m];
            }
            if (OUT) {
#pragma unroll
                for (int r = 0; r < SR; ++r)
                    *reinterpret_cast<float4 *>(&sm.S[rg * SR + r][c4]) =
                        make_float4(S[r][0], S[r][1], S[r][2], S[r][3]);
            }
            if (tid < 32) {
                const float x = ng;
                if (!log_decay_ok(x) && blk == 0)
                    report(st, KDA_ERR_DECAY_RANGE, g_per_token ? (t0 + tid) * p.H + h : h, 30);
                float pre = x < kLogZero ? kLogZero : x;   // (a comparison, so that NaN spreads)
                float pre_lo = 0.f, suf = x;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const float a = __shfl_up_sync(0xffffffffu, pre, d);
                    const float a_lo = __shfl_up_sync(0xffffffffu, pre_lo, d);
                    const float b = __shfl_down_sync(0xffffffffu, suf, d);
                    if (tid >= d) add2(pre, pre_lo, a, a_lo);
                    if (tid + d < 32) suf += b;
                }
                const float after = __shfl_down_sync(0xffffffffu, suf, 1);
                sm.G[tid] = pre;
                sm.Glo[tid] = pre_lo;
                sm.eG[tid] = expf(pre + pre_lo);
                sm.w[tid] = tid == 31 ? 1.f : expf(after);
                if (tid == 0) {
                    sm.total_log = suf;
                    sm.total = expf(suf);
                }
            }
            __syncthreads();
            if (t0 + C < it.t1) fetch(t0 + C);
            if (OUT) {
                // rows ta, ta + 16 and columns sa, sa + 16 of P
                const int ta = tid / 16, sa = tid % 16;
                float acc[2][2] = {};
#pragma unroll 4
                for (int d = 0; d < DK; d += 4) {
                    float4 a[2], b[2];
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        a[m] = *reinterpret_cast<const float4 *>(&sm.q[ta + 16 * m][d]);
                        b[m] = *reinterpret_cast<const float4 *>(&sm.k[sa + 16 * m][d]);
                    }
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int n = 0; n < 2; ++n)
                            acc[m][n] += a[m].x * b[n].x + a[m].y * b[n].y + a[m].z * b[n].z + a[m].w * b[n].w;
                }
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        const int t = ta + 16 * m, s = sa + 16 * n;
                        sm.p[t][s] = t >= s ? acc[m][n] * expf((sm.G[t] - sm.G[s]) + (sm.Glo[t] - sm.Glo[s])) : 0.f;
                    }
                __syncthreads();
                float oi[OR][4] = {}, oa[OR][4] = {};
#pragma unroll 2
                for (int i = 0; i < DK; i += 4) {
                    float4 s4[4];
#pragma unroll
                    for (int m = 0; m < 4; ++m) s4[m] = *reinterpret_cast<const float4 *>(&sm.S[i + m][c4]);
#pragma unroll
                    for (int r = 0; r < OR; ++r) {
                        const float4 a = *reinterpret_cast<const float4 *>(&sm.q[rg * OR + r][i]);
                        fma4(oi[r], a.x, s4[0]);
                        fma4(oi[r], a.y, s4[1]);
                        fma4(oi[r], a.z, s4[2]);
                        fma4(oi[r], a.w, s4[3]);
                    }
                }
#pragma unroll 2
                for (int s = 0; s < C; s += 4) {
                    float4 v4[4];
#pragma unroll
                    for (int m = 0; m < 4; ++m) v4[m] = *reinterpret_cast<const float4 *>(&sm.v[s + m][c4]);
#pragma unroll
                    for (int r = 0; r < OR; ++r) {
                        const float4 a = *reinterpret_cast<const float4 *>(&sm.p[rg * OR + r][s]);
                        fma4(oa[r], a.x, v4[0]);
                        fma4(oa[r], a.y, v4[1]);
                        fma4(oa[r], a.z, v4[2]);
                        fma4(oa[r], a.w, v4[3]);
                    }
                }
#pragma unroll
                for (int r = 0; r < OR; ++r) {
                    const int row = rg * OR + r;
                    if (row < len) {
                        const float e = sm.eG[row];
                        *reinterpret_cast<float4 *>(o + ((t0 + row) * p.H + h) * (int64_t)DV + j0 + c4) =
                            make_float4(oa[r][0] + e * oi[r][0], oa[r][1] + e * oi[r][1],
                                        oa[r][2] + e * oi[r][2], oa[r][3] + e * oi[r][3]);
                    }
                }
            }
            float add[SR][4] = {};
#pragma unroll 4
            for (int s = 0; s < C; ++s) {
                float4 v4 = *reinterpret_cast<const float4 *>(&sm.v[s][c4]);
                const float w = sm.w[s];
                v4.x *= w; v4.y *= w; v4.z *= w; v4.w *= w;
#pragma unroll
                for (int r = 0; r < SR; ++r) fma4(add[r], sm.k[s][rg * SR + r], v4);
            }
            const float e = sm.total;
            log_sum += sm.total_log;
#pragma unroll
            for (int r = 0; r < SR; ++r)
#pragma unroll
                for (int j = 0; j < 4; ++j) S[r][j] = e * S[r][j] + add[r][j];
            __syncthreads();
        }
        float *dst = OUT ? (it.c1 == it.nc && hT ? hT + nh : nullptr)
                         : bnd + cut_state(p, range + 1, 0) * dkdv;
        if (dst) {
#pragma unroll
            for (int r = 0; r < SR; ++r)
                *reinterpret_cast<float4 *>(dst + (int64_t)(rg * SR + r) * DV + j0 + c4) =
                    make_float4(S[r][0], S[r][1], S[r][2], S[r][3]);
        }
        if (!OUT && blk == 0 && tid == 0) bnd_log[cut_state(p, range + 1, 0)] = log_sum;
    }
}

template <int DK, int DV, int DVB>
static cudaError_t launch_columns(bool out, const Plan &p, const float *q, const float *k,
                                  const float *v, int64_t qs, int64_t ks, int64_t vs, const float *g,
                                  int gpt, const float *h0, float *hT, float *o, float *bnd,
                                  float *bnd_log, StatusWord *st, cudaStream_t s) {
    constexpr size_t bytes = sizeof(Smem<DK, DVB>);
    auto *f = out ? la_chunk_simt_kernel<DK, DV, DVB, true> : la_chunk_simt_kernel<DK, DV, DVB, false>;
    cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return e;
    const int ranges = out ? p.ranges : p.ranges - 1;   // (the last ends at the row's end)
    f<<<ranges * (DV / DVB), kThreads, bytes, s>>>(p, q, k, v, qs, ks, vs, g, gpt, h0, hT, o, bnd,
                                                   bnd_log, st);
    return cudaGetLastError();
}

// Columns in blocks of at most 64, a CTA each; or, where two blocks of every range that holds work
// would be more CTAs than SMs, all columns in one, so that the scores are formed once.  (All, in
// blocks: 20 sequences of 500 tokens, 8 heads of 128 x 128: 267 us, 360; 3 of 1000, 37 and 513, 4
// heads of 64 x 128, 96 busy ranges: 39, 41; 4 of 300, 4 heads of 128 x 128, 80 busy: 43, 53; one of
// 2500, 2 heads, 78 busy: 63, 70.  With fewer, blocks keep more SMs busy: one of 2432, 76 busy: 52,
// 42; one of 600, 8 heads, 72 busy: 54, 42.)
template <int DK, int DV, typename... A>
static cudaError_t launch_dims(bool whole, A... args) {
    if (DV > 64 && whole) return launch_columns<DK, DV, DV>(args...);
    return launch_columns<DK, DV, (DV < 64 ? DV : 64)>(args...);
}

}  // namespace la

cudaError_t launch_la_plan(const int32_t *cu, int N, int64_t T_tot, int32_t *off, int unit_cost,
                           int chunk, int uncut, la::Cut *cuts, int ranges, int split, uint32_t *flags, int n_flags, StatusWord *st, const float *h0, float *hT,
                           int H, int lanes, int64_t dkdv, cudaStream_t s) {
    float *S_out = hT != h0 ? hT : nullptr;   // an in-place update leaves empty ones as they are
    const int64_t nh = (int64_t)N * H;
    const int grid = S_out ? 1 + (int)(nh < 255 ? nh : 255) : 1;
    la::la_plan_kernel<<<grid, la::kPlanThreads, 0, s>>>(
        cu, N, T_tot, off, off + N + 1, off + 2 * (N + 1), unit_cost, chunk, uncut, cuts, ranges, split,
        flags, n_flags, st, h0, S_out, H, H / lanes, dkdv / 4);
    return cudaGetLastError();
}

cudaError_t launch_la_scan(const la::Plan &p, const float *h0, float *bnd, const float *bnd_log,
                           int64_t dkdv, cudaStream_t s) {
    const dim3 grid((unsigned)((dkdv / 4 + la::kScanThreads - 1) / la::kScanThreads),
                    (unsigned)((p.ranges - 1) * p.lanes));
    return la::launch_after(la::la_scan_kernel, grid, dim3(la::kScanThreads), 0, s, p, h0, bnd, bnd_log,
                            dkdv / 4);
}

cudaError_t launch_la_simt(bool out, bool whole, int dk, int dv, const la::Plan &p, const float *q,
                           const float *k, const float *v, int64_t qs, int64_t ks, int64_t vs,
                           const float *g, int gpt, const float *h0, float *hT, float *o,
                           float *bnd, float *bnd_log, StatusWord *st, cudaStream_t s) {
#define KDA_LA(DK_, DV_)                                                                       \
    if (dk == DK_ && dv == DV_)                                                                \
        return la::launch_dims<DK_, DV_>(whole, out, p, q, k, v, qs, ks, vs, g, gpt, h0, hT, o, bnd,  \
                                         bnd_log, st, s);
    KDA_LA(32, 32) KDA_LA(32, 64) KDA_LA(32, 128)
    KDA_LA(64, 32) KDA_LA(64, 64) KDA_LA(64, 128)
    KDA_LA(128, 32) KDA_LA(128, 64) KDA_LA(128, 128)
#undef KDA_LA
    return cudaErrorInvalidValue;
}

}  // namespace kda
