// la_decode.cu -- one token of the decayed linear attention against resident fp32 states.
//
//   S <- exp(g) S + k v^T,   o = S^T q       (after the update)
// Memory-bound: the state is read once and written once (2 dk dv fp32 a sequence and head),
// everything else is 1% of that.  A CTA owns a block of value columns of one (sequence,
// head); a thread holds R rows x 4 columns, so a warp's loads are whole 128-byte lines, all
// issued before the first is used, and the columns' outputs are joined in shared memory.
// 256 sequences of 32 heads (1.08 GB): 159 us, 6.8 TB/s, a plain copy's rate.  One sequence: 4 us,
// launch and memory latency.
#include "kda_common.cuh"

namespace kda {
namespace la {

constexpr int kThreads = 128;

template <int DK, int DV, int DVC, typename T>
__global__ void __launch_bounds__(kThreads)
la_decode_kernel(const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v,
                 const float *__restrict__ g, float *__restrict__ state, T *__restrict__ o,
                 int H, int group, int64_t qs, int64_t ks, int64_t vs, int g_per_token,
                 const int32_t *__restrict__ slot_idx, int P, StatusWord *st) {
    constexpr int TPR = DVC / 4, RPP = kThreads / TPR, R = DK / RPP, NCB = DV / DVC;
    static_assert(DVC % 4 == 0 && DV % DVC == 0 && kThreads % TPR == 0 && DK % RPP == 0 && R > 0,
                  "shape");
    __shared__ float s_k[DK], s_q[DK];
    __shared__ __align__(16) float s_o[RPP][DVC];
    const int64_t nh = blockIdx.x / NCB;
    const int j0 = (int)(blockIdx.x % NCB) * DVC;
    const int64_t n = nh / H;
    const int h = (int)(nh - n * H), hk = h / group;
    const int tid = threadIdx.x;
    const int64_t slot = slot_idx ? (int64_t)slot_idx[n] : n;
    if (slot < 0 || slot >= P) {
        if (tid == 0 && h == 0 && j0 == 0) report(st, KDA_ERR_INVALID_ARG, n, 31);
        return;
    }
    const int c4 = tid % TPR, rg = tid / TPR;
    float4 *S4 = reinterpret_cast<float4 *>(state + (slot * H + h) * DK * DV + j0);
    float4 s[R];
#pragma unroll
    for (int p = 0; p < R; ++p) s[p] = __ldcs(S4 + (int64_t)(rg + p * RPP) * (DV / 4) + c4);

    float vj[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) vj[j] = to_f(v[n * vs + (int64_t)h * DV + j0 + c4 * 4 + j]);
    const float a = expf(g_per_token ? g[nh] : g[h]);
    for (int i = tid; i < DK; i += kThreads) {
        s_k[i] = to_f(k[n * ks + (int64_t)hk * DK + i]);
        s_q[i] = to_f(q[n * qs + (int64_t)hk * DK + i]);
    }
    __syncthreads();
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int p = 0; p < R; ++p) {
        const int row = rg + p * RPP;
        const float kr = s_k[row], qr = s_q[row];
        float4 w = s[p];
        w.x = a * w.x + kr * vj[0];
        w.y = a * w.y + kr * vj[1];
        w.z = a * w.z + kr * vj[2];
        w.w = a * w.w + kr * vj[3];
        S4[(int64_t)row * (DV / 4) + c4] = w;
        acc[0] += qr * w.x; acc[1] += qr * w.y; acc[2] += qr * w.z; acc[3] += qr * w.w;
    }
    *reinterpret_cast<float4 *>(&s_o[rg][c4 * 4]) = make_float4(acc[0], acc[1], acc[2], acc[3]);
    __syncthreads();
    for (int j = tid; j < DVC; j += kThreads) {
        float x = 0.f;
#pragma unroll 8
        for (int r = 0; r < RPP; ++r) x += s_o[r][j];
        o[nh * DV + j0 + j] = from_f<T>(x);
    }
}

template <int DK, int DV, typename T>
static cudaError_t launch_dims(const void *q, const void *k, const void *v, const float *g,
                               float *state, void *o, int N, int H, int Hk, int64_t qs, int64_t ks,
                               int64_t vs, int gpt, const int32_t *idx, int P, StatusWord *st,
                               cudaStream_t s) {
    constexpr int DVC = DV == 128 ? 64 : DV;
    la_decode_kernel<DK, DV, DVC, T><<<(unsigned)((int64_t)N * H * (DV / DVC)), kThreads, 0, s>>>(
        (const T *)q, (const T *)k, (const T *)v, g, state, (T *)o, H, H / Hk, qs, ks, vs, gpt, idx,
        P, st);
    return cudaGetLastError();
}

}  // namespace la

cudaError_t launch_la_decode(int dtype, int dk, int dv, const void *q, const void *k,
                             const void *v, const float *g, float *state, void *o, int N, int H,
                             int Hk, int64_t qs, int64_t ks, int64_t vs, int gpt,
                             const int32_t *idx, int P, StatusWord *st, cudaStream_t s) {
#define KDA_LA(DK_, DV_)                                                                        \
    if (dk == DK_ && dv == DV_)                                                                 \
        return dtype == KDA_BF16                                                                \
                   ? la::launch_dims<DK_, DV_, __nv_bfloat16>(q, k, v, g, state, o, N, H, Hk, qs, ks, \
                                                              vs, gpt, idx, P, st, s)           \
                   : la::launch_dims<DK_, DV_, float>(q, k, v, g, state, o, N, H, Hk, qs, ks, vs, \
                                                      gpt, idx, P, st, s);
    KDA_LA(32, 32) KDA_LA(32, 64) KDA_LA(32, 128)
    KDA_LA(64, 32) KDA_LA(64, 64) KDA_LA(64, 128)
    KDA_LA(128, 32) KDA_LA(128, 64) KDA_LA(128, 128)
#undef KDA_LA
    return cudaErrorInvalidValue;
}

}  // namespace kda
