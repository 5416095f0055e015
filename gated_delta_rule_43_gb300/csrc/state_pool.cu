// state_pool.cu -- copying, forking, clearing and compacting the slots of a state pool.
//
// Memory-bound: a source is read once (a forked one comes from L2 after its first copy) and
// a destination written once.  Copies run as parts of slots, so that a few copies of large
// slots still fill the GPU.
#include "kda_common.cuh"

namespace kda {
namespace pool {

constexpr int kThreads = 256;
constexpr int kAhead = 4;   // 16-byte loads a thread has in flight

// vec4 values [begin, end) of one slot
__device__ __forceinline__ void copy_part(float4 *dst, const float4 *src, int64_t begin,
                                          int64_t end) {
    for (int64_t i = begin + threadIdx.x; i < end; i += kThreads * kAhead) {
        float4 x[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (i + j * kThreads < end)
                x[j] = src ? src[i + j * kThreads] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (i + j * kThreads < end) dst[i + j * kThreads] = x[j];
    }
}

// Copies src_idx[i] -> dst_idx[i] for i < n (n_dev[0] where the count is on the device),
// each as `parts` parts.  With `check`, a copy whose indices break the rules is left out:
// every CTA looks through the n indices for another copy with this destination, or one that
// reads it.
__global__ void __launch_bounds__(kThreads)
copy_kernel(float4 *__restrict__ pool, int P, int64_t vecs, const int32_t *__restrict__ src_idx,
            const int32_t *__restrict__ dst_idx, int n, const int32_t *__restrict__ n_dev,
            int parts, int check, StatusWord *st) {
    const int64_t count = n_dev ? *n_dev : n;
    const int64_t per = (vecs + parts - 1) / parts;
    for (int64_t task = blockIdx.x; task < count * parts; task += gridDim.x) {
        const int64_t i = task / parts, part = task - i * parts;
        const int src = src_idx[i], dst = dst_idx[i];
        if (check) {
            bool bad = src < -1 || src >= P || dst < 0 || dst >= P;
            for (int64_t m = threadIdx.x; m < count && !bad; m += kThreads)
                bad = m != i && (dst_idx[m] == dst || src_idx[m] == dst);
            if (__syncthreads_or(bad)) {
                if (threadIdx.x == 0 && part == 0) report(st, KDA_ERR_INVALID_ARG, i, 32);
                continue;
            }
        }
        if (src == dst) continue;
        copy_part(pool + dst * vecs, src >= 0 ? pool + src * vecs : nullptr, part * per,
                  min(vecs, (part + 1) * per));
    }
}

// One CTA: the moves that pack the live slots, the new index of each slot and the count.
constexpr int kPlanThreads = 1024;
__global__ void __launch_bounds__(kPlanThreads)
plan_kernel(const uint8_t *__restrict__ live, int P, int32_t *__restrict__ new_index,
            int32_t *__restrict__ n_live, int32_t *__restrict__ src_idx,
            int32_t *__restrict__ dst_idx, int32_t *__restrict__ n_moves) {
    __shared__ int s_holes[32], s_movers[32], s_total;
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    int mine = 0;
    for (int i = tid; i < P; i += kPlanThreads) mine += live[i] != 0;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, d);
    if (lane == 0) s_holes[wid] = mine;
    __syncthreads();
    if (tid < 32) {
        int x = s_holes[tid];
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
        if (tid == 0) s_total = x;
    }
    __syncthreads();
    const int L = s_total;
    int holes = 0, movers = 0;   // before this tile
    for (int base = 0; base < P; base += kPlanThreads) {
        const int i = base + tid;
        const bool on = i < P && live[i] != 0;
        const bool hole = i < P && !on && i < L, mover = on && i >= L;
        const unsigned hb = __ballot_sync(0xffffffffu, hole), mb = __ballot_sync(0xffffffffu, mover);
        if (lane == 0) {
            s_holes[wid] = __popc(hb);
            s_movers[wid] = __popc(mb);
        }
        __syncthreads();
        int hn = holes, mn = movers;
        for (int w = 0; w < 32; ++w) {
            if (w < wid) { hn += s_holes[w]; mn += s_movers[w]; }
            holes += s_holes[w];
            movers += s_movers[w];
        }
        const unsigned below = (1u << lane) - 1u;
        if (hole) dst_idx[hn + __popc(hb & below)] = i;
        if (mover) src_idx[mn + __popc(mb & below)] = i;
        if (i < P && !mover) new_index[i] = on ? i : -1;
        __syncthreads();   // (also: the lists are complete after the last tile)
    }
    for (int m = tid; m < movers; m += kPlanThreads) new_index[src_idx[m]] = dst_idx[m];
    if (tid == 0) {
        *n_live = L;
        *n_moves = movers;
    }
}

// Parts per slot: about four tasks an SM, and no part under 16 KB
static int parts_of(int64_t vecs, int64_t copies, int sms) {
    const int64_t want = (4LL * sms + copies - 1) / (copies > 0 ? copies : 1);
    const int64_t most = vecs / 1024;
    const int64_t p = want < most ? want : most;
    return (int)(p < 1 ? 1 : p);
}

}  // namespace pool

cudaError_t launch_pool_copy(float *p, int P, int64_t elems, const int32_t *src,
                             const int32_t *dst, int n, StatusWord *st, int sms, cudaStream_t s) {
    const int64_t vecs = elems / 4;
    const int parts = pool::parts_of(vecs, n, sms);
    const int64_t tasks = (int64_t)n * parts, cap = 8LL * sms;
    pool::copy_kernel<<<(unsigned)(tasks < cap ? tasks : cap), pool::kThreads, 0, s>>>(
        (float4 *)p, P, vecs, src, dst, n, nullptr, parts, 1, st);
    return cudaGetLastError();
}

cudaError_t launch_pool_compact(float *p, int P, int64_t elems, const uint8_t *live,
                                int32_t *new_index, int32_t *n_live, int32_t *moves, int sms,
                                cudaStream_t s) {
    // moves: the count, then P / 2 sources and P / 2 destinations (no more slots can move)
    const int half = P / 2 + 1;
    int32_t *src = moves + 4, *dst = src + half;
    pool::plan_kernel<<<1, pool::kPlanThreads, 0, s>>>(live, P, new_index, n_live, src, dst, moves);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int64_t vecs = elems / 4;
    const int parts = pool::parts_of(vecs, P / 4, sms);
    pool::copy_kernel<<<(unsigned)(8 * sms), pool::kThreads, 0, s>>>(
        (float4 *)p, P, vecs, src, dst, 0, moves, parts, 0, nullptr);
    return cudaGetLastError();
}

}  // namespace kda
