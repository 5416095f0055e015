// state_pool.cu -- copying, forking, clearing and compacting the slots of a state pool.
//
// Memory-bound: a source is read once (a forked one comes from L2 after its first copy) and
// a destination written once.  Copies run as parts of slots, so that a few copies of large
// slots still fill the GPU.  12 slots of 2 MB forked six times: 28 us for 176 MB, 6.3 TB/s.
// Compacting with 60 slots to move: 44 us for 252 MB, 5.7 TB/s, of which the plan takes 4.
#include "kda_common.cuh"

namespace kda {
namespace pool {

constexpr int kThreads = 256;
constexpr int kAhead = 8;   // 16-byte loads a thread has in flight
constexpr int kPart = kThreads * kAhead;   // 16-byte values of a task: 32 KB

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

// A copy whose indices break the rules is left out: one with another copy that has its destination,
// or that reads it (which a copy of a slot to itself does not disturb).  Up to kLooked copies,
// every CTA looks through all of them.  That is quadratic, so beyond, each slot gets a mark first,
// where the workspace has room for them (two more launches).  Looked through and marked, copies of
// 128 bytes: 2049: 13 us, 12; 4097: 26, 15; 16384: 219, 35; 65536: 9.7 ms, 0.11.
constexpr int kLooked = 2048;
constexpr uint32_t kRead = 0x80000000u;   // of a mark: read by a copy to another slot; below: writers

__global__ void __launch_bounds__(kThreads)
mark_kernel(uint32_t *__restrict__ marks, int P, const int32_t *__restrict__ src_idx,
            const int32_t *__restrict__ dst_idx, int n) {
    const int i = blockIdx.x * kThreads + threadIdx.x;
    if (i >= n) return;
    const int src = src_idx[i], dst = dst_idx[i];
    if (dst >= 0 && dst < P) atomicAdd(marks + dst, 1u);
    if (src >= 0 && src < P && src != dst) atomicOr(marks + src, kRead);
}

// Copy i = task / parts of n, its part task % parts: a CTA a task.
__global__ void __launch_bounds__(kThreads)
copy_kernel(float4 *__restrict__ pool, int P, int64_t vecs, const int32_t *__restrict__ src_idx,
            const int32_t *__restrict__ dst_idx, int n, const uint32_t *__restrict__ marks, int parts,
            int64_t per, StatusWord *st) {
    const int64_t i = blockIdx.x / parts, part = blockIdx.x - i * parts;
    const int src = src_idx[i], dst = dst_idx[i];
    bool bad = src < -1 || src >= P || dst < 0 || dst >= P;
    if (marks) {
        const uint32_t mark = bad ? 0u : marks[dst];
        bad = bad || (mark & ~kRead) > 1u || (mark >= kRead && src != dst);
    } else {
        for (int m = threadIdx.x; m < n && !bad; m += kThreads)
            bad = m != i && (dst_idx[m] == dst || (src_idx[m] == dst && src != dst));
    }
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0 && part == 0) report(st, KDA_ERR_INVALID_ARG, i, 32);
        return;
    }
    if (src == dst) return;
    copy_part(pool + dst * vecs, src >= 0 ? pool + src * vecs : nullptr, part * per,
              min(vecs, (part + 1) * per));
}

// The moves that plan_kernel found.  Their number is on the device, so the CTAs of a fixed grid
// draw tasks from a counter.
struct Moves {
    int32_t count;
    uint32_t next;     // task to be drawn
};
__global__ void __launch_bounds__(kThreads)
move_kernel(float4 *__restrict__ pool, int64_t vecs, Moves *moves, const int32_t *__restrict__ src_idx,
            const int32_t *__restrict__ dst_idx, int parts, int64_t per) {
    __shared__ uint32_t s_task;
    asm volatile("griddepcontrol.wait;" ::: "memory");   // (plan_kernel)
    const uint32_t tasks = (uint32_t)moves->count * (uint32_t)parts;
    while (true) {
        __syncthreads();
        if (threadIdx.x == 0) s_task = atomicAdd(&moves->next, 1u);
        __syncthreads();
        const uint32_t task = s_task;
        if (task >= tasks) return;
        const uint32_t i = task / parts, part = task - i * parts;
        copy_part(pool + dst_idx[i] * vecs, pool + src_idx[i] * vecs, part * per,
                  min(vecs, (part + 1) * per));
    }
}

// One CTA: the moves that pack the live slots, the new index of each slot and the count.
constexpr int kPlanThreads = 1024;
__global__ void __launch_bounds__(kPlanThreads)
plan_kernel(const uint8_t *__restrict__ live, int P, int32_t *__restrict__ new_index,
            int32_t *__restrict__ n_live, int32_t *__restrict__ src_idx,
            int32_t *__restrict__ dst_idx, Moves *__restrict__ moves) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
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
        moves->count = movers;
        moves->next = 0;
    }
}

// 16-byte values a task copies: 32 KB, more where a task first looks through many indices
static int64_t part_of(int64_t vecs, int64_t looked_through) {
    const int64_t p = looked_through * 2 > kPart ? (looked_through * 2 + kPart - 1) / kPart * kPart : kPart;
    return p < vecs ? p : vecs;
}

}  // namespace pool

// marks: room for one a slot, or null
cudaError_t launch_pool_copy(float *p, int P, int64_t elems, const int32_t *src,
                             const int32_t *dst, int n, uint32_t *marks, StatusWord *st,
                             cudaStream_t s) {
    const int64_t vecs = elems / 4;
    if (n <= pool::kLooked) marks = nullptr;
    if (marks) {
        const cudaError_t e = cudaMemsetAsync(marks, 0, sizeof(uint32_t) * P, s);
        if (e != cudaSuccess) return e;
        pool::mark_kernel<<<(n + pool::kThreads - 1) / pool::kThreads, pool::kThreads, 0, s>>>(
            marks, P, src, dst, n);
    }
    int64_t per = pool::part_of(vecs, marks ? 0 : n);
    while ((vecs + per - 1) / per * n > 0x7fffffffLL) per *= 2;
    const int64_t parts = (vecs + per - 1) / per;
    pool::copy_kernel<<<(unsigned)(n * parts), pool::kThreads, 0, s>>>(
        (float4 *)p, P, vecs, src, dst, n, marks, (int)parts, per, st);
    return cudaGetLastError();
}

cudaError_t launch_pool_compact(float *p, int P, int64_t elems, const uint8_t *live,
                                int32_t *new_index, int32_t *n_live, int32_t *moves, int sms,
                                cudaStream_t s) {
    // moves: the header, then P / 2 sources and P / 2 destinations (no more slots can move)
    const int half = P / 2 + 1;
    pool::Moves *m = reinterpret_cast<pool::Moves *>(moves);
    int32_t *src = moves + 4, *dst = src + half;
    pool::plan_kernel<<<1, pool::kPlanThreads, 0, s>>>(live, P, new_index, n_live, src, dst, m);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int64_t vecs = elems / 4;
    int64_t per = pool::part_of(vecs, 0);
    while ((vecs + per - 1) / per * half > 0x7fffffffLL) per *= 2;
    const int64_t parts = (vecs + per - 1) / per;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(half * parts < 8LL * sms ? half * parts : 8LL * sms));
    cfg.blockDim = dim3(pool::kThreads);
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, pool::move_kernel, (float4 *)p, vecs, m, (const int32_t *)src,
                              (const int32_t *)dst, (int)parts, per);
}

}  // namespace kda
