// kda_la.cuh -- what the translation units of the decayed linear attention share: the plan
// of the packed sequences, the work items of a launch, and the gate's values in a chunk.
//
// Every sequence is cut into segments of seg_tokens tokens.  seg_off[n] counts the segments
// of the sequences before n, bnd_off[n] the inner boundaries (a sequence of s segments has
// s - 1); boundary bnd_off[n] + j lies between the segments j and j + 1 of sequence n.
// When the final states overwrite the initial ones, the last segment of a sequence may write
// before the first one has read: then the scan keeps a copy of the initial state of every
// sequence of several segments behind the boundaries' states, at index
// bnd_off[N] + multi_off[n] (multi_off counts such sequences before n).
#pragma once

#include "kda_common.cuh"

namespace kda {
namespace la {

struct Plan {
    const int32_t *cu;        // [N + 1]
    const int32_t *seg_off;   // [N + 1]
    const int32_t *bnd_off;   // [N + 1]
    const int32_t *multi_off; // [N + 1]
    int N;
    int H, Hk;
    int64_t seg_tokens;
    int in_place;             // the final states overwrite the initial ones
};

struct Item {
    int n, seg, nseg;
    int64_t t0, t1;           // tokens [t0, t1) of the packed tensors
    int64_t bnd;              // boundary that ends this segment (the one before starts it)
};

// The largest n with off[n] <= x (off is non-decreasing, off[0] = 0, x < off[N]).
__device__ __forceinline__ int find_owner(const int32_t *off, int N, int32_t x) {
    int lo = 0, hi = N - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (off[mid] <= x) lo = mid; else hi = mid - 1;
    }
    return lo;
}

__device__ __forceinline__ Item segment(const Plan &p, int32_t slot) {
    Item it;
    it.n = p.N == 1 ? 0 : find_owner(p.seg_off, p.N, slot);
    const int32_t first = p.seg_off[it.n];
    it.seg = slot - first;
    it.nseg = p.seg_off[it.n + 1] - first;
    it.t0 = p.cu[it.n] + it.seg * p.seg_tokens;
    it.t1 = min(it.t0 + p.seg_tokens, (int64_t)p.cu[it.n + 1]);
    it.bnd = p.bnd_off[it.n] + it.seg;
    return it;
}

// Segment j < bnd_off[N] of those that end at an inner boundary.
__device__ __forceinline__ Item inner_segment(const Plan &p, int32_t j) {
    Item it;
    it.n = p.N == 1 ? 0 : find_owner(p.bnd_off, p.N, j);
    it.seg = j - p.bnd_off[it.n];
    it.nseg = p.seg_off[it.n + 1] - p.seg_off[it.n];
    it.t0 = p.cu[it.n] + it.seg * p.seg_tokens;
    it.t1 = it.t0 + p.seg_tokens;
    it.bnd = j;
    return it;
}

// Where segment `it` of head h starts from: boundary states, the initial state or its copy;
// NULL for zeros.
__device__ __forceinline__ const float *start_state(const Plan &p, const Item &it, int h,
                                                    const float *h0, const float *bnd,
                                                    int64_t dkdv) {
    if (it.seg > 0) return bnd + ((it.bnd - 1) * p.H + h) * dkdv;
    if (!h0) return nullptr;
    if (it.nseg > 1 && p.in_place)
        return bnd + ((int64_t)(p.bnd_off[p.N] + p.multi_off[it.n]) * p.H + h) * dkdv;
    return h0 + ((int64_t)it.n * p.H + h) * dkdv;
}

// A log decay below this is e^g = 0 in fp32.  Prefix sums, whose differences give the decay
// between two tokens of a chunk, take g no lower than this, so that a reset (-inf) leaves
// no inf - inf; sums that are only ever exponentiated take g as it is.
constexpr float kLogZero = -104.0f;

__device__ __forceinline__ bool log_decay_ok(float g) { return g <= 0.0f; }   // false for NaN

}  // namespace la
}  // namespace kda
