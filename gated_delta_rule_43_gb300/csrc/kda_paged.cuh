// kda_paged.cuh -- what the kernels of the paged key/value cache share (not part of the ABI).
//
// Pages are [P, Hk, page size, D] (a head's tokens of a page are one run of memory, what a tile
// load wants), P pages `stride` elements apart, so that keys and values may be halves of one pool.
// Position j of sequence n lies in slot j % size of page table[n][j / size].  Of the sequence's
// kv_lens[n] tokens the last are the `len` new ones that the call is about: token i of them stands at
// position kv_lens[n] - len + i.  A position below 0 is padding: it is written nowhere, reads as
// zeros and attends to nothing.
#pragma once

#include <cuda_fp8.h>

#include "kda_common.cuh"

namespace kda {
namespace paged {

struct Cache {
    const int32_t *cu;        // [N + 1], or null: one new token a sequence
    const int32_t *kv_lens;   // [N]
    const int32_t *table;     // [N, width]
    int N, width;
    int T;                    // rows of the packed tensors
    int P, Hk, shift;         // pages; heads; log2 of the page size
    void *k, *v;
    int64_t stride;           // elements from one page to the next
    float *ks, *vs;           // [P, Hk, page size] scales of an e4m3 cache, or null
    int64_t scale_stride;
};

// The new tokens of sequence n and where they stand: rows [begin, begin + len), the first at position
// `pos`.  A sequence that does not fit (the first one also where it does not begin at 0) has len 0.
struct Span {
    int begin, len, pos;
};
__device__ __forceinline__ bool lens_ok(const Cache &c, int n, int begin, int end, int ctx) {
    return (n > 0 || begin == 0) && begin >= 0 && begin <= end && end <= c.T && ctx >= 0 && ctx <= ((int64_t)c.width << c.shift);
}
__device__ __forceinline__ Span span_of(const Cache &c, int n) {
    const int ctx = c.kv_lens[n], begin = c.cu ? c.cu[n] : n, end = c.cu ? c.cu[n + 1] : n + 1;
    if (!lens_ok(c, n, begin, end, ctx)) return Span{0, 0, 0};
    return Span{begin, end - begin, ctx - (end - begin)};
}

// Reports sequences that do not fit; all threads of one block.
__device__ __forceinline__ void check_spans(const Cache &c, StatusWord *st) {
    if (!st) return;
    for (int n = threadIdx.x; n < c.N; n += blockDim.x) {
        const int begin = c.cu ? c.cu[n] : n, end = c.cu ? c.cu[n + 1] : n + 1;
        if (!lens_ok(c, n, begin, end, c.kv_lens[n])) report(st, KDA_ERR_SEQLENS, n, 61);
    }
}

// The sequence whose rows hold row t (cu must be ascending; where it is not, some sequence or -1);
// a whole warp, 32 places a step.
__device__ __forceinline__ int sequence_of(const Cache &c, int t) {
    const int lane = threadIdx.x & 31;
    int lo = 0, count = c.N;   // the last n in [lo, lo + count) with cu[n] <= t
    while (count > 1) {
        const int step = (count + 31) / 32, at = lo + lane * step;
        const bool here = lane * step < count && c.cu[at] <= t;
        const uint32_t m = __ballot_sync(0xffffffffu, here);
        if (m == 0) return -1;
        const int last = 31 - __clz(m);
        lo += last * step;
        count = min(step, count - last * step);
    }
    return lo;
}

// The least power of two s with top / s <= 448, the largest e4m3: 448 = 1.75 * 2^8.  Multiplying
// and dividing by it is exact, so a stored value is off by its one rounding to e4m3 alone, and s
// times an e4m3 is a bf16 exactly (2^-100 keeps the smallest of them above bf16's own).
__device__ __forceinline__ int scale_exponent(float top) {
    const uint32_t b = __float_as_uint(top);
    const int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
    return min(max(e, -100), 119);
}
__device__ __forceinline__ float two_to(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Blocks of `size` keys that rows at positions first .. last see: `sinks` of them from the sequence's
// start, then those from block `from` on.
struct KeyBlocks {
    int sinks, from, count;
    __device__ __forceinline__ int block(int i) const { return i < sinks ? i : from + i - sinks; }
};
__device__ __forceinline__ KeyBlocks key_blocks(int first, int last, int window, int sinks, int size) {
    KeyBlocks b{0, 0, 0};
    if (last < 0) return b;
    if (window > 0) {
        b.from = max(0, first - window + 1) / size;
        b.sinks = min(b.from, (int)(((int64_t)sinks + size - 1) / size));
    }
    b.count = b.sinks + last / size + 1 - b.from;
    return b;
}

}  // namespace paged
}  // namespace kda
