// kda_la.cuh -- how a prefill of the decayed linear attention is cut over the GPU.
//
// A unit is one head of one sequence, a run of chunks; the units of all sequences,
// heads inside sequences, stand in one row of `total` chunks.  The row is cut into `ranges`
// equal parts, one for each CTA (CTA group on the CUDA cores), wherever that falls: every SM
// has the same work whatever the lengths are.  (A unit counts as `unit_cost` chunks more than it
// has, for its states.)  The state at a cut inside a unit comes from one of these:
//   - the unit is cut once and its first part is handed on (see Items);
//   - else a first pass forms what the tokens before the cut, back to the unit's start or the cut
//     before, leave there, and the range behind starts from all of the unit's cuts up to its own
//     (p.compose), or, where those can be many or the initial states are overwritten, a scan
//     along the cuts has put them together (6 us).
// A cut moves out of a unit of at most 512 tokens (64 on the CUDA cores) to its nearer end: for
// so few another start costs more than the evener load gives (40 sequences of 700 tokens, 4 heads:
// with 256, 512, 1024 tokens 55, 55, 63 us; 8 heads of 8192, whose pieces it bounds: 51, 48, 48).
// Nothing is cut in calls of at most 1024 tokens (128): the kernels it takes cost as much as it
// gives (8 heads of 600 tokens: 27 us, cut 29; of 1000: 31 and 29).  When there are more SMs than work,
// every unit has a range of its own, and a longer one several.  On the tensor cores these are of
// sqrt(chunks) / 2 chunks, since every range adds a state that others read (8 heads of 2000 tokens
// in pieces of 2, 4, 8 chunks: 32, 38, 51 us; 2 heads of 16384: 55, 48, 55); on the CUDA cores,
// where a chunk takes longest, of two (a head of 4096 tokens in pieces of 1, 2, 4: 69, 51, 67 us).
// Chunks are 128 tokens on the tensor cores and 32 on the CUDA cores.
//
// Value heads that share queries and keys are walked side by side: `lanes` CTAs take the same
// range of the row of every lanes-th head, so that what one of them reads the others find in
// L2.  (With four heads a query/key head, tiles read and written without any arithmetic:
// head after head 5.8k cycles a chunk, side by side 3.9k.)
#pragma once

#include "kda_common.cuh"

namespace kda {
namespace la {

constexpr int kTcChunk = 128, kTcUncut = 512, kTcSplit = 1024;
constexpr int kSimtChunk = 32, kSimtUncut = 64, kSimtSplit = 128;
constexpr int kMaxRanges = 512;   // (the plan's shared memory)

// A place in the row of chunks: before chunk c of head h of sequence n.  (What a walk needs of the
// sequence stands beside it: one read from memory less before anything can begin.)
struct Cut {
    int64_t x;
    int32_t nc;               // chunks of sequence n, 0 at the row's end
    int32_t begin, stop;      // its tokens
    int32_t n, h, c;
    int32_t inner;            // inside a unit: 1 + the inner cuts of this unit that follow; else 0
    int32_t before;           // the inner cuts of this unit before it
    int32_t handed;           // the range before hands the state on (see Items)
};

struct Plan {
    const int32_t *cu;        // [N + 1]
    const int32_t *off;       // [N + 1]: chunks of the sequences before n
    const Cut *cuts;          // [ranges + 1], the last at the row's end
    int N, H, Hk;
    int lanes;                // divides H / Hk
    int ranges;               // of a lane
    int chunk;                // tokens
    int in_place;             // the final states overwrite the initial ones
    int compose;              // no scan: ranges put their start states together themselves
    uint32_t *flags;          // states handed on, as the states of the cuts; then the CTAs begun (or null)
    int left_out;             // tests: the range (times lanes, plus lane) whose first load of keys is left out, or -1
};

// The chunks [c0, c1) of one unit.
struct Item {
    enum Part { kWhole, kHead, kTail };
    int n, h;
    int part;                 // kHead, kTail: of a unit whose one cut is handed on
    int c0, c1, nc;           // of nc
    int t0, t1;               // tokens [t0, t1) of the packed tensors
};

__device__ __forceinline__ void set_tokens(Item &it, int chunk, int begin, int stop) {
    it.t0 = begin + it.c0 * chunk;
    it.t1 = it.c1 == it.nc ? stop : begin + it.c1 * chunk;
}

// Walks the items of the range between two cuts.  The heads of a sequence follow each other, so
// what is known of the sequence is kept: its reads take microseconds beside a busy memory.  (Little
// of it, in 32 bits: every role holds one in registers.)
struct Walk {
    int left;                 // chunks of the range
    int n, h, c;
    int nc;                   // chunks of sequence n, 0: not read yet
    int begin, stop;          // its tokens
    __device__ __forceinline__ Walk(const Plan &p, int range, int lane) {
        const Cut &b = p.cuts[range];
        left = (int)(p.cuts[range + 1].x - b.x);
        n = b.n;
        h = b.h * p.lanes + lane;
        c = b.c;
        nc = b.nc;
        begin = b.begin;
        stop = b.stop;
    }
    __device__ __forceinline__ void skip(const Plan &p, int chunks) {   // to the end of the unit
        left -= chunks;
        c = 0;
        if ((h += p.lanes) >= p.H) {
            h -= p.H;
            ++n;
            nc = 0;
        }
    }
    __device__ __forceinline__ bool next(const Plan &p, Item &it) {
        if (left <= 0) return false;
        if (nc == 0) {
            while ((nc = p.off[n + 1] - p.off[n]) == 0) ++n;   // (sequences without tokens)
            begin = p.cu[n];
            stop = p.cu[n + 1];
        }
        it.part = Item::kWhole;
        it.n = n;
        it.h = h;
        it.c0 = c;
        it.nc = nc;
        it.c1 = min(nc, c + left);
        set_tokens(it, p.chunk, begin, stop);
        skip(p, it.c1 - c);
        return true;
    }
};

// Programmatic launches: a kernel may be on the GPU before the one that it depends on has ended.
__device__ __forceinline__ void wait_for_previous() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void let_next_start() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
template <typename... P, typename... A>
inline cudaError_t launch_after(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem,
                                cudaStream_t s, A... args) {
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

// What the range before cut `i` (1 ..) contributes to it; false when that cut is none inside
// a unit.
__device__ __forceinline__ bool before_cut(const Plan &p, int i, int lane, Item &it) {
    const Cut e = p.cuts[i];
    if (!e.inner) return false;
    it.part = Item::kHead;
    it.n = e.n;
    it.h = e.h * p.lanes + lane;
    it.c1 = e.c;
    it.c0 = (int)max((int64_t)0, e.c - (e.x - p.cuts[i - 1].x));
    it.nc = e.nc;
    set_tokens(it, p.chunk, e.begin, e.stop);
    return true;
}

// The states of the inner boundaries, cuts 1 .. of each lane.  Where the final states overwrite
// the initial ones, the last range of a unit may write before the first one has read: the
// scan keeps a copy of the initial state of such a unit, for the range that it begins in.
__device__ __forceinline__ int64_t cut_state(const Plan &p, int i, int lane) {
    return (int64_t)(i - 1) * p.lanes + lane;
}
__device__ __forceinline__ int64_t initial_copy(const Plan &p, int range, int lane) {
    return (int64_t)(p.ranges + range) * p.lanes + lane;
}

// Where an item starts from: `steps` states, each taken after the decay of what lies between it
// and the one before.  A unit's start: none (zeros) or the initial state (its copy).  A cut
// after the scan: the state there.  A cut without it (p.compose): the unit's initial state and
// what the cuts up to this one hold.
struct Start {
    int steps;
    int32_t h0;               // index of the first step's initial state, -1: it is a cut's
    bool h0_copied;
    int32_t first, lanes;     // the first cut's state; from one to the next
    __device__ __forceinline__ bool in_bnd(int s) const { return s > 0 || h0 < 0 || h0_copied; }
    __device__ __forceinline__ int32_t index(int s) const {
        return s == 0 && h0 >= 0 ? h0 : first + (s - (h0 >= 0 ? 1 : 0)) * lanes;
    }
};
__device__ __forceinline__ Start start_state(const Plan &p, const Item &it, int range, int lane, bool h0) {
    Start r{0, -1, false, 0, p.lanes};
    if (it.part == Item::kTail) {
        r.steps = 1;
        r.first = (int32_t)cut_state(p, range, lane);
    } else if (it.c0 > 0) {
        const int before = p.compose ? p.cuts[range].before : 0;
        r.first = (int32_t)cut_state(p, range - before, lane);
        r.steps = before + 1;
        if (p.compose && h0) {
            r.h0 = it.n * p.H + it.h;
            ++r.steps;
        }
    } else if (h0) {
        r.steps = 1;
        r.h0_copied = it.c1 < it.nc && it.part != Item::kHead && p.in_place;
        r.h0 = r.h0_copied ? (int32_t)initial_copy(p, range, lane) : it.n * p.H + it.h;
    }
    return r;
}

// The items of a range, in the order in which they are walked.  A unit with one cut needs no
// first pass where the range behind the cut has as much else to do as lies before it: the
// range before takes its part (the head) first of all and hands the state on, the range
// behind takes the rest (the tail) last.  A head waits for nothing, and ranges are dealt out in
// the order in which CTAs begin, so that the one before has begun: the wait ends however few
// CTAs run at a time.  (16 packed sequences of 18 chunks in the mean, 66 chunks a range: the first pass
// took 34 of 224 us.)
struct Items {
    Walk walk;
    enum { kFirst, kWalk, kLast } at;
    __device__ __forceinline__ Items(const Plan &p, int range, int lane) : walk(p, range, lane) {
        at = p.cuts[range + 1].handed ? kFirst : kWalk;
        if (p.cuts[range].handed) walk.skip(p, walk.nc - walk.c);
        if (at == kFirst) walk.left -= p.cuts[range + 1].c;
    }
    __device__ __forceinline__ bool next(const Plan &p, int range, int lane, Item &it) {
        if (at == kFirst) {
            at = kWalk;
            return before_cut(p, range + 1, lane, it);
        }
        if (at == kLast) return false;
        if (walk.next(p, it)) return true;
        at = kLast;
        const Cut &b = p.cuts[range];
        if (!b.handed) return false;
        it.part = Item::kTail;
        it.n = b.n;
        it.h = b.h * p.lanes + lane;
        it.c0 = b.c;
        it.c1 = it.nc = b.nc;
        set_tokens(it, p.chunk, b.begin, b.stop);
        return true;
    }
};

// A log decay below this is e^g = 0 in fp32.  Prefix sums, whose differences give the decay
// between two tokens of a chunk, take g no lower than this, so that a reset (-inf) leaves
// no inf - inf; sums that are only ever exponentiated take g as it is.
constexpr float kLogZero = -104.0f;

__device__ __forceinline__ bool log_decay_ok(float g) { return g <= 0.0f; }   // false for NaN

}  // namespace la
}  // namespace kda
