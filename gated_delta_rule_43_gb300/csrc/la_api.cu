// la_api.cu -- C ABI of the decayed linear attention, the query/key preparation and the
// state pool (declared in include/kda.h): argument checks, workspace layout, dispatch.
#include <cuda.h>
#include <stdint.h>

#include <atomic>
#include <cmath>

#include "kda_la.cuh"

namespace kda {
cudaError_t launch_la_plan(const int32_t *cu, int N, int64_t T_tot, int32_t *off, int unit_cost,
                           int chunk, int uncut, la::Cut *cuts, int ranges, int split, uint32_t *flags, int n_flags, StatusWord *st, const float *h0, float *hT,
                           int H, int lanes, int64_t dkdv, cudaStream_t s);
cudaError_t launch_la_scan(const la::Plan &p, const float *h0, float *bnd, const float *bnd_log,
                           int64_t dkdv, cudaStream_t s);
cudaError_t launch_la_simt(bool out, bool whole, int dk, int dv, const la::Plan &p, const float *q,
                           const float *k, const float *v, int64_t qs, int64_t ks, int64_t vs,
                           const float *g, int gpt, const float *h0, float *hT, float *o,
                           float *bnd, float *bnd_log, StatusWord *st, cudaStream_t s);
cudaError_t la_tensor_maps(CUtensorMap (&m)[8], const void *q, const void *k, const void *v,
                           const void *o, const float *h0, const float *hT, const float *bnd,
                           const la::Plan &p, int64_t T, int dk, int dv, int64_t qs, int64_t ks,
                           int64_t vs);
cudaError_t launch_la_tc(bool out, const la::Plan &p, const CUtensorMap (&m)[8], const float *g,
                         int gpt, int has_h0, int has_hT, void *o, int dk, int dv, float *bnd,
                         float *bnd_log, StatusWord *st, cudaStream_t s);
cudaError_t launch_la_decode(int dtype, int dk, int dv, const void *q, const void *k,
                             const void *v, const float *g, float *state, void *o, int N, int H,
                             int Hk, int64_t qs, int64_t ks, int64_t vs, int gpt,
                             const int32_t *idx, int P, StatusWord *st, cudaStream_t s);
cudaError_t launch_qk(int dtype, int D, const void *q, const void *k, void *qo, void *ko,
                      int64_t T_tot, int Hq, int Hk, int64_t qs, int64_t ks, int64_t qos,
                      int64_t kos, const float *qw, const float *kw, int norm, float eps,
                      float q_scale, float k_scale, const int32_t *pos, const float *inv_freq,
                      int rot, int interleaved, float rope_scale, int sms, cudaStream_t s);
cudaError_t launch_pool_copy(float *p, int P, int64_t elems, const int32_t *src,
                             const int32_t *dst, int n, uint32_t *marks, StatusWord *st,
                             cudaStream_t s);
cudaError_t launch_pool_compact(float *p, int P, int64_t elems, const uint8_t *live,
                                int32_t *new_index, int32_t *n_live, int32_t *moves, int sms,
                                cudaStream_t s);
}  // namespace kda

using namespace kda;

namespace {

inline size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
inline bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }
inline bool head_ok(int32_t d) { return d == 32 || d == 64 || d == 128; }
inline bool dtype_ok(int32_t d) { return d == KDA_F32 || d == KDA_BF16; }
inline int64_t elt(int32_t dtype) { return dtype == KDA_BF16 ? 2 : 4; }
kda_status cuda_status(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }

// SMs of the current device; a GB300's where there is none (sizing on a host without a GPU).
int sm_count() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 152;
    return sms;
}

// A strided [T, heads, D] tensor: rows in 16-byte steps, no overlap between tokens (an input
// of plain loads may repeat one token, stride 0), and no offset past 2^62 bytes.
bool stride_ok(int64_t stride, int64_t T, int32_t heads, int32_t D, int32_t dtype,
               bool repeat = false) {
    return (stride >= (int64_t)heads * D || (repeat && stride == 0)) && (stride * elt(dtype)) % 16 == 0 &&
           (T == 0 || stride <= ((int64_t)1 << 59) / T);
}

struct LaLayout {
    int lanes, ranges, chunk, uncut;   // uncut: chunks
    bool split;
    int flags;                // states that may be handed on, and a count of CTAs (tensor cores)
    size_t cuts_off, off_off, log_off, flag_off, bnd_off, total;
};

// One range of one lane an SM, and no more than there can be chunks.  On the
// tensor cores all heads that share queries and keys are lanes, or as many of them as leave no
// more than 1/24 of the SMs over; the CUDA cores are not bound by what they read.
LaLayout la_layout(int64_t T, int32_t N, int32_t H, int32_t Hk, int32_t dk, int32_t dv, int32_t dtype, int sms) {
    LaLayout L{};
    L.chunk = dtype == KDA_BF16 ? la::kTcChunk : la::kSimtChunk;
    L.uncut = (dtype == KDA_BF16 ? la::kTcUncut : la::kSimtUncut) / L.chunk;
    if (sms > la::kMaxRanges) sms = la::kMaxRanges;
    L.lanes = dtype == KDA_BF16 ? H / Hk : 1;
    while ((H / Hk) % L.lanes != 0 || L.lanes > sms || sms % L.lanes * 24 > sms) --L.lanes;
    const int64_t most = (T / L.chunk + N) * (int64_t)(H / L.lanes);
    sms /= L.lanes;
    L.ranges = (int)(most < 1 ? 1 : most < sms ? most : sms);
    L.split = L.ranges > 1 && T > (dtype == KDA_BF16 ? la::kTcSplit : la::kSimtSplit);
    const size_t all = (size_t)L.ranges * L.lanes;
    L.cuts_off = kHeaderBytes;
    L.off_off = L.cuts_off + round_up(sizeof(la::Cut) * ((size_t)L.ranges + 1), 256);
    L.log_off = L.off_off + round_up(3 * sizeof(int32_t) * ((size_t)N + 1), 256);
    // With fewer units than ranges nearly all cuts are in units of several: nothing to hand on.
    L.flags = dtype == KDA_BF16 && L.split && (int64_t)N * (H / L.lanes) >= L.ranges ? (int)all + 1 : 0;
    L.flag_off = L.log_off + round_up(sizeof(float) * all, 256);
    L.bnd_off = L.flag_off + round_up(sizeof(uint32_t) * L.flags, 256);
    L.total = L.bnd_off + (L.split ? sizeof(float) * 2 * all * dk * dv : 0);
    return L;
}

// Ranges that hold work, on the CUDA cores: all, or with SMs to spare the pieces that the plan
// cuts, counted for sequences of the mean length (the lengths are on the device).
int64_t busy_ranges(const LaLayout &L, int64_t T, int32_t N, int32_t H) {
    const int64_t each = (T + (int64_t)N * L.chunk - 1) / ((int64_t)N * L.chunk);   // chunks
    const int64_t pieces = N * (int64_t)H * (L.split && each >= 4 ? each / 2 : 1);
    return pieces < L.ranges ? pieces : L.ranges;
}

// Test hook (kda_test_la_fault): what the next call leaves out.
std::atomic<int> g_la_left_out{-1};

bool la_sizes_ok(int64_t T, int32_t N, int32_t H, int32_t Hk, int32_t dk, int32_t dv) {
    return N >= 0 && T >= 0 && H > 0 && Hk > 0 && H % Hk == 0 && (T == 0 || N > 0) &&
           T < ((int64_t)1 << 31) && T <= ((int64_t)1 << 40) / ((int64_t)H * (dk > dv ? dk : dv)) &&
           (int64_t)N * H <= 0x7fffffffLL &&
           (T / la::kSimtChunk + N) * (int64_t)H <= 0x7fffffffLL;   // (chunks are counted in 32 bits)
}

}  // namespace

extern "C" {

size_t kda_la_chunk_fwd_workspace_size(int64_t total_tokens, int32_t num_seqs, int32_t H,
                                       int32_t Hk, int32_t dk, int32_t dv, int32_t dtype) {
    if (!dtype_ok(dtype) || !head_ok(dk) || !head_ok(dv) ||
        !la_sizes_ok(total_tokens, num_seqs, H, Hk, dk, dv))
        return 0;
    return la_layout(total_tokens, num_seqs, H, Hk, dk, dv, dtype, sm_count()).total;
}

kda_status kda_la_chunk_fwd(const void *q, const void *k, const void *v, const float *g,
                            const int32_t *cu_seqlens, int32_t num_seqs, int64_t total_tokens,
                            int32_t H, int32_t Hk, int32_t dk, int32_t dv, int32_t dtype,
                            int64_t q_stride, int64_t k_stride, int64_t v_stride,
                            int32_t g_per_token, const float *initial_state,
                            float *final_state, void *o, void *workspace,
                            size_t workspace_bytes, void *stream) {
    if (!dtype_ok(dtype) || !head_ok(dk) || !head_ok(dv)) return KDA_ERR_UNSUPPORTED;
    if (!la_sizes_ok(total_tokens, num_seqs, H, Hk, dk, dv)) return KDA_ERR_INVALID_ARG;
    if (!stride_ok(q_stride, total_tokens, Hk, dk, dtype) ||
        !stride_ok(k_stride, total_tokens, Hk, dk, dtype) ||
        !stride_ok(v_stride, total_tokens, H, dv, dtype))
        return KDA_ERR_INVALID_ARG;
    if (!cu_seqlens || !workspace) return KDA_ERR_INVALID_ARG;
    if (total_tokens > 0 && (!q || !k || !v || !g || !o)) return KDA_ERR_INVALID_ARG;
    const void *al16[] = {q, k, v, o, initial_state, final_state};
    for (const void *p : al16)
        if (!aligned(p, 16)) return KDA_ERR_INVALID_ARG;
    if (!aligned(g, 4) || !aligned(cu_seqlens, 4) || !aligned(workspace, 256))
        return KDA_ERR_INVALID_ARG;
    if (o && (o == q || o == k || o == v)) return KDA_ERR_INVALID_ARG;
    const LaLayout L = la_layout(total_tokens, num_seqs, H, Hk, dk, dv, dtype, sm_count());
    if (workspace_bytes < L.total) return KDA_ERR_INVALID_ARG;

    cudaStream_t s = (cudaStream_t)stream;
    StatusWord *st = (StatusWord *)workspace;
    if (num_seqs == 0) return cuda_status(cudaMemsetAsync(st, 0, sizeof(StatusWord), s));
    uint8_t *ws = (uint8_t *)workspace;
    la::Cut *cuts = (la::Cut *)(ws + L.cuts_off);
    int32_t *off = (int32_t *)(ws + L.off_off);
    float *bnd_log = (float *)(ws + L.log_off), *bnd = (float *)(ws + L.bnd_off);
    const int64_t dkdv = (int64_t)dk * dv;
    // On the tensor cores a range can put its start state together from what the cuts before it
    // hold: 64 KB a cut (0.8 us) against a scan of about 7 us.  A unit has at most ranges * lanes / H + 1 cuts (the
    // cuts are even, and H units are as long as the longest).  In place the initial states may
    // be gone by then; the scan keeps copies.
    const bool in_place = initial_state && initial_state == final_state;
    const bool compose = dtype == KDA_BF16 && !in_place && L.ranges * L.lanes / H + 1 <= 12;
    const int left_out = dtype == KDA_BF16 ? g_la_left_out.exchange(-1) : -1;
    const la::Plan p{cu_seqlens, off, cuts, num_seqs, H, Hk, L.lanes, L.ranges, L.chunk,
                     in_place, compose, L.flags ? (uint32_t *)(ws + L.flag_off) : nullptr,
                     left_out};
    // A unit's states cost about as much as a chunk each (64 KB in, 64 KB out; measured on 16
    // packed sequences: 11.6k cycles beside 5.4k of a chunk).
    const int unit_cost = (initial_state ? 1 : 0) + (final_state ? 1 : 0);
    cudaError_t e = launch_la_plan(cu_seqlens, num_seqs, total_tokens, off, unit_cost, L.chunk,
                                   L.uncut, cuts, L.ranges, L.split, p.flags, L.flags, st, initial_state, final_state, H, L.lanes, dkdv, s);
    if (e != cudaSuccess) return KDA_ERR_CUDA;
    if (total_tokens == 0) return KDA_OK;
    CUtensorMap maps[8];
    if (dtype == KDA_BF16 &&
        la_tensor_maps(maps, q, k, v, o, initial_state, final_state, L.split ? bnd : nullptr, p,
                       total_tokens, dk, dv, q_stride, k_stride, v_stride) != cudaSuccess)
        return KDA_ERR_CUDA;
    // With two column blocks a range, one wave of CTAs: see launch_dims
    const bool whole = busy_ranges(L, total_tokens, num_seqs, H) * 2 > sm_count();
    auto pass = [&](bool out) {
        if (dtype == KDA_BF16)
            return launch_la_tc(out, p, maps, g, g_per_token, initial_state != nullptr,
                                final_state != nullptr, o, dk, dv, bnd, bnd_log, st, s);
        return launch_la_simt(out, whole, dk, dv, p, (const float *)q, (const float *)k, (const float *)v,
                              q_stride, k_stride, v_stride, g, g_per_token, initial_state,
                              final_state, (float *)o, bnd, bnd_log, st, s);
    };
    if (L.split) {
        e = pass(false);
        if (e == cudaSuccess && !compose) e = launch_la_scan(p, initial_state, bnd, bnd_log, dkdv, s);
        if (e != cudaSuccess) return KDA_ERR_CUDA;
    }
    return cuda_status(pass(true));
}

kda_status kda_test_la_fault(int32_t part) {
    if (part < -1) return KDA_ERR_INVALID_ARG;
    g_la_left_out = part;
    return KDA_OK;
}

static kda_status la_decode_impl(const void *q, const void *k, const void *v, const float *g,
                                 float *state, const int32_t *idx, int32_t P, void *o, int32_t N,
                                 int32_t H, int32_t Hk, int32_t dk, int32_t dv, int32_t dtype,
                                 int64_t qs, int64_t ks, int64_t vs, int32_t gpt, StatusWord *st,
                                 void *stream) {
    if (!dtype_ok(dtype) || !head_ok(dk) || !head_ok(dv)) return KDA_ERR_UNSUPPORTED;
    if (N < 0 || P < 0 || H <= 0 || Hk <= 0 || H % Hk != 0 || (int64_t)N * H > 0x1fffffffLL)
        return KDA_ERR_INVALID_ARG;
    if (!stride_ok(qs, N, Hk, dk, dtype, true) || !stride_ok(ks, N, Hk, dk, dtype, true) ||
        !stride_ok(vs, N, H, dv, dtype, true))
        return KDA_ERR_INVALID_ARG;
    if (N > 0 && (!q || !k || !v || !g || !state || !o)) return KDA_ERR_INVALID_ARG;
    const void *al16[] = {q, k, v, o, state};
    for (const void *p : al16)
        if (!aligned(p, 16)) return KDA_ERR_INVALID_ARG;
    if (!aligned(g, 4) || !aligned(idx, 4)) return KDA_ERR_INVALID_ARG;
    if (o && (o == q || o == k || o == v || o == (void *)state)) return KDA_ERR_INVALID_ARG;
    if (st && cudaMemsetAsync(st, 0, sizeof(StatusWord), (cudaStream_t)stream) != cudaSuccess)
        return KDA_ERR_CUDA;
    if (N == 0) return KDA_OK;
    return cuda_status(launch_la_decode(dtype, dk, dv, q, k, v, g, state, o, N, H, Hk, qs, ks, vs,
                                        gpt, idx, P, st, (cudaStream_t)stream));
}

kda_status kda_la_decode_step(const void *q, const void *k, const void *v, const float *g,
                              float *state, void *o, int32_t N, int32_t H, int32_t Hk,
                              int32_t dk, int32_t dv, int32_t dtype, int64_t q_stride,
                              int64_t k_stride, int64_t v_stride, int32_t g_per_token,
                              void *stream) {
    return la_decode_impl(q, k, v, g, state, nullptr, N, o, N, H, Hk, dk, dv, dtype, q_stride,
                          k_stride, v_stride, g_per_token, nullptr, stream);
}

kda_status kda_la_decode_step_indexed(const void *q, const void *k, const void *v,
                                      const float *g, float *state_pool,
                                      const int32_t *state_idx, int32_t P, void *o, int32_t N,
                                      int32_t H, int32_t Hk, int32_t dk, int32_t dv,
                                      int32_t dtype, int64_t q_stride, int64_t k_stride,
                                      int64_t v_stride, int32_t g_per_token, void *workspace,
                                      size_t workspace_bytes, void *stream) {
    if (N > 0 && !state_idx) return KDA_ERR_INVALID_ARG;
    if (workspace && (workspace_bytes < kHeaderBytes || !aligned(workspace, 256)))
        return KDA_ERR_INVALID_ARG;
    return la_decode_impl(q, k, v, g, state_pool, state_idx, P, o, N, H, Hk, dk, dv, dtype,
                          q_stride, k_stride, v_stride, g_per_token, (StatusWord *)workspace,
                          stream);
}

kda_status kda_qk_norm_rope(const void *q, const void *k, void *q_out, void *k_out,
                            int64_t total_tokens, int32_t Hq, int32_t Hk, int32_t D,
                            int32_t dtype, int64_t q_stride, int64_t k_stride,
                            int64_t q_out_stride, int64_t k_out_stride, const float *q_weight,
                            const float *k_weight, int32_t norm, float eps, float q_scale,
                            float k_scale, const int32_t *positions, const float *inv_freq,
                            int32_t rot_dim, int32_t layout, float rope_scale, void *stream) {
    if (!dtype_ok(dtype) || !head_ok(D)) return KDA_ERR_UNSUPPORTED;
    if (norm < KDA_NORM_NONE || norm > KDA_NORM_RMS ||
        (layout != KDA_ROPE_HALF && layout != KDA_ROPE_INTERLEAVED))
        return KDA_ERR_INVALID_ARG;
    if (rot_dim < 0 || rot_dim > D) return KDA_ERR_INVALID_ARG;
    if (rot_dim % 16 != 0) return KDA_ERR_UNSUPPORTED;
    if (total_tokens < 0 || total_tokens >= ((int64_t)1 << 31) || Hq <= 0 || Hk < 0 ||
        (int64_t)Hq + Hk > 65536 || !(eps >= 0.f) || std::isinf(eps))
        return KDA_ERR_INVALID_ARG;
    if (!stride_ok(q_stride, total_tokens, Hq, D, dtype, true) ||
        !stride_ok(q_out_stride, total_tokens, Hq, D, dtype) ||
        (Hk > 0 && (!stride_ok(k_stride, total_tokens, Hk, D, dtype, true) ||
                    !stride_ok(k_out_stride, total_tokens, Hk, D, dtype))))
        return KDA_ERR_INVALID_ARG;
    if (total_tokens == 0) return KDA_OK;
    if (!q || !q_out || (Hk > 0 && (!k || !k_out)) || (rot_dim > 0 && (!positions || !inv_freq)))
        return KDA_ERR_INVALID_ARG;
    const void *al16[] = {q, k, q_out, k_out, q_weight, k_weight};
    for (const void *p : al16)
        if (!aligned(p, 16)) return KDA_ERR_INVALID_ARG;
    if (!aligned(positions, 4) || !aligned(inv_freq, 4)) return KDA_ERR_INVALID_ARG;
    // in place only with the input's own stride
    if ((q_out == q && q_out_stride != q_stride) || (Hk > 0 && k_out == k && k_out_stride != k_stride))
        return KDA_ERR_INVALID_ARG;
    if (Hk > 0 && (q_out == k || k_out == q || q_out == k_out)) return KDA_ERR_INVALID_ARG;
    return cuda_status(launch_qk(dtype, D, q, k, q_out, k_out, total_tokens, Hq, Hk, q_stride,
                                 k_stride, q_out_stride, k_out_stride, q_weight, k_weight, norm,
                                 eps, q_scale, k_scale, positions, inv_freq, rot_dim,
                                 layout == KDA_ROPE_INTERLEAVED, rope_scale, sm_count(),
                                 (cudaStream_t)stream));
}

size_t kda_state_pool_workspace_size(int32_t P) {
    return P < 0 ? 0 : kHeaderBytes + round_up(sizeof(int32_t) * (4 + 2 * ((size_t)P / 2 + 1)), 256);
}

static bool pool_ok(const float *pool, int32_t P, int64_t slot_elems) {
    return P >= 0 && slot_elems > 0 && slot_elems % 4 == 0 &&
           (P == 0 || slot_elems <= ((int64_t)1 << 58) / P) && (P == 0 || pool) && aligned(pool, 16);
}

kda_status kda_state_pool_copy(float *pool, int32_t P, int64_t slot_elems,
                               const int32_t *src_idx, const int32_t *dst_idx, int32_t n,
                               void *workspace, size_t workspace_bytes, void *stream) {
    if (!pool_ok(pool, P, slot_elems) || n < 0 || n > (1 << 24)) return KDA_ERR_INVALID_ARG;
    if (n > 0 && (!src_idx || !dst_idx || !aligned(src_idx, 4) || !aligned(dst_idx, 4)))
        return KDA_ERR_INVALID_ARG;
    // Without room for marks the check of the copies against each other is quadratic: 2^16 of them
    // take 10 ms
    const bool room = workspace && workspace_bytes >= kda_state_pool_workspace_size(P);
    if (n > (1 << 16) && !room) return KDA_ERR_INVALID_ARG;
    if (workspace && (workspace_bytes < kHeaderBytes || !aligned(workspace, 256)))
        return KDA_ERR_INVALID_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    if (workspace && cudaMemsetAsync(workspace, 0, sizeof(StatusWord), s) != cudaSuccess)
        return KDA_ERR_CUDA;
    if (n == 0) return KDA_OK;
    uint32_t *marks = room ? (uint32_t *)((uint8_t *)workspace + kHeaderBytes) : nullptr;
    return cuda_status(launch_pool_copy(pool, P, slot_elems, src_idx, dst_idx, n, marks,
                                        (StatusWord *)workspace, s));
}

kda_status kda_state_pool_compact(float *pool, int32_t P, int64_t slot_elems,
                                  const uint8_t *live, int32_t *new_index, int32_t *n_live,
                                  void *workspace, size_t workspace_bytes, void *stream) {
    if (!pool_ok(pool, P, slot_elems) || !n_live || !aligned(n_live, 4)) return KDA_ERR_INVALID_ARG;
    if (P > 0 && (!live || !new_index || !aligned(new_index, 4))) return KDA_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < kda_state_pool_workspace_size(P) || !aligned(workspace, 256))
        return KDA_ERR_INVALID_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    if (P == 0) return cuda_status(cudaMemsetAsync(n_live, 0, sizeof(int32_t), s));
    return cuda_status(launch_pool_compact(pool, P, slot_elems, live, new_index, n_live,
                                           (int32_t *)((uint8_t *)workspace + kHeaderBytes),
                                           sm_count(), s));
}

}  // extern "C"
