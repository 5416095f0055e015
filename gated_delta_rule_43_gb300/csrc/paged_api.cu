// paged_api.cu -- C ABI of the paged key/value cache and its attention (declared in include/kda.h):
// argument checks, workspace layout, dispatch.
#include <stdint.h>

#include <atomic>
#include <cmath>

#include "kda_paged.cuh"

namespace kda {
cudaError_t launch_kv_cache(bool write, int dtype, int cache_dtype, int D, const paged::Cache &c, void *k, void *v,
                            int64_t ks, int64_t vs, StatusWord *st, cudaStream_t s);
size_t paged_simt_bytes(const paged::Cache &c, int group, int D, int sms);
cudaError_t launch_paged_simt(int cache_dtype, int D, const paged::Cache &c, const void *q, int64_t qs, void *o, int group,
                              float scale, int window, int sinks, float *part, int sms, StatusWord *st, cudaStream_t s);
cudaError_t launch_paged_none(int64_t row_bytes, const paged::Cache &c, void *o, int group, StatusWord *st, cudaStream_t s);
size_t paged_tc_bytes(const paged::Cache &c, int group, int D, int sms);
cudaError_t launch_paged_tc(bool e4m3, int D, const paged::Cache &c, const void *q, int64_t qs, void *o, int group,
                            float scale, int window, int sinks, void *ws, int sms, int left_out, cudaStream_t s);
size_t paged_decode_bytes(int group, int D, int sms);
cudaError_t launch_paged_decode(bool e4m3, int D, const paged::Cache &c, const void *q, int64_t qs, void *o, int group,
                                float scale, int window, int sinks, void *ws, int sms, int left_out, cudaStream_t s);
size_t paged_decode_simt_bytes(bool e4m3, int group, int D, int sms);
cudaError_t launch_paged_decode_simt(bool e4m3, int D, const paged::Cache &c, const void *q, int64_t qs, void *o, int group,
                                     float scale, int window, int sinks, void *ws, int sms, cudaStream_t s);
}  // namespace kda

using namespace kda;

namespace {

inline bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }
kda_status cuda_status(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }

int sm_count() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 152;
    return sms;
}

inline int64_t bytes_of(int32_t dtype) { return dtype == KDA_E4M3 ? 1 : dtype == KDA_BF16 ? 2 : 4; }

kda_status types_ok(const kda_paged_cache *p, int32_t dtype) {
    if (!p) return KDA_ERR_INVALID_ARG;
    if (dtype != KDA_F32 && dtype != KDA_BF16) return KDA_ERR_UNSUPPORTED;
    if (p->dtype != dtype && p->dtype != KDA_E4M3) return KDA_ERR_UNSUPPORTED;
    if (p->D != 32 && p->D != 64 && p->D != 128) return KDA_ERR_UNSUPPORTED;
    const int32_t s = p->page_size;
    return s >= 16 && s <= 1024 && (s & (s - 1)) == 0 ? KDA_OK : KDA_ERR_UNSUPPORTED;
}

bool sizes_ok(const kda_paged_cache *p, int64_t T) {
    return p->num_seqs >= 0 && p->table_width >= 0 && p->num_pages >= 0 && p->Hk > 0 && p->Hk <= 65536 && T >= 0 &&
           T < ((int64_t)1 << 31) && (p->cu_seqlens || T == p->num_seqs) &&
           (int64_t)p->table_width * p->page_size < ((int64_t)1 << 31) && p->num_seqs < 0x7fffffff;
}

// q rows of all heads in 16-byte steps, tokens apart or (an input) one token for all
bool stride_ok(int64_t stride, int64_t T, int64_t row, int32_t dtype) {
    return (stride >= row || stride == 0) && stride * bytes_of(dtype) % 16 == 0 &&
           (T == 0 || stride <= ((int64_t)1 << 59) / T);
}

// The cache's pointers and strides, for a call that touches it.
bool cache_ok(const kda_paged_cache *p) {
    const int64_t page = (int64_t)p->Hk * p->page_size * p->D;
    if (!p->kv_lens || !aligned(p->kv_lens, 4) || !aligned(p->cu_seqlens, 4) || !aligned(p->block_table, 4) ||
        (p->table_width > 0 && !p->block_table))
        return false;
    if (p->num_pages > 0 && (!p->k_pages || !p->v_pages || p->k_pages == p->v_pages)) return false;
    if (!aligned(p->k_pages, 16) || !aligned(p->v_pages, 16)) return false;
    if (p->page_stride < page || p->page_stride % ((int64_t)p->page_size * p->D) != 0 ||
        (p->num_pages > 0 && p->page_stride / ((int64_t)p->page_size * p->D) > 0x7fffffff / p->num_pages) ||
        (p->num_pages > 0 && p->page_stride > ((int64_t)1 << 58) / p->num_pages))
        return false;
    if (p->dtype == KDA_E4M3)
        return (p->num_pages == 0 || (p->k_scales && p->v_scales && p->k_scales != p->v_scales)) &&
               aligned(p->k_scales, 16) && aligned(p->v_scales, 16) &&
               p->scale_stride >= (int64_t)p->Hk * p->page_size && p->scale_stride % 4 == 0 &&
               (p->num_pages == 0 || p->scale_stride <= ((int64_t)1 << 58) / p->num_pages);
    return !p->k_scales && !p->v_scales;
}

paged::Cache make(const kda_paged_cache *p, int64_t T) {
    int shift = 0;
    while ((1 << shift) < p->page_size) ++shift;
    return paged::Cache{p->cu_seqlens, p->kv_lens, p->block_table, p->num_seqs, p->table_width, (int)T,
                        p->num_pages, p->Hk, shift, p->k_pages, p->v_pages, p->page_stride,
                        p->k_scales, p->v_scales, p->scale_stride};
}

kda_status clear(StatusWord *st, cudaStream_t s) {
    return st ? cuda_status(cudaMemsetAsync(st, 0, sizeof(StatusWord), s)) : KDA_OK;
}

bool attn_sizes_ok(const kda_paged_cache *p, int64_t T, int32_t H) {
    return sizes_ok(p, T) && H > 0 && H <= 65536 && H % p->Hk == 0 && T * (H / p->Hk) < ((int64_t)1 << 31);
}

// Test hook (kda_test_paged_fault): what the next call leaves out.
std::atomic<int> g_left_out{-1};

// bf16 goes to the tensor cores, fp32 to the CUDA cores; a pool without pages has nothing to load (and no tensor
// map).
size_t attn_bytes(const kda_paged_cache *p, int64_t T, int32_t H, int32_t dtype) {
    if (p->num_pages == 0) return kHeaderBytes;
    const paged::Cache c = make(p, T);
    const int group = H / p->Hk, sms = sm_count();
    if (dtype == KDA_BF16) return p->cu_seqlens ? paged_tc_bytes(c, group, p->D, sms) : paged_decode_bytes(group, p->D, sms);
    if (!p->cu_seqlens) return paged_decode_simt_bytes(p->dtype == KDA_E4M3, group, p->D, sms);
    return kHeaderBytes + paged_simt_bytes(c, group, p->D, sms);
}

kda_status attn(const kda_paged_cache *p, const void *q, int64_t qs, void *o, int64_t T, int32_t H, int32_t dtype,
                float scale, int32_t window, int32_t sinks, void *workspace, size_t workspace_bytes, void *stream) {
    const kda_status t = types_ok(p, dtype);
    if (t != KDA_OK) return t;
    if (!attn_sizes_ok(p, T, H)) return KDA_ERR_INVALID_ARG;
    if (!stride_ok(qs, T, (int64_t)H * p->D, dtype) || !(scale > 0.f) || std::isinf(scale) || window < 0 || sinks < 0)
        return KDA_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < attn_bytes(p, T, H, dtype)) return KDA_ERR_INVALID_ARG;
    if (T > 0 && (!q || !o || q == o)) return KDA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(o, 16)) return KDA_ERR_INVALID_ARG;
    if (p->num_seqs > 0 && !cache_ok(p)) return KDA_ERR_INVALID_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    StatusWord *st = (StatusWord *)workspace;
    const bool e4m3 = p->dtype == KDA_E4M3, some = T > 0 && p->num_seqs > 0;
    const int group = H / p->Hk;
    if (some && p->num_pages > 0 && dtype == KDA_BF16)
        return cuda_status((p->cu_seqlens ? launch_paged_tc : launch_paged_decode)(
            e4m3, p->D, make(p, T), q, qs, o, group, scale, window, sinks, workspace, sm_count(), g_left_out.exchange(-1), s));
    if (some && p->num_pages > 0 && !p->cu_seqlens)
        return cuda_status(launch_paged_decode_simt(e4m3, p->D, make(p, T), q, qs, o, group, scale, window, sinks, workspace,
                                                    sm_count(), s));
    const kda_status e = clear(st, s);
    if (e != KDA_OK || !some) return e;
    if (p->num_pages == 0) return cuda_status(launch_paged_none(p->D * bytes_of(dtype), make(p, T), o, group, st, s));
    return cuda_status(launch_paged_simt(p->dtype, p->D, make(p, T), q, qs, o, group, scale, window, sinks,
                                         (float *)((uint8_t *)workspace + kHeaderBytes), sm_count(), st, s));
}

kda_status move(bool write, const kda_paged_cache *p, const void *k, const void *v, int64_t T, int32_t dtype, int64_t ks,
                int64_t vs, void *workspace, size_t workspace_bytes, void *stream) {
    const kda_status t = types_ok(p, dtype);
    if (t != KDA_OK) return t;
    if (!sizes_ok(p, T)) return KDA_ERR_INVALID_ARG;
    const int64_t row = (int64_t)p->Hk * p->D;
    if (!stride_ok(ks, T, row, dtype) || !stride_ok(vs, T, row, dtype)) return KDA_ERR_INVALID_ARG;
    if (workspace && (workspace_bytes < kHeaderBytes || !aligned(workspace, 256))) return KDA_ERR_INVALID_ARG;
    if (T > 0 && (!k || !v)) return KDA_ERR_INVALID_ARG;
    if (!aligned(k, 16) || !aligned(v, 16)) return KDA_ERR_INVALID_ARG;
    if (!write && T > 0 && (k == v || k == p->k_pages || k == p->v_pages || v == p->k_pages || v == p->v_pages))
        return KDA_ERR_INVALID_ARG;
    if (p->num_seqs > 0 && !cache_ok(p)) return KDA_ERR_INVALID_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    const kda_status e = clear((StatusWord *)workspace, s);
    if (e != KDA_OK || T == 0 || p->num_seqs == 0) return e;
    return cuda_status(launch_kv_cache(write, dtype, p->dtype, p->D, make(p, T), const_cast<void *>(k),
                                       const_cast<void *>(v), ks, vs, (StatusWord *)workspace, s));
}

}  // namespace

extern "C" {

kda_status kda_kv_cache_write(const kda_paged_cache *cache, const void *k, const void *v, int64_t total_tokens,
                              int32_t dtype, int64_t k_stride, int64_t v_stride, void *workspace,
                              size_t workspace_bytes, void *stream) {
    return move(true, cache, k, v, total_tokens, dtype, k_stride, v_stride, workspace, workspace_bytes, stream);
}

kda_status kda_kv_cache_read(const kda_paged_cache *cache, void *k, void *v, int64_t total_tokens, int32_t dtype,
                             void *workspace, size_t workspace_bytes, void *stream) {
    const int64_t row = cache ? (int64_t)cache->Hk * cache->D : 0;
    return move(false, cache, k, v, total_tokens, dtype, row, row, workspace, workspace_bytes, stream);
}

size_t kda_paged_attn_workspace_size(const kda_paged_cache *cache, int64_t total_tokens, int32_t H, int32_t dtype) {
    if (types_ok(cache, dtype) != KDA_OK || !attn_sizes_ok(cache, total_tokens, H)) return 0;
    return attn_bytes(cache, total_tokens, H, dtype);
}

kda_status kda_paged_attn_fwd(const kda_paged_cache *cache, const void *q, int64_t q_stride, void *o,
                              int64_t total_tokens, int32_t H, int32_t dtype, float scale, int32_t window,
                              int32_t sinks, void *workspace, size_t workspace_bytes, void *stream) {
    if (!cache || !cache->cu_seqlens) return KDA_ERR_INVALID_ARG;
    return attn(cache, q, q_stride, o, total_tokens, H, dtype, scale, window, sinks, workspace, workspace_bytes, stream);
}

kda_status kda_paged_attn_decode_step(const kda_paged_cache *cache, const void *q, int64_t q_stride, void *o, int32_t H,
                                      int32_t dtype, float scale, int32_t window, int32_t sinks, void *workspace,
                                      size_t workspace_bytes, void *stream) {
    if (!cache || cache->cu_seqlens) return KDA_ERR_INVALID_ARG;
    return attn(cache, q, q_stride, o, cache->num_seqs, H, dtype, scale, window, sinks, workspace, workspace_bytes, stream);
}

kda_status kda_test_paged_fault(int32_t part) {
    if (part < -1) return KDA_ERR_INVALID_ARG;
    g_left_out = part;
    return KDA_OK;
}

}  // extern "C"
