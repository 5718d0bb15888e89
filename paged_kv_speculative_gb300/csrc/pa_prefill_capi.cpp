// C ABI of the prompt-side operators: page operations, rotary cache writes,
// chunk attention. Arguments are checked before anything is enqueued; a
// refused call launches nothing.
#include <cmath>

#include "../../include/pa_verify.h"
#include "pa_prefill.h"

using namespace pav;

namespace {

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
template <typename... T>
int check_ints(const T*... p) {
  return (aligned(p, 4) && ...) ? PA_OK : report_error(PA_ERR_INVALID, "int32 arrays, scales and error_flags must be 4-byte aligned");
}

int ok() { return report_error(PA_OK, ""); }

int launched(cudaError_t e) {
  return e == cudaSuccess ? PA_OK : report_error(PA_ERR_CUDA, cudaGetErrorString(e));
}

int check_pages_desc(const pa_pages_desc* d) {
  if (!d) return report_error(PA_ERR_INVALID, "desc must not be NULL");
  if (d->num_seqs < 0 || d->block_table_stride < 1 || d->num_pages < 1)
    return report_error(PA_ERR_INVALID, "need num_seqs >= 0, block_table_stride >= 1 and num_pages >= 1");
  if (d->num_seqs > kMaxBatch) return report_error(PA_ERR_UNSUPPORTED, "num_seqs above 1024");
  // lengths are int32 tokens
  if (d->block_table_stride >= (1 << 27)) return report_error(PA_ERR_UNSUPPORTED, "block_table_stride must stay below 2^27");
  return PA_OK;
}

PagesDesc pages_desc(const pa_pages_desc* d) { return PagesDesc{d->num_seqs, d->block_table_stride, d->num_pages}; }

int check_workspace(const void* ws, size_t bytes, size_t need) {
  if (!ws) return report_error(PA_ERR_INVALID, "a required pointer is NULL");
  if (!aligned(ws, 256)) return report_error(PA_ERR_INVALID, "workspace must be 256-byte aligned");
  if (bytes < need) return report_error(PA_ERR_WORKSPACE, "workspace smaller than the call needs");
  return PA_OK;
}

// Checks shared by the chunk desc's two users; *sms gets the SM count when `query` is set.
int check_chunk_desc(const pa_chunk_desc* d, int* sms) {
  if (!d) return report_error(PA_ERR_INVALID, "desc must not be NULL");
  if (d->num_seqs < 0 || d->num_tokens < 0) return report_error(PA_ERR_INVALID, "num_seqs and num_tokens must be >= 0");
  if (d->num_seqs > kMaxBatch) return report_error(PA_ERR_UNSUPPORTED, "num_seqs above 1024");
  if (d->num_q_heads < 1 || d->num_kv_heads < 1 || d->num_q_heads % d->num_kv_heads != 0)
    return report_error(PA_ERR_INVALID, "need num_q_heads >= 1, num_kv_heads >= 1 and num_q_heads % num_kv_heads == 0");
  if (d->num_q_heads / d->num_kv_heads > kMaxRows) return report_error(PA_ERR_UNSUPPORTED, "num_q_heads / num_kv_heads above 128");
  if (d->page_size != kPage) return report_error(PA_ERR_UNSUPPORTED, "page_size must be 16");
  if (d->kv_dtype != PA_KV_BF16 && d->kv_dtype != PA_KV_FP8_E4M3) return report_error(PA_ERR_INVALID, "unknown kv_dtype");
  if (d->kv_dtype == PA_KV_FP8_E4M3) {
    if (d->head_dim != 128 && d->head_dim != 256) return report_error(PA_ERR_UNSUPPORTED, "FP8 KV needs head_dim 128 or 256");
  } else if (d->head_dim != 64 && d->head_dim != 128 && d->head_dim != 256) {
    return report_error(PA_ERR_UNSUPPORTED, "bf16 KV needs head_dim 64, 128 or 256");
  }
  if (d->num_pages < 1 || d->block_table_stride < 1)
    return report_error(PA_ERR_INVALID, "num_pages and block_table_stride must be >= 1");
  if (static_cast<int64_t>(d->num_pages) * d->num_kv_heads * kPage >= (int64_t(1) << 31))
    return report_error(PA_ERR_UNSUPPORTED, "num_pages * num_kv_heads * 16 must stay below 2^31");
  if (static_cast<int64_t>(d->num_tokens) * d->num_q_heads >= (int64_t(1) << 31))
    return report_error(PA_ERR_UNSUPPORTED, "num_tokens * num_q_heads must stay below 2^31");
  if (d->sm_count < 0) return report_error(PA_ERR_INVALID, "sm_count must be >= 0");
  const int64_t row = static_cast<int64_t>(d->num_q_heads) * d->head_dim;
  if (d->q_stride != 0 && (d->q_stride < row || d->q_stride % 8 != 0))
    return report_error(PA_ERR_INVALID, "q_stride must be 0 or a multiple of 8 of at least num_q_heads * head_dim");
  *sms = d->sm_count;
  if (*sms == 0) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return report_error(PA_ERR_CUDA, cudaGetErrorString(e));
  }
  return PA_OK;
}

}  // namespace

extern "C" {

int pa_pages_fork(const pa_pages_desc* desc, int32_t* block_table, int32_t* context_lens, int32_t* ref_counts,
                  const int32_t* parents, const int32_t* children, int32_t num_forks, uint32_t* error_flags,
                  pa_stream_t stream) {
  ok();
  if (int rc = check_pages_desc(desc)) return rc;
  if (num_forks < 0) return report_error(PA_ERR_INVALID, "num_forks must be >= 0");
  if (num_forks > kMaxBatch) return report_error(PA_ERR_UNSUPPORTED, "num_forks above 1024");
  if (num_forks == 0) return PA_OK;
  if (!block_table || !context_lens || !ref_counts || !parents || !children)
    return report_error(PA_ERR_INVALID, "a required pointer is NULL");
  if (int rc = check_ints(block_table, context_lens, ref_counts, parents, children, error_flags)) return rc;
  return launched(launch_pages_fork(pages_desc(desc), block_table, context_lens, ref_counts, parents, children, num_forks,
                                    error_flags, reinterpret_cast<cudaStream_t>(stream)));
}

size_t pa_pages_workspace_bytes(const pa_pages_desc* desc) {
  ok();
  return check_pages_desc(desc) ? 0 : pages_workspace_bytes(pages_desc(desc));
}

int pa_pages_resize(const pa_pages_desc* desc, int32_t* block_table, int32_t* context_lens, int32_t* ref_counts,
                    const int32_t* new_lens, int32_t* copy_src, int32_t* copy_dst, uint32_t* error_flags,
                    void* workspace, size_t workspace_bytes, pa_stream_t stream) {
  ok();
  if (int rc = check_pages_desc(desc)) return rc;
  if (desc->num_seqs == 0) return PA_OK;
  if (!block_table || !context_lens || !ref_counts || !new_lens || !copy_src || !copy_dst)
    return report_error(PA_ERR_INVALID, "a required pointer is NULL");
  if (int rc = check_ints(block_table, context_lens, ref_counts, new_lens, copy_src, copy_dst, error_flags)) return rc;
  const PagesDesc d = pages_desc(desc);
  if (int rc = check_workspace(workspace, workspace_bytes, pages_workspace_bytes(d))) return rc;
  return launched(launch_pages_resize(d, block_table, context_lens, ref_counts, new_lens, copy_src, copy_dst, error_flags,
                                      workspace, reinterpret_cast<cudaStream_t>(stream)));
}

int pa_pages_compact(const pa_pages_desc* desc, const int32_t* block_table, const int32_t* context_lens,
                     const int32_t* ref_counts, int32_t* block_table_out, int32_t* ref_counts_out, int32_t* copy_src,
                     int32_t* copy_dst, int32_t* num_moves, uint32_t* error_flags, void* workspace,
                     size_t workspace_bytes, pa_stream_t stream) {
  ok();
  if (int rc = check_pages_desc(desc)) return rc;
  const bool lists = desc->num_pages >= 2;  // with one page there is no move to list
  if ((desc->num_seqs > 0 && (!block_table || !context_lens || !block_table_out)) || !ref_counts || !ref_counts_out ||
      (lists && (!copy_src || !copy_dst)) || !num_moves)
    return report_error(PA_ERR_INVALID, "a required pointer is NULL");
  if (int rc = check_ints(block_table, context_lens, ref_counts, block_table_out, ref_counts_out, copy_src, copy_dst, num_moves, error_flags))
    return rc;
  const PagesDesc d = pages_desc(desc);
  if (int rc = check_workspace(workspace, workspace_bytes, pages_workspace_bytes(d))) return rc;
  return launched(launch_pages_compact(d, block_table, context_lens, ref_counts, block_table_out, ref_counts_out, copy_src,
                                       copy_dst, num_moves, error_flags, workspace, reinterpret_cast<cudaStream_t>(stream)));
}

int pa_pages_copy(const pa_pool_desc* desc, const int32_t* copy_src, const int32_t* copy_dst, int32_t max_pairs,
                  const int32_t* num_pairs, void* const* k_caches, void* const* v_caches, float* const* k_scales,
                  float* const* v_scales, uint32_t* error_flags, pa_stream_t stream) {
  ok();
  if (!desc) return report_error(PA_ERR_INVALID, "desc must not be NULL");
  const pa_pool_desc& d = *desc;
  if (d.num_pages < 1 || d.num_kv_heads < 1 || d.num_layers < 1 || max_pairs < 0)
    return report_error(PA_ERR_INVALID, "need num_pages >= 1, num_kv_heads >= 1, num_layers >= 1 and max_pairs >= 0");
  if (d.num_layers > kMaxCopyLayers) return report_error(PA_ERR_UNSUPPORTED, "num_layers above 64");
  if (d.kv_dtype != PA_KV_BF16 && d.kv_dtype != PA_KV_FP8_E4M3) return report_error(PA_ERR_INVALID, "unknown kv_dtype");
  if (d.head_dim != 64 && d.head_dim != 128 && d.head_dim != 256)
    return report_error(PA_ERR_UNSUPPORTED, "head_dim must be 64, 128 or 256");
  const bool fp8 = d.kv_dtype == PA_KV_FP8_E4M3;
  const int64_t page_units = static_cast<int64_t>(d.num_kv_heads) * d.head_dim * (fp8 ? 1 : 2);  // x 16 tokens / 16 bytes
  if (page_units >= (int64_t(1) << 30)) return report_error(PA_ERR_UNSUPPORTED, "pages too large");
  if (max_pairs == 0) return PA_OK;
  if (!copy_src || !copy_dst || !k_caches || !v_caches) return report_error(PA_ERR_INVALID, "a required pointer is NULL");
  if (fp8 && (!k_scales || !v_scales)) return report_error(PA_ERR_INVALID, "FP8 KV needs k_scales and v_scales");
  if (int rc = check_ints(copy_src, copy_dst, num_pairs, error_flags)) return rc;
  PoolCopy c{};
  for (int l = 0; l < d.num_layers; ++l) {
    c.data[2 * l] = k_caches[l];
    c.data[2 * l + 1] = v_caches[l];
    if (fp8) {
      c.scale[2 * l] = k_scales[l];
      c.scale[2 * l + 1] = v_scales[l];
    }
  }
  for (int w = 0; w < 2 * d.num_layers; ++w) {
    if (!c.data[w] || (fp8 && !c.scale[w])) return report_error(PA_ERR_INVALID, "a layer's pointer is NULL");
    if (!aligned(c.data[w], 16) || !aligned(c.scale[w], 16))
      return report_error(PA_ERR_INVALID, "caches and scales must be 16-byte aligned");
  }
  c.src = copy_src;
  c.dst = copy_dst;
  c.num_pairs = num_pairs;
  c.err = error_flags;
  c.max_pairs = max_pairs;
  c.num_pages = d.num_pages;
  c.layers = d.num_layers;
  c.page_units = static_cast<int32_t>(page_units);
  c.scale_units = fp8 ? d.num_kv_heads * kPage * 4 / 16 : 0;
  return launched(launch_pages_copy(c, reinterpret_cast<cudaStream_t>(stream)));
}

int pa_rope_write(const pa_rope_desc* desc, const void* q, const void* k, const void* v, const int32_t* positions,
                  const double* inv_freq, const int32_t* pair_axis, const int64_t* slot_mapping, void* q_out,
                  void* k_cache, void* v_cache, float* k_scale, float* v_scale, uint32_t* error_flags,
                  pa_stream_t stream) {
  ok();
  if (!desc) return report_error(PA_ERR_INVALID, "desc must not be NULL");
  const pa_rope_desc& d = *desc;
  if (d.num_tokens < 0 || d.num_q_heads < 1 || d.num_kv_heads < 1 || d.num_pages < 0)
    return report_error(PA_ERR_INVALID, "need num_tokens >= 0, num_q_heads >= 1, num_kv_heads >= 1 and num_pages >= 0");
  if (d.head_dim != 64 && d.head_dim != 128 && d.head_dim != 256)
    return report_error(PA_ERR_UNSUPPORTED, "head_dim must be 64, 128 or 256");
  if (d.rot_dim < 0 || d.rot_dim > d.head_dim || d.rot_dim % 16 != 0)
    return report_error(PA_ERR_INVALID, "rot_dim must be a multiple of 16 in 0 .. head_dim");
  if (d.num_axes < 1 || d.num_axes > 4) return report_error(PA_ERR_INVALID, "num_axes must lie in 1..4");
  if (d.pairs != PA_ROPE_HALVES && d.pairs != PA_ROPE_NEIGHBOURS) return report_error(PA_ERR_INVALID, "unknown pairs");
  if (d.kv_dtype != PA_KV_BF16 && d.kv_dtype != PA_KV_FP8_E4M3) return report_error(PA_ERR_INVALID, "unknown kv_dtype");
  const int64_t qrow = static_cast<int64_t>(d.num_q_heads) * d.head_dim, krow = static_cast<int64_t>(d.num_kv_heads) * d.head_dim;
  if (static_cast<int64_t>(d.num_tokens) * (d.num_q_heads + 2 * static_cast<int64_t>(d.num_kv_heads)) >= (int64_t(1) << 31))
    return report_error(PA_ERR_UNSUPPORTED, "too many tokens for one call");
  const int64_t strides[4] = {d.q_stride ? d.q_stride : qrow, d.k_stride ? d.k_stride : krow, d.v_stride ? d.v_stride : krow,
                              d.q_out_stride ? d.q_out_stride : qrow};
  for (int i = 0; i < 4; ++i)
    if (strides[i] % 8 != 0 || strides[i] < (i == 1 || i == 2 ? krow : qrow))
      return report_error(PA_ERR_INVALID, "strides must be 0 or multiples of 8 of at least a token's row");
  if (d.num_tokens == 0) return PA_OK;
  if (!q || !k || !v || !positions || !slot_mapping || !q_out || !k_cache || !v_cache || (d.rot_dim > 0 && (!inv_freq || !pair_axis)))
    return report_error(PA_ERR_INVALID, "a required pointer is NULL");
  const bool fp8 = d.kv_dtype == PA_KV_FP8_E4M3;
  if (fp8 && (!k_scale || !v_scale)) return report_error(PA_ERR_INVALID, "FP8 KV needs k_scale and v_scale");
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16))
    return report_error(PA_ERR_INVALID, "q, k, v, q_out and caches must be 16-byte aligned");
  if (!aligned(positions, 4) || !aligned(inv_freq, 8) || !aligned(pair_axis, 4) || !aligned(slot_mapping, 8))
    return report_error(PA_ERR_INVALID, "positions, inv_freq, pair_axis and slot_mapping must be aligned to their type");
  if (int rc = check_ints(k_scale, v_scale, error_flags)) return rc;
  if (q == q_out && strides[0] != strides[3]) return report_error(PA_ERR_INVALID, "q_out = q needs equal strides");
  RopeParams p{};
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.positions = positions;
  p.inv_freq = inv_freq;
  p.pair_axis = pair_axis;
  p.slots = slot_mapping;
  p.q_out = static_cast<uint16_t*>(q_out);
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.err = error_flags;
  p.q_stride = strides[0];
  p.k_stride = strides[1];
  p.v_stride = strides[2];
  p.q_out_stride = strides[3];
  p.num_tokens = d.num_tokens;
  p.num_q_heads = d.num_q_heads;
  p.num_kv_heads = d.num_kv_heads;
  p.rot_dim = d.rot_dim;
  p.num_axes = d.num_axes;
  p.neighbours = d.pairs == PA_ROPE_NEIGHBOURS;
  p.num_pages = d.num_pages;
  return launched(launch_rope_write(d.head_dim, fp8 ? 1 : 0, p, reinterpret_cast<cudaStream_t>(stream)));
}

size_t pa_chunk_workspace_bytes(const pa_chunk_desc* desc) {
  ok();
  int sms = 0;
  if (check_chunk_desc(desc, &sms)) return 0;
  return chunk_workspace_bytes(desc->head_dim, sms);
}

int pa_chunk_attention(const pa_chunk_desc* desc, const void* q, const void* k_cache, const void* v_cache,
                       const float* k_scale, const float* v_scale, const int32_t* block_table,
                       const int32_t* context_lens, const int32_t* query_lens, float softmax_scale, void* out,
                       void* workspace, size_t workspace_bytes, pa_stream_t stream) {
  ok();
  int sms = 0;
  if (int rc = check_chunk_desc(desc, &sms)) return rc;
  const pa_chunk_desc& d = *desc;
  if (d.num_seqs == 0 || d.num_tokens == 0) return PA_OK;
  const bool fp8 = d.kv_dtype == PA_KV_FP8_E4M3;
  if (!q || !k_cache || !v_cache || !block_table || !context_lens || !query_lens || !out)
    return report_error(PA_ERR_INVALID, "a required pointer is NULL");
  if (fp8 && (!k_scale || !v_scale)) return report_error(PA_ERR_INVALID, "FP8 KV needs k_scale and v_scale");
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16))
    return report_error(PA_ERR_INVALID, "q, k_cache, v_cache and out must be 16-byte aligned");
  if (fp8 && (!aligned(k_scale, 16) || !aligned(v_scale, 16)))
    return report_error(PA_ERR_INVALID, "k_scale and v_scale must be 16-byte aligned");
  if (!aligned(block_table, 4) || !aligned(context_lens, 4) || !aligned(query_lens, 4))
    return report_error(PA_ERR_INVALID, "int32 arrays must be 4-byte aligned");
  if (!(std::isfinite(softmax_scale) && softmax_scale > 0.f))
    return report_error(PA_ERR_INVALID, "softmax_scale must be finite and > 0");
  if (int rc = check_workspace(workspace, workspace_bytes, chunk_workspace_bytes(d.head_dim, sms))) return rc;
  ChunkParams p{};
  p.q = static_cast<const uint16_t*>(q);
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.block_table = block_table;
  p.ctx = context_lens;
  p.ql = query_lens;
  p.out = static_cast<uint16_t*>(out);
  p.ws = static_cast<uint8_t*>(workspace);
  p.q_stride = d.q_stride && d.num_tokens > 1 ? d.q_stride : static_cast<int64_t>(d.num_q_heads) * d.head_dim;  // one row has none
  p.scale = softmax_scale;
  p.num_seqs = d.num_seqs;
  p.num_tokens = d.num_tokens;
  p.num_q_heads = d.num_q_heads;
  p.num_kv_heads = d.num_kv_heads;
  p.num_pages = d.num_pages;
  p.bt_stride = d.block_table_stride;
  p.sms = sms;
  return launched(launch_chunk(d.head_dim, fp8 ? 1 : 0, p, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
