// Internal declarations of the prompt-side operators: page operations, rotary
// cache writes, chunk attention.
#pragma once

#include "pa_internal.h"

namespace pav {

// Bits of the device error word (the header's PA_DEVERR_*).
constexpr uint32_t kErrPageRange = 1u, kErrLengths = 2u, kErrTimeout = 4u, kErrNoPages = 8u, kErrRefs = 16u;

// These kernels are short and follow one another, so each may be brought up while the one before it in the stream ends
// (programmatic dependent launch): it lets its own follower come (chained_start) once all its blocks run, and touches
// memory only when the kernel before it, and by the same rule all before that, have ended (the wait). Every thread passes it.
template <typename... Params, typename... Args>
inline cudaError_t launch_chained(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, Params(args)...);
}
#ifdef __CUDACC__
__device__ __forceinline__ void chained_let_follow() { asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory"); }
__device__ __forceinline__ void chained_wait() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }
__device__ __forceinline__ void chained_start() {
  chained_let_follow();
  chained_wait();
}
#endif

struct PagesDesc {
  int32_t num_seqs, stride, num_pages;
};

constexpr int kMaxCopyLayers = 64;  // layers of one pages_copy call (their pointers travel in the kernel parameters)

struct PoolCopy {
  const int32_t* src;
  const int32_t* dst;
  const int32_t* num_pairs;  // device, or null: max_pairs
  uint32_t* err;
  int32_t max_pairs, num_pages, layers;
  int32_t page_units, scale_units;  // 16-byte units of a page's K (or V) and of its scales (0: none)
  void* data[2 * kMaxCopyLayers];   // K of layer 0, V of layer 0, K of layer 1, ...
  float* scale[2 * kMaxCopyLayers];
};

size_t pages_workspace_bytes(const PagesDesc& d);
cudaError_t launch_pages_fork(const PagesDesc& d, int32_t* table, int32_t* lens, int32_t* ref, const int32_t* parents,
                              const int32_t* children, int n, uint32_t* err, cudaStream_t stream);
cudaError_t launch_pages_resize(const PagesDesc& d, int32_t* table, int32_t* lens, int32_t* ref, const int32_t* new_lens,
                                int32_t* copy_src, int32_t* copy_dst, uint32_t* err, void* ws, cudaStream_t stream);
cudaError_t launch_pages_compact(const PagesDesc& d, const int32_t* table, const int32_t* lens, const int32_t* ref,
                                 int32_t* table_out, int32_t* ref_out, int32_t* copy_src, int32_t* copy_dst,
                                 int32_t* num_moves, uint32_t* err, void* ws, cudaStream_t stream);
cudaError_t launch_pages_copy(const PoolCopy& c, cudaStream_t stream);

struct RopeParams {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  const int32_t* positions;  // [axes, tokens]
  const double* inv_freq;
  const int32_t* pair_axis;
  const int64_t* slots;
  uint16_t* q_out;
  void* k_cache;
  void* v_cache;
  float* k_scale;
  float* v_scale;
  uint32_t* err;
  int64_t q_stride, k_stride, v_stride, q_out_stride;
  int32_t num_tokens, num_q_heads, num_kv_heads, rot_dim, num_axes, neighbours, num_pages;
};
cudaError_t launch_rope_write(int head_dim, int fp8, const RopeParams& p, cudaStream_t stream);

struct ChunkParams {
  const uint16_t* q;
  const void* k_cache;
  const void* v_cache;
  const float* k_scale;
  const float* v_scale;
  const int32_t* block_table;
  const int32_t* ctx;
  const int32_t* ql;
  uint16_t* out;
  uint8_t* ws;       // error word, records, partials
  float* part_o;
  float* part_lse;
  int64_t q_stride;
  float scale;
  int32_t num_seqs, num_tokens, num_q_heads, num_kv_heads, num_pages, bt_stride, sms;
  int32_t group, tq;  // q heads of a KV head; tokens of a 128-row tile, floor(128 / group)
};
size_t chunk_workspace_bytes(int head_dim, int sms);
cudaError_t launch_chunk(int head_dim, int fp8, const ChunkParams& p, cudaStream_t stream);

}  // namespace pav
