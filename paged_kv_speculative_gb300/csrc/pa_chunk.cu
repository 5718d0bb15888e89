// Launches of chunk attention: tensor maps, the kernel (one CTA an SM), the combine.
#include <cudaTypedefs.h>

#include "pa_chunk.cuh"

namespace pav {

namespace {

bool encode(CUtensorMap* map, uint32_t rank, const void* base, const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box) {
  auto enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encoder());
  const cuuint32_t ones[3] = {1, 1, 1};
  return enc && enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), dims, strides, box, ones,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }
size_t records_bytes(int sms) { return up256(static_cast<size_t>(sms) * sizeof(ChunkRecord)); }
// Rows of the partial slots: two slots a CTA.
size_t part_rows(int head_dim, int sms) { return static_cast<size_t>(sms) * 2 * (head_dim <= 128 ? 2 : 1) * 128; }

template <int FP8, int D>
cudaError_t launch(const ChunkParams& p, cudaStream_t stream) {
  using C = ChunkCfg<FP8, D>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = ensure_smem_attr(pa_chunk_kernel<FP8, D>, C::kSmem, done);
  if (e != cudaSuccess) return e;
  CUtensorMap k{}, v{}, q{};
  if constexpr (!FP8) {  // (8-bit caches and their queries are read by plain loads)
    const cuuint64_t kv_dims[2] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(p.num_pages) * p.num_kv_heads * kPage};
    const cuuint64_t kv_strides[1] = {static_cast<cuuint64_t>(C::kRowB)};
    const cuuint32_t kv_box[2] = {64, static_cast<cuuint32_t>(kPage)};
    const cuuint64_t q_dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(p.num_q_heads), static_cast<cuuint64_t>(p.num_tokens)};
    const cuuint64_t q_strides[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(p.q_stride) * 2};
    const cuuint32_t q_box[3] = {64, static_cast<cuuint32_t>(p.group), static_cast<cuuint32_t>(p.tq)};
    if (!encode(&k, 2, p.k_cache, kv_dims, kv_strides, kv_box) || !encode(&v, 2, p.v_cache, kv_dims, kv_strides, kv_box) ||
        !encode(&q, 3, p.q, q_dims, q_strides, q_box))
      return cudaErrorInvalidValue;
  }
  e = launch_chained(pa_chunk_kernel<FP8, D>, dim3(p.sms), dim3(C::kThreads), C::kSmem, stream, k, v, q, p);
  if (e != cudaSuccess) return e;
  // a row a warp
  return launch_chained(pa_chunk_combine_kernel<FP8, D>, dim3(p.sms, 128 * C::NT / (kChunkCombineThreads / 32)),
                        dim3(kChunkCombineThreads), 0, stream, p);
}

}  // namespace

size_t chunk_workspace_bytes(int head_dim, int sms) {
  const size_t rows = part_rows(head_dim, sms);
  return kWsHeader + records_bytes(sms) + rows * 4 + rows * head_dim * 4;
}

cudaError_t launch_chunk(int head_dim, int fp8, const ChunkParams& p_in, cudaStream_t stream) {
  ChunkParams p = p_in;
  p.part_lse = reinterpret_cast<float*>(p.ws + kWsHeader + records_bytes(p.sms));
  p.part_o = p.part_lse + part_rows(head_dim, p.sms);
  p.group = p.num_q_heads / p.num_kv_heads;
  p.tq = 128 / p.group;
  if (fp8) return head_dim == 128 ? launch<1, 128>(p, stream) : launch<1, 256>(p, stream);
  return head_dim == 64 ? launch<0, 64>(p, stream) : head_dim == 128 ? launch<0, 128>(p, stream) : launch<0, 256>(p, stream);
}

}  // namespace pav
