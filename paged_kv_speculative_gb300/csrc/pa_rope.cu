// Rotary positions with several axes, fused with the paged KV write.
//
// Pair p of token t turns by angle = pos[axis_p][t] * w_p. In turns, with f_p = w_p / 2 pi as a 64-bit fixed-point
// fraction F_p = round(f_p 2^64), the angle modulo one turn is the low 64 bits of pos * F_p: the reduction is exact for
// every int32 position (also negative ones: two's complement wraps the same way). What remains is f_p's own rounding, twice
// (1 / 2 pi and the product): |pos w_p| 2^-52 radians, 2^-21 at position 2^31 and w_p = 1. The reduced angle in fp32, in
// [-pi, pi), is off by three roundings, up to 3 pi 2^-24; its sine and cosine are the approximate ones, documented to 2^-21.19
// there. Together within 2^-19: the outputs keep 8 bits, or 4, and the accurate forms took 40 instructions a pair.
//
// Memory bound: every q, k, v entry is read and written once. A thread owns 8 pairs of a head (16 entries, two 16-byte
// accesses), so D / 16 threads cover a head and a warp several heads at once, kBatch such groups of heads with all their loads
// in flight. A block takes the table F_p into shared memory once (double precision is slow here).
#include <cuda_runtime.h>
#include <stdint.h>

#include "pa_device.cuh"
#include "pa_prefill.h"

namespace pav {

namespace {

__device__ __forceinline__ void unpack8(uint4 w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[2 * e] = bf16_lo(u[e]);
    x[2 * e + 1] = bf16_hi(u[e]);
  }
}
__device__ __forceinline__ void store8(uint16_t* dst, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(dst) =
      make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(hi) : "f"(d), "f"(c));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

// (a, b): the thread's two 8-entry units of a head; turned in place.
__device__ __forceinline__ void turn(float (&a)[8], float (&b)[8], const float (&c)[8], const float (&s)[8], bool neighbours) {
  if (neighbours) {  // pairs (2i, 2i + 1) of the 16 consecutive entries a, b
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = a[2 * i], y = a[2 * i + 1], z = b[2 * i], w = b[2 * i + 1];
      a[2 * i] = x * c[i] - y * s[i];
      a[2 * i + 1] = x * s[i] + y * c[i];
      b[2 * i] = z * c[4 + i] - w * s[4 + i];
      b[2 * i + 1] = z * s[4 + i] + w * c[4 + i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = a[i], y = b[i];
      a[i] = x * c[i] - y * s[i];
      b[i] = x * s[i] + y * c[i];
    }
  }
}

// Eight warps a block, four groups an item, two blocks an SM (GB300's 152): 8192 tokens of 32/4 heads of 128 (168 MB) in 32.5 us, where a
// plain copy of as many bytes takes 32.8. When it took 35.6: 2 groups an item 41.0, 3 37.8; three blocks an SM with 2 groups 49.3.
constexpr int kRopeWarps = 8;
constexpr int kRopeBatch = 4;
constexpr int kRopeGrid = 2 * 152;

template <int D, bool FP8, int kBatch>
__global__ void __launch_bounds__(32 * kRopeWarps) pa_rope_write_kernel(const RopeParams p, int parts) {
  chained_start();
  constexpr int kTph = D / 16;        // threads of a head
  constexpr int kHeads = 32 / kTph;   // heads a warp covers at once: a group
  __shared__ uint64_t s_freq[D / 2];  // 64-bit turns per position
  __shared__ int s_axis[D / 2];       // -1: no such axis
  __shared__ __align__(16) float2 s_turn[kRopeWarps][D / 2];  // a token's (cos, sin), one warp's
  const int half = p.rot_dim / 2;
  const int lane = threadIdx.x & 31, j = lane % kTph;
  float2* turn_of = s_turn[threadIdx.x >> 5];
  const bool turns = j < half / 8;
  // entry offsets of the thread's two units
  const int ua = p.neighbours || !turns ? 16 * j : 8 * j;
  const int ub = p.neighbours || !turns ? ua + 8 : ua + half;
  const int heads = p.num_q_heads + 2 * p.num_kv_heads;
  const int groups = (heads + kHeads - 1) / kHeads;
  // items (token, part of its groups), dealt to the warps in turn; this warp's first, and the step to its next
  const uint32_t warps = gridDim.x * kRopeWarps, first = blockIdx.x * kRopeWarps + (threadIdx.x >> 5);
  const int step_t = static_cast<int>(warps / parts), step_part = static_cast<int>(warps % parts);
  int t = static_cast<int>(first / parts), part = static_cast<int>(first % parts);

  struct Item {
    int64_t slot;
    uint4 a[kBatch], b[kBatch];
  };
  auto load = [&](int t, int part, Item& x) {
    x.slot = -1;
    if (t >= p.num_tokens) return;
    x.slot = p.slots[t];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int g = part * kBatch + k, h = g * kHeads + lane / kTph;
      x.a[k] = x.b[k] = make_uint4(0, 0, 0, 0);
      if (h < heads) {
        const int hk = h - p.num_q_heads, hv = hk - p.num_kv_heads;
        const uint16_t* src = hk < 0   ? p.q + t * p.q_stride + static_cast<int64_t>(h) * D
                              : hv < 0 ? p.k + t * p.k_stride + static_cast<int64_t>(hk) * D
                                       : p.v + t * p.v_stride + static_cast<int64_t>(hv) * D;
        x.a[k] = *reinterpret_cast<const uint4*>(src + ua);
        x.b[k] = *reinterpret_cast<const uint4*>(src + ub);
      }
    }
  };
  Item cur, next;
  load(t, part, cur);  // on its way while the table is made
  for (int i = threadIdx.x; i < half; i += blockDim.x) {
    const double turns_per_pos = p.inv_freq[i] * 0.15915494309189533577;                                    // 1 / (2 pi)
    s_freq[i] = static_cast<uint64_t>(__double2ll_rn(turns_per_pos * 9223372036854775808.0)) << 1;  // 2^63, then 2^64
    const int axis = p.pair_axis[i];
    s_axis[i] = axis >= 0 && axis < p.num_axes ? axis : -1;
    if (s_axis[i] < 0 && blockIdx.x == 0 && p.err) atomicOr(p.err, kErrLengths);
  }
  __syncthreads();
  for (int nt, npart; t < p.num_tokens; t = nt, part = npart, cur = next) {
    nt = t + step_t;
    npart = part + step_part;
    if (npart >= parts) {
      npart -= parts;
      ++nt;
    }
    load(nt, npart, next);
    const int64_t slot = cur.slot;
    if (slot < 0) continue;
    const bool stored = slot < static_cast<int64_t>(p.num_pages) * kPage;
    if (!stored && part == 0 && lane == 0 && p.err) atomicOr(p.err, kErrPageRange);
    // the token's angles, a few pairs a lane
    __syncwarp();
#pragma unroll
    for (int i0 = 0; i0 < D / 2; i0 += 32) {
      const int i = i0 + lane;
      if (i < half) {
        const int axis = s_axis[i];
        const int64_t pos = axis < 0 ? 0 : p.positions[static_cast<int64_t>(axis) * p.num_tokens + t];
        const uint64_t a = static_cast<uint64_t>(pos) * s_freq[i];
        // the top 32 bits as a signed fraction: [-1, 1) half turns, in radians
        const float x = static_cast<float>(static_cast<int32_t>(static_cast<uint32_t>(a >> 32))) * (4.656612873077393e-10f * 3.14159265358979f);
        turn_of[i] = make_float2(__cosf(x), __sinf(x));
      }
    }
    __syncwarp();
    float cs[8], sn[8];
    if (turns) {
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const float4 x = *reinterpret_cast<const float4*>(turn_of + 8 * j + i);
        cs[i] = x.x;
        sn[i] = x.y;
        cs[i + 1] = x.z;
        sn[i + 1] = x.w;
      }
    }
    const size_t page = static_cast<size_t>(slot >> 4);
    const int off = static_cast<int>(slot & 15);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int g = part * kBatch + k, h = g * kHeads + lane / kTph;
      if (g >= groups) break;  // of the last part
      const bool on = h < heads;
      const int hk = h - p.num_q_heads, hv = hk - p.num_kv_heads;
      float a[8], b[8];
      unpack8(cur.a[k], a);
      unpack8(cur.b[k], b);
      if (turns && hv < 0) turn(a, b, cs, sn, p.neighbours);
      if (on && hk < 0) {
        uint16_t* dst = p.q_out + t * p.q_out_stride + static_cast<int64_t>(h) * D;
        store8(dst + ua, a);
        store8(dst + ub, b);
      }
      if ((g + 1) * kHeads <= p.num_q_heads) continue;  // q heads only
      const size_t row = (page * p.num_kv_heads + (hv < 0 ? hk : hv)) * kPage + off;
      if (FP8) {
        // largest magnitude of the head, over its kTph threads (every lane takes part)
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, fmaxf(fabsf(a[i]), fabsf(b[i])));
#pragma unroll
        for (int w = kTph / 2; w >= 1; w >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, w));
        if (on && hk >= 0 && stored) {
          const float s = m > 0.f ? __fdiv_rn(m, 448.f) : 1.f;
          uint8_t* dst = static_cast<uint8_t*>(hv < 0 ? p.k_cache : p.v_cache) + row * D;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            a[i] = __fdiv_rn(a[i], s);
            b[i] = __fdiv_rn(b[i], s);
          }
          *reinterpret_cast<uint2*>(dst + ua) = make_uint2(e4m3x4(a[0], a[1], a[2], a[3]), e4m3x4(a[4], a[5], a[6], a[7]));
          *reinterpret_cast<uint2*>(dst + ub) = make_uint2(e4m3x4(b[0], b[1], b[2], b[3]), e4m3x4(b[4], b[5], b[6], b[7]));
          if (j == 0) (hv < 0 ? p.k_scale : p.v_scale)[row] = s;
        }
      } else if (on && hk >= 0 && stored) {
        uint16_t* dst = static_cast<uint16_t*>(hv < 0 ? p.k_cache : p.v_cache) + row * D;
        store8(dst + ua, a);
        store8(dst + ub, b);
      }
    }
  }
}

template <int D, bool FP8, int kBatch>
cudaError_t launch(const RopeParams& p, cudaStream_t stream) {
  constexpr int kHeads = 32 / (D / 16);
  const int groups = (p.num_q_heads + 2 * p.num_kv_heads + kHeads - 1) / kHeads, parts = (groups + kBatch - 1) / kBatch;
  const int64_t blocks = (static_cast<int64_t>(p.num_tokens) * parts + kRopeWarps - 1) / kRopeWarps;
  const int grid = static_cast<int>(blocks < kRopeGrid ? blocks : kRopeGrid);
  return launch_chained(pa_rope_write_kernel<D, FP8, kBatch>, grid, 32 * kRopeWarps, 0, stream, p, parts);
}

template <int D, bool FP8>
cudaError_t launch_any(const RopeParams& p, cudaStream_t stream) {
  // While each group of heads of each token can have a warp of its own, it has: they spread over the SMs. Beyond, four share a token's
  // angles and have their loads in flight at once. us, one and four groups an item, bf16, 128: 32/4 heads, 64 tokens (640 groups) 2.95
  // and 3.19, 192 (1920) 3.34 and 3.56, 256 (2560) 4.20 and 3.75, 1024 8.6 and 6.1; 8/2 heads, 768 (2304) 3.44 and 3.63, 1024
  // 4.4 and 3.7; 64/8 heads, 128 (2560) 4.2 and 3.8; heads of 256, FP8, 192 (1920) 4.35 and 4.88, 256 (2560) 5.3 and 5.0.
  constexpr int kHeads = 32 / (D / 16);
  const int64_t groups = (p.num_q_heads + 2 * p.num_kv_heads + kHeads - 1) / kHeads;
  return p.num_tokens * groups <= kRopeGrid * kRopeWarps ? launch<D, FP8, 1>(p, stream) : launch<D, FP8, kRopeBatch>(p, stream);
}

}  // namespace

cudaError_t launch_rope_write(int head_dim, int fp8, const RopeParams& p, cudaStream_t stream) {
  if (head_dim == 64) return fp8 ? launch_any<64, true>(p, stream) : launch_any<64, false>(p, stream);
  if (head_dim == 128) return fp8 ? launch_any<128, true>(p, stream) : launch_any<128, false>(p, stream);
  if (head_dim == 256) return fp8 ? launch_any<256, true>(p, stream) : launch_any<256, false>(p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace pav
