// Chunk attention over the paged cache on 5th-generation tensor cores.
//
// Work. A unit is (sequence, KV head, block of query rows): its rows are the (token, head of the group) pairs of NT x TQ
// consecutive tokens, TQ = floor(128 / G), packed token-major so that a K/V tile read once serves the whole GQA group.
// NT = 2 row tiles of 128 at head_dim 64 and 128; one at 256, whose output fills the tensor memory. A unit walks the keys
// it can see, 0 .. E - 1, in tiles of kTok tokens. Units laid end to end (sequence, head, block) form one line whose
// length counts visible keys plus a fixed cost per unit, and CTA c works the piece [W c / n, W (c + 1) / n) of it, rounded
// to tiles. Long contexts with few rows are thereby split over all SMs and prompts are balanced whatever their lengths;
// a CTA has at most two units that it shares with others. Those leave normalised fp32 partials and log2-sum-exps in the
// workspace, which pa_chunk_combine_kernel joins in the order of the CTAs (no atomics: the same bits every time). Every CTA
// derives its piece from the device lengths by itself (prefix sums over the sequences, then a search in closed form), so
// there is no plan, no launch for one, and a captured graph serves every batch that fits.
//
// Roles. Warps 0-3 feed: bf16 K and V pages come through the block table by 2-D TMA boxes (16 tokens x 128 bytes, one lane a
// box; warps 0 and 2) into a ring of tile slots, K_0 V_0 K_1 V_1 ..., and the unit's query rows by TMA (warp 3); warp 1 issues the
// MMAs. Then NH = 2 warpgroups of softmax for each row tile, two threads a row, each with half of a tile's columns:
//   S = Q K^T   A = Q (shared memory), B = K, accumulator S in tensor memory
//   O += P V    A = P (tensor memory, in the columns of the S it came from), B = V, accumulator O
// With two row tiles the order PV_0(i) S_0(i+1) PV_1(i) S_1(i+1) gives each softmax the other tile's MMAs to hide behind; with
// one tile, S alternates between two buffers: S(i+1) PV(i).
//
// Softmax. A row keeps a reference M and P = 2^(y - M), y the score in log2 units. M rises only when a score passes it by
// more than 8 (2^8 in P), so O is rescaled rarely, and the two threads of a row need only a vote per tile (they meet in shared
// memory when one of them wants M raised); O / l is the same whatever M was. Sums stay fp32; P is rounded to bf16 (the output's
// type; l sums the unrounded values).
// FP8. The tiles are widened to 16 bits on their way into the ring, once for all rows of the unit, by the softmax warps in the time
// they wait for their next scores: one page of K or V a warp and tile, read from global memory (which warp 0, a few tiles
// ahead, brings into L2), codes times scale, written in the layout of the bf16 tiles; everything behind is the bf16 path. K and Q are
// f16: 11 bits (a key's entry is off by 2^-11 of itself at most, where E4M3 left 2^-4), so a K tile is scaled by 2^(4 - e), 2^e just
// above its largest scale, which its scores are multiplied back by, and a row of Q by the power of two that puts its largest entry in
// [1, 2): bf16's 8 bits then stay down to 2^-17 of that power, below it entries count in steps of 2^-24.
// P and V are bf16, as there: P has to reach as far down as l does. In f16 a weight below 2^-25 of the reference is 0, and behind one
// key that stands 17.4 nats above the others their whole part of the output goes (the cost: single tokens 159.5 to 167 us,
// 512 tokens over 16384, 8/1 heads of 256, 110 to 114, 1024 over 8192 170.5 either way). V counts in 2^30, so that scales of
// up to 1e30 sum in fp32 and those down to 2^-87 keep every code.
// Measured, us, calls back to back: 1024 tokens over 8192, 32/4 heads of 128: bf16 115, 8 bits 170.5; 512 over 16384, 8/1 heads of 256, 8
// bits 114; 1024 over 8192, 32/4 heads of 64: 101.5. Single tokens, 32 sequences of 8192 keys: bf16 107.6 (537 MB; the verify kernel
// 95), 8 bits 167 (the verify kernel 75: it widens nothing). With L2 emptied before each call 121.5, 176, 119, 107, 118 and 172.
// Tried for 8 bits and slower when the first of these took 177, L2 emptied: V alone widened, by two warps of their own, 204; six
// warps of their own for both 181 to 185; the second softmax group taking every other key tile of single tokens 175 for 169 (and
// prompts lost 10 % to the registers that it took). 8 bits throughout, P in two E4M3 terms, took 297 with one thread a row, when bf16
// took 158: scales at every score are 160 16-byte shared loads a warp and tile.
#pragma once

#include "pa_device.cuh"
#include "pa_prefill.h"
#include "pa_tc.cuh"

namespace pav {

// The MMA warp issues as one: every lane computes the (uniform) operands and waits, and `go`, set on one elected lane, guards
// the instruction. The operands of tcgen05.mma are uniform registers; from a branch that one lane takes alone, each of them
// is moved there for every MMA, which cost 90 clocks an MMA where the tensor cores need 64.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r;
}
__device__ __forceinline__ void mma_f16_ss(uint32_t go, uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(id), "r"(acc), "r"(go)
      : "memory");
}
// O += P V with P in tensor memory: `a` is a tensor-memory address.
__device__ __forceinline__ void mma_f16_ts(uint32_t go, uint32_t d_tmem, uint32_t a, uint64_t b, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a), "l"(b), "r"(id), "r"(acc), "r"(go)
      : "memory");
}
__device__ __forceinline__ void commit_if(uint32_t go, uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(smem_addr(bar)),
      "r"(go)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}
__device__ __forceinline__ void mbar_arrive_one(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void named_sync(int id, int nthreads) {
  asm volatile("bar.sync %0, %1;\n" ::"r"(id), "r"(nthreads) : "memory");
}
// OR of `pred` over the `nthreads` threads of named barrier `id`.
__device__ __forceinline__ bool named_or(int id, int nthreads, bool pred) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred pi, po;\n setp.ne.u32 pi, %3, 0;\n barrier.red.or.pred po, %1, %2, pi;\n selp.u32 %0, 1, 0, po;\n}\n"
      : "=r"(r)
      : "r"(id), "r"(nthreads), "r"(static_cast<uint32_t>(pred))
      : "memory");
  return r != 0;
}
// Four E4M3 codes to two f16 pairs; exact.
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t x, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, h;\n}\n" : "=r"(lo), "=r"(hi) : "r"(x));
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t fma_f16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;\n" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
__device__ __forceinline__ float2 f16x2_to_f32x2(uint32_t x) {
  float2 f;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.f32.f16 %0, l;\n cvt.f32.f16 %1, h;\n}\n" : "=f"(f.x), "=f"(f.y) : "r"(x));
  return f;
}
// Maximum of v over the 32 lanes of the warp (NaN never wins).
__device__ __forceinline__ float chunk_warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;\n" : "=f"(r) : "f"(v));
  return r;
}
// 32 consecutive 32-bit columns of this thread's tensor-memory lane.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,"
      "%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

// ---------------------------------------------------------------- geometry
template <int FP8, int D>
struct ChunkCfg {
  static constexpr int NT = D <= 128 ? 2 : 1;             // row tiles of a unit
  static constexpr int NS = D <= 128 ? 1 : 2;             // S buffers of a row tile
  static constexpr int NH = 2;                            // threads a row
  static constexpr int kTok = D == 256 ? 64 : 128;        // tokens of a K/V tile (at 256: 64, so that slots stay 32 KB)
  static constexpr int kCols = kTok / NH;                 // columns of a softmax thread
  static constexpr int kRowB = 2 * D;                     // bytes of a token's row in the ring
  static constexpr int kPlanes = kRowB / 128;             // 128-byte planes of a tile
  static constexpr int kPlane = kTok * 128;
  static constexpr int kStage = kTok * kRowB;
  static constexpr int kPages = kTok / kPage;
  static constexpr int kBoxes = kPages * kPlanes;         // TMA boxes of a tile (one lane each)
  static constexpr int kQPlanes = D / 64;                 // 16 KB planes of a Q tile
  static constexpr int kQTile = kQPlanes * 16384;
  static constexpr int kTileSlots = FP8 ? 8 : 0;          // tiles that warp 0 describes ahead
  static constexpr int kWarps = 4 * NT * NH;              // softmax warps
  static constexpr int kAhead = FP8 ? kWarps / 2 : 0;     // of them, those that widen K (the others widen V): one page each
  static constexpr int kLimit = 227 * 1024 - 1024 - 1024 - NT * NH * 128 * 8 - kTileSlots * 64;  // alignment slack, barriers, exchange
  static constexpr int kFit = (kLimit - NT * kQTile) / kStage;
  static constexpr int kSlots = FP8 ? 4 : kFit < 10 ? kFit : 10;
  static constexpr int kOffKV = 0;
  static constexpr int kOffQ = kSlots * kStage;
  static constexpr int kOffTile = kOffQ + NT * kQTile;
  static constexpr int kOffEx = kOffTile + kTileSlots * 64;  // [NT][max, sum][NH][128] floats: the two threads of a row meet here
  static constexpr int kOffBar = kOffEx + NT * NH * 128 * 8;
  static constexpr int kSmem = kOffBar + 1024 + 1024;
  static constexpr int kThreads = 128 * (1 + NT * NH);
  static_assert(kBoxes <= 32, "one box a lane");
  static_assert(!FP8 || kAhead == kPages, "one page a widening warp");
  static_assert(kSlots >= 4 && kSlots <= kFit, "a V slot's previous tile is consumed when the softmax looks at it");
  static_assert(kSlots * kStage >= kMaxBatch * 20 + 64, "the set-up's tables fit the ring");
  static_assert((2 * kSlots + 2 * kTileSlots + 12) * 8 + 112 + 28 * kWarps <= 1024, "barriers and walks fit");
};

// FP8: what the widening warps and the softmax know of a tile.
struct __align__(16) ChunkTile {
  int page[8];        // page x KV heads + head; -1: none (zeros)
  int keys;           // tokens of the tile that exist; -1: there is no such tile
  float k_up;         // 2^(4 - e) of K
  float k_factor;     // 2^(e - 4): what its scores count in
  int pad[5];
};
constexpr float kChunkVUnit = 1073741824.f;  // FP8: what V, and with it O, counts in (2^30)

// Line length of a unit: its visible keys plus this many tokens for its start and end (three tiles; 32 ragged sequences 71.3 us,
// with two 72.8, four 72.9; 64 prompts of 300 tokens 137.4, 142.9, 137.3).
constexpr int kChunkUnitCost = 384;
// A CTA gets at least this much of the line: below it, splitting costs more than it saves (us with 128, 256, 384, 512, 1024: two
// sequences of 1500 keys, 40 tokens each, 22.7, 22.2, 22.9, 24.0, 29.4; four decode tokens over 3000 17.2, 17.2, 17.1, 18.0, 23.5; two
// short sequences 10.3, 10.3, 10.2, 12.5, 12.5).
constexpr int kChunkMinPiece = 256;

struct ChunkPos {  // a place on the line: tile t of unit (b, g, j); b = num_seqs: the end
  int b, g, j, t;
};
__device__ __forceinline__ bool same_unit(const ChunkPos& x, const ChunkPos& y) { return x.b == y.b && x.g == y.g && x.j == y.j; }

// What a CTA did with units that it shares with others (8 ints in the workspace): its first unit if that began in an
// earlier CTA (head: 1 it goes on after this CTA, 2 it ends here; partial slot 2 c), its last if it begins here and does not
// end here (tail = 1; partial slot 2 c + 1; first token row, tokens, KV head).
struct ChunkRecord {
  int head, tail, tok0, ntok, g, pad[3];
};

// A sequence of the batch as the units see it.
struct ChunkSeq {
  int ctx, q, off;  // off: first token row
};
constexpr int kChunkMaxContext = 1 << 30;
// Rows are packed by max(query_lens, 0); past num_tokens the sum stays at num_tokens + 1, so no garbage length wraps it.
__device__ __forceinline__ int chunk_off_after(const ChunkParams& p, int off, int q) {
  return static_cast<int>(min(static_cast<long long>(off) + max(q, 0), static_cast<long long>(p.num_tokens) + 1));
}
__device__ __forceinline__ bool chunk_live(const ChunkParams& p, const ChunkSeq& s) {
  return s.q > 0 && s.ctx >= s.q && s.ctx <= kChunkMaxContext && s.ctx <= static_cast<long long>(p.bt_stride) * kPage &&
         s.off + static_cast<long long>(s.q) <= p.num_tokens;
}

// One role's walk over its CTA's units.
template <int NT, int TOK>
struct ChunkWalk {
  const ChunkParams& p;
  const ChunkPos& end;  // in shared memory
  ChunkPos& at;         // the softmax warps' place stands in shared memory too: registers are scarce there
  ChunkSeq& s;
  __device__ __forceinline__ ChunkWalk(const ChunkParams& p_, const ChunkPos* cuts, const ChunkSeq* seqs, ChunkPos& a, ChunkSeq& q,
                                       bool mine = true)
      : p(p_), end(cuts[1]), at(a), s(q) {
    if (mine) {
      at = cuts[0];
      s = seqs[0];
      if (!done() && at.t >= tiles()) next();  // the cut fell on the unit's end
    }
  }
  __device__ __forceinline__ int R() const { return NT * p.tq; }  // tokens of a unit
  __device__ __forceinline__ bool done() const { return at.b >= p.num_seqs || (same_unit(at, end) && at.t >= end.t); }
  __device__ __forceinline__ int ntok() const { return min(R(), s.q - at.j * R()); }          // tokens of the unit
  __device__ __forceinline__ int tok0() const { return s.off + at.j * R(); }                // its first token row
  __device__ __forceinline__ int first_key() const { return s.ctx - s.q + at.j * R(); }     // last key its first token sees
  __device__ __forceinline__ int keys() const { return first_key() + ntok(); }            // E: keys its last token sees
  __device__ __forceinline__ int tiles() const { return (keys() + TOK - 1) / TOK; }
  __device__ __forceinline__ int t1() const { return same_unit(at, end) ? end.t : tiles(); }  // this CTA's tiles are [at.t, t1)
  __device__ __forceinline__ void next() {
    at.t = 0;
    if (same_unit(at, end)) {  // the range ended inside this unit
      at = end;
      return;
    }
    if (++at.j * R() < s.q) return;
    at.j = 0;
    if (++at.g < p.num_kv_heads) return;
    at.g = 0;
    while (true) {
      s.off = chunk_off_after(p, s.off, s.q);
      if (++at.b >= p.num_seqs) return;
      s.ctx = __ldg(p.ctx + at.b);
      s.q = __ldg(p.ql + at.b);
      if (chunk_live(p, s)) return;
    }
  }
};

// Line length of one head's units of a sequence: blocks j < J of min(R, q - j R) tokens, each seeing P + its last token keys.
__device__ __forceinline__ long long chunk_blocks_length(int ctx, int q, int R, int J) {  // J <= ceil(q / R)
  const long long P = ctx - q;
  const long long full = static_cast<long long>(J) * (P + kChunkUnitCost) + static_cast<long long>(R) * J * (J + 1) / 2;
  const long long over = static_cast<long long>(J) * R - q;  // the last block of the chunk is shorter
  return over > 0 ? full - over : full;
}

// ---------------------------------------------------------------- kernel
template <int FP8, int D>
__global__ void __launch_bounds__(ChunkCfg<FP8, D>::kThreads, 1)
    pa_chunk_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                    const __grid_constant__ CUtensorMap tmq, const __grid_constant__ ChunkParams p) {
  using C = ChunkCfg<FP8, D>;
  using Walk = ChunkWalk<C::NT, C::kTok>;
  constexpr int NT = C::NT, NS = C::NS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* kvfull = reinterpret_cast<uint64_t*>(sm + C::kOffBar);
  uint64_t* kvempty = kvfull + C::kSlots;
  uint64_t* tfull = kvempty + C::kSlots;     // [kTileSlots]
  uint64_t* tempty = tfull + C::kTileSlots;
  uint64_t* qfull = tempty + C::kTileSlots;  // [NT]
  uint64_t* qfree = qfull + 2;               // bf16: the unit's last S is done
  uint64_t* sfull = qfree + 1;               // [NT * NS]
  uint64_t* pfull = sfull + 2;               // [NT * NS]: a warp may be a tile ahead of its group, so one for each S buffer
  uint64_t* odone = pfull + 2;               // [NT * NS]: a PV is done
  uint64_t* drain = odone + 2;
  uint32_t* tbase = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tbase + 1);
  volatile int* progress = reinterpret_cast<volatile int*>(tbase + 2);  // bf16: ring entries of V that have been filled
  ChunkPos* s_pos = reinterpret_cast<ChunkPos*>(tbase + 4);  // [2]
  ChunkSeq* s_seq = reinterpret_cast<ChunkSeq*>(s_pos + 2);  // [2]: the cuts' sequences
  struct WalkState {
    ChunkPos at;
    ChunkSeq s;
  };
  WalkState* s_walk = reinterpret_cast<WalkState*>(s_seq + 2);  // [softmax warps]

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint32_t* err = reinterpret_cast<uint32_t*>(p.ws);
  const int G = p.group, TQ = p.tq, R = NT * TQ;

  // ------------------------------------------------------------ this CTA's piece of the line
  // Warp 0 finds it while warp 1 takes tensor memory and warp 2 sets the barriers up. Up to 32 sequences stand in warp 0's
  // lanes; more go through tables in the shared memory that is the ring later.
  chained_let_follow();  // the combine may be brought up meanwhile
  int* t_ctx = reinterpret_cast<int*>(sm);
  int* t_q = t_ctx + kMaxBatch;
  int* t_off = t_q + kMaxBatch;
  long long* t_pre = reinterpret_cast<long long*>(t_off + kMaxBatch);  // [num_seqs + 1]
  const bool many = p.num_seqs > 32;
  if (many || warp == 0 || warp == 3) chained_wait();  // (the others wait when they have set up what touches no memory)
  if (many) {
    for (int b = tid; b < p.num_seqs; b += C::kThreads) {
      t_ctx[b] = __ldg(p.ctx + b);
      t_q[b] = __ldg(p.ql + b);
    }
    __syncthreads();
  }
  if (warp == 0 || warp == 3) {  // warp 0 finds the piece's start, warp 3 its end
    const int side = warp == 3;
    const uint32_t cap = static_cast<uint32_t>(p.num_tokens) + 1;  // at most 2^31
    long long pre = 0, my_pre = 0;
    uint32_t off = 0;
    ChunkSeq s{0, 0, 0};
    for (int b0 = 0; b0 < p.num_seqs; b0 += 32) {
      const int b = b0 + lane;
      s = ChunkSeq{0, 0, 0};
      if (b < p.num_seqs) s = many ? ChunkSeq{t_ctx[b], t_q[b], 0} : ChunkSeq{__ldg(p.ctx + b), __ldg(p.ql + b), 0};
      const uint32_t q = min(static_cast<uint32_t>(max(s.q, 0)), cap);
      uint32_t x = q;  // rows up to and with this sequence; past the end the sum stays at cap
#pragma unroll
      for (int m = 1; m < 32; m <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, x, m);
        if (lane >= m) x = min(x + y, cap);
      }
      uint32_t before = __shfl_up_sync(0xffffffffu, x, 1);
      if (lane == 0) before = 0;
      s.off = static_cast<int>(min(off + before, cap));
      off = min(off + __shfl_sync(0xffffffffu, x, 31), cap);
      const bool live = chunk_live(p, s);
      if (blockIdx.x == 0 && warp == 0 && b < p.num_seqs && !live && (s.q != 0 || s.ctx < 0)) atomicOr(err, kErrLengths);
      const long long n = live ? p.num_kv_heads * chunk_blocks_length(s.ctx, s.q, R, (s.q + R - 1) / R) : 0;
      long long z = n;
      if (__all_sync(0xffffffffu, n < (1 << 26))) {
        uint32_t z32 = static_cast<uint32_t>(n);
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
          const uint32_t y = __shfl_up_sync(0xffffffffu, z32, m);
          if (lane >= m) z32 += y;
        }
        z = z32;
      } else {
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
          const long long y = __shfl_up_sync(0xffffffffu, z, m);
          if (lane >= m) z += y;
        }
      }
      my_pre = pre + z - n;
      if (many && warp == 0 && b < p.num_seqs) {
        t_off[b] = s.off;
        t_pre[b] = my_pre;
      }
      pre += __shfl_sync(0xffffffffu, z, 31);
    }
    if (!many && lane >= p.num_seqs) my_pre = pre + 1;  // behind every place on the line
    if (many) named_sync(15, 64);                       // both warps: the tables are there
    const long long n = max(1ll, min(static_cast<long long>(gridDim.x), pre / kChunkMinPiece));
    const long long c = blockIdx.x + side;
    const long long x = c < n ? (pre < (1 << 23) && n <= 256 ? static_cast<uint32_t>(pre) * static_cast<uint32_t>(c) / static_cast<uint32_t>(n) : pre * c / n) : pre;
    ChunkPos at{p.num_seqs, 0, 0, 0};
    ChunkSeq q{0, 0, 0};
    if (x < pre) {
      // the last sequence that starts at or before x (and so is not empty)
      long long start;
      if (many) {
        int lo = 0, hi = p.num_seqs - 1;
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (t_pre[mid] <= x) lo = mid;
          else hi = mid - 1;
        }
        at.b = lo;
        start = t_pre[lo];
        q = ChunkSeq{t_ctx[lo], t_q[lo], t_off[lo]};
      } else {
        at.b = 31 - __clz(__ballot_sync(0xffffffffu, my_pre <= x));
        start = __shfl_sync(0xffffffffu, my_pre, at.b);
        q = ChunkSeq{__shfl_sync(0xffffffffu, s.ctx, at.b), __shfl_sync(0xffffffffu, s.q, at.b), __shfl_sync(0xffffffffu, s.off, at.b)};
      }
      const int J = (q.q + R - 1) / R;
      const long long head = chunk_blocks_length(q.ctx, q.q, R, J);
      long long in = x - start;
      at.g = in < (1ll << 31) && head < (1ll << 31) ? static_cast<uint32_t>(in) / static_cast<uint32_t>(head) : static_cast<int>(in / head);
      in -= at.g * head;
      int jl = 0, jh = J - 1;
      while (jl < jh) {
        const int mid = (jl + jh + 1) >> 1;
        if (chunk_blocks_length(q.ctx, q.q, R, mid) <= in) jl = mid;
        else jh = mid - 1;
      }
      at.j = jl;
      // half of the unit's fixed cost stands before its keys, half behind them; to the nearest tile, 0 .. all of them
      in -= chunk_blocks_length(q.ctx, q.q, R, jl) + kChunkUnitCost / 2;
      const int tiles = (q.ctx - q.q + min((jl + 1) * R, q.q) + C::kTok - 1) / C::kTok;
      at.t = in <= 0 ? 0 : min(tiles, static_cast<int>((in + C::kTok / 2) / C::kTok));
    }
    if (lane == 0) {
      s_pos[side] = at;
      s_seq[side] = q;
    }
  } else if (warp == 1) {
    tc::tmem_alloc(tbase, 512);
    tc::tmem_relinquish();
  } else if (warp == 2 && lane == 0) {
    for (int i = 0; i < C::kSlots; ++i) {
      mbar_init(smem_addr(&kvfull[i]), FP8 ? C::kAhead : 1);
      mbar_init(smem_addr(&kvempty[i]), 1);
    }
    for (int i = 0; i < C::kTileSlots; ++i) { mbar_init(smem_addr(&tfull[i]), 1); mbar_init(smem_addr(&tempty[i]), C::kWarps); }
    for (int i = 0; i < NT; ++i) mbar_init(smem_addr(&qfull[i]), FP8 ? 4 * C::NH : 1);
    for (int i = 0; i < NT * NS; ++i) {
      mbar_init(smem_addr(&sfull[i]), 1);
      mbar_init(smem_addr(&pfull[i]), 4 * C::NH);
      mbar_init(smem_addr(&odone[i]), 1);
    }
    mbar_init(smem_addr(qfree), 1);
    mbar_init(smem_addr(drain), 1);
    *abort_flag = 0;
    *progress = 0;
    fence_mbar_init();
    if constexpr (!FP8) {
      prefetch_tmap(&tmk);
      prefetch_tmap(&tmv);
      prefetch_tmap(&tmq);
    }
  }
  chained_wait();
  __syncwarp();
  fence_proxy_async();  // the tables' shared memory becomes the TMA ring
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (tid == 0) {  // for the combine
    const ChunkPos first = s_pos[0], last = s_pos[1];
    ChunkPos at;
    ChunkSeq q;
    const Walk w(p, s_pos, s_seq, at, q);
    const bool inside = same_unit(first, last);
    auto tiles_of = [&](const ChunkPos& at, const ChunkSeq& q) { return (q.ctx - q.q + min((at.j + 1) * R, q.q) + C::kTok - 1) / C::kTok; };
    ChunkRecord r{};
    if (!w.done()) {
      const bool ends = last.b >= p.num_seqs || last.t >= tiles_of(last, s_seq[1]);  // its last unit ends here
      if (first.t > 0 && first.t < tiles_of(first, s_seq[0])) r.head = inside && !ends ? 1 : 2;
      r.tail = !ends && last.t > 0 && (!inside || first.t == 0) ? 1 : 0;
      r.tok0 = s_seq[1].off + last.j * R;
      r.ntok = min(R, s_seq[1].q - last.j * R);
      r.g = last.g;
    }
    reinterpret_cast<ChunkRecord*>(p.ws + kWsHeader)[blockIdx.x] = r;
  }
  const uint32_t tmem = *tbase;
  auto tS = [&](int s, int buf) { return tmem + (s * NS + buf) * 128; };
  auto tO = [&](int s) { return tmem + 256 + s * D; };
  // A wait that runs out is recorded and ends its role; nobody waits for long after that, since every wait is bounded.
  auto wait = [&](uint64_t* bar, int phase) {
    if (mbar_wait_bounded(smem_addr(bar), static_cast<uint32_t>(phase) & 1u)) return true;
    *abort_flag = 1;
    atomicOr(err, kErrTimeout);
    return false;
  };
  // Two waits of the bf16 path may span a whole unit, whose keys can take many times the limit: for its query rows' place, and by the
  // softmax of row tile 1 behind a unit that has none. They run out when the limit passes without a new tile. (The other waits span a
  // tile or two; all of them in this form took 3 to 8 % more time.)
  auto wait_unit = [&](uint64_t* bar, int phase) {
    for (int seen = -1;;) {
      if (mbar_wait_bounded(smem_addr(bar), static_cast<uint32_t>(phase) & 1u)) return true;
      const int now = *progress;
      if (now == seen || *abort_flag) return wait(bar, phase);
      seen = now;
    }
  };
  uint8_t* sKV = sm + C::kOffKV;
  uint8_t* sQ = sm + C::kOffQ;
  ChunkTile* tiles = reinterpret_cast<ChunkTile*>(sm + C::kOffTile);

  if (warp < 4) {
    ChunkPos at;
    ChunkSeq seq;
    Walk w(p, s_pos, s_seq, at, seq);
    if (warp != 1) {
      if constexpr (FP8) {
        if (warp == 0) {
          // ====================================================== the tiles ahead: pages, exponents, and their bytes into L2
          int n = 0;
          bool ok = true;
          auto put = [&](const ChunkTile& x, int pg, int slot) {  // lanes 0 .. 7 hold the pages
            if (n >= C::kTileSlots) {
              int free = 1;
              if (lane == 0) free = !*abort_flag && wait(&tempty[slot], n / C::kTileSlots - 1);
              if (!__shfl_sync(0xffffffffu, free, 0)) return false;
            }
            if (lane == 0) tiles[slot] = x;
            __syncwarp();
            if (lane < C::kPages) tiles[slot].page[lane] = pg;
            __syncwarp();
            if (lane == 0) mbar_arrive_one(smem_addr(&tfull[slot]));
            return true;
          };
          for (; ok && !w.done(); w.next()) {
            const int E = w.keys(), t1 = w.t1();
            const int32_t* row = p.block_table + static_cast<size_t>(w.at.b) * p.bt_stride;
            // page ids are read two tiles ahead, scales one
            auto page_id = [&](int t) {  // -1: none, -2: outside the pool
              if (lane >= C::kPages || t >= t1 || t * C::kTok + lane * kPage >= E) return -1;
              const int pg = __ldg(row + t * C::kPages + lane);
              return static_cast<unsigned>(pg) < static_cast<unsigned>(p.num_pages) ? pg : -2;
            };
            auto scales = [&](int t, int pg) {  // K's, of this lane's four tokens; what lies behind E is read as 0
              const int id = __shfl_sync(0xffffffffu, pg, lane / 4);
              const int left = E - t * C::kTok - 4 * lane;
              if (lane >= C::kTok / 4 || t >= t1 || left <= 0 || id < 0) return make_float4(0.f, 0.f, 0.f, 0.f);
              const size_t at = (static_cast<size_t>(id) * p.num_kv_heads + w.at.g) * kPage + (4 * lane) % kPage;
              return *reinterpret_cast<const float4*>(p.k_scale + at);
            };
            auto largest = [&](int t, const float4& x) {
              const int left = E - t * C::kTok - 4 * lane;
              float m = fabsf(x.x);
              m = left > 1 ? fmaxf(m, fabsf(x.y)) : m;
              m = left > 2 ? fmaxf(m, fabsf(x.z)) : m;
              return chunk_warp_max(left > 3 ? fmaxf(m, fabsf(x.w)) : m);
            };
            auto exponent = [](float top) { return top > 1e-30f ? ilogbf(fminf(top, 1e30f)) + 1 : -98; };  // top < 2^e
            int t = w.at.t;
            int pg = page_id(t), pg1 = page_id(t + 1);
            float4 sc = scales(t, pg);
            for (; t < t1; ++t, ++n) {
              const int pg2 = page_id(t + 2);
              const float4 sc1 = scales(t + 1, pg1);
              // the page's codes into L2: lanes 0 .. 7 K, 16 .. 23 V; V's scales: lanes 8 .. 15
              const int far = __shfl_sync(0xffffffffu, pg, lane & 7);
              if (lane >= 8 && lane < 8 + C::kPages && far >= 0)
                asm volatile("prefetch.global.L2 [%0];\n" ::"l"(p.v_scale + (static_cast<size_t>(far) * p.num_kv_heads + w.at.g) * kPage));
              if ((lane & 15) < C::kPages && far >= 0)
                asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;\n" ::"l"(
                                 static_cast<const uint8_t*>(lane < 16 ? p.k_cache : p.v_cache) +
                                 (static_cast<size_t>(far) * p.num_kv_heads + w.at.g) * (kPage * D)),
                             "r"(kPage * D)
                             : "memory");
              if (pg == -2) atomicOr(err, kErrPageRange);
              ChunkTile x;
              x.keys = min(C::kTok, E - t * C::kTok);
              const int ek = exponent(largest(t, sc));
              x.k_up = exp2f(static_cast<float>(4 - ek));
              x.k_factor = exp2f(static_cast<float>(ek - 4));
              if (!(ok = put(x, pg < 0 ? -1 : pg * p.num_kv_heads + w.at.g, n % C::kTileSlots))) break;
              pg = pg1;
              pg1 = pg2;
              sc = sc1;
            }
          }
          if (ok) {
            ChunkTile x{};
            x.keys = -1;
            (void)put(x, -1, n % C::kTileSlots);
          }
        }
      } else if (warp != 3) {
        // ======================================================== pages of K (warp 0) and V (warp 2): ring entries 2 n and 2 n + 1
        const bool is_v = warp == 2;
        const CUtensorMap* map = is_v ? &tmv : &tmk;
        const int jl = lane / C::kPlanes, plane = lane - jl * C::kPlanes;  // this lane's box: page of the tile, plane
        const bool boxed = lane < C::kBoxes;
        int e = is_v;
        bool ok = true;
        for (; ok && !w.done(); w.next()) {
          const int E = w.keys(), t1 = w.t1();
          const int32_t* row = p.block_table + static_cast<size_t>(w.at.b) * p.bt_stride;
          // page ids are read two tiles ahead: they are not waited for at the ring
          auto page_id = [&](int t) { return boxed && t < t1 && t * C::kTok + jl * kPage < E ? __ldg(row + t * C::kPages + jl) : -1; };
          int t = w.at.t;
          int pg = page_id(t), pg1 = page_id(t + 1);
          for (; t < t1; ++t, e += 2) {
            const int pages = min(C::kPages, (E - t * C::kTok + kPage - 1) / kPage);
            const int pg2 = page_id(t + 2);
            const int slot = e % C::kSlots;
            int good = 1;
            if (lane == 0) {
              if (e >= C::kSlots) good = !*abort_flag && wait(&kvempty[slot], e / C::kSlots - 1);
              if (good) mbar_arrive_expect_tx(smem_addr(&kvfull[slot]), pages * (kPage * C::kRowB));
              if (is_v) *progress = e;
            }
            if (!__shfl_sync(0xffffffffu, good, 0)) {
              ok = false;
              break;
            }
            if (boxed && jl < pages) {
              // an id outside the pool is flagged and read past the tensor's end, where TMA fills zeros
              const bool bad = static_cast<unsigned>(pg) >= static_cast<unsigned>(p.num_pages);
              if (bad) atomicOr(err, kErrPageRange);
              const int at = (bad ? p.num_pages * p.num_kv_heads : pg * p.num_kv_heads + w.at.g) * kPage;
              tma_load_2d(smem_addr(sKV + slot * C::kStage + plane * C::kPlane + jl * (kPage * 128)), map, smem_addr(&kvfull[slot]), plane * 64, at);
            }
            pg = pg1;
            pg1 = pg2;
          }
        }
        // no copy may land after the CTA exits
        if (lane == 0)
          for (int k = max(static_cast<int>(is_v), e - 2 * C::kSlots); k < e; k += 2)
            if (k >= e - C::kSlots) (void)mbar_wait_bounded(smem_addr(&kvfull[k % C::kSlots]), static_cast<uint32_t>(k / C::kSlots) & 1u);
      } else if (lane == 0) {
        // ======================================================== query rows: box = 64 entries x G heads x TQ tokens
        int u = 0;
        uint32_t qphase[2] = {0, 0};
        for (; !w.done(); w.next(), ++u) {
          if (u > 0 && (*abort_flag || !wait_unit(qfree, u - 1))) break;
          for (int s = 0; s < NT; ++s) {
            if (s * TQ >= w.ntok()) break;
            const uint32_t bar = smem_addr(&qfull[s]);
            mbar_arrive_expect_tx(bar, C::kQPlanes * 128 * G * TQ);
            for (int pl = 0; pl < C::kQPlanes; ++pl)
              tma_load_3d(smem_addr(sQ + s * C::kQTile + pl * 16384), &tmq, bar, pl * 64, w.at.g * G, w.tok0() + s * TQ);
            ++qphase[s];
          }
        }
        for (int s = 0; s < NT; ++s)
          if (qphase[s]) (void)mbar_wait_bounded(smem_addr(&qfull[s]), (qphase[s] - 1) & 1u);
      }
    } else {
      // ========================================================== MMA issuer
      const uint32_t go = elect_one();
      auto all_wait = [&](uint64_t* bar, int phase) { return __all_sync(0xffffffffu, wait(bar, phase)) != 0; };
      constexpr uint32_t fmt = FP8 ? tc::kF16 : tc::kBF16;
      constexpr uint32_t idS = tc::idesc(fmt, fmt, tc::kKMajor, tc::kKMajor, 128, C::kTok);
      constexpr uint32_t idPV = tc::idesc(tc::kBF16, tc::kBF16, tc::kKMajor, tc::kMNMajor, 128, D);
      const uint32_t aKV = smem_addr(sKV), aQ = smem_addr(sQ);
      int n = 0;              // tiles so far: K at ring entry 2 n, V at 2 n + 1
      int ns[2] = {0, 0};     // S products issued for each row tile
      int np[2] = {0, 0};     // PV products
      auto issue_s = [&](int s, int k) {  // S of row tile s, K at ring entry k (landed)
        const int buf = NS == 1 ? 0 : ns[s] & 1;
        const uint64_t dK = tc::sdesc(aKV + (k % C::kSlots) * C::kStage, 16, 1024, tc::kSwizzle128B);
        const uint64_t dQ = tc::sdesc(aQ + s * C::kQTile, 16, 1024, tc::kSwizzle128B);
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
          mma_f16_ss(go, tS(s, buf), tc::desc_plus(dQ, (i / 4) * 16384 + (i & 3) * 32),
                     tc::desc_plus(dK, (i / 4) * C::kPlane + (i & 3) * 32), idS, i > 0);
        commit_if(go, &sfull[s * NS + buf]);
        ++ns[s];
      };
      auto issue_pv = [&](int s, int k, bool first, int tokens) {  // tile k's V (landed), P of tile np[s] written
        const uint32_t tP = tS(s, NS == 1 ? 0 : np[s] & 1);
        const uint64_t dV = tc::sdesc(aKV + (2 * k + 1) % C::kSlots * C::kStage, C::kPlane, 1024, tc::kSwizzle128B);
        if (tokens >= C::kTok) {
#pragma unroll
          for (int i = 0; i < C::kTok / 16; ++i)
            mma_f16_ts(go, tO(s), tP + i * 8, tc::desc_plus(dV, i * 2048), idPV, i > 0 ? 1u : !first);
        } else {
          // only the k-steps that hold keys: what lies behind them was never loaded
          const int steps = (tokens + 15) / 16;
          for (int i = 0; i < steps; ++i) mma_f16_ts(go, tO(s), tP + i * 8, tc::desc_plus(dV, i * 2048), idPV, i > 0 ? 1u : !first);
        }
        commit_if(go, &odone[NS == 1 ? s : np[s] & 1]);
        ++np[s];
      };
      auto landed = [&](int k) { return all_wait(&kvfull[k % C::kSlots], k / C::kSlots); };
      bool ok = true;
      int uq[2] = {0, 0};
      for (; ok && !w.done(); w.next()) {
        const int t0 = w.at.t, t1 = w.t1(), E = w.keys();
        const int nt = NT == 2 && w.ntok() > TQ ? 2 : 1;
        for (int s = 0; ok && s < nt; ++s) ok = all_wait(&qfull[s], uq[s]++);
        ok = ok && landed(2 * n);
        if (!ok) break;
        tc::fence_after_sync();
        for (int s = 0; s < nt; ++s) issue_s(s, 2 * n);
        commit_if(go, &kvempty[(2 * n) % C::kSlots]);
        for (int t = t0; t < t1; ++t, ++n) {
          const bool more = t + 1 < t1;
          if (!more && !FP8) commit_if(go, qfree);  // every S of the unit has been issued
          if (NS == 2 && more) {
            if (!(ok = landed(2 * n + 2))) break;
            tc::fence_after_sync();
            issue_s(0, 2 * n + 2);
            commit_if(go, &kvempty[(2 * n + 2) % C::kSlots]);
          }
          if (!(ok = landed(2 * n + 1))) break;
          for (int s = 0; s < nt; ++s) {
            if (!(ok = NS == 1 ? all_wait(&pfull[s], np[s]) : all_wait(&pfull[np[s] & 1], np[s] >> 1))) break;
            tc::fence_after_sync();
            issue_pv(s, n, t == t0, E - t * C::kTok);
            if (s == nt - 1) commit_if(go, &kvempty[(2 * n + 1) % C::kSlots]);
            if (NS == 1 && more) {
              if (s == 0 && !(ok = landed(2 * n + 2))) break;
              tc::fence_after_sync();
              issue_s(s, 2 * n + 2);
              if (s == nt - 1) commit_if(go, &kvempty[(2 * n + 2) % C::kSlots]);
            }
          }
          if (!ok || __any_sync(0xffffffffu, *abort_flag)) {
            ok = false;
            break;
          }
        }
      }
      // MMAs still running (after a failure) must end before tensor memory is freed
      commit_if(go, drain);
      (void)mbar_wait_bounded(smem_addr(drain), 0u);
    }
  } else {
    // ============================================================ softmax: row tile s, half h of the columns; row = tensor-memory lane
    // The warp's place stands in shared memory, where lane 0 moves it on; at head_dim 64 in registers (1024 tokens over 8192, 32/4 heads:
    // 101.7 us, in shared memory 103.4; at 128 two sequences of 1500 keys 22.7 and 22.3, prompts the same).
    constexpr bool kOwn = D == 64;
    ChunkPos own_at;
    ChunkSeq own_seq;
    Walk w(p, s_pos, s_seq, kOwn ? own_at : s_walk[warp - 4].at, kOwn ? own_seq : s_walk[warp - 4].s, kOwn || lane == 0);
    __syncwarp();
    auto next_unit = [&]() {
      __syncwarp();
      if (kOwn || lane == 0) w.next();
      __syncwarp();
    };
    const int s = ((warp - 4) >> 2) / C::NH, h = ((warp - 4) >> 2) % C::NH;
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const int tok = r / G, head = r - tok * G;  // of the row inside its tile
    const int pair = 1 + s * 4 + (warp & 3);    // named barrier of the two warps that share 32 rows
    float* ex_max = reinterpret_cast<float*>(sm + C::kOffEx) + s * 2 * C::NH * 128;  // [NH][128]
    float* ex_sum = ex_max + C::NH * 128;
    // A wait that failed ends this warp's later waits, but the named barriers are still reached in order: no warp is left at one.
    bool ok = true;
    auto await = [&](uint64_t* bar, int phase) { ok = __all_sync(0xffffffffu, ok && wait(bar, phase)) != 0; };
    // PV of this row tile's tile i. A parity wait tells a phase only from the one before it. With one S buffer, S(i) done says
    // PV(i - 1) is; with two it says so of PV(i - 2) only, so the PVs take turns on two barriers.
    auto pv_done = [&](int i) { await(NS == 1 ? &odone[s] : &odone[i & 1], NS == 1 ? i : i >> 1); };
    int i_s = 0;  // tiles of this row tile so far
    int n = 0;    // tiles of the CTA so far
    // FP8: this warp's page of tile m, K's (the first kAhead warps; two tiles ahead of the softmax) or V's (one ahead), widened into
    // the ring. A lane takes 16 codes of a token, D / 16 lanes a row, so a warp's loads are whole rows; lanes whose entries lie in an
    // odd plane take the neighbouring row, whose chunks stand in the other banks: the stores have no conflicts.
    // In three steps: peek reads the tile's description, fetch starts the loads, store converts and writes. At head_dim 256, where a
    // thread has registers to spare, a tile's description is read, and its loads are started, before the exponentials of the tile
    // before (129 to 119 us for 512 tokens over 16384, 8/1 heads); at 128 that spills, and the three follow one another (193 us against 205).
    constexpr bool kEarly = D == 256;
    const int job = warp - 4 - (warp - 4 >= C::kAhead ? C::kAhead : 0);
    const bool widens_v = warp - 4 >= C::kAhead;
    constexpr int kLanes = D / 16, kStep = 32 / kLanes, kLoads = kPage / kStep;
    const int c16 = lane % kLanes, sub = (lane / kLanes) ^ ((c16 >> 2) & 1);  // its 16 codes; its row of kStep
    bool more_tiles = FP8 != 0;
    struct Job {
      int page, keys;
      float up;
    };
    auto peek = [&](int m, Job& j) {
      if (!more_tiles) return;
      await(&tfull[m % 8], m / 8);
      const ChunkTile& x = tiles[m % 8];
      j.page = x.page[job];
      j.keys = x.keys;
      j.up = widens_v ? 1.f / kChunkVUnit : x.k_up;
      more_tiles = ok && j.keys >= 0;
    };
    auto fetch = [&](const Job& j, uint4 (&code)[kLoads], float (&f)[kLoads]) {
      const size_t at = static_cast<size_t>(max(j.page, 0)) * kPage + sub;
      const uint8_t* src = static_cast<const uint8_t*>(widens_v ? p.v_cache : p.k_cache) + at * D + c16 * 16;
      const float* scale = (widens_v ? p.v_scale : p.k_scale) + at;
#pragma unroll
      for (int k = 0; k < kLoads; ++k) {
        code[k] = __ldg(reinterpret_cast<const uint4*>(src + k * kStep * D));
        f[k] = __ldg(scale + k * kStep);
      }
    };
    auto store = [&](int m, const Job& j, uint4 (&code)[kLoads], float (&f)[kLoads]) {
      const int e = 2 * m + (widens_v ? 1 : 0), slot = e % C::kSlots;
      if (e >= C::kSlots) await(&kvempty[slot], e / C::kSlots - 1);
      uint8_t* dst = sKV + slot * C::kStage + (c16 >> 2) * C::kPlane + (job * kPage + sub) * 128;
      // behind the unit's last key, or outside the pool: zeros
      const int live = j.page < 0 ? 0 : j.keys - job * kPage - sub;
      if (__any_sync(0xffffffffu, live <= kPage - kStep)) {
#pragma unroll
        for (int k = 0; k < kLoads; ++k)
          if (k * kStep >= live) {
            code[k] = make_uint4(0, 0, 0, 0);
            f[k] = 0.f;
          }
      }
#pragma unroll
      for (int k = 0; k < kLoads; ++k) {
        const float fs = f[k] * j.up;
        const uint32_t u[4] = {code[k].x, code[k].y, code[k].z, code[k].w};
        uint32_t o[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) e4m3x4_to_f16x4(u[i], o[2 * i], o[2 * i + 1]);
        if (widens_v) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 v = __fmul2_rn(f16x2_to_f32x2(o[i]), make_float2(fs, fs));
            o[i] = pack_bf16(v.x, v.y);
          }
        } else {
          const uint32_t hi = pack_f16(fs, fs);
          // K: the scale as two f16 terms (one would put the same 2^-11 on all of a key's products, and so on its score): code x low,
          // then one rounding of code x high + that
          const float rest = fs - f16x2_to_f32x2(hi).x;
          const uint32_t lo = pack_f16(rest, rest);
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = fma_f16x2(o[i], hi, mul_f16x2(o[i], lo));
        }
        // entries 16 c ..: plane c / 4, chunks 2 (c % 4) and the next
        const int row = (k * kStep + sub) & 7, ch = 2 * (c16 & 3);  // a page is two swizzle periods
        *reinterpret_cast<uint4*>(dst + k * kStep * 128 + ((ch ^ row) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4*>(dst + k * kStep * 128 + (((ch + 1) ^ row) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive_one(smem_addr(&kvfull[slot]));
    };
    auto widen = [&](int m) {
      Job j;
      peek(m, j);
      if (!more_tiles) return;
      uint4 code[kLoads];
      float f[kLoads];
      fetch(j, code, f);
      store(m, j, code, f);
    };
    Job next_job;
    uint4 code[kEarly ? kLoads : 1];
    float f[kEarly ? kLoads : 1];
    const int ahead = widens_v ? 1 : 2;
    if constexpr (FP8) {
      for (int m = 0; m < ahead; ++m) widen(m);
      if (kEarly) peek(ahead, next_job);
    }
    for (; !w.done(); next_unit()) {
      const int t0 = w.at.t, t1 = w.t1(), ntok = w.ntok();
      if (s * TQ >= ntok) {  // no rows for this tile in the unit
        if constexpr (FP8) {
          for (int t = t0; t < t1; ++t, ++n) {
            await(&tfull[n % 8], n / 8);
            if (lane == 0) mbar_arrive_one(smem_addr(&tempty[n % 8]));
            if constexpr (kEarly) {
              if (more_tiles) {
                fetch(next_job, code, f);
                store(n + ahead, next_job, code, f);
                peek(n + ahead + 1, next_job);
              }
            } else {
              widen(n + ahead);
            }
          }
        }
        continue;
      }
      const bool valid = tok < TQ && s * TQ + tok < ntok;
      const int lim = valid ? w.first_key() + s * TQ + tok : -1;  // last key the row sees
      float cr = p.scale * 1.4426950408889634f;
      if constexpr (FP8) {
        // this half of the row's Q in f16, scaled by a power of two so that the row's largest entry lies in [1, 2); the unit
        // before has done its last S (this thread has read it)
        uint8_t* dst = sQ + s * C::kQTile + r * 128;
        const uint16_t* src = p.q + static_cast<int64_t>(w.tok0() + s * TQ + tok) * p.q_stride + static_cast<int64_t>(w.at.g * G + head) * D;
        // eight loads at a time; at head_dim 128 that is all, held for the second pass (1024 tokens
        // over 8192: 177 us; read twice, four and two loads at a time, 183)
        constexpr int kBatches = D / 128;
        uint4 own[8];
        auto read = [&](int at) {
#pragma unroll
          for (int e = 0; e < 8; ++e) own[e] = valid ? *reinterpret_cast<const uint4*>(src + h * (D / 2) + 64 * at + 8 * e) : make_uint4(0, 0, 0, 0);
        };
        float mx = 0.f;
#pragma unroll 1
        for (int b = 0; b < kBatches; ++b) {
          read(b);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint32_t u[4] = {own[e].x, own[e].y, own[e].z, own[e].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) mx = fmaxf(mx, fmaxf(fabsf(bf16_lo(u[k])), fabsf(bf16_hi(u[k]))));
          }
        }
        ex_max[h * 128 + r] = mx;
        named_sync(pair, 64);
        mx = fmaxf(ex_max[r], ex_max[128 + r]);
        const int ex = mx > 0.f && mx < INFINITY ? -ilogbf(mx) : 0;
#pragma unroll 1
        for (int b = kBatches - 1; b >= 0; --b) {  // the last batch is still here
          if (b < kBatches - 1) read(b);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int e = h * (D / 2) + 64 * b + 8 * i;
            const uint32_t u[4] = {own[i].x, own[i].y, own[i].z, own[i].w};
            uint32_t o[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) o[k] = pack_f16(ldexpf(bf16_lo(u[k]), ex), ldexpf(bf16_hi(u[k]), ex));
            *reinterpret_cast<uint4*>(dst + (e >> 6) * 16384 + ((((e & 63) >> 3) ^ (r & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
          }
        }
        cr = ldexpf(cr, -ex);
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive_one(smem_addr(&qfull[s]));
      }
      if constexpr (!FP8 && NT == 2) {
        if (s == 1) ok = __all_sync(0xffffffffu, ok && wait_unit(&sfull[1], i_s)) != 0;
      }
      float M = -INFINITY, l = 0.f;
      for (int t = t0; t < t1; ++t, ++n, ++i_s) {
        const int buf = NS == 1 ? 0 : i_s & 1;
        const uint32_t tSb = tS(s, buf) + lanes;
        await(&sfull[s * NS + buf], NS == 1 ? i_s : i_s >> 1);
        tc::fence_after_sync();
        uint32_t x[C::kCols];
#pragma unroll
        for (int c = 0; c < C::kCols; c += 32) tmem_ld32(tSb + h * C::kCols + c, x + c);
        tc::wait_ld();
        float cr_t = cr;  // FP8: the tile's scores count in k_factor
        if constexpr (FP8) {
          cr_t = cr * tiles[n % 8].k_factor;  // this warp has seen its barrier when it peeked at the tile
          __syncwarp();
          if (lane == 0) mbar_arrive_one(smem_addr(&tempty[n % 8]));
        }
        const int vis = lim - t * C::kTok - h * C::kCols;  // last visible column of this half
        if (__any_sync(0xffffffffu, vis < C::kCols - 1)) {
#pragma unroll
          for (int c = 0; c < C::kCols; ++c)
            if (c > vis) x[c] = 0xFF800000u;  // -infinity
        }
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < C::kCols; c += 2)
          m4[(c >> 1) & 3] = fmaxf(fmaxf(m4[(c >> 1) & 3], __uint_as_float(x[c])), __uint_as_float(x[c + 1]));
        float mx = cr_t * fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
        // both halves' scores are in registers once both warps have voted: P may then overwrite S
        if (named_or(pair, 64, mx > M + 8.f)) {
          ex_max[h * 128 + r] = mx;
          named_sync(pair, 64);
          mx = fmaxf(ex_max[r], ex_max[128 + r]);
          const bool up = mx > M + 8.f;
          const float f = up ? fast_exp2(M - mx) : 1.f;  // 0 on the row's first tile
          l *= f;
          M = up ? mx : M;
          if (t > t0) {
            pv_done(i_s - 1);
            tc::fence_after_sync();
#pragma unroll 1
            for (int c = h * (D / 2); c < (h + 1) * (D / 2); c += 8) {  // few columns at a time: the scores are live
              uint32_t o[8];
              tc::ld8(tO(s) + lanes + c, o);
              tc::wait_ld();
#pragma unroll
              for (int k = 0; k < 8; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
              tc::st8(tO(s) + lanes + c, o);
            }
          }
        }
        const float shift = M == -INFINITY ? 0.f : -M;  // a row without a visible key so far: P = 2^-inf = 0
        const float2 cr2 = make_float2(cr_t, cr_t), sh2 = make_float2(shift, shift);
        float2 l2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        if constexpr (FP8 && kEarly) {
          if (more_tiles) fetch(next_job, code, f);
        }
#pragma unroll
        for (int c0 = 0; c0 < C::kCols; c0 += 32) {
          uint32_t pw[16];
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            const float2 d = __ffma2_rn(make_float2(__uint_as_float(x[c0 + c]), __uint_as_float(x[c0 + c + 1])), cr2, sh2);
            const float2 e = make_float2(fast_exp2(d.x), fast_exp2(d.y));
            l2[(c >> 1) & 1] = __fadd2_rn(l2[(c >> 1) & 1], e);
            pw[c / 2] = pack_bf16(e.x, e.y);
          }
          tc::st16(tSb + (h * C::kCols + c0) / 2, pw);
        }
        l += (l2[0].x + l2[0].y) + (l2[1].x + l2[1].y);
        const int nv = w.keys() - t * C::kTok;
        if (!FP8 && s == 0 && h == 0 && nv < C::kTok) {
          // V rows behind the unit's last key, up to the end of the last k-step, may hold anything, and P = 0 times NaN
          // would still reach O: they become zeros
          await(&kvfull[(2 * n + 1) % C::kSlots], (2 * n + 1) / C::kSlots);
          if (r >= nv && r < (nv + 15) / 16 * 16) {
#pragma unroll
            for (int pl = 0; pl < C::kPlanes; ++pl) {
              uint4* z = reinterpret_cast<uint4*>(sKV + ((2 * n + 1) % C::kSlots) * C::kStage + pl * C::kPlane + r * 128);
#pragma unroll
              for (int k = 0; k < 8; ++k) z[k] = make_uint4(0, 0, 0, 0);
            }
          }
          fence_proxy_async();
        }
        tc::wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive_one(smem_addr(&pfull[s * NS + buf]));
        if constexpr (FP8) {
          if constexpr (kEarly) {
            if (more_tiles) {
              store(n + ahead, next_job, code, f);
              peek(n + ahead + 1, next_job);
            }
          } else {
            widen(n + ahead);
          }
        }
      }
      // ---- the unit's rows, or this CTA's part of them: this half of the head's entries
      ex_sum[h * 128 + r] = l;
      named_sync(pair, 64);
      l = ex_sum[r] + ex_sum[128 + r];
      pv_done(i_s - 1);
      tc::fence_after_sync();
      const bool whole = t0 == 0 && t1 == w.tiles();
      const float inv = whole || l != 0.f ? (FP8 ? kChunkVUnit : 1.f) / l : 0.f;  // a part may hold no key that the row sees
      if (whole) {
        uint16_t* dst = p.out + (static_cast<int64_t>(w.tok0() + s * TQ + tok) * p.num_q_heads + w.at.g * G + head) * D;
#pragma unroll 1
        for (int c = h * (D / 2); c < (h + 1) * (D / 2); c += 32) {
          uint32_t o[32];
          tmem_ld32(tO(s) + lanes + c, o);
          tc::wait_ld();
          if (valid && ok) {
#pragma unroll
            for (int k = 0; k < 32; k += 8) {
              uint4 v;
              v.x = pack_bf16(__uint_as_float(o[k]) * inv, __uint_as_float(o[k + 1]) * inv);
              v.y = pack_bf16(__uint_as_float(o[k + 2]) * inv, __uint_as_float(o[k + 3]) * inv);
              v.z = pack_bf16(__uint_as_float(o[k + 4]) * inv, __uint_as_float(o[k + 5]) * inv);
              v.w = pack_bf16(__uint_as_float(o[k + 6]) * inv, __uint_as_float(o[k + 7]) * inv);
              *reinterpret_cast<uint4*>(dst + c + k) = v;
            }
          }
        }
      } else {
        const int slot = 2 * blockIdx.x + (t0 == 0 ? 1 : 0);
        const size_t row = (static_cast<size_t>(slot) * NT + s) * 128 + r;
        float* dst = p.part_o + row * D;
        if (valid && h == 0) p.part_lse[row] = l == 0.f ? -INFINITY : M + __log2f(l);
#pragma unroll 1
        for (int c = h * (D / 2); c < (h + 1) * (D / 2); c += 32) {
          uint32_t o[32];
          tmem_ld32(tO(s) + lanes + c, o);
          tc::wait_ld();
          if (valid) {
#pragma unroll
            for (int k = 0; k < 32; k += 4)
              *reinterpret_cast<float4*>(dst + c + k) = make_float4(__uint_as_float(o[k]) * inv, __uint_as_float(o[k + 1]) * inv,
                                                                    __uint_as_float(o[k + 2]) * inv, __uint_as_float(o[k + 3]) * inv);
          }
        }
      }
      tc::fence_before_sync();  // the next unit's first PV overwrites O, after this warp's next arrival on pfull
    }
  }
  __syncwarp();
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

constexpr int kChunkCombineThreads = 512;

// Joins the partials of the unit that begins in CTA blockIdx.x and goes on behind it: with M the largest lse,
// out = sum 2^(lse_k - M) O_k / sum 2^(lse_k - M), one warp a row, the pieces in the order of their CTAs.
template <int FP8, int D>
__global__ void __launch_bounds__(kChunkCombineThreads) pa_chunk_combine_kernel(const __grid_constant__ ChunkParams p) {
  using C = ChunkCfg<FP8, D>;
  constexpr int NT = C::NT;
  const ChunkRecord* records = reinterpret_cast<const ChunkRecord*>(p.ws + kWsHeader);
  constexpr int kWarps = kChunkCombineThreads / 32;
  const int c = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  chained_start();
  const ChunkRecord rec = records[c];
  if (!rec.tail) return;
  const int G = p.group, TQ = p.tq;
  const int rows = rec.ntok * G;
  if (static_cast<int>(blockIdx.y) * kWarps >= rows) return;
  // the CTA where the unit ends
  int end = c;
  for (int k0 = c + 1; k0 < static_cast<int>(gridDim.x); k0 += 32) {
    const uint32_t hit = __ballot_sync(0xffffffffu, k0 + lane < static_cast<int>(gridDim.x) && records[k0 + lane].head == 2);
    if (hit) {
      end = k0 + __ffs(hit) - 1;
      break;
    }
  }
  for (int i = blockIdx.y * kWarps + warp; i < rows; i += gridDim.y * kWarps) {
    const int tok = i / G, h = i - tok * G, s = tok / TQ;
    const size_t at = static_cast<size_t>(s) * 128 + (tok - s * TQ) * G + h;  // row of a partial slot
    auto row_of = [&](int k) { return static_cast<size_t>(k == c ? 2 * c + 1 : 2 * k) * NT * 128 + at; };
    auto lse_of = [&](int k) { return k == c || records[k].head ? p.part_lse[row_of(k)] : -INFINITY; };
    float M = -INFINITY;
    for (int k = c + lane; k <= end; k += 32) M = fmaxf(M, lse_of(k));
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, m));
    const float base = M == -INFINITY ? 0.f : M;
    float o[D / 32], sum = 0.f;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) o[e] = 0.f;
    for (int k0 = c; k0 <= end; k0 += 32) {
      const float mine = k0 + lane <= end ? fast_exp2(lse_of(k0 + lane) - base) : 0.f;
      const int n = min(32, end - k0 + 1);
#pragma unroll 4
      for (int k = 0; k < n; ++k) {
        const float wk = __shfl_sync(0xffffffffu, mine, k);
        if (wk == 0.f) continue;
        sum += wk;
        const float2* src = reinterpret_cast<const float2*>(p.part_o + row_of(k0 + k) * D);
#pragma unroll
        for (int e = 0; e < D / 64; ++e) {
          const float2 v = src[32 * e + lane];
          o[2 * e] += wk * v.x;
          o[2 * e + 1] += wk * v.y;
        }
      }
    }
    const float inv = 1.f / sum;
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + (static_cast<int64_t>(rec.tok0 + tok) * p.num_q_heads + rec.g * G + h) * D);
#pragma unroll
    for (int e = 0; e < D / 64; ++e) dst[32 * e + lane] = pack_bf16(o[2 * e] * inv, o[2 * e + 1] * inv);
  }
}

}  // namespace pav
