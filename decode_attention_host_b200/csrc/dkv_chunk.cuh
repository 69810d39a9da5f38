// dkv_chunk.cuh -- attention of a chunk of new tokens per sequence over the
// paged cache, on the 5th-generation tensor cores.
//
// Query i of sequence b sits at position L_b + i.  With hi = L_b + i + self it
// sees the cached tokens t < hi, and under a window only those with
// t >= hi - window or t < sinks:
//     s_t = scale * (R(L_b + i) q) . (R(t) k_t),   o = sum_t softmax(s)_t v_t.
// A row that sees nothing is zero.
//
// Work.  The G query heads of a kv head share its K and V, so the rows of a
// (sequence, kv head) are its tokens times G, token-major, and a CTA takes 256
// of them as two tiles of 128 (the M of one tcgen05.mma).  It walks the 128-
// token tiles that some row of it sees: the tiles that hold sinks, then those
// from the first row's window start to the last row's end.  With few row tiles
// the walk is cut into splits whose partial results a second kernel joins.
//
// One CTA per SM, 16 warps:
//   warps 0, 2  copy K and V tiles, one tensor copy per run of rows that lies
//               in one block (16 to 128 rows) and 64-element half
//   warp 1      issues the matrix instructions: S = Q K^T into TMEM, then
//               O += P V with P read from TMEM; the two row tiles alternate, so
//               one's softmax runs under the other's products
//   warps 4-7   rotate each K tile in place: keys are cached un-rotated, and a
//               tile that is rotated once serves 256 rows
//   warps 8-11, 12-15  the softmax of row tile 0 and 1, a thread per row: no
//               value leaves its thread, the running maximum is raised lazily
//               (only past 2^8, or 2^4 with fp16 weights, so O is rescaled
//               rarely), P goes back to TMEM over the S it came from
// A chunk of at most 128 rows a kv head takes CTAs of 128 rows (DUAL, below).
//
// Measured on a B200, 32 query heads over 8 kv heads, D = 128, bf16, in a burst
// and in a loop at lower clocks: 2048 rows on 30720 tokens in 1.08 and 1.23 ms,
// 0.99 and 0.87 PFLOP/s (0.6 of a plain matrix product; without rotation 0.89
// ms, 1.2 PFLOP/s); 8 rows on four 64k contexts in 202 and 246 us, 5.3 and 4.4
// TB/s.  A K/V tile takes about 3900 cycles where its products take 2100: the
// softmax warps and the rotating one share the schedulers, 47% of whose slots
// issue, and the tensor core waits for P.  The long case's 256 CTAs are 1.73
// waves of 148 SMs and take two; its rows are too many for the workspace that
// splits need.  The 128 x 128 tiles are what TMEM's 512 columns hold twice (S
// and O); N = 64 halves the products' rate.
//
// Roundings to 16 bits: rotated queries and keys are held in fp16 for both
// cache types (fp32 rotation, one rounding to 2^-11; bf16 operands would be
// off by 2^-8, the largest error of the whole computation), unrotated ones as
// stored; the weights P take V's type, as one instruction multiplies equal
// types.  Everything else is fp32.  A rotated component beyond fp16's range, or
// a block id outside the pools, makes the rows that see it NaN (the kernel
// notes the first and the last such token of a CTA) and sets a status bit.
#pragma once

#include <type_traits>

#include "dkv_kernels.cuh"

namespace dkv {

constexpr int kChunkTokens = 128;                  // tokens of a K/V tile, the N of S = Q K^T
constexpr int kChunkThreads = 512;
constexpr int kSubTile = kChunkTokens * 128;       // bytes of 128 rows x 64 elements, 128-byte swizzle
constexpr int kRopeChain = 8;                      // K tiles that may follow one seed of the rotation
// Registers per thread of the four warp groups, out of the 128 per thread the
// block is launched with: the shares add up to exactly those.
constexpr int kRegsLaunch = 128;
constexpr int kRegsIssue = 64;
constexpr int kRegsRotate = 96;
constexpr int kRegsSoftmax = 176;
static_assert(kRegsIssue + kRegsRotate + 2 * kRegsSoftmax <= 4 * kRegsLaunch, "setmaxnreg.inc would wait for ever");
constexpr float kMostOperand = 65504.f;            // fp16's largest value; what rounds to it is in range too
// Weights are 2^(score - reference + kWeightBias), the reference raised once a score passes it by kWeightLag.  fp16
// has 29 binades of normal numbers below 2^15: held there, a weight keeps its 11 bits down to 2^-25 of the
// reference, and one below that is off by 2^-25 (half a subnormal step), 2^-36 of the reference.  Held around 2^0,
// 64k weights of 2^-25 beside one dominating token went missing from the product and not from the sum.
// bf16 has fp32's range and needs no bias.
template <bool BF16>
constexpr float kWeightLag = BF16 ? kLazyMax : 4.f;
template <bool BF16>
constexpr float kWeightBias = BF16 ? 0.f : 11.f;
constexpr int kStatusRange = 64;                   // DKV_STATUS_RANGE

struct ChunkParams {
  const uint16_t* q;          // [total_rows] of hq * D elements, q_stride elements apart
  uint16_t* out;              // [total_rows][hq][D]
  const int32_t* q_start;     // [batch + 1]
  const int32_t* seq_lens;    // [batch]
  const int32_t* table;       // [batch][stride]
  const uint64_t* turns;      // [D / 2] turns per position, 2^-64 turns
  float* part_o;              // [total_rows][hq][nsplit][D], nsplit > 1
  float* part_lse;            // [total_rows][hq][nsplit], log2 domain
  int32_t* status;
  long long q_stride;
  int32_t total_rows, batch, stride, hq, hkv, block_size, host_split, id_total, max_len;
  int32_t group_shift;        // log2(hq / hkv)
  int32_t nsplit;
  int32_t box;                // rows of one tensor copy: the largest power of two that divides the block, up to 128
  int32_t oob_row;            // a row outside the pool of `oob_host`: copies from there fill with zeros
  int32_t oob_host;
  int32_t window, sinks, self;
  float qscale;               // softmax scale * log2(e)
  int32_t stall_first_copy;   // test hook: CTA 0 arms the barrier of its first key tile but issues no copy
  InvDiv div_bs, div_hkv, div_split;
};

// Tensor maps of the four pools: boxes of `box` rows x 64 elements, 128-byte swizzle.
struct ChunkMaps {
  CUtensorMap k_dev, v_dev, k_host, v_host;
};

template <int D>
struct ChunkShape {
  static constexpr int kSub = D / 64;                       // 64-element halves of a row
  static constexpr int kTile = kSub * kSubTile;             // bytes of a Q, K or V tile
  static constexpr int kStagesK = D == 128 ? 3 : 4;
  static constexpr int kStagesV = D == 128 ? 2 : 4;
  static constexpr int kMoreV = D == 128 ? 1 : 0;            // in the place of an unused second Q tile
};

struct ChunkTail {
  uint64_t k_full[4], k_ready[4], k_free[4];   // copied, rotated, read by the products of both row tiles
  uint64_t v_full[4], v_free[4];
  uint64_t q_ready[2], s_full[2], p_ready[2];  // per row tile
  uint64_t done;                               // every product has completed
  uint32_t tmem;
  int32_t b, tile;                             // the CTA's sequence (-1: none) and row tile
  int32_t q0, n, len;                          // its first row, rows and cached tokens
  int32_t bad_lo, bad_hi;                      // first and last token of an invalid block or with a key out of range
  uint32_t bad_rows[8];                        // a query out of range, by softmax warp and lane
  int32_t broken;                              // a wait ran out: every role gives up
};

template <int D>
__host__ __device__ constexpr size_t chunk_smem_bytes() {
  using C = ChunkShape<D>;
  return static_cast<size_t>(2 + C::kStagesK + C::kStagesV) * C::kTile + sizeof(ChunkTail);
}

// ----------------------------------------------------------------------------- tensor core helpers

// Shared-memory matrix descriptor, 128-byte swizzle: start address and the two
// strides in 16-byte units, descriptor version 1, swizzle mode 2.  Held as its
// two words: the high one is the same for every operand here (8-row groups
// 1024 bytes apart), the low one moves by plain additions.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_low(uint32_t addr, uint32_t lead) { return (addr >> 4) | ((lead >> 4) << 16); }

// Instruction descriptor of kind::f16: fp32 accumulator, A and B both fp16 or
// both bf16, A K-major, B K-major or (mn) N-major.
__host__ __device__ constexpr uint32_t umma_idesc(int m, int n, bool bf16, bool mn) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (mn ? 1u << 16 : 0u) |
         (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

// The issuing warp stays converged and one lane's predicate `on` issues: the
// operands are then warp-uniform values, which the instruction takes from
// uniform registers, and need no moves there one by one (a branch around the
// instruction costs those: 97 cycles from one to the next, where the tensor
// core needs 64).
__device__ __forceinline__ void umma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool acc, uint32_t on) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "mov.b64 a, {%1, %6};\n\tmov.b64 b, {%2, %6};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d), "r"(a), "r"(b), "r"(idesc),
      "r"(static_cast<uint32_t>(acc)), "r"(on), "r"(kDescHigh)
      : "memory");
}
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool acc, uint32_t on) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "mov.b64 b, {%2, %6};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d), "r"(a), "r"(b), "r"(idesc),
      "r"(static_cast<uint32_t>(acc)), "r"(on), "r"(kDescHigh)
      : "memory");
}
// One arrival on `bar` when all matrix instructions the issuing lane has issued are complete.
__device__ __forceinline__ void umma_commit(uint32_t bar, uint32_t on) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar), "r"(on)
      : "memory");
}
__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

#define DKV_R8(r, i) "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]), \
                     "+r"(r[i + 6]), "+r"(r[i + 7])
#define DKV_O8(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), "=r"(r[i + 5]), \
                     "=r"(r[i + 6]), "=r"(r[i + 7])
#define DKV_I8(r, i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), "r"(r[i + 5]), \
                     "r"(r[i + 6]), "r"(r[i + 7])

// 32 columns of this warp's 32 TMEM lanes, one lane per thread.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : DKV_O8(r, 0), DKV_O8(r, 8), DKV_O8(r, 16), DKV_O8(r, 24)
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : DKV_O8(r, 0), DKV_O8(r, 8)
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};"
      ::DKV_I8(r, 0), DKV_I8(r, 8), "r"(addr)
      : "memory");
}
// Completes this thread's loads; the registers pass through, so no use of them moves above it.
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : DKV_R8(r, 0), DKV_R8(r, 8), DKV_R8(r, 16), DKV_R8(r, 24)::"memory");
}
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : DKV_R8(r, 0), DKV_R8(r, 8)::"memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
#undef DKV_R8
#undef DKV_O8
#undef DKV_I8

// ----------------------------------------------------------------------------- small helpers

// The angle of position pos for a pair of `turns` per position: the product
// modulo 2^64 is the angle modulo one turn, its top 32 bits as a signed number
// the angle in [-1/2, 1/2) turns; in radians, off by 2^-24 of its value in fp32.
__device__ __forceinline__ float turn_angle(int pos, uint64_t turns) {
  const int32_t frac = static_cast<int32_t>((static_cast<uint64_t>(static_cast<uint32_t>(pos)) * turns) >> 32);
  return static_cast<float>(frac) * 1.4629180792671596e-9f;   // 2 pi / 2^32
}
__device__ __forceinline__ void turn_cs(int pos, uint64_t turns, float& c, float& s) {
  __sincosf(turn_angle(pos, turns), &s, &c);
}

template <bool BF16>
__device__ __forceinline__ uint32_t narrow2(float x, float y) {
  if constexpr (BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

// The n lowest bits set, n clamped to [0, 32].
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? kFull : (1u << n) - 1u; }

// max(|a|, |b|) of fp16 pairs; a NaN is ignored.
__device__ __forceinline__ uint32_t hmax_abs2(uint32_t m, uint32_t v) {
  const uint32_t a = v & 0x7fff7fffu;
  const __half2 r = __hmax2(*reinterpret_cast<const __half2*>(&m), *reinterpret_cast<const __half2*>(&a));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ bool has_inf2(uint32_t m) { return (m & 0xffffu) == 0x7c00u || (m >> 16) == 0x7c00u; }

// A wait of the chunk kernel: bounded, and given up as soon as another role has.
__device__ __forceinline__ bool chunk_wait(uint64_t* bar, uint32_t parity, ChunkTail& t, int32_t* status) {
  const uint32_t b = smem_u32(bar);
  if (mbar_try_wait(b, parity)) return true;
  const unsigned long long t0 = global_ns();
  for (unsigned i = 1;; ++i) {
    if (mbar_try_wait(b, parity)) return true;
    if ((i & 63u) == 0) {
      if (*reinterpret_cast<volatile int32_t*>(&t.broken)) return false;
      if (global_ns() - t0 > kWaitLimitNs) {
        *reinterpret_cast<volatile int32_t*>(&t.broken) = 1;
        atomicOr(status, kStatusTimeout);
        return false;
      }
    }
  }
}

// Ring position: stage and the parity of its current use.
struct Ring {
  int stage = 0;
  uint32_t parity = 0;
  template <int N>
  __device__ __forceinline__ void next() {
    if (++stage == N) {
      stage = 0;
      parity ^= 1u;
    }
  }
};

// ----------------------------------------------------------------------------- the kernel

// DUAL: a CTA takes 128 rows instead of 256.  Both softmax groups and both halves
// of TMEM then serve the same rows: the first has the even K/V tiles, the second
// the odd ones, and their results are joined at the end.  A group's tile goes
// through product, softmax and product in turn, so with one group alone the
// tensor core and the copies idle most of the time (8 rows on four 64k contexts:
// 243 us, 201 with two).
template <int D, bool BF16, bool ROPE, bool DUAL>
__global__ void __launch_bounds__(kChunkThreads, 1)
    chunk_kernel(const ChunkParams p, const __grid_constant__ ChunkMaps maps) {
  using C = ChunkShape<D>;
  constexpr int kRows = DUAL ? 128 : 256;    // rows of a CTA
  constexpr int kStagesV = C::kStagesV + (DUAL ? C::kMoreV : 0);
  constexpr bool kOpBf16 = BF16 && !ROPE;    // type of the Q K^T operands
  extern __shared__ __align__(1024) char chunk_smem[];
  char* const sq = chunk_smem;
  // V's stages follow the two Q tiles, the second of which is one more of them under DUAL
  char* const sv = sq + (DUAL && C::kMoreV ? 1 : 2) * C::kTile;
  char* const sk = sv + kStagesV * C::kTile;
  ChunkTail& t = *reinterpret_cast<ChunkTail*>(sk + C::kStagesK * C::kTile);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(kFull, tid >> 5, 0);   // warp-uniform, and known to be

  if (smem_u32(chunk_smem) & 1023u) {   // the swizzled tiles need a 1024-byte aligned base
    if (tid == 0) atomicOr(p.status, kStatusLayout);
    return;
  }

  // ---- which rows: CTA = (row tile, kv head, split).  CTAs start in order, so
  // the long ones come first: of up to 32 sequences the one that ends last (in
  // tokens) first, and of a sequence its last row tile first, as that sees the
  // most tokens.  More sequences are taken from the last one on.
  const int unit = p.div_split.div(static_cast<int>(blockIdx.x));
  const int split = static_cast<int>(blockIdx.x) - unit * p.nsplit;
  const int slot = p.div_hkv.div(unit);
  const int h = unit - slot * p.hkv;
  if (warp == 0) {
    // 32 sequences at a time, each lane with its rows and length in hand
    int before = 0, fb = -1, ft = 0, fq = 0, fn = 0, fl = 0;
    for (int b0 = p.batch - 1; b0 >= 0 && fb < 0; b0 -= 32) {
      const int b = b0 - lane;
      const int q = b >= 0 ? p.q_start[b] : 0;
      const int n = b >= 0 ? p.q_start[b + 1] - q : 0;
      const int len = b >= 0 ? p.seq_lens[b] : 0;
      const bool rank = p.batch <= 32;
      const int tiles =
          n > 0 ? static_cast<int>(((static_cast<long long>(n) << p.group_shift) + kRows - 1) / kRows) : 0;
      int inc = tiles;
      if (rank) {   // row tiles of this sequence and of those before it in the order
        const unsigned key = static_cast<unsigned>(max(len, 0)) + static_cast<unsigned>(max(n, 0));
        for (int o = 0; o < p.batch; ++o) {
          const unsigned other = __shfl_sync(kFull, key, o);
          const int more = __shfl_sync(kFull, tiles, o);
          if (other > key || (other == key && o < lane)) inc += more;
        }
      } else {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int u = __shfl_up_sync(kFull, inc, o);
          if (lane >= o) inc += u;
        }
      }
      const unsigned hit = __ballot_sync(kFull, slot < before + inc && slot >= before + inc - tiles);
      if (hit) {
        const int src = __ffs(hit) - 1;
        fb = b0 - src;
        ft = __shfl_sync(kFull, before + inc - 1 - slot, src);
        fq = __shfl_sync(kFull, q, src);
        fn = __shfl_sync(kFull, n, src);
        fl = __shfl_sync(kFull, len, src);
      }
      before += __shfl_sync(kFull, inc, 31);
    }
    if (lane == 0) {
      t.b = fb;
      t.tile = ft;
      t.q0 = fq;
      t.n = fn;
      t.len = fl;
      t.bad_lo = INT32_MAX;
      t.bad_hi = -1;
      for (int i = 0; i < 8; ++i) t.bad_rows[i] = 0;
      t.broken = 0;
    }
  } else if (warp == 1 && lane == 0) {
    for (int i = 0; i < 4; ++i) {
      mbar_init(smem_u32(&t.k_full[i]), 1);
      mbar_init(smem_u32(&t.k_ready[i]), 4);
      mbar_init(smem_u32(&t.k_free[i]), 1);
      mbar_init(smem_u32(&t.v_full[i]), 1);
      mbar_init(smem_u32(&t.v_free[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&t.q_ready[i]), 4);
      mbar_init(smem_u32(&t.s_full[i]), 1);
      mbar_init(smem_u32(&t.p_ready[i]), 4);
    }
    mbar_init(smem_u32(&t.done), 1);
    mbar_init_fence();
    t.tmem = 0;
  }
  __syncthreads();
  const int b = t.b;
  if (b < 0) return;
  const int q0 = t.q0, n = t.n, L = t.len;
  const int row0 = t.tile * kRows;
  const int rows = min((n << p.group_shift) - row0, kRows);
  const bool bad_len = L < 0 || L > p.max_len - n;

  // ---- which tokens: [0, sk_end) and [lo_min, hi_max), in tiles of 128
  const int hi_min = L + (row0 >> p.group_shift) + p.self;
  const int hi_max = L + ((row0 + rows - 1) >> p.group_shift) + p.self;
  const int lo_min = p.window ? max(0, hi_min - p.window) : 0;
  const int sk_end = min(p.sinks, lo_min);
  const int tb = lo_min / kChunkTokens;
  const int na = min((sk_end + kChunkTokens - 1) / kChunkTokens, tb);
  const int total = bad_len ? 0 : na + max(0, (hi_max + kChunkTokens - 1) / kChunkTokens - tb);
  const int per = (total + p.nsplit - 1) / p.nsplit;
  const int j0 = min(split * per, total);
  const int nt = min(j0 + per, total) - j0;
  auto tile_pos = [&](int j) { return (j0 + j < na ? j0 + j : tb + j0 + j - na) * kChunkTokens; };

  // this thread's row (softmax warps)
  const int m = (warp >> 2) - 2;                 // softmax: group 0 or 1
  const int row_m = row0 + (DUAL ? 0 : 128 * m); // first row of the group's row tile
  const int idx = row_m + (tid & 127);
  const int tok = idx >> p.group_shift;
  const int head = (h << p.group_shift) + (idx & ((1 << p.group_shift) - 1));
  // tokens whose rows exist: all n, unless q_start names rows outside the buffers
  const int n_rows = q0 < 0 || q0 > p.total_rows ? 0 : min(n, p.total_rows - q0);
  const bool live = m >= 0 && tok < n_rows;
  auto place_of_row = [&] { return static_cast<size_t>(live ? q0 + tok : 0) * p.hq + head; };   // of all rows' heads

  // this thread's row with one value: zero (an empty split), or NaN
  auto one_value = [&](bool nan) {
    if (!live) return;
    const size_t at = place_of_row();
    if (p.nsplit == 1) {
      const uint32_t f = nan ? 0x7fff7fffu : 0u;
      for (int c = 0; c < D / 8; ++c) reinterpret_cast<uint4*>(p.out + at * D)[c] = make_uint4(f, f, f, f);
    } else {
      const float f = nan ? __int_as_float(0x7fc00000) : 0.f;
      float4* o = reinterpret_cast<float4*>(p.part_o + (at * p.nsplit + split) * D);
      for (int c = 0; c < D / 4; ++c) o[c] = make_float4(f, f, f, f);
      p.part_lse[at * p.nsplit + split] = nan ? f : -INFINITY;
    }
  };
  if (nt == 0 || p.id_total == 0) {
    // no token to see: zero rows; an invalid length, or no pool to look in: NaN rows
    const bool nan = bad_len || (p.id_total == 0 && total > 0);
    if (nan && tid == 0) atomicOr(p.status, bad_len ? 2 : 1);
    one_value(nan);
    return;
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the joining kernel waits for the results itself
  // TMEM columns: S (and P over its first half) of row tile i at 128 i, O at 256 + D i.
  // The issuing warp allocates them; the others learn the address with their first S.

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
    if (warp == 0 || warp == 2) {
      // ------------------------------------------------------------ copies
      // A warp each for K and V, so that neither waits for the other's stages (K
      // runs ahead, as it is rotated before its product: with one warp for both
      // the rotated key tile came last and set the pace, 4280 cycles a tile).
      // The block ids of the next tile are read while this one's stage is waited for.
      const bool is_v = warp == 2;
      const int stages = is_v ? kStagesV : C::kStagesK;
      uint64_t* const full = is_v ? t.v_full : t.k_full;
      uint64_t* const free_ = is_v ? t.v_free : t.k_free;
      const CUtensorMap* const dev_map = is_v ? &maps.v_dev : &maps.k_dev;
      const CUtensorMap* const host_map = is_v ? &maps.v_host : &maps.k_host;
      const int nbox = kChunkTokens / p.box;
      const uint32_t box_bytes = static_cast<uint32_t>(p.box) * 128;
      const int32_t* trow = p.table + static_cast<size_t>(b) * p.stride;
      auto read_id = [&](int j) {   // of the run of rows that this lane copies; -2: nothing there to see
        if (lane >= nbox || j >= nt) return -2;
        const int t0 = tile_pos(j) + lane * p.box;
        return t0 < hi_max && (t0 + p.box > lo_min || t0 < sk_end) ? max(trow[p.div_bs.div(t0)], -1) : -2;
      };
      int stage = 0;
      uint32_t parity = 0;
      int next_id = read_id(0);
      for (int j = 0; j < nt; ++j) {
        const int id = next_id;
        next_id = read_id(j + 1);
        // the rows to copy: in this pool, or outside it, which fills with zeros
        int y = p.oob_row;
        bool host = p.oob_host != 0;
        if (id >= 0 && id < p.id_total) {
          const int t0 = tile_pos(j) + lane * p.box;
          host = id < p.host_split;
          y = ((host ? id : id - p.host_split) * p.hkv + h) * p.block_size + (t0 - p.div_bs.div(t0) * p.block_size);
        } else if (id != -2) {   // the run's tokens that some row sees
          const int t0 = tile_pos(j) + lane * p.box, t1 = t0 + p.box;
          atomicMin(&t.bad_lo, t0 < sk_end ? t0 : max(t0, lo_min));
          atomicMax(&t.bad_hi, (t1 > lo_min ? min(t1, hi_max) : min(t1, sk_end)) - 1);
          atomicOr(p.status, 1);
        }
        __syncwarp();
        if (!__all_sync(kFull, chunk_wait(&free_[stage], parity ^ 1u, t, p.status))) break;
        const uint32_t bar = smem_u32(&full[stage]);
        if (lane == 0) mbar_arrive_expect_tx(bar, C::kTile);
        __syncwarp();
        if (lane < nbox && !(p.stall_first_copy && blockIdx.x == 0 && j == 0 && !is_v)) {
          const uint32_t dst = smem_u32((is_v ? sv : sk) + stage * C::kTile) + lane * box_bytes;
#pragma unroll
          for (int x = 0; x < C::kSub; ++x) tma_load_2d(dst + x * kSubTile, host ? host_map : dev_map, 64 * x, y, bar);
        }
        if (++stage == stages) {
          stage = 0;
          parity ^= 1u;
        }
      }
      // copies still in flight after a wait ran out get a bounded time to land
      // before the block's shared memory is released (a barrier's completed
      // phase is the parity before the next use's)
      if (*reinterpret_cast<volatile int32_t*>(&t.broken)) {
        for (int i = 0; i < stages; ++i) {
          mbar_wait_bounded(smem_u32(&full[stage]), parity ^ 1u);
          if (++stage == stages) {
            stage = 0;
            parity ^= 1u;
          }
        }
      }
    } else if (warp == 1) {
      // ------------------------------------------------------------ matrix products
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&t.tmem))
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
      __syncwarp();
      constexpr uint32_t kIdQK = umma_idesc(128, kChunkTokens, kOpBf16, false);
      constexpr uint32_t kIdPV = umma_idesc(128, D, BF16, true);
      const uint32_t on = lane == 0;
      const int tiles = __shfl_sync(kFull, nt, 0);
      const uint32_t tm = __shfl_sync(kFull, *reinterpret_cast<volatile uint32_t*>(&t.tmem), 0);
      const uint32_t q_low = desc_low(smem_u32(sq), 16), k_low = desc_low(smem_u32(sk), 16);
      const uint32_t v_low = desc_low(smem_u32(sv), kSubTile);
      // S of group g = Q K^T, both K-major
      auto qk = [&](int g, uint32_t a, int stage) {
        const uint32_t k = k_low + stage * (C::kTile >> 4);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const uint32_t o = ((i >> 2) * kSubTile + (i & 3) * 32) >> 4;
          umma_ss(tm + 128 * g, a + o, k + o, kIdQK, i > 0, on);
        }
        umma_commit(smem_u32(&t.s_full[g]), on);
      };
      // O of group g += P V: V is N-major, 64-column blocks kSubTile apart
      auto pv = [&](int g, uint32_t v, bool acc) {
#pragma unroll
        for (int i = 0; i < kChunkTokens / 16; ++i)
          umma_ts(tm + 256 + D * g, tm + 128 * g + 8 * i, v + i * (2048 >> 4), kIdPV, acc || i > 0, on);
      };
      // V rows that no row of the CTA sees hold anything: their weights are 0, but
      // 0 * NaN is not, so they are zeroed.  Here, as this warp waits for every use
      // of V's stages in turn; the rotating warps, which run ahead, cannot tell a
      // stage's use from the one two before it by the barrier's parity.
      auto clear_unseen = [&](int j, int stage) {
        const int p0 = tile_pos(j);
        if (p0 + kChunkTokens <= hi_max && (p0 >= lo_min || p0 + kChunkTokens <= sk_end)) return;
#pragma unroll 1
        for (int r = lane; r < kChunkTokens; r += 32) {
          const int tt = p0 + r;
          if (tt < hi_max && (tt >= lo_min || tt < sk_end)) continue;
          char* const v = sv + stage * C::kTile + r * 128;
#pragma unroll
          for (int e = 0; e < 8 * C::kSub; ++e)
            *reinterpret_cast<uint4*>(v + (e >> 3) * kSubTile + (e & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async();
        __syncwarp();
      };
      Ring rk, rv;
      bool ok = chunk_wait(&t.q_ready[0], 0, t, p.status);
      const int row_tiles = __shfl_sync(kFull, rows > 128 ? 2 : 1, 0);
      if (!DUAL && row_tiles == 2) ok = ok && chunk_wait(&t.q_ready[1], 0, t, p.status);
      ok = ok && chunk_wait(&t.k_ready[0], 0, t, p.status);
      ok = __all_sync(kFull, ok);
      if (!DUAL && ok) {
        // two row tiles (or one, if no rows are left for the second): each K/V tile
        // is group 0's turn, then group 1's; a group's next S is issued right
        // behind its O
        tmem_fence_after();
        qk(0, q_low, 0);
        if (row_tiles == 2) qk(1, q_low + (C::kTile >> 4), 0);
        umma_commit(smem_u32(&t.k_free[0]), on);
        rk.next<C::kStagesK>();
        for (int j = 0; j < tiles; ++j) {
          const bool more = j + 1 < tiles;
          ok = __all_sync(kFull, chunk_wait(&t.v_full[rv.stage], rv.parity, t, p.status));
          if (ok) clear_unseen(j, rv.stage);
#pragma unroll 1   // unrolled, its operands no longer fit in uniform registers: 4% slower
          for (int g = 0; g < row_tiles && ok; ++g) {
            ok = chunk_wait(&t.p_ready[g], j & 1, t, p.status);
            if (g == 0 && more) ok = ok && chunk_wait(&t.k_ready[rk.stage], rk.parity, t, p.status);
            if (!(ok = __all_sync(kFull, ok))) break;
            tmem_fence_after();
            pv(g, v_low + rv.stage * (C::kTile >> 4), j > 0);
            if (g == row_tiles - 1) umma_commit(smem_u32(&t.v_free[rv.stage]), on);
            if (more) {
              qk(g, q_low + g * (C::kTile >> 4), rk.stage);
              if (g == row_tiles - 1) umma_commit(smem_u32(&t.k_free[rk.stage]), on);
            }
            __syncwarp();
          }
          if (!ok) break;
          rv.next<kStagesV>();
          rk.next<C::kStagesK>();
        }
      } else if (DUAL && ok) {
        // one row tile: K/V tile j is group (j mod 2)'s turn, tile j + 2 its next
        auto next_s = [&](int j) {
          if (!__all_sync(kFull, chunk_wait(&t.k_ready[rk.stage], rk.parity, t, p.status))) return false;
          tmem_fence_after();
          qk(j & 1, q_low, rk.stage);
          umma_commit(smem_u32(&t.k_free[rk.stage]), on);
          rk.next<C::kStagesK>();
          return true;
        };
        ok = next_s(0) && (tiles == 1 || next_s(1));
#pragma unroll 1
        for (int j = 0; j < tiles && ok; ++j) {
          ok = chunk_wait(&t.v_full[rv.stage], rv.parity, t, p.status);
          ok = ok && chunk_wait(&t.p_ready[j & 1], (j >> 1) & 1, t, p.status);
          if (!(ok = __all_sync(kFull, ok))) break;
          clear_unseen(j, rv.stage);
          tmem_fence_after();
          pv(j & 1, v_low + rv.stage * (C::kTile >> 4), j > 1);
          umma_commit(smem_u32(&t.v_free[rv.stage]), on);
          rv.next<kStagesV>();
          if (j + 2 < tiles) ok = next_s(j + 2);
          __syncwarp();
        }
      }
      // also after a wait ran out: what was issued completes before TMEM is given back
      umma_commit(smem_u32(&t.done), on);
      mbar_wait_bounded(smem_u32(&t.done), 0);
    }
  } else if (warp < 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRotate));
    // -------------------------------------------------------------- rotation of K, in place
    // A thread owns 8 consecutive pairs (one 16-byte chunk of each half) of
    // every kStep-th row; its cos / sin advance kStep positions from row to
    // row, across tiles too while positions continue, with a fresh seed at
    // least every kRopeChain tiles (64 fp32 steps at most, 2^-18).
    constexpr int kChunks = D / 16;             // chunks of a half row
    constexpr int kStep = 128 / kChunks;
    const int r = tid - 128;
    const int c = r % kChunks, rr = r / kChunks;
    float2 E[4], F[4], Cc[4], Sc[4];
    if constexpr (ROPE) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // to the last bit, as the recurrence repeats their error
        sincosf(turn_angle(kStep, p.turns[8 * c + 2 * i]), &F[i].x, &E[i].x);
        sincosf(turn_angle(kStep, p.turns[8 * c + 2 * i + 1]), &F[i].y, &E[i].y);
      }
    }
    int next_pos = -1, chain = 0;
    Ring rk;
    for (int j = 0; j < nt; ++j) {
      const int p0 = tile_pos(j);
      const bool edge = p0 + kChunkTokens > hi_max || (p0 < lo_min && p0 + kChunkTokens > sk_end);
      if constexpr (ROPE) {
        if (p0 != next_pos || chain == kRopeChain) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            turn_cs(p0 + rr, p.turns[8 * c + 2 * i], Cc[i].x, Sc[i].x);
            turn_cs(p0 + rr, p.turns[8 * c + 2 * i + 1], Cc[i].y, Sc[i].y);
          }
          chain = 0;
        }
        ++chain;
        next_pos = p0 + kChunkTokens;
      }
      if (!__all_sync(kFull, chunk_wait(&t.k_full[rk.stage], rk.parity, t, p.status))) break;
      if constexpr (ROPE) {
        char* const k = sk + rk.stage * C::kTile;
        float mx = 0.f;
#pragma unroll
        for (int i = 0; i < 128 / kStep; ++i) {
          const int rw = rr + kStep * i;
          uint4* const px = reinterpret_cast<uint4*>(k + rw * 128 + ((c ^ (rw & 7)) << 4));
          uint4* const py = D == 128 ? px + kSubTile / 16
                                     : reinterpret_cast<uint4*>(k + rw * 128 + (((c + 4) ^ (rw & 7)) << 4));
          const uint4 ux = *px, uy = *py;
          float2 X[4] = {widen2<BF16>(ux.x), widen2<BF16>(ux.y), widen2<BF16>(ux.z), widen2<BF16>(ux.w)};
          float2 Y[4] = {widen2<BF16>(uy.x), widen2<BF16>(uy.y), widen2<BF16>(uy.z), widen2<BF16>(uy.w)};
          rope_rotate_advance<4>(X, Y, Cc, Sc, E, F);
          uint32_t o[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            o[e] = narrow2<false>(X[e].x, X[e].y);
            o[4 + e] = narrow2<false>(Y[e].x, Y[e].y);
          }
          // range: only of tokens that some row sees, the others hold anything
          const int tt = p0 + rw;
          if (!edge || (tt < hi_max && (tt >= lo_min || tt < sk_end))) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              mx = fmaxf(mx, fmaxf(fabsf(X[e].x), fabsf(X[e].y)));
              mx = fmaxf(mx, fmaxf(fabsf(Y[e].x), fabsf(Y[e].y)));
            }
          }
          *px = make_uint4(o[0], o[1], o[2], o[3]);
          *py = make_uint4(o[4], o[5], o[6], o[7]);
        }
        if (mx > kMostOperand) {   // rare: which of this thread's rows hold an infinity now
#pragma unroll 1
          for (int rw = rr; rw < kChunkTokens; rw += kStep) {
            const int tt = p0 + rw;
            if (tt >= hi_max || (tt < lo_min && tt >= sk_end)) continue;
            const char* const at = k + rw * 128;
            const uint4 ux = *reinterpret_cast<const uint4*>(at + ((c ^ (rw & 7)) << 4));
            const uint4 uy = D == 128 ? *reinterpret_cast<const uint4*>(at + kSubTile + ((c ^ (rw & 7)) << 4))
                                      : *reinterpret_cast<const uint4*>(at + (((c + 4) ^ (rw & 7)) << 4));
            const uint32_t mu = hmax_abs2(hmax_abs2(hmax_abs2(hmax_abs2(0u, ux.x), ux.y), ux.z), ux.w);
            if (!has_inf2(hmax_abs2(hmax_abs2(hmax_abs2(hmax_abs2(mu, uy.x), uy.y), uy.z), uy.w))) continue;
            atomicMin(&t.bad_lo, tt);
            atomicMax(&t.bad_hi, tt);
            atomicOr(p.status, kStatusRange);
          }
        }
      }
      fence_proxy_async();   // the products read what was written here
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&t.k_ready[rk.stage]));
      rk.next<C::kStagesK>();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    // -------------------------------------------------------------- softmax, a thread per row
    if (DUAL || m == 0 || rows > 128) {
      // The warp's 32 queries: rotated, to their place in the swizzled tile; rows
      // past the end are zero.  A lane takes 8 pairs of every kPer-th row (one
      // 16-byte chunk of each half), so that a load covers whole lines, and its
      // cos / sin advance from row to row as those of the keys do.
      const int pos = L + tok;
      if (!DUAL || m == 0) {
        constexpr int kC = D / 16, kPer = 32 / kC;
        const int c = lane % kC, r0 = 32 * (warp & 3) + lane / kC;
        const int first_row = row_m + r0;
        const int step = kPer >> p.group_shift;
        uint4 ux[kC], uy[kC];   // every load in flight at once: the first product waits for the last
#pragma unroll
        for (int i = 0; i < kC; ++i) {
          const int id = first_row + kPer * i, tk = id >> p.group_shift;
          ux[i] = uy[i] = make_uint4(0u, 0u, 0u, 0u);
          if (tk < n_rows) {
            const uint16_t* const src = p.q + (q0 + tk) * p.q_stride +
                                        ((h << p.group_shift) + (id & ((1 << p.group_shift) - 1))) * D + 8 * c;
            ux[i] = *reinterpret_cast<const uint4*>(src);
            uy[i] = *reinterpret_cast<const uint4*>(src + D / 2);
          }
        }
        float2 E[4], F[4], Cc[4], Sc[4];
        if constexpr (ROPE) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint64_t t0 = p.turns[8 * c + 2 * i], t1 = p.turns[8 * c + 2 * i + 1];
            turn_cs(L + (first_row >> p.group_shift), t0, Cc[i].x, Sc[i].x);
            turn_cs(L + (first_row >> p.group_shift), t1, Cc[i].y, Sc[i].y);
            turn_cs(step, t0, E[i].x, F[i].x);
            turn_cs(step, t1, E[i].y, F[i].y);
          }
        }
        char* const dst = sq + m * C::kTile;
#pragma unroll
        for (int i = 0; i < kC; ++i) {
          const int r = r0 + kPer * i;
          if constexpr (ROPE) {
            float2 X[4] = {widen2<BF16>(ux[i].x), widen2<BF16>(ux[i].y), widen2<BF16>(ux[i].z), widen2<BF16>(ux[i].w)};
            float2 Y[4] = {widen2<BF16>(uy[i].x), widen2<BF16>(uy[i].y), widen2<BF16>(uy[i].z), widen2<BF16>(uy[i].w)};
            rope_rotate_advance<4>(X, Y, Cc, Sc, E, F);
            uint32_t o[8], mx = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              o[e] = narrow2<false>(X[e].x, X[e].y);
              o[4 + e] = narrow2<false>(Y[e].x, Y[e].y);
              mx = hmax_abs2(hmax_abs2(mx, o[e]), o[4 + e]);
            }
            // lanes [kC g, kC (g + 1)) hold row kPer i + g of the warp's 32; in shared
            // memory, as a register held over the walk cost 3% with few rows
            const unsigned inf = __ballot_sync(kFull, has_inf2(mx));
            if (inf && lane / kPer == i && (inf >> (kC * (lane % kPer)) & ((1u << kC) - 1u)) != 0) {
              atomicOr(&t.bad_rows[warp - 8], 1u << lane);
              atomicOr(p.status, kStatusRange);
            }
            ux[i] = make_uint4(o[0], o[1], o[2], o[3]);
            uy[i] = make_uint4(o[4], o[5], o[6], o[7]);
          }
          *reinterpret_cast<uint4*>(dst + r * 128 + ((c ^ (r & 7)) << 4)) = ux[i];
          if constexpr (D == 128) *reinterpret_cast<uint4*>(dst + kSubTile + r * 128 + ((c ^ (r & 7)) << 4)) = uy[i];
          else *reinterpret_cast<uint4*>(dst + r * 128 + (((c + 4) ^ (r & 7)) << 4)) = uy[i];
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&t.q_ready[m]));
      }
      const int hi = live ? pos + p.self : 0;
      const int lo = p.window ? max(0, hi - p.window) : 0;
      // the row tile's tightest bounds: a K/V tile inside them needs no mask
      const int first = L + (row_m >> p.group_shift) + p.self;
      const int last = L + (min(row0 + rows, row_m + 128) - 1 >> p.group_shift) + p.self;
      const int lo_last = p.window ? max(0, last - p.window) : 0;
      const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
      uint32_t ts = 0, to = 0;
      float ref = -1e30f, sum = 0.f;
      bool ok = true;
      const int turns = DUAL ? (nt + 1 - m) >> 1 : nt;
      for (int j = 0; j < turns; ++j) {
        const int p0 = tile_pos(DUAL ? 2 * j + m : j);
        ok = __all_sync(kFull, chunk_wait(&t.s_full[m], j & 1, t, p.status));
        if (!ok) break;
        tmem_fence_after();
        if (j == 0) {
          const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&t.tmem);
          ts = tmem + lanes + 128 * m;
          to = tmem + lanes + 256 + D * m;
        }
        uint32_t s[4][32];
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_ld32(ts + 32 * i, s[i]);
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_ld_wait(s[i]);
        if (p0 + kChunkTokens > first || (p0 < lo_last && p0 + kChunkTokens > p.sinks)) {
          // one bit per token, so that a token costs a test and a select
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c = p0 + 32 * i;
            const uint32_t seen = low_bits(hi - c) & (~low_bits(lo - c) | low_bits(p.sinks - c));
#pragma unroll
            for (int e = 0; e < 32; ++e) s[i][e] = (seen >> e) & 1u ? s[i][e] : 0xff800000u;   // -inf
          }
        }
        float mx[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          mx[i] = __uint_as_float(s[i][0]);
#pragma unroll
          for (int e = 1; e < 32; ++e) mx[i] = fmaxf(mx[i], __uint_as_float(s[i][e]));
        }
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.qscale;
        // a higher reference, once some score exceeds the old one by 2^kWeightLag
        const bool raise = top > ref + kWeightLag<BF16>;
        if (__any_sync(kFull, raise)) {
          const float now = raise ? top : ref;
          const float a = ex2(ref - now);
          ref = now;
          sum *= a;
          if (j > 0) {   // the product that last added to O has completed: it precedes this S
#pragma unroll 1
            for (int i = 0; i < D / 16; ++i) {
              uint32_t o[16];
              tmem_ld16(to + 16 * i, o);
              tmem_ld_wait(o);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * a);
              tmem_st16(to + 16 * i, o);
            }
          }
        }
        const float2 sc = f2(p.qscale), off = f2(kWeightBias<BF16> - ref);
        float2 acc[2] = {f2(0.f), f2(0.f)};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // in three sweeps, so that 32 exponentials are in flight at a time
          float2 y[16];
#pragma unroll
          for (int e = 0; e < 16; ++e)
            y[e] = __ffma2_rn(make_float2(__uint_as_float(s[i][2 * e]), __uint_as_float(s[i][2 * e + 1])), sc, off);
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            y[e] = make_float2(ex2(y[e].x), ex2(y[e].y));
          }
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            acc[e & 1] = __fadd2_rn(acc[e & 1], y[e]);
            w[e] = narrow2<BF16>(y[e].x, y[e].y);
          }
          tmem_st16(ts + 16 * i, w);
        }
        tmem_st_wait();
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&t.p_ready[m]));
        sum += (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
      }
      ok = ok && __all_sync(kFull, chunk_wait(&t.done, 0, t, p.status));
      tmem_fence_after();
      // ---- the row's result
      // A thread's row goes through the block's shared memory, which nothing reads
      // any more, so that the warp writes whole lines: row by row from the
      // threads themselves, a CTA's 256 rows of fp32 took 10,600 cycles.
      char* const buf = chunk_smem + (warp - 8) * (32 * D * 4);
      float2* const other = reinterpret_cast<float2*>(chunk_smem + 8 * (32 * D * 4));   // the second group's (ref, sum)
      float mine = 1.f, theirs = 0.f;   // factors of the two groups' O
      if (DUAL) {
        if (m == 1) {
          if (ok && turns > 0) {
#pragma unroll 1
            for (int i = 0; i < D / 32; ++i) {
              uint32_t o[32];
              tmem_ld32(to + 32 * i, o);
              tmem_ld_wait(o);
#pragma unroll
              for (int e = 0; e < 8; ++e)
                *reinterpret_cast<uint4*>(buf + lane * (D * 4) + (((8 * i + e) ^ (lane & 7)) << 4)) =
                    make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
            }
            other[tid & 127] = make_float2(ref, sum);
          }
        }
        asm volatile("bar.sync 1, 256;" ::: "memory");   // both groups come here, after a wait that ran out too
        if (m == 0 && nt > 1 && ok) {
          const float2 o = other[tid & 127];
          const float top = fmaxf(ref, o.x);
          mine = ex2(ref - top);
          theirs = ex2(o.x - top);
          sum = sum * mine + o.y * theirs;
          ref = top;
        }
      }
      ok = ok && *reinterpret_cast<volatile int32_t*>(&t.broken) == 0;
      // NaN: the row sees an invalid token (of several, the first and the last are known)
      const int bad_lo = *reinterpret_cast<volatile int32_t*>(&t.bad_lo);
      const int bad_hi = *reinterpret_cast<volatile int32_t*>(&t.bad_hi);
      const uint32_t bad_rows = *reinterpret_cast<volatile uint32_t*>(&t.bad_rows[warp - 8]);
      const bool nan = !ok || (bad_rows >> lane & 1u) || (hi > bad_lo && (lo <= bad_hi || bad_lo < p.sinks));
      const float inv = nan ? __int_as_float(0x7fc00000) : (sum == 0.f ? 0.f : 1.f / sum);
      auto flush = [&](auto bytes, auto&& place) {   // the warp's 32 rows of `bytes` bytes to place(row of the warp)
        constexpr int kRow = decltype(bytes)::value, kC = kRow / 16, kPer = 32 / kC;
        __syncwarp();
#pragma unroll 4
        for (int i = 0; i < kC; ++i) {
          const int r = kPer * i + lane / kC, c = lane % kC;
          const int id = row_m + 32 * (warp & 3) + r, tk = id >> p.group_shift;
          const int hd = (h << p.group_shift) + (id & ((1 << p.group_shift) - 1));
          if (tk < n_rows)
            reinterpret_cast<uint4*>(place(static_cast<size_t>(q0 + tk) * p.hq + hd))[c] =
                *reinterpret_cast<const uint4*>(buf + r * kRow + ((c ^ (r & 7)) << 4));
        }
      };
      const bool writes = !DUAL || m == 0;
      if (ok && writes) {
#pragma unroll 1
        for (int i = 0; i < D / 32; ++i) {
          uint32_t o[32];
          tmem_ld32(to + 32 * i, o);
          tmem_ld_wait(o);
          if (DUAL && nt > 1) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float4 x = *reinterpret_cast<const float4*>(buf + 4 * (32 * D * 4) + lane * (D * 4) +
                                                                 (((8 * i + e) ^ (lane & 7)) << 4));
              o[4 * e] = __float_as_uint(__uint_as_float(o[4 * e]) * mine + x.x * theirs);
              o[4 * e + 1] = __float_as_uint(__uint_as_float(o[4 * e + 1]) * mine + x.y * theirs);
              o[4 * e + 2] = __float_as_uint(__uint_as_float(o[4 * e + 2]) * mine + x.z * theirs);
              o[4 * e + 3] = __float_as_uint(__uint_as_float(o[4 * e + 3]) * mine + x.w * theirs);
            }
          }
          if (p.nsplit == 1) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t w[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                w[k] = narrow2<BF16>(__uint_as_float(o[8 * e + 2 * k]) * inv,
                                     __uint_as_float(o[8 * e + 2 * k + 1]) * inv);
              *reinterpret_cast<uint4*>(buf + lane * (D * 2) + (((4 * i + e) ^ (lane & 7)) << 4)) =
                  make_uint4(w[0], w[1], w[2], w[3]);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              *reinterpret_cast<float4*>(buf + lane * (D * 4) + (((8 * i + e) ^ (lane & 7)) << 4)) =
                  make_float4(__uint_as_float(o[4 * e]) * inv, __uint_as_float(o[4 * e + 1]) * inv,
                              __uint_as_float(o[4 * e + 2]) * inv, __uint_as_float(o[4 * e + 3]) * inv);
          }
        }
      } else if (!ok) {   // a wait ran out: copies may still be landing in shared memory
        one_value(true);
      }
      if (ok && writes && p.nsplit == 1)
        flush(std::integral_constant<int, D * 2>{}, [&](size_t at) { return p.out + at * D; });
      if (ok && writes && p.nsplit > 1)
        flush(std::integral_constant<int, D * 4>{}, [&](size_t at) { return p.part_o + (at * p.nsplit + split) * D; });
      if (ok && writes && live && p.nsplit > 1)
        p.part_lse[place_of_row() * p.nsplit + split] =
            nan ? __int_as_float(0x7fc00000) : (sum == 0.f ? -INFINITY : ref - kWeightBias<BF16> + __log2f(sum));
    }
  }
  tmem_fence_before();
  __syncthreads();
  if (warp == 1) {
    tmem_fence_after();
    const uint32_t tmem = __shfl_sync(kFull, *reinterpret_cast<volatile uint32_t*>(&t.tmem), 0);
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
}

// ----------------------------------------------------------------------------- joining the splits

// One warp per (row, head): o = sum_i 2^(lse_i - top) o_i / sum_i 2^(lse_i - top).
// A NaN split makes the row NaN; a row whose splits are all empty is zero.
template <int D, bool BF16>
__global__ void __launch_bounds__(128) chunk_merge_kernel(const ChunkParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const long long w = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (w >= static_cast<long long>(min(p.total_rows, p.q_start[p.batch])) * p.hq) return;
  const float* const lse = p.part_lse + w * p.nsplit;
  const float* const o = p.part_o + w * p.nsplit * D;
  float top = -INFINITY;
  bool nan = false;
  for (int i = lane; i < p.nsplit; i += 32) {
    const float l = lse[i];
    nan |= isnan(l);
    top = fmaxf(top, l);
  }
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, k));
  nan = __any_sync(kFull, nan);
  float z = 0.f, acc[D / 32];
#pragma unroll
  for (int k = 0; k < D / 32; ++k) acc[k] = 0.f;
  if (top != -INFINITY) {
    for (int i = 0; i < p.nsplit; ++i) {
      const float f = ex2(lse[i] - top);
      z += f;
#pragma unroll
      for (int k = 0; k < D / 64; ++k) {
        const float2 x = *reinterpret_cast<const float2*>(o + static_cast<size_t>(i) * D + 64 * k + 2 * lane);
        acc[2 * k] = fmaf(f, x.x, acc[2 * k]);
        acc[2 * k + 1] = fmaf(f, x.y, acc[2 * k + 1]);
      }
    }
  }
  const float inv = nan ? __int_as_float(0x7fc00000) : (z > 0.f ? 1.f / z : 0.f);
#pragma unroll
  for (int k = 0; k < D / 64; ++k)
    *reinterpret_cast<uint32_t*>(p.out + w * D + 64 * k + 2 * lane) =
        narrow2<BF16>(acc[2 * k] * inv, acc[2 * k + 1] * inv);
}

}  // namespace dkv
