// dkv_chunk.cuh -- attention of a chunk of new tokens per sequence over the
// paged cache.
//
// Query i of sequence b sits at position L_b + i.  With hi = L_b + i + self it
// sees the cached tokens t < hi, and under a window only those with
// t >= hi - window or t < sinks:
//     s_t = scale * (R(L_b + i) q) . (R(t) k_t),   o = sum_t softmax(s)_t v_t.
// A row that sees nothing is zero.
#pragma once

#include "dkv_kernels.cuh"

namespace dkv {

struct ChunkParams {
  const uint16_t* q;          // [total_rows] of hq * D elements, q_stride elements apart
  uint16_t* out;              // [total_rows][hq][D]
  const uint16_t* k_host;     // block ids [0, host_split)
  const uint16_t* v_host;
  const uint16_t* k_dev;      // block ids [host_split, id_total)
  const uint16_t* v_dev;
  const int32_t* q_start;     // [batch + 1]
  const int32_t* seq_lens;    // [batch]
  const int32_t* table;       // [batch][stride]
  const uint64_t* turns;      // [D / 2] turns per position, 2^-64 turns
  int32_t* status;
  long long q_stride;
  int32_t total_rows, batch, stride, hq, hkv, block_size, host_split, id_total, max_len;
  int32_t window, sinks, self;
  float qscale;               // softmax scale * log2(e)
};

// cos / sin of position pos for a pair of `turns` per position: the product
// modulo 2^64 is the angle modulo one turn, its top 32 bits as a signed number
// the angle in [-1/2, 1/2) turns (off by 2^-24 of a half turn in fp32).
__device__ __forceinline__ void turn_cs(int pos, uint64_t turns, float& c, float& s) {
  const int32_t frac = static_cast<int32_t>((static_cast<uint64_t>(static_cast<uint32_t>(pos)) * turns) >> 32);
  __sincosf(static_cast<float>(frac) * 1.4629180792671596e-9f, &s, &c);   // 2 pi / 2^32
}

template <bool BF16>
__device__ __forceinline__ float widen1(uint16_t x) {
  return BF16 ? __uint_as_float(static_cast<uint32_t>(x) << 16) : __half2float(__ushort_as_half(x));
}
template <bool BF16>
__device__ __forceinline__ uint16_t narrow1(float x) {
  return BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(x)) : __half_as_ushort(__float2half_rn(x));
}

// One warp per (row, kv head): lane l holds the pairs l, l + 32 of the G
// queries and walks the visible tokens one by one with an online softmax.
template <int D, int G, bool BF16, bool ROPE>
__global__ void __launch_bounds__(128) chunk_row_kernel(const ChunkParams p) {
  constexpr int NP = D / 64;
  const long long w = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int row = static_cast<int>(w / p.hkv), h = static_cast<int>(w % p.hkv);
  if (row >= p.total_rows || row >= p.q_start[p.batch]) return;
  int b = 0, e = p.batch;
  while (e - b > 1) {
    const int mid = (b + e) >> 1;
    if (p.q_start[mid] <= row) b = mid;
    else e = mid;
  }
  const int i = row - p.q_start[b], n = p.q_start[b + 1] - p.q_start[b];
  const int L = p.seq_lens[b];
  bool poison = false;
  if (L < 0 || L > p.max_len - n) {
    if (lane == 0) atomicOr(p.status, 2);
    poison = true;
  }
  const int hi = poison ? 0 : L + i + p.self;
  const int lo = p.window ? max(0, hi - p.window) : 0;
  const int sk = min(p.sinks, lo);
  uint64_t tn[NP];
  float qx[G][NP], qy[G][NP], m[G], l[G], ox[G][NP], oy[G][NP];
#pragma unroll
  for (int j = 0; j < NP; ++j) {
    tn[j] = ROPE ? p.turns[lane + 32 * j] : 0;
    float c = 1.f, s = 0.f;
    if (ROPE) turn_cs(L + i, tn[j], c, s);
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const uint16_t* q = p.q + row * p.q_stride + (h * G + g) * D;
      const float x = widen1<BF16>(q[lane + 32 * j]), y = widen1<BF16>(q[lane + 32 * j + D / 2]);
      qx[g][j] = (x * c - y * s) * p.qscale;
      qy[g][j] = (y * c + x * s) * p.qscale;
      ox[g][j] = oy[g][j] = 0.f;
      m[g] = -1e30f;
      l[g] = 0.f;
    }
  }
  for (int t = sk > 0 ? 0 : lo; t < hi; t = t + 1 == sk ? lo : t + 1) {
    const int blk = t / p.block_size;
    const int id = p.table[static_cast<size_t>(b) * p.stride + blk];
    if (id < 0 || id >= p.id_total) {
      if (lane == 0) atomicOr(p.status, 1);
      poison = true;
      break;
    }
    const bool host = id < p.host_split;
    const size_t at = ((static_cast<size_t>(host ? id : id - p.host_split) * p.hkv + h) * p.block_size +
                       (t - blk * p.block_size)) * D;
    const uint16_t* k = (host ? p.k_host : p.k_dev) + at;
    const uint16_t* v = (host ? p.v_host : p.v_dev) + at;
    float sc[G];
#pragma unroll
    for (int g = 0; g < G; ++g) sc[g] = 0.f;
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      const float x = widen1<BF16>(k[lane + 32 * j]), y = widen1<BF16>(k[lane + 32 * j + D / 2]);
      float c = 1.f, s = 0.f;
      if (ROPE) turn_cs(t, tn[j], c, s);
      const float kx = x * c - y * s, ky = y * c + x * s;
#pragma unroll
      for (int g = 0; g < G; ++g) sc[g] = fmaf(qx[g][j], kx, fmaf(qy[g][j], ky, sc[g]));
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sc[g] += __shfl_xor_sync(kFull, sc[g], o);
      const float mx = fmaxf(m[g], sc[g]);
      const float a = exp2f(m[g] - mx), pw = exp2f(sc[g] - mx);
      m[g] = mx;
      l[g] = l[g] * a + pw;
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        ox[g][j] = ox[g][j] * a + pw * widen1<BF16>(v[lane + 32 * j]);
        oy[g][j] = oy[g][j] * a + pw * widen1<BF16>(v[lane + 32 * j + D / 2]);
      }
    }
  }
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const float inv = poison ? __int_as_float(0x7fc00000) : (l[g] > 0.f || isnan(l[g]) ? 1.f / l[g] : 0.f);
    uint16_t* o = p.out + (static_cast<size_t>(row) * p.hq + h * G + g) * D;
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      o[lane + 32 * j] = narrow1<BF16>(ox[g][j] * inv);
      o[lane + 32 * j + D / 2] = narrow1<BF16>(oy[g][j] * inv);
    }
  }
}

}  // namespace dkv
