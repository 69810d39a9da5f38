// dkv_tables.cuh -- the block tables and slot maps of a step, and the store of
// its K/V rows through them.
//
// extend_tables_kernel: sequence b holds ctx_b tokens in ceil(ctx_b / S)
// blocks and gets new_b more.  With the two prefix sums
//     q_start[b] = sum_{a < b} new_a,
//     first[b]   = sum_{a < b} ceil((ctx_a + new_a) / S) - ceil(ctx_a / S)
// every output is a function of its own index: the k-th new block of sequence
// b is the free list's entry (top - first[b] - k), and token i of sequence b,
// at position p = ctx_b + i, has slot id(p / S) * S + p mod S.  A CTA computes
// both sums for itself (the lengths are a few KB) and then takes its share of
// the table entries and slots, each of which looks its sequence up in shared
// memory, so one launch does all of it.
//
// store_kv_kernel: one warp moves (a part of) one token's K and V row to its
// slot, 4 chunks of K and of V in flight per lane.  Bound by HBM: 8192 rows of
// 32 heads (267 MB) in 45 us, 5.9 TB/s, 0.9 of a plain copy, with 256-byte
// pieces at random slots.  Streaming loads (evict first) took 47 us; streaming
// stores are as fast as these but would put the new rows out of L2, where the
// attention that follows reads them.
#pragma once

#include <stdint.h>

#include "dkv_kernels.cuh"

namespace dkv {

constexpr int kTableThreads = 512;
constexpr int kTableMaxBatch = 8192;        // both prefix sums and the lengths fit in 96 KB of shared memory
constexpr int kTableCtasPerSm = 3;
constexpr int kTableRun = 4;                // consecutive slots a thread maps at a time
constexpr int kStatusBadId = 1;             // DKV_STATUS_BAD_BLOCK_ID
constexpr int kStatusBadLen = 2;            // DKV_STATUS_BAD_SEQ_LEN
constexpr int kStatusNoBlocks = 16;         // DKV_STATUS_NO_FREE_BLOCKS
constexpr int kStatusNoSlots = 32;          // DKV_STATUS_NO_SLOTS

struct TableParams {
  const int32_t* seq_lens;    // [batch]
  const int32_t* new_lens;    // [batch]
  int32_t* table;             // [batch][stride]
  const int32_t* free_ids;    // [free_capacity], a stack: the top is entry free_count - 1
  const int32_t* free_count;  // [1]
  int32_t* free_left;         // [1], may be free_count itself
  int32_t* q_start;           // [batch + 1]
  int64_t* slot_map;          // [max_slots]
  int32_t* status;
  int32_t* done;              // CTAs finished; zero between launches
  int32_t batch, stride, block_size, max_len, free_capacity, max_slots;
  int32_t wide;               // slot_map is 16-byte aligned
  InvDiv div_bs;
};

__host__ __device__ constexpr size_t table_smem_bytes(int batch) {
  return 3 * sizeof(int32_t) * (static_cast<size_t>(batch) + 1);
}

// Component-wise sum, saturating at 2^30 + 1: more than max_slots or the free list may hold.
__device__ __forceinline__ uint2 sat_add(uint2 a, uint2 b) {
  constexpr uint32_t kTop = (1u << 30) + 1;
  return make_uint2(min(a.x + b.x, kTop), min(a.y + b.y, kTop));
}

// Largest b with start[b] <= x, for start[0] = 0 <= x < start[n].
__device__ __forceinline__ int owner_of(const int32_t* start, int n, int x) {
  int lo = 0, hi = n;   // start[lo] <= x < start[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kTableThreads, kTableCtasPerSm) extend_tables_kernel(const TableParams p) {
  constexpr int NW = kTableThreads / 32;
  extern __shared__ int32_t table_smem[];
  int32_t* const s_start = table_smem;                  // [batch + 1] q_start
  int32_t* const s_first = table_smem + p.batch + 1;    // [batch + 1] first new block
  int32_t* const s_ctx = s_first + p.batch + 1;         // [batch] tokens before the step
  __shared__ uint2 s_sum[NW];
  __shared__ int s_bad;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) s_bad = 0;
  const int top = *p.free_count;
  __syncthreads();

  // both prefix sums, kTableThreads sequences at a time, in 32 bits that
  // saturate above every count a call may reach (2^30)
  uint2 base = make_uint2(0u, 0u);
  for (int b0 = 0; b0 < p.batch; b0 += kTableThreads) {
    const int b = b0 + tid;
    uint2 mine = make_uint2(0u, 0u);
    if (b < p.batch) {
      const long long ctx = p.seq_lens[b], add = p.new_lens[b];
      s_ctx[b] = static_cast<int32_t>(ctx);
      if (ctx < 0 || add < 0 || ctx + add > p.max_len) {
        s_bad = 1;
      } else {
        mine.x = static_cast<uint32_t>(add);
        mine.y = static_cast<uint32_t>(p.div_bs.div(static_cast<int>(ctx + add) + p.block_size - 1) -
                                       p.div_bs.div(static_cast<int>(ctx) + p.block_size - 1));
      }
    }
    uint2 inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint2 u = make_uint2(__shfl_up_sync(kFull, inc.x, o), __shfl_up_sync(kFull, inc.y, o));
      if (lane >= o) inc = sat_add(inc, u);
    }
    if (lane == 31) s_sum[warp] = inc;
    __syncthreads();
    uint2 before = base, all = make_uint2(0u, 0u);
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const uint2 u = s_sum[w];
      if (w < warp) before = sat_add(before, u);
      all = sat_add(all, u);
    }
    // sums that saturate are refused below; the stored values are then unused
    if (b < p.batch) {
      s_start[b] = static_cast<int32_t>(before.x + inc.x - mine.x);
      s_first[b] = static_cast<int32_t>(before.y + inc.y - mine.y);
    }
    base = sat_add(base, all);
    __syncthreads();
  }
  if (tid == 0) {
    s_start[p.batch] = static_cast<int32_t>(base.x);
    s_first[p.batch] = static_cast<int32_t>(base.y);
  }
  __syncthreads();
  // all or nothing: a call that cannot be served in full changes no table
  // entry, takes no block and maps no slot
  int why = 0;
  if (s_bad) why |= kStatusBadLen;
  if (base.x > static_cast<uint32_t>(p.max_slots)) why |= kStatusNoSlots;
  if (top < 0 || top > p.free_capacity || base.y > static_cast<uint32_t>(top)) why |= kStatusNoBlocks;
  const int n_new = why ? 0 : static_cast<int>(base.x);
  const int n_blk = why ? 0 : static_cast<int>(base.y);

  const int gid = blockIdx.x * kTableThreads + tid;
  const int gsz = gridDim.x * kTableThreads;
  for (int k = gid; k < n_blk; k += gsz) {
    const int b = owner_of(s_first, p.batch, k);
    const int held = p.div_bs.div(s_ctx[b] + p.block_size - 1);
    p.table[static_cast<size_t>(b) * p.stride + held + (k - s_first[b])] = p.free_ids[top - 1 - k];
  }
  int bad_id = 0;
  // Runs of kTableRun slots: one search for the first, the next ones move to the
  // next sequence or block when they leave theirs (a million slots took 15 us
  // with a search and two dependent loads for each).
  for (int i0 = gid * kTableRun; i0 < p.max_slots; i0 += gsz * kTableRun) {
    int64_t slot[kTableRun];
    int b = i0 < n_new ? owner_of(s_start, p.batch, i0) : p.batch;
    int blk = -1, id = -1;
#pragma unroll
    for (int r = 0; r < kTableRun; ++r) {
      const int i = i0 + r;
      slot[r] = -1;
      if (i >= n_new) continue;
      while (s_start[b + 1] <= i) {   // past the end of b, and over sequences without new tokens
        ++b;
        blk = -1;
      }
      const int pos = s_ctx[b] + (i - s_start[b]);
      const int at = p.div_bs.div(pos);
      if (at != blk) {
        blk = at;
        const int held = p.div_bs.div(s_ctx[b] + p.block_size - 1);
        // entries below `held` were there before the call; the others are being
        // written by this launch and are taken from the free list instead
        id = blk < held ? p.table[static_cast<size_t>(b) * p.stride + blk]
                        : p.free_ids[top - 1 - (s_first[b] + blk - held)];
        if (id < 0) bad_id = kStatusBadId;
      }
      if (id >= 0) slot[r] = static_cast<int64_t>(id) * p.block_size + (pos - blk * p.block_size);
    }
    if (p.wide && i0 + kTableRun <= p.max_slots) {
      longlong2* const o = reinterpret_cast<longlong2*>(p.slot_map + i0);
      o[0] = make_longlong2(slot[0], slot[1]);
      o[1] = make_longlong2(slot[2], slot[3]);
    } else {
#pragma unroll
      for (int r = 0; r < kTableRun; ++r)
        if (i0 + r < p.max_slots) p.slot_map[i0 + r] = slot[r];
    }
  }
  for (int b = gid; b <= p.batch; b += gsz) p.q_start[b] = why ? 0 : s_start[b];
  if (bad_id) atomicOr(p.status, bad_id);

  // free_left may be free_count, which every CTA reads at its start: the last
  // CTA to finish writes it
  __syncthreads();
  if (tid == 0) {
    if (blockIdx.x == 0 && why) atomicOr(p.status, why);
    __threadfence();
    const unsigned done = atomicAdd(reinterpret_cast<unsigned*>(p.done), 1u);
    if (done == gridDim.x - 1) {
      *p.free_left = top - n_blk;
      atomicExch(p.done, 0);
    }
  }
}

// ----------------------------------------------------------------------------- K/V store

struct StoreParams {
  const uint16_t* k_new;      // [rows] of hkv * D elements, row_stride elements apart
  const uint16_t* v_new;
  const int64_t* slot_map;    // [rows]
  uint16_t* k_host;           // mapped host pools: block ids [0, host_split)
  uint16_t* v_host;
  uint16_t* k_dev;            // HBM pools: block ids [host_split, id_total)
  uint16_t* v_dev;
  int32_t* status;
  long long row_stride;
  int32_t rows, hkv, block_size, host_split, id_total;
  int32_t parts;              // warps per row
};

constexpr int kStoreWarps = 4;
constexpr int kStoreUnroll = 4;   // 16-byte K chunks (and as many V chunks) a lane has in flight

template <int D>
__global__ void __launch_bounds__(kStoreWarps * 32) store_kv_kernel(const StoreParams p) {
  constexpr int CPH = D / 8;      // 16-byte chunks per head
  const long long w = static_cast<long long>(blockIdx.x) * kStoreWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int row = static_cast<int>(w / p.parts);
  const int part = static_cast<int>(w - static_cast<long long>(row) * p.parts);
  if (row >= p.rows) return;
  const long long slot = p.slot_map[row];
  if (slot < 0) return;
  const long long id = slot / p.block_size;
  const int r = static_cast<int>(slot - id * p.block_size);
  if (id >= p.id_total) {
    if (lane == 0 && part == 0) atomicOr(p.status, kStatusBadId);
    return;
  }
  const bool on_host = id < p.host_split;
  uint16_t* const kd = on_host ? p.k_host : p.k_dev;
  uint16_t* const vd = on_host ? p.v_host : p.v_dev;
  const long long blk = on_host ? id : id - p.host_split;
  const uint16_t* const ks = p.k_new + row * p.row_stride;
  const uint16_t* const vs = p.v_new + row * p.row_stride;
  const int chunks = p.hkv * CPH;
  for (int c0 = part * (32 * kStoreUnroll) + lane; c0 < chunks; c0 += p.parts * (32 * kStoreUnroll)) {
    uint4 k[kStoreUnroll], v[kStoreUnroll];
#pragma unroll
    for (int u = 0; u < kStoreUnroll; ++u) {
      const int c = c0 + 32 * u;
      if (c < chunks) {
        k[u] = __ldg(reinterpret_cast<const uint4*>(ks + 8 * c));
        v[u] = __ldg(reinterpret_cast<const uint4*>(vs + 8 * c));
      }
    }
#pragma unroll
    for (int u = 0; u < kStoreUnroll; ++u) {
      const int c = c0 + 32 * u;
      if (c < chunks) {
        const int h = c / CPH;
        const size_t o = ((static_cast<size_t>(blk) * p.hkv + h) * p.block_size + r) * D + (c - h * CPH) * 8;
        *reinterpret_cast<uint4*>(kd + o) = k[u];
        *reinterpret_cast<uint4*>(vd + o) = v[u];
      }
    }
  }
}

}  // namespace dkv
