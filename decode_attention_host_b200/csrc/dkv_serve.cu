// dkv_serve.cu -- C ABI of the entry points an engine calls around the decode
// step: block tables and slot maps, the store of new K/V rows, attention of a
// chunk of new tokens, and decode under a sliding window.
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>
#include <string>

#include "dkv.h"
#include "dkv_chunk.cuh"
#include "dkv_error.h"
#include "dkv_handle.h"
#include "dkv_kernels.cuh"
#include "dkv_plan.h"
#include "dkv_tables.cuh"
#include "dkv_tma.h"

namespace {

using dkv::set_error;

// Ring depth of the windowed split kernel: 229 us with 2 stages, 232 with 3, for 64 sequences of 8 kv heads (32
// query heads) and a 4096-token window.
constexpr int kWinStages = 2;
// Units per resident warp when some blocks sit in host memory: a unit that reads one waits for the PCIe link, and
// short units let the others go on (16 ragged sequences with their sinks on the host: 74 us with 2 splits, 60 with 9).
constexpr int kWinHostUnits = 4;

bool misaligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

// Whether one of the arrays of 4-byte numbers could not be loaded from.
template <class... P>
bool misaligned4(P... p) {
  return (misaligned(p, 4) || ...);
}

template <int D, int G, bool BF16, bool ROPE>
void launch_window(dim3 grid, size_t smem, cudaStream_t s, const dkv::SplitParams& p, const dkv::TileMaps& m) {
  dkv::split_kernel<D, G, BF16, kWinStages, ROPE, false, true><<<grid, dkv::kThreads, smem, s>>>(p, m);
}

template <int D, int G, bool BF16, bool ROPE>
dkv::SplitEntry window_entry() {
  return {&launch_window<D, G, BF16, ROPE>,
          reinterpret_cast<const void*>(&dkv::split_kernel<D, G, BF16, kWinStages, ROPE, false, true>)};
}

template <int D, bool BF16, bool ROPE>
cudaError_t launch_chunk(cudaStream_t s, const dkv::ChunkParams& p, const dkv::ChunkMaps& m, int ctas,
                         int rows) {
  constexpr size_t kSmem = dkv::chunk_smem_bytes<D>();
  if (rows == 128) dkv::chunk_kernel<D, BF16, ROPE, true><<<ctas, dkv::kChunkThreads, kSmem, s>>>(p, m);
  else dkv::chunk_kernel<D, BF16, ROPE, false><<<ctas, dkv::kChunkThreads, kSmem, s>>>(p, m);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || p.nsplit == 1) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>((static_cast<long long>(p.total_rows) * p.hq + 3) / 4));
  cfg.blockDim = dim3(128);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, dkv::chunk_merge_kernel<D, BF16>, p);
}

template <int D, bool BF16, bool ROPE, bool DUAL>
cudaError_t prepare_chunk() {
  auto* const k = dkv::chunk_kernel<D, BF16, ROPE, DUAL>;
  cudaFuncAttributes a{};
  cudaError_t e = cudaFuncGetAttributes(&a, k);
  if (e != cudaSuccess) return e;
  // the warp groups divide the launch's registers among themselves; with fewer
  // of them the softmax warps would wait for registers that do not exist
  if (a.numRegs < dkv::kRegsLaunch) return cudaErrorInvalidKernelImage;
  return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(dkv::chunk_smem_bytes<D>()));
}

// Calls f.template operator()<D, G, BF16, ROPE>() for a handle's shape.
template <class F>
auto by_shape(const dkv_config& c, F&& f) {
  const int G = c.num_q_heads / c.num_kv_heads;
  auto tail = [&](auto d, auto g) {
    constexpr int D = decltype(d)::value, GG = decltype(g)::value;
    const bool rope = c.rope_base > 0.0;
    if (c.kv_dtype == DKV_KV_BF16)
      return rope ? f.template operator()<D, GG, true, true>() : f.template operator()<D, GG, true, false>();
    return rope ? f.template operator()<D, GG, false, true>() : f.template operator()<D, GG, false, false>();
  };
  auto group = [&](auto d) {
    if (G == 1) return tail(d, std::integral_constant<int, 1>{});
    if (G == 2) return tail(d, std::integral_constant<int, 2>{});
    return tail(d, std::integral_constant<int, 4>{});
  };
  return c.head_dim == 64 ? group(std::integral_constant<int, 64>{}) : group(std::integral_constant<int, 128>{});
}

struct PickWindow {
  template <int D, int G, bool BF16, bool ROPE>
  dkv::SplitEntry operator()() const {
    return window_entry<D, G, BF16, ROPE>();
  }
};
struct LaunchChunk {
  cudaStream_t s;
  const dkv::ChunkParams& p;
  const dkv::ChunkMaps& m;
  int ctas, rows;
  template <int D, int G, bool BF16, bool ROPE>
  cudaError_t operator()() const {
    return launch_chunk<D, BF16, ROPE>(s, p, m, ctas, rows);
  }
};
struct PrepareChunk {
  template <int D, int G, bool BF16, bool ROPE>
  cudaError_t operator()() const {
    const cudaError_t e = prepare_chunk<D, BF16, ROPE, false>();
    return e != cudaSuccess ? e : prepare_chunk<D, BF16, ROPE, true>();
  }
};

// Splits of every row tile's walk over the cache.  A CTA takes one (row tile,
// kv head, split) and holds its SM; the time is the number of waves times a
// CTA's share of the walk and its start and end, about 10 us, which is 12
// tiles' time with 128 rows to a CTA (0.8 us a tile) and 5 with 256 (2 us),
// and about one tile's for joining.  `tiles` goes by the table's capacity, as
// the lengths are on the device.  16 rows of 4 heads on 4096 tokens: 40 us
// whole, 17 in 5 splits, 14.5 in 9 to 32; 8 sequences of 16 rows of 32 heads:
// 62 us whole, 43 in 2 (one wave), 55 in 4; 8 rows of 32 heads on four 64k
// contexts: 201 in 4 or 9, 338 in 2, 264 in 32.
int chunk_splits(long long units, int sms, long long tiles, int rows, long long max_splits) {
  const double ends = rows == 128 ? 12.0 : 5.0;
  int best = 1;
  double best_cost = 0.0;
  for (int n = 1; n <= 64 && n <= max_splits && (n == 1 || n <= tiles); ++n) {
    const double waves = static_cast<double>((units * n + sms - 1) / sms);
    const double cost = waves * (static_cast<double>((tiles + n - 1) / n) + ends) + (n > 1 ? 1.0 : 0.0);
    if (n == 1 || cost < 0.97 * best_cost) {
      best = n;
      best_cost = cost;
    }
  }
  return best;
}

// The checks of the two attention entry points that do not depend on the
// query layout: batch, table, ids, pools (aligned, and of the right kind).
int check_cache(dkv_handle* h, const char* who, const void* k_host, const void* v_host, const void* k_dev,
                const void* v_dev, int32_t host_split, int32_t num_dev_blocks) {
  const std::string w(who);
  if (host_split < 0 || num_dev_blocks < 0 || static_cast<long long>(host_split) + num_dev_blocks > INT_MAX)
    return set_error(DKV_ERR_INVALID_ARG, w + ": host_split / num_dev_blocks out of range");
  if ((host_split > 0 && (!k_host || !v_host)) || (num_dev_blocks > 0 && (!k_dev || !v_dev)))
    return set_error(DKV_ERR_INVALID_ARG, w + ": pool pointers are null");
  if ((host_split > 0 && (misaligned(k_host, 16) || misaligned(v_host, 16))) ||
      (num_dev_blocks > 0 && (misaligned(k_dev, 16) || misaligned(v_dev, 16))))
    return set_error(DKV_ERR_INVALID_ARG, w + ": K/V pools must be 16-byte aligned");
  int rc;
  if (host_split > 0) {
    if ((rc = dkv::check_host_pool(h, k_host, 0)) != DKV_OK) return rc;
    if ((rc = dkv::check_host_pool(h, v_host, 1)) != DKV_OK) return rc;
  }
  if (num_dev_blocks > 0) {
    if ((rc = dkv::check_dev_pool(h, k_dev, 0)) != DKV_OK) return rc;
    if ((rc = dkv::check_dev_pool(h, v_dev, 1)) != DKV_OK) return rc;
  }
  return DKV_OK;
}

int check_mask(const char* who, int32_t window, int32_t sinks, int32_t include_self, int32_t min_window) {
  if (window < min_window || sinks < 0 || (include_self != 0 && include_self != 1))
    return set_error(DKV_ERR_INVALID_ARG, std::string(who) + ": window, sinks or include_self out of range");
  return DKV_OK;
}

}  // namespace

cudaError_t dkv::prepare_serving(dkv_handle* h) {
  h->window_kernel = by_shape(h->cfg, PickWindow{});
  cudaError_t e = cudaFuncSetAttribute(h->window_kernel.ptr, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(split_smem_bytes(h->cfg.head_dim, kWinStages)));
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(h->window_kernel.ptr, cudaFuncAttributePreferredSharedMemoryCarveout,
                           cudaSharedmemCarveoutMaxShared);
  if (e != cudaSuccess) return e;
  int per_sm = 0;
  e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, h->window_kernel.ptr, kThreads,
                                                    split_smem_bytes(h->cfg.head_dim, kWinStages));
  if (e != cudaSuccess) return e;
  h->window_ctas = (per_sm > 0 ? per_sm : 1) * h->sm_count;
  e = by_shape(h->cfg, PrepareChunk{});
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(extend_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(table_smem_bytes(kTableMaxBatch)));
}

extern "C" {

int dkv_extend_tables(dkv_handle* h, const int32_t* seq_lens, const int32_t* new_lens, int32_t batch,
                      int32_t* block_table, int32_t block_table_stride, const int32_t* free_ids,
                      int32_t free_capacity, const int32_t* free_count, int32_t* free_left, int32_t* q_start,
                      int64_t* slot_map, int32_t max_slots, dkv_stream_t stream) {
  if (!h) return set_error(DKV_ERR_INVALID_ARG, "dkv_extend_tables: null handle");
  const dkv_config& c = h->cfg;
  if (batch < 1 || batch > c.max_batch)
    return set_error(DKV_ERR_INVALID_ARG, "dkv_extend_tables: batch outside [1, max_batch]");
  if (batch > dkv::kTableMaxBatch) return set_error(DKV_ERR_UNSUPPORTED, "dkv_extend_tables: batch above 8192");
  if (!seq_lens || !new_lens || !block_table || !free_count || !free_left || !q_start ||
      (!free_ids && free_capacity > 0) || (!slot_map && max_slots > 0))
    return set_error(DKV_ERR_INVALID_ARG, "dkv_extend_tables: null pointer");
  if (block_table_stride < 1 || free_capacity < 0 || free_capacity > (1 << 30) || max_slots < 0 ||
      max_slots > (1 << 30))
    return set_error(DKV_ERR_INVALID_ARG, "dkv_extend_tables: stride, free_capacity or max_slots out of range");
  if (misaligned(slot_map, 8))
    return set_error(DKV_ERR_INVALID_ARG, "dkv_extend_tables: slot_map must be 8-byte aligned");
  if (misaligned4(seq_lens, new_lens, block_table, free_ids, free_count, free_left, q_start))
    return set_error(DKV_ERR_INVALID_ARG, "dkv_extend_tables: the int32 arrays must be 4-byte aligned");
  dkv::DeviceGuard guard(c.device);
  if (!guard.ok) return set_error(DKV_ERR_CUDA, "cudaSetDevice failed");
  dkv::TableParams p{};
  p.seq_lens = seq_lens;
  p.new_lens = new_lens;
  p.table = block_table;
  p.free_ids = free_ids;
  p.free_count = free_count;
  p.free_left = free_left;
  p.q_start = q_start;
  p.slot_map = slot_map;
  p.status = h->status;
  p.done = h->work + dkv::kWorkTables;
  p.batch = batch;
  p.stride = block_table_stride;
  p.block_size = c.block_size;
  p.max_len = (block_table_stride < c.max_blocks_per_seq ? block_table_stride : c.max_blocks_per_seq) * c.block_size;
  p.free_capacity = free_capacity;
  p.max_slots = max_slots;
  p.div_bs = dkv::make_invdiv(c.block_size);
  p.wide = !misaligned(slot_map, 16);
  // a run of slots per thread, up to one wave
  constexpr long long kRun = dkv::kTableRun * dkv::kTableThreads;
  const long long want = (static_cast<long long>(max_slots) + kRun - 1) / kRun;
  const long long wave = dkv::kTableCtasPerSm * h->sm_count;
  const int ctas = static_cast<int>(want < 1 ? 1 : want > wave ? wave : want);
  dkv::extend_tables_kernel<<<ctas, dkv::kTableThreads, dkv::table_smem_bytes(batch),
                              reinterpret_cast<cudaStream_t>(stream)>>>(p);
  DKV_CUDA(cudaGetLastError());
  return DKV_OK;
}

int dkv_store_kv(dkv_handle* h, const void* k_new, const void* v_new, int64_t row_stride, const int64_t* slot_map,
                 int32_t num_rows, int32_t host_split, void* k_host, void* v_host, void* k_dev, void* v_dev,
                 dkv_stream_t stream, int32_t num_dev_blocks) {
  if (!h) return set_error(DKV_ERR_INVALID_ARG, "dkv_store_kv: null handle");
  const dkv_config& c = h->cfg;
  if (num_rows < 0) return set_error(DKV_ERR_INVALID_ARG, "dkv_store_kv: num_rows < 0");
  if (num_rows == 0) return DKV_OK;
  if (!k_new || !v_new || !slot_map) return set_error(DKV_ERR_INVALID_ARG, "dkv_store_kv: null pointer");
  const int64_t width = static_cast<int64_t>(c.num_kv_heads) * c.head_dim;
  if (row_stride < width || row_stride % 8 != 0)
    return set_error(DKV_ERR_INVALID_ARG, "dkv_store_kv: row_stride must be a multiple of 8, at least Hkv * D");
  if (misaligned(k_new, 16) || misaligned(v_new, 16) || misaligned(slot_map, 8))
    return set_error(DKV_ERR_INVALID_ARG, "dkv_store_kv: k_new and v_new must be 16-byte, slot_map 8-byte aligned");
  dkv::DeviceGuard guard(c.device);
  if (!guard.ok) return set_error(DKV_ERR_CUDA, "cudaSetDevice failed");
  int rc = check_cache(h, "dkv_store_kv", k_host, v_host, k_dev, v_dev, host_split, num_dev_blocks);
  if (rc != DKV_OK) return rc;
  dkv::StoreParams p{};
  p.k_new = static_cast<const uint16_t*>(k_new);
  p.v_new = static_cast<const uint16_t*>(v_new);
  p.slot_map = slot_map;
  p.k_host = static_cast<uint16_t*>(k_host);
  p.v_host = static_cast<uint16_t*>(v_host);
  p.k_dev = static_cast<uint16_t*>(k_dev);
  p.v_dev = static_cast<uint16_t*>(v_dev);
  p.status = h->status;
  p.row_stride = row_stride;
  p.rows = num_rows;
  p.hkv = c.num_kv_heads;
  p.block_size = c.block_size;
  p.host_split = host_split;
  p.id_total = host_split + num_dev_blocks;
  const int per = 32 * dkv::kStoreUnroll;
  p.parts = static_cast<int>((width / 8 + per - 1) / per);
  const long long warps = static_cast<long long>(num_rows) * p.parts;
  const long long ctas = (warps + dkv::kStoreWarps - 1) / dkv::kStoreWarps;
  if (ctas > INT_MAX) return set_error(DKV_ERR_INVALID_ARG, "dkv_store_kv: too many rows");
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (c.head_dim == 64) dkv::store_kv_kernel<64><<<static_cast<unsigned>(ctas), dkv::kStoreWarps * 32, 0, s>>>(p);
  else dkv::store_kv_kernel<128><<<static_cast<unsigned>(ctas), dkv::kStoreWarps * 32, 0, s>>>(p);
  DKV_CUDA(cudaGetLastError());
  return DKV_OK;
}

int dkv_attn_chunk(dkv_handle* h, const void* q, int64_t q_stride, const int32_t* q_start, int32_t total_rows,
                   const void* k_host, const void* v_host, const void* k_dev, const void* v_dev,
                   const int32_t* block_table, const int32_t* seq_lens, int32_t host_split, void* out, int32_t window,
                   int32_t sinks, int32_t include_self, dkv_stream_t stream, int32_t batch,
                   int32_t block_table_stride, int32_t num_dev_blocks, void* k_stage, void* v_stage) {
  if (!h) return set_error(DKV_ERR_INVALID_ARG, "dkv_attn_chunk: null handle");
  const dkv_config& c = h->cfg;
  if (batch < 0 || batch > c.max_batch)
    return set_error(DKV_ERR_INVALID_ARG, "dkv_attn_chunk: batch outside [0, max_batch]");
  if (total_rows < 0 || total_rows > (1 << 28))
    return set_error(DKV_ERR_INVALID_ARG, "dkv_attn_chunk: total_rows outside [0, 2^28]");
  int rc = check_mask("dkv_attn_chunk", window, sinks, include_self, 0);
  if (rc != DKV_OK) return rc;
  if (batch == 0 || total_rows == 0) {
    h->last_launches = 0;
    return DKV_OK;
  }
  if (!q || !out || !q_start || !block_table || !seq_lens)
    return set_error(DKV_ERR_INVALID_ARG, "dkv_attn_chunk: null pointer");
  if (block_table_stride < 1) return set_error(DKV_ERR_INVALID_ARG, "dkv_attn_chunk: block_table_stride must be >= 1");
  const int64_t width = static_cast<int64_t>(c.num_q_heads) * c.head_dim;
  if (q_stride < width || q_stride % 8 != 0)
    return set_error(DKV_ERR_INVALID_ARG, "dkv_attn_chunk: q_stride must be a multiple of 8, at least Hq * D");
  if (misaligned(q, 16) || misaligned(out, 16))
    return set_error(DKV_ERR_INVALID_ARG, "dkv_attn_chunk: q and out must be 16-byte aligned");
  if (misaligned4(q_start, block_table, seq_lens))
    return set_error(DKV_ERR_INVALID_ARG, "dkv_attn_chunk: q_start, the table and seq_lens must be 4-byte aligned");
  const bool staged = k_stage != nullptr || v_stage != nullptr;
  if (staged && (!k_stage || !v_stage || misaligned(k_stage, 16) || misaligned(v_stage, 16)))
    return set_error(DKV_ERR_INVALID_ARG, "dkv_attn_chunk: staging pools must both be given, 16-byte aligned");
  dkv::DeviceGuard guard(c.device);
  if (!guard.ok) return set_error(DKV_ERR_CUDA, "cudaSetDevice failed");
  if ((rc = check_cache(h, "dkv_attn_chunk", k_host, v_host, k_dev, v_dev, host_split, num_dev_blocks)) != DKV_OK)
    return rc;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool copies = staged && host_split > 0;
  if (copies) {
    if ((rc = dkv::check_dev_pool(h, k_stage, 2)) != DKV_OK) return rc;
    if ((rc = dkv::check_dev_pool(h, v_stage, 3)) != DKV_OK) return rc;
  }
  dkv::ChunkParams p{};
  p.q = static_cast<const uint16_t*>(q);
  p.out = static_cast<uint16_t*>(out);
  p.q_start = q_start;
  p.seq_lens = seq_lens;
  p.table = block_table;
  p.turns = reinterpret_cast<const uint64_t*>(h->inv_freq + c.head_dim / 2);
  p.part_o = h->part_o;
  p.part_lse = h->part_lse;
  p.status = h->status;
  p.q_stride = q_stride;
  p.total_rows = total_rows;
  p.batch = batch;
  p.stride = block_table_stride;
  p.hq = c.num_q_heads;
  p.hkv = c.num_kv_heads;
  p.block_size = c.block_size;
  p.host_split = host_split;
  p.id_total = host_split + num_dev_blocks;
  const int nblk = block_table_stride < c.max_blocks_per_seq ? block_table_stride : c.max_blocks_per_seq;
  p.max_len = nblk * c.block_size;
  p.group_shift = h->G == 4 ? 2 : h->G - 1;
  p.box = 16;
  while (p.box < dkv::kChunkTokens && c.block_size % (2 * p.box) == 0) p.box *= 2;
  p.window = window;
  p.sinks = window ? sinks : 0;
  p.self = include_self;
  p.qscale = h->qscale;
  // 128 rows to a CTA while a sequence has no more of them on average (a kv head's rows: its tokens times G)
  const int rows = static_cast<long long>(total_rows) * h->G <= 128LL * batch ? 128 : 256;
  // sum over b of ceil(rows_b G / rows), rows_b unknown here, is at most this
  const long long row_tiles =
      (static_cast<long long>(total_rows) * h->G + static_cast<long long>(batch) * (rows - h->G)) / rows;
  const long long units = row_tiles * c.num_kv_heads;
  long long see = p.max_len;   // tokens that a row tile may walk over
  if (window && static_cast<long long>(window) + sinks + 512 < see)
    see = static_cast<long long>(window) + sinks + 512;
  // the plan counts the row tiles to expect: one for each sequence, or as many
  // as the rows fill and half a tile more for each sequence's last one
  const long long fill = static_cast<long long>(total_rows) * h->G / rows + batch / 2;
  const long long expect = fill < batch ? batch : fill > row_tiles ? row_tiles : fill;
  const long long walk = (see + dkv::kChunkTokens - 1) / dkv::kChunkTokens;
  const long long room = static_cast<long long>(h->part_rows) / (static_cast<long long>(total_rows) * c.num_q_heads);
  p.nsplit = chunk_splits((expect < row_tiles ? expect : row_tiles) * c.num_kv_heads, h->sm_count, walk, rows, room);
  if (units * p.nsplit > INT_MAX) return set_error(DKV_ERR_INVALID_ARG, "dkv_attn_chunk: too many rows");
  p.div_bs = dkv::make_invdiv(c.block_size);
  p.div_hkv = dkv::make_invdiv(c.num_kv_heads);
  p.div_split = dkv::make_invdiv(p.nsplit);
  dkv::ChunkMaps maps{};
  const long long block_rows = static_cast<long long>(c.num_kv_heads) * c.block_size;
  const long long host_rows = host_split * block_rows, dev_rows = num_dev_blocks * block_rows;
  if (host_rows >= (1LL << 31) || dev_rows >= (1LL << 31))
    return set_error(DKV_ERR_INVALID_ARG, "dkv_attn_chunk: a pool holds 2^31 or more token rows");
  p.oob_host = dev_rows == 0;
  p.oob_row = static_cast<int32_t>(dev_rows ? dev_rows : host_rows);
  const int D = c.head_dim;
  int code = 0;
  if (dev_rows) {
    code = dkv::encode_box_map(&maps.k_dev, k_dev, dev_rows, D, p.box);
    if (code == 0) code = dkv::encode_box_map(&maps.v_dev, v_dev, dev_rows, D, p.box);
  }
  if (code == 0 && host_rows) {
    code = dkv::encode_box_map(&maps.k_host, copies ? k_stage : k_host, host_rows, D, p.box);
    if (code == 0) code = dkv::encode_box_map(&maps.v_host, copies ? v_stage : v_host, host_rows, D, p.box);
  }
  if (code != 0)
    return set_error(DKV_ERR_CUDA,
                     "cuTensorMapEncodeTiled rejected the pool's tensor map (" + std::to_string(code) + ")");
  // from here on nothing refuses the call: only now is anything put on the stream, or the test hook taken
  if (copies) {
    const size_t bytes = static_cast<size_t>(host_rows) * D * 2;
    DKV_CUDA(cudaMemcpyAsync(k_stage, k_host, bytes, cudaMemcpyHostToDevice, s));
    DKV_CUDA(cudaMemcpyAsync(v_stage, v_host, bytes, cudaMemcpyHostToDevice, s));
  }
  p.stall_first_copy = dkv::take_stall_copy() ? 1 : 0;
  DKV_CUDA(by_shape(c, LaunchChunk{s, p, maps, static_cast<int>(units * p.nsplit), rows}));
  h->last_launches = p.nsplit > 1 ? 2 : 1;
  return DKV_OK;
}

int dkv_attn_decode_window(dkv_handle* h, int32_t window, int32_t sinks, int32_t include_self, const float* q,
                           const void* k_host, const void* v_host, const void* k_dev, const void* v_dev,
                           const int32_t* block_table, const int32_t* seq_lens, int32_t host_split, float* out,
                           dkv_stream_t stream, int32_t batch, int32_t block_table_stride, int32_t num_dev_blocks) {
  if (!h) return set_error(DKV_ERR_INVALID_ARG, "dkv_attn_decode_window: null handle");
  const dkv_config& c = h->cfg;
  if (batch < 0 || batch > c.max_batch)
    return set_error(DKV_ERR_INVALID_ARG, "dkv_attn_decode_window: batch outside [0, max_batch]");
  int rc = check_mask("dkv_attn_decode_window", window, sinks, include_self, 1);
  if (rc != DKV_OK) return rc;
  if (batch == 0) {
    h->last_launches = 0;
    return DKV_OK;
  }
  if (!q || !out || !block_table || !seq_lens)
    return set_error(DKV_ERR_INVALID_ARG, "dkv_attn_decode_window: null q / out / table / seq_lens");
  if (block_table_stride < 1)
    return set_error(DKV_ERR_INVALID_ARG, "dkv_attn_decode_window: block_table_stride must be >= 1");
  if (misaligned(q, 8)) return set_error(DKV_ERR_INVALID_ARG, "dkv_attn_decode_window: q must be 8-byte aligned");
  if (misaligned4(out, block_table, seq_lens))
    return set_error(DKV_ERR_INVALID_ARG, "dkv_attn_decode_window: out, the table and seq_lens must be 4-byte aligned");
  dkv::DeviceGuard guard(c.device);
  if (!guard.ok) return set_error(DKV_ERR_CUDA, "cudaSetDevice failed");
  if ((rc = check_cache(h, "dkv_attn_decode_window", k_host, v_host, k_dev, v_dev, host_split, num_dev_blocks)) !=
      DKV_OK)
    return rc;

  const int nblk = block_table_stride < c.max_blocks_per_seq ? block_table_stride : c.max_blocks_per_seq;
  // the most blocks with a visible token that a sequence can have: the window
  // may straddle one more than it fills
  const long long wb = static_cast<long long>(window) / c.block_size + 2;
  const long long sb = (static_cast<long long>(sinks) + c.block_size - 1) / c.block_size;
  const int vis = static_cast<int>(wb + sb < nblk ? wb + sb : nblk);
  const long per = static_cast<long>(batch) * c.num_kv_heads;
  const dkv::SplitPlan pl =
      dkv::plan_split_even(vis, per, c.block_size,
                           static_cast<long>(dkv::kWarps) * h->window_ctas * (host_split > 0 ? kWinHostUnits : 1),
                           static_cast<long>(h->part_rows / (static_cast<size_t>(batch) * c.num_q_heads)));
  if (static_cast<size_t>(batch) * c.num_q_heads * pl.nsplit > h->part_rows)
    return set_error(DKV_ERR_INVALID_ARG, "internal: split plan exceeds the workspace");
  dkv::SplitParams sp{};
  sp.work = h->work + dkv::kWorkWindow;
  sp.q = q;
  sp.k_pool = static_cast<const uint16_t*>(k_dev);
  sp.v_pool = static_cast<const uint16_t*>(v_dev);
  sp.k_host = static_cast<const uint16_t*>(k_host);
  sp.v_host = static_cast<const uint16_t*>(v_host);
  sp.host_split = host_split;
  sp.window = window;
  sp.sinks = sinks;
  sp.table = block_table;
  sp.seq_lens = seq_lens;
  sp.inv_freq = h->inv_freq;
  sp.part_o = h->part_o;
  sp.part_lse = h->part_lse;
  sp.status = h->status;
  sp.hq = c.num_q_heads;
  sp.hkv = c.num_kv_heads;
  sp.block_size = c.block_size;
  sp.stride = block_table_stride;
  sp.nsplit = pl.nsplit;
  sp.nslots = pl.nsplit;
  sp.bps = dkv::min_blocks_per_split(c.block_size);
  sp.id_total = host_split + num_dev_blocks;
  sp.max_len = nblk * c.block_size;
  sp.n_units = batch * pl.nsplit * c.num_kv_heads;
  sp.rope = c.rope_base > 0.0 ? 1 : 0;
  sp.qscale = h->qscale;
  sp.extra_tokens = include_self;
  sp.num_queries = 1;
  dkv::set_divisors(sp);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int need = (sp.n_units + dkv::kWarps - 1) / dkv::kWarps;
  const int ctas = need < h->window_ctas ? need : h->window_ctas;
  static const dkv::TileMaps no_maps{};
  h->window_kernel.fn(dim3(ctas), dkv::split_smem_bytes(c.head_dim, kWinStages), s, sp, no_maps);
  DKV_CUDA(cudaGetLastError());
  // joined by a kernel of its own: a warp that joins the splits it finished
  // last, behind a fence and a counter, took 249 us instead of 229 on 64
  // sequences and 15.5 us instead of 10.7 on a single short one
  dkv::MergeParams mp{};
  mp.part_o = h->part_o;
  mp.part_lse = h->part_lse;
  mp.out = out;
  mp.nslots = pl.nsplit;
  mp.nsplit = 0;
  mp.has_dev = 1;
  DKV_CUDA(h->merge(batch * c.num_q_heads, s, mp, true));
  h->last_launches = 2;
  return DKV_OK;
}

}  // extern "C"
