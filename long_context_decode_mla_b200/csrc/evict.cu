// Eviction from one shard's cache by accumulated attention weight: of every
// request's rows the `budget` of largest mass stay, in place.
//
// Row j of a request has its mass and a token position t; rows with t < sink
// or t >= L - recent are kept before all others.  Ties go to the lowest row.
// Attention does not depend on the order of the rows (the rope is in the keys
// already), so a kept row below the budget does not move: the kept rows at or
// past it, in order, fill the places below it that were given up, in order.
// Reads 4 to 8 bytes a row and moves only the rows that have to move: sources
// are at or past the budget and targets below it, so no order of the copies
// can matter.
//
// One cluster per request picks the rows (select_topk.cuh) and writes the
// lists of freed places and moving rows with the new masses and positions; a
// second kernel copies the rows, launched ahead as the first one's dependent.
// The picking is bound by its passes' barriers (64 requests of 2,112 rows 8 us, 24
// of up to 50,250 rows 18.5 us), the moving by HBM (78,000 bf16
// rows move in 34 us after the picking, 5.2 TB/s read and written).
#include "dcpmla.h"

#include <algorithm>
#include <climits>
#include <mutex>

#include "common.cuh"
#include "kernels.h"
#include "select_topk.cuh"
#include "tc_ptx.cuh"

namespace dcpmla {
namespace {

struct EvictParams {
  uint8_t* kv;
  long long num_blocks;
  const int* block_table;
  int bt_stride;
  const int* seq_lens;
  const int* rows;             // rows a request holds; nullptr: the shard's share of its length
  const float* mass;
  const int* positions;        // nullptr: row j is token j * nshards + shard
  int mass_stride;
  int batch, shard, nshards;
  int budget, sink, recent;
  float* mass_out;
  int* positions_out;
  int* rows_out;
  int* flags;
  int* count;                  // [batch] rows to move
  int* holes;                  // [batch][budget] places given up, ascending
  int* movers;                 // [batch][budget] rows that move, ascending
};

// Rows of request b, clipped to its table row and to the mass array.
__device__ __forceinline__ int rows_of(const EvictParams& p, int b, int* length) {
  int L = __ldg(p.seq_lens + b);
  bool bad = L < 0;
  L = max(L, 0);
  int n = p.rows ? __ldg(p.rows + b) : local_len(L, p.shard, p.nshards);
  if (n < 0) {
    bad = true;
    n = 0;
  }
  const long long room = min((long long)p.bt_stride * kBlock, (long long)p.mass_stride);
  if (n > room) {
    bad = true;
    n = (int)room;
  }
  if (bad && p.flags && threadIdx.x == 0) atomicOr(p.flags, kFlagBadLength);
  *length = L;
  return n;
}

__device__ __forceinline__ int position_of(const EvictParams& p, size_t base, int j) {
  if (p.positions) return __ldg(p.positions + base + j);
  return (int)min((long long)INT_MAX, (long long)j * p.nshards + p.shard);
}

__global__ void __launch_bounds__(topk::kThreads) pick_kernel(const EvictParams p) {
  extern __shared__ __align__(16) uint32_t bits[];
  __shared__ topk::Ctl c;
  topk::cg::cluster_group cl = topk::cg::this_cluster();
  ptx::launch_dependents();
  const int b = blockIdx.y;
  int L;
  const int n = rows_of(p, b, &L);
  const int keep = min(n, p.budget);
  const size_t base = (size_t)b * p.mass_stride;
  int lo, hi;
  topk::slice(n, cl.block_rank(), cl.num_blocks(), &lo, &hi);
  if (cl.block_rank() == 0 && threadIdx.x == 0) p.rows_out[b] = keep;
  if (n <= p.budget) {               // nothing to give up (the same for the whole cluster)
    if (cl.block_rank() == 0 && threadIdx.x == 0) p.count[b] = 0;
    for (int j = lo + threadIdx.x; j < hi; j += topk::kThreads) {
      p.mass_out[base + j] = p.mass[base + j];
      if (p.positions_out) p.positions_out[base + j] = position_of(p, base, j);
    }
    return;
  }
  const int fresh = L - p.recent;    // positions from here on are recent
  const bool put_mass = p.mass_out != p.mass;
  const bool put_pos = p.positions_out && p.positions_out != p.positions;
  struct Row {
    float mass;
    int position;
  };
  topk::mark(
      cl, c, lo, hi, keep, bits, [&](int j) { return Row{p.mass[base + j], position_of(p, base, j)}; },
      [&](int j, const Row& row, bool first) {
        if (first && j < p.budget) {
          // as if the row stayed; the move kernel corrects the freed places
          if (put_mass) p.mass_out[base + j] = row.mass;
          if (put_pos) p.positions_out[base + j] = row.position;
        }
        return row.position < p.sink || row.position >= fresh ? 0xFFFFFFFFu : topk::key_of(row.mass);
      });
  // Freed places (below the budget, not taken) and moving rows (taken, at or
  // past it) of this slice; every mass has been read by now.
  auto word = [&](int list, int w) {
    const int j0 = lo + 32 * w;
    const uint32_t live = hi - j0 >= 32 ? 0xFFFFFFFFu : (1u << (hi - j0)) - 1u;
    const int d = p.budget - j0;     // rows of this word below the budget
    const uint32_t below = d >= 32 ? 0xFFFFFFFFu : d <= 0 ? 0u : (1u << d) - 1u;
    return list == 0 ? ~bits[w] & live & below : bits[w] & live & ~below;
  };
  int pos[2] = {0, 0};
  if (cl.num_blocks() > 1) {
    int holes = 0, movers = 0, th, tm;
    for (int w = threadIdx.x; w < (hi - lo + 31) / 32; w += topk::kThreads) {
      holes += __popc(word(0, w));
      movers += __popc(word(1, w));
    }
    block_exclusive_scan(holes, c.warp_sums, &th);
    block_exclusive_scan(movers, c.warp_sums, &tm);
    if (threadIdx.x == 0) {
      c.share[0] = th;
      c.share[1] = tm;
    }
    topk::sync(cl);
    pos[0] = topk::before(cl, c, 0);
    pos[1] = topk::before(cl, c, 1);
    topk::sync(cl);      // shared memory stays until every CTA has read it
  }
  topk::emit<2>(c, lo, hi, pos, word, [&](int list, int j, int at) {
    (list == 0 ? p.holes : p.movers)[(size_t)b * p.budget + at] = j;
  });
  if (cl.block_rank() == cl.num_blocks() - 1 && threadIdx.x == 0) p.count[b] = pos[1];
}

// Physical row address, or nullptr (flagged) for a table entry outside the pool.
template <int kRowBytes>
__device__ __forceinline__ uint8_t* row_at(const EvictParams& p, int b, int j) {
  const int blk = __ldg(p.block_table + (size_t)b * p.bt_stride + j / kBlock);
  if (blk < 0 || (long long)blk >= p.num_blocks) {
    if (p.flags) atomicOr(p.flags, kFlagBadBlock);
    return nullptr;
  }
  return p.kv + ((size_t)blk * kBlock + j % kBlock) * kRowBytes;
}

constexpr int kMoveWarps = 8;
constexpr int kMoveRows = 4;       // rows a warp copies at once, eight lanes each

// Moving rows: the bytes, the mass and the position.  A row's copy starts with
// three dependent loads (place, table entry, row), so a warp takes four rows at
// once, all of their bytes in flight before the first store.
template <int kRowBytes>
__global__ void __launch_bounds__(32 * kMoveWarps) move_kernel(const EvictParams p) {
  constexpr int kUnits = kRowBytes / 16, kPer = (kUnits + 7) / 8;
  const int b = blockIdx.y, sub = (threadIdx.x & 31) >> 3, l = threadIdx.x & 7;
  ptx::wait_primary();
  const int n = __ldcg(p.count + b);
  const size_t base = (size_t)b * p.mass_stride;
  const int stride = gridDim.x * kMoveWarps * kMoveRows;
  for (int i = (blockIdx.x * kMoveWarps + (threadIdx.x >> 5)) * kMoveRows + sub; i < n; i += stride) {
    const int src = __ldcg(p.movers + (size_t)b * p.budget + i);
    const int dst = __ldcg(p.holes + (size_t)b * p.budget + i);
    const uint4* s = reinterpret_cast<const uint4*>(row_at<kRowBytes>(p, b, src));
    uint4* d = reinterpret_cast<uint4*>(row_at<kRowBytes>(p, b, dst));
    if (l == 0) {
      p.mass_out[base + dst] = p.mass[base + src];
      if (p.positions_out) p.positions_out[base + dst] = position_of(p, base, src);
    }
    if (!s || !d) continue;
    uint4 v[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k)
      if (l + 8 * k < kUnits) v[k] = s[l + 8 * k];
#pragma unroll
    for (int k = 0; k < kPer; ++k)
      if (l + 8 * k < kUnits) d[l + 8 * k] = v[k];
  }
}

bool aligned16(const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0; }
size_t round256(size_t x) { return (x + 255) & ~(size_t)255; }

// Workspace: 256-byte header (flag word), counts, freed places, moving rows.
size_t evict_bytes(int batch, int budget) {
  return kWsHeader + round256((size_t)batch * 4) + 2 * round256((size_t)batch * budget * 4);
}

constexpr long long kMaxRows = 8ll << 20;     // rows of a request: a bit each in the cluster

std::mutex g_mutex;
bool g_done[kMaxDevicesConfigured] = {};

}  // namespace
}  // namespace dcpmla

using namespace dcpmla;

extern "C" {

int mla_cache_evict_workspace_size(int batch, int budget, size_t* bytes) {
  if (!bytes || batch < 0 || budget < 1) return DCPMLA_ERR_INVALID_ARGUMENT;
  *bytes = evict_bytes(batch, budget);
  return DCPMLA_OK;
}

int mla_cache_evict(void* kv_cache, int kv_dtype, int64_t num_blocks, int block_size,
                    const int32_t* block_table, int block_table_stride, const int32_t* seq_lens,
                    const int32_t* rows, int batch, int shard_id, int num_shards,
                    const float* mass, const int32_t* positions, int64_t mass_stride, int budget,
                    int sink, int recent, float* mass_out, int32_t* positions_out,
                    int32_t* rows_out, void* workspace, size_t workspace_bytes, void* stream) {
  if (batch < 0 || block_table_stride < 1 || num_shards < 1 || shard_id < 0 ||
      shard_id >= num_shards || num_blocks < 1 || block_size < 1 || mass_stride < 1 ||
      budget < 1 || sink < 0 || recent < 0 || (long long)sink + recent > budget)
    return DCPMLA_ERR_INVALID_ARGUMENT;
  if (kv_dtype != DCPMLA_KV_BF16 && kv_dtype != DCPMLA_KV_FP8) return DCPMLA_ERR_INVALID_ARGUMENT;
  if (block_size != kBlock || batch > 65535 || mass_stride > INT32_MAX ||
      std::min<long long>((long long)block_table_stride * kBlock, mass_stride) > kMaxRows)
    return DCPMLA_ERR_UNSUPPORTED;
  if (batch == 0) return DCPMLA_OK;
  if (!kv_cache || !block_table || !seq_lens || !mass || !mass_out || !rows_out ||
      rows_out == rows || rows_out == seq_lens)
    return DCPMLA_ERR_INVALID_ARGUMENT;
  if (!aligned16(kv_cache) || (workspace && !aligned16(workspace))) return DCPMLA_ERR_ALIGNMENT;
  if (!workspace || workspace_bytes < evict_bytes(batch, budget)) return DCPMLA_ERR_WORKSPACE;
  int dev = 0, sms = 0;
  int rc = dcpmla_device_sm_count(&sms);
  if (rc != DCPMLA_OK) return rc;
  if (cudaGetDevice(&dev) != cudaSuccess) return DCPMLA_ERR_CUDA;
  EvictParams p{};
  p.kv = static_cast<uint8_t*>(kv_cache);
  p.num_blocks = num_blocks;
  p.block_table = block_table;
  p.bt_stride = block_table_stride;
  p.seq_lens = seq_lens;
  p.rows = rows;
  p.mass = mass;
  p.positions = positions;
  p.mass_stride = (int)mass_stride;
  p.batch = batch;
  p.shard = shard_id;
  p.nshards = num_shards;
  p.budget = budget;
  p.sink = sink;
  p.recent = recent;
  p.mass_out = mass_out;
  p.positions_out = positions_out;
  p.rows_out = rows_out;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.flags = reinterpret_cast<int*>(ws);
  p.count = reinterpret_cast<int*>(ws + kWsHeader);
  p.holes = p.count + round256((size_t)batch * 4) / 4;
  p.movers = p.holes + round256((size_t)batch * budget * 4) / 4;
  {
    std::lock_guard<std::mutex> lock(g_mutex);
    if (!g_done[dev]) {
      if (cudaFuncSetAttribute(pick_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               (int)(kMaxRows / topk::kMaxCluster / 8 + 256)) != cudaSuccess)
        return DCPMLA_ERR_CUDA;
      g_done[dev] = true;
    }
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const long long most = std::min<long long>((long long)block_table_stride * kBlock, mass_stride);
  int size = topk::cluster_size(most, batch, sms);
  while ((most + size - 1) / size > kMaxRows / topk::kMaxCluster) size *= 2;   // bits in shared memory
  const size_t smem = (size_t)topk::slice_words(most, size) * 4;
  if (launch_kernel(pick_kernel, dim3(size, batch), topk::kThreads, smem, st, size, false, p) !=
      cudaSuccess)
    return DCPMLA_ERR_CUDA;
  const int most_moves = (int)std::min<long long>(budget, std::max<long long>(most - budget, 0));
  if (most_moves > 0) {
    constexpr int kCtaRows = kMoveWarps * kMoveRows;
    // several waves: requests move very different numbers of rows (24 requests of 0 to
    // 6,800: 62.7, 57.3 and 54.2 us for the call at 4, 8 and 32 CTAs an SM)
    const int gx = std::max(1, std::min((most_moves + kCtaRows - 1) / kCtaRows, sms * 32 / batch));
    const dim3 grid(gx, batch);
    auto move = kv_dtype == DCPMLA_KV_BF16 ? move_kernel<kRowBytesBf16> : move_kernel<kRowBytesFp8>;
    if (launch_kernel(move, grid, 32 * kMoveWarps, 0, st, 0, true, p) != cudaSuccess)
      return DCPMLA_ERR_CUDA;
  }
  return cudaGetLastError() == cudaSuccess ? DCPMLA_OK : DCPMLA_ERR_CUDA;
}

}  // extern "C"
