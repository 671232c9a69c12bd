// Choice of the cache blocks that a query token reads, from the block
// summaries (int8 codes of the mean key and their scales), and the decode over
// the chosen blocks.
//
//   q codes: per head and scale group, step = max|q| / 127 (1 if 0), code =
//            rint(q / step)                                 (values not finite: 0)
//   s_hb   = sum over the five groups, in order, of
//            fp32(codes_q . codes_b) * (step_hg * scale_bg)  (fp32, no fusing)
//   rank_b = max_h (s_hb - max_b' s_hb')
//
// The code products are whole numbers below 2^24, exact in fp32 and in any
// order, and every other step is one rounded fp32 operation: the choice is the
// same bits for every launch shape.  Ranking by the distance to the head's own
// best block lets every head speak on its own softmax's scale: a block is left
// out only if it is far from the best for all of them.  The first
// `sink` and last `recent` blocks are always taken; ties go to the lowest
// index.
#include "dcpmla.h"

#include <cmath>
#include <mutex>

#include "common.cuh"
#include "kernels.h"
#include "select_topk.cuh"

namespace dcpmla {
namespace {

constexpr int kGroups = 5;
constexpr int kQCodes = 64 * kHeadDim;              // q codes of a row, 64 heads
constexpr int kQBytes = kQCodes + 64 * kGroups * 4; // then the steps [group][head]
constexpr int kTile = 128;                          // blocks per scoring tile

struct SelectParams {
  const __nv_bfloat16* q;      // [rows][heads][576]
  const uint8_t* summaries;
  long long num_blocks;
  const int* block_table;
  int bt_stride;
  const int* seq_lens;
  int batch, heads, q_len, shard, nshards;
  int topk, sink, recent;
  int tiles;                   // scoring tiles per row (from the table's stride)
  uint8_t* q_codes;            // [rows][kQBytes]
  float* scores;               // [rows][tiles][heads][kTile]
  float* tile_max;             // [rows][tiles][heads]
  int* out_blocks;             // [rows][topk] or nullptr
  int* out_table;              // [rows][topk]
  int* out_lens;               // [rows]
  int* flags;
};

// Rows of this shard that query row r sees; sets flag bits on a bad length.
__device__ __forceinline__ int rows_of(const SelectParams& p, int r, int* blocks) {
  const int b = r / p.q_len, i = r % p.q_len;
  int L = __ldg(p.seq_lens + b);
  bool bad = L < 0;
  L = max(0, L - (p.q_len - 1 - i));
  int n = local_len(L, p.shard, p.nshards);
  int nb = n > 0 ? (n - 1) / kBlock + 1 : 0;
  if (nb > p.bt_stride) {
    bad = true;
    nb = p.bt_stride;
    n = nb * kBlock;
  }
  if (bad && p.flags && threadIdx.x == 0) atomicOr(p.flags, kFlagBadLength);
  *blocks = nb;
  return n;
}

// int8 codes of one query row: a warp per (head, group).
__global__ void __launch_bounds__(160) q_codes_kernel(const SelectParams p) {
  const int r = blockIdx.x, h = blockIdx.y, g = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const __nv_bfloat16* q = p.q + ((size_t)r * p.heads + h) * kHeadDim;
  const int v = g < 4 ? 4 : 2, d = g < 4 ? 128 * g + 4 * lane : kVDim + 2 * lane;
  float x[4] = {0.f, 0.f, 0.f, 0.f};
  float amax = 0.f;
  for (int e = 0; e < v; ++e) {
    x[e] = __bfloat162float(q[d + e]);
    if (!(fabsf(x[e]) <= 3.4028234663852886e38f)) x[e] = 0.f;
    amax = fmaxf(amax, fabsf(x[e]));
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const float step = amax > 0.f ? __fdiv_rn(amax, 127.f) : 1.f;
  uint8_t* out = p.q_codes + (size_t)r * kQBytes;
  for (int e = 0; e < v; ++e)
    out[h * kHeadDim + d + e] = (uint8_t)min(127, max(-127, __float2int_rn(__fdiv_rn(x[e], step))));
  if (lane == 0) reinterpret_cast<float*>(out + kQCodes)[g * 64 + h] = step;
}

// Scores of one tile of blocks of one row: a thread per block.
__global__ void __launch_bounds__(kTile) score_kernel(const SelectParams p) {
  const int r = blockIdx.y, tile = blockIdx.x;
  int nb;
  rows_of(p, r, &nb);
  if (tile * kTile >= nb) return;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float wmax[kTile / 32][64];
  const uint8_t* qc = p.q_codes + (size_t)r * kQBytes;
  for (int i = threadIdx.x; i < kQBytes / 16; i += kTile)
    reinterpret_cast<uint4*>(smem)[i] = reinterpret_cast<const uint4*>(qc)[i];
  __syncthreads();
  const float* steps = reinterpret_cast<const float*>(smem + kQCodes);
  const int k = tile * kTile + threadIdx.x;
  const int b = r / p.q_len;
  int blk = -1;
  if (k < nb) {
    blk = __ldg(p.block_table + (size_t)b * p.bt_stride + k);
    if (blk < 0 || (long long)blk >= p.num_blocks) {
      if (p.flags) atomicOr(p.flags, kFlagBadBlock);
      blk = -1;
    }
  }
  const uint8_t* rec = p.summaries + (size_t)max(blk, 0) * kSummaryBytes;
  float sc[kGroups];
  for (int g = 0; g < kGroups; ++g) sc[g] = reinterpret_cast<const float*>(rec + kHeadDim)[g];
  float* out = p.scores + ((size_t)r * p.tiles + tile) * p.heads * kTile;
  for (int h = 0; h < p.heads; ++h) {
    float s = 0.f;
    for (int g = 0; g < kGroups; ++g) {
      int dot = 0;
      const int words = g < 4 ? 32 : 16;
      for (int w = 0; w < words; ++w)
        dot = __dp4a(reinterpret_cast<const int*>(smem + h * kHeadDim + 128 * g)[w],
                     reinterpret_cast<const int*>(rec + 128 * g)[w], dot);
      const float t = __fmul_rn((float)dot, __fmul_rn(steps[g * 64 + h], sc[g]));
      s = g == 0 ? t : __fadd_rn(s, t);
    }
    if (blk < 0) s = -INFINITY;
    out[h * kTile + threadIdx.x] = s;
    float m = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if ((threadIdx.x & 31) == 0) wmax[threadIdx.x >> 5][h] = m;
  }
  __syncthreads();
  if (threadIdx.x < p.heads)
    p.tile_max[((size_t)r * p.tiles + tile) * p.heads + threadIdx.x] =
        fmaxf(fmaxf(wmax[0][threadIdx.x], wmax[1][threadIdx.x]),
              fmaxf(wmax[2][threadIdx.x], wmax[3][threadIdx.x]));
}

// Ranks and the choice of one row: one cluster.
__global__ void __launch_bounds__(topk::kThreads) choose_kernel(const SelectParams p, int bit_words) {
  extern __shared__ __align__(16) uint32_t dyn[];
  __shared__ topk::Ctl c;
  __shared__ float hmax[64];
  __shared__ int s_pos;
  topk::cg::cluster_group cl = topk::cg::this_cluster();
  const int r = blockIdx.y, b = r / p.q_len;
  int nb;
  const int n = rows_of(p, r, &nb);
  uint32_t* bits = dyn;
  uint32_t* keys = dyn + bit_words;
  int lo, hi;
  topk::slice(nb, cl.block_rank(), cl.num_blocks(), &lo, &hi);
  const int want = min(nb, p.topk);
  const int tiles = (nb + kTile - 1) / kTile;
  if (threadIdx.x < p.heads) {
    float m = -INFINITY;
    for (int t = 0; t < tiles; ++t)
      m = fmaxf(m, p.tile_max[((size_t)r * p.tiles + t) * p.heads + threadIdx.x]);
    hmax[threadIdx.x] = m;
  }
  __syncthreads();
  for (int k = lo + threadIdx.x; k < hi; k += topk::kThreads) {
    uint32_t key = 0xFFFFFFFFu;
    if (k >= p.sink && k < nb - p.recent) {
      const float* s = p.scores + ((size_t)r * p.tiles + k / kTile) * p.heads * kTile + k % kTile;
      float rank = -INFINITY;
      for (int h = 0; h < p.heads; ++h) {
        const float v = s[h * kTile];
        // equal infinities: no distance
        rank = fmaxf(rank, v == hmax[h] ? 0.f : __fsub_rn(v, hmax[h]));
      }
      key = topk::key_of(rank);
    }
    keys[k - lo] = key;
  }
  __syncthreads();
  if (want > 0)
    topk::mark(cl, c, lo, hi, want, bits, [&](int i) { return keys[i - lo]; });
  // places of this slice's blocks in the list
  int mine = 0;
  for (int w = threadIdx.x; w < (hi - lo + 31) / 32; w += topk::kThreads) mine += __popc(bits[w]);
  int tot;
  block_exclusive_scan(mine, c.warp_sums, &tot);
  if (threadIdx.x == 0) c.share[0] = tot;
  cl.sync();
  int pos = topk::before(cl, c, 0);
  cl.sync();          // shared memory stays until every CTA has read it
  for (int base = lo; base < hi; base += topk::kThreads) {
    const int k = base + threadIdx.x;
    const bool take = k < hi && ((bits[(k - lo) >> 5] >> ((k - lo) & 31)) & 1u);
    const int at = pos + block_exclusive_scan(take ? 1 : 0, c.warp_sums, &tot);
    pos += tot;
    if (take) {
      if (p.out_blocks) p.out_blocks[(size_t)r * p.topk + at] = k;
      p.out_table[(size_t)r * p.topk + at] = __ldg(p.block_table + (size_t)b * p.bt_stride + k);
    }
  }
  if (cl.block_rank() == 0) {
    for (int i = want + threadIdx.x; i < p.topk; i += topk::kThreads) {
      if (p.out_blocks) p.out_blocks[(size_t)r * p.topk + i] = -1;
      p.out_table[(size_t)r * p.topk + i] = -1;
    }
    // every chosen block is full but the last of the row, which is always chosen
    if (threadIdx.x == 0) p.out_lens[r] = n - (nb - want) * kBlock;
  }
}

bool aligned16(const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0; }
size_t round256(size_t x) { return (x + 255) & ~(size_t)255; }

// Workspace: 256-byte header (flag word), q codes, scores, tile maxima.
struct SelectLayout {
  size_t q_codes, scores, tile_max, total;
};
SelectLayout layout(int rows, int heads, int stride) {
  const size_t tiles = ((size_t)stride + kTile - 1) / kTile;
  SelectLayout l;
  l.q_codes = kWsHeader;
  l.scores = l.q_codes + round256((size_t)rows * kQBytes);
  l.tile_max = l.scores + round256((size_t)rows * tiles * heads * kTile * 4);
  l.total = l.tile_max + round256((size_t)rows * tiles * heads * 4);
  return l;
}

// Largest table stride: a row's keys and bits fit one cluster's shared memory.
constexpr int kMaxCluster = 8;
constexpr int kMaxStride = kMaxCluster * 49152;

int check_sizes(int batch, int heads, int q_len, int stride) {
  if (batch < 0 || heads < 1 || q_len < 1 || q_len > kMaxQueryLen || stride < 1)
    return DCPMLA_ERR_INVALID_ARGUMENT;
  if (heads > kMaxHeads || stride > kMaxStride ||
      (long long)batch * q_len > 65535)      // grid y
    return DCPMLA_ERR_UNSUPPORTED;
  return DCPMLA_OK;
}

std::mutex g_mutex;
bool g_done[kMaxDevicesConfigured] = {};

cudaError_t prepare_device(int dev) {
  std::lock_guard<std::mutex> lock(g_mutex);
  if (g_done[dev]) return cudaSuccess;
  cudaError_t e = cudaFuncSetAttribute(choose_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       208 * 1024);
  if (e != cudaSuccess) return e;
  g_done[dev] = true;
  return cudaSuccess;
}

struct SelectArgs {
  const void* q;
  const void* summaries;
  int64_t num_blocks;
  int block_size;
  const int32_t* block_table;
  int stride;
  const int32_t* seq_lens;
  int batch, heads, q_len, shard, nshards, topk, sink, recent;
};

// Checks of the choice's arguments; fills p with them.
int check_select(const SelectArgs& a, SelectParams* p) {
  if (a.nshards < 1 || a.shard < 0 || a.shard >= a.nshards || a.num_blocks < 1 ||
      a.block_size < 1 || a.topk < 1 || a.sink < 0 || a.recent < 1 ||
      (long long)a.sink + a.recent > a.topk)
    return DCPMLA_ERR_INVALID_ARGUMENT;
  const int rc = check_sizes(a.batch, a.heads, a.q_len, a.stride);
  if (rc != DCPMLA_OK) return rc;
  if (a.block_size != kBlock) return DCPMLA_ERR_UNSUPPORTED;
  *p = SelectParams{};
  if (a.batch == 0) return DCPMLA_OK;
  if (!a.q || !a.summaries || !a.block_table || !a.seq_lens) return DCPMLA_ERR_INVALID_ARGUMENT;
  if (!aligned16(a.q) || !aligned16(a.summaries)) return DCPMLA_ERR_ALIGNMENT;
  p->q = static_cast<const __nv_bfloat16*>(a.q);
  p->summaries = static_cast<const uint8_t*>(a.summaries);
  p->num_blocks = a.num_blocks;
  p->block_table = a.block_table;
  p->bt_stride = a.stride;
  p->seq_lens = a.seq_lens;
  p->batch = a.batch;
  p->heads = a.heads;
  p->q_len = a.q_len;
  p->shard = a.shard;
  p->nshards = a.nshards;
  p->topk = a.topk;
  p->sink = a.sink;
  p->recent = a.recent;
  p->tiles = (a.stride + kTile - 1) / kTile;
  return DCPMLA_OK;
}

cudaError_t launch_select(const SelectParams& p, cudaStream_t st) {
  const int rows = p.batch * p.q_len;
  q_codes_kernel<<<dim3(rows, p.heads), 160, 0, st>>>(p);
  score_kernel<<<dim3(p.tiles, rows), kTile, kQBytes, st>>>(p);
  const int size = p.bt_stride <= 4096 ? 1 : kMaxCluster;
  const int words = topk::slice_words(p.bt_stride, size);
  return topk::launch(choose_kernel, rows, size, (size_t)words * 33 * 4, st, p, words);
}

// The choice on a workspace part `ws` (laid out by layout()).
int run_select(SelectParams& p, uint8_t* ws, cudaStream_t st) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return DCPMLA_ERR_CUDA;
  if (dev < 0 || dev >= kMaxDevicesConfigured) return DCPMLA_ERR_UNSUPPORTED;
  if (prepare_device(dev) != cudaSuccess) return DCPMLA_ERR_CUDA;
  const SelectLayout l = layout(p.batch * p.q_len, p.heads, p.bt_stride);
  p.q_codes = ws + l.q_codes;
  p.scores = reinterpret_cast<float*>(ws + l.scores);
  p.tile_max = reinterpret_cast<float*>(ws + l.tile_max);
  return launch_select(p, st) == cudaSuccess ? DCPMLA_OK : DCPMLA_ERR_CUDA;
}

}  // namespace
}  // namespace dcpmla

using namespace dcpmla;

extern "C" {

int mla_block_select_workspace_size(int batch, int num_heads, int q_len, int block_table_stride,
                                    size_t* bytes) {
  if (!bytes) return DCPMLA_ERR_INVALID_ARGUMENT;
  const int rc = check_sizes(batch, num_heads, q_len, block_table_stride);
  if (rc != DCPMLA_OK) return rc;
  *bytes = layout(batch * q_len, num_heads, block_table_stride).total;
  return DCPMLA_OK;
}

int mla_block_select(const void* q, const void* summaries, int64_t num_blocks, int block_size,
                     const int32_t* block_table, int block_table_stride, const int32_t* seq_lens,
                     int batch, int num_heads, int q_len, int shard_id, int num_shards,
                     int block_topk, int sink_blocks, int recent_blocks, int32_t* out_blocks,
                     int32_t* out_table, int32_t* out_lens, void* workspace,
                     size_t workspace_bytes, void* stream) {
  SelectArgs a{q, summaries, num_blocks, block_size, block_table, block_table_stride, seq_lens,
               batch, num_heads, q_len, shard_id, num_shards, block_topk, sink_blocks,
               recent_blocks};
  SelectParams p;
  int rc = check_select(a, &p);
  if (rc != DCPMLA_OK || batch == 0) return rc;
  if (!out_table || !out_lens) return DCPMLA_ERR_INVALID_ARGUMENT;
  if (workspace && !aligned16(workspace)) return DCPMLA_ERR_ALIGNMENT;
  if (!workspace || workspace_bytes < layout(batch * q_len, num_heads, block_table_stride).total)
    return DCPMLA_ERR_WORKSPACE;
  p.out_blocks = out_blocks;
  p.out_table = out_table;
  p.out_lens = out_lens;
  p.flags = static_cast<int*>(workspace);
  return run_select(p, static_cast<uint8_t*>(workspace), static_cast<cudaStream_t>(stream));
}

// Workspace of mla_decode_blocks: the decode's own (its flag word is the
// call's: the choice reports into it too), the choice's, the chosen tables and
// lengths.
int mla_decode_blocks_workspace_size(int batch, int num_heads, int q_len, int block_table_stride,
                                     int block_topk, int num_splits, size_t* bytes) {
  if (!bytes || block_topk < 1) return DCPMLA_ERR_INVALID_ARGUMENT;
  int rc = check_sizes(batch, num_heads, q_len, block_table_stride);
  if (rc != DCPMLA_OK) return rc;
  size_t dec = 0;
  const int rows = batch * q_len;
  rc = mla_decode_workspace_size(rows, num_heads, num_splits, 0, &dec);
  if (rc != DCPMLA_OK) return rc;
  *bytes = round256(dec) + layout(rows, num_heads, block_table_stride).total +
           round256((size_t)rows * block_topk * 4) + round256((size_t)rows * 4);
  return DCPMLA_OK;
}

int mla_decode_blocks(const void* q, const void* kv_cache, int kv_dtype, const void* summaries,
                      int64_t num_blocks, int block_size, const int32_t* block_table,
                      int block_table_stride, const int32_t* seq_lens, int batch, int num_heads,
                      int q_len, int shard_id, int num_shards, int block_topk, int sink_blocks,
                      int recent_blocks, float softmax_scale, float* out_partial, float* out_lse,
                      int32_t* out_blocks, void* workspace, size_t workspace_bytes,
                      int num_splits, int impl, void* stream) {
  // everything the decode below would refuse is refused here, before the choice is launched
  SelectArgs a{q, summaries, num_blocks, block_size, block_table, block_table_stride, seq_lens,
               batch, num_heads, q_len, shard_id, num_shards, block_topk, sink_blocks,
               recent_blocks};
  SelectParams p;
  int rc = check_select(a, &p);
  if (rc != DCPMLA_OK) return rc;
  if ((kv_dtype != DCPMLA_KV_BF16 && kv_dtype != DCPMLA_KV_FP8) || num_splits < 0 ||
      !std::isfinite(softmax_scale) ||
      (impl != DCPMLA_IMPL_AUTO && impl != DCPMLA_IMPL_SIMT && impl != DCPMLA_IMPL_TC &&
       impl != DCPMLA_IMPL_TC_F16))
    return DCPMLA_ERR_INVALID_ARGUMENT;
  if (batch == 0) return DCPMLA_OK;
  if (!kv_cache || !out_partial || !out_lse) return DCPMLA_ERR_INVALID_ARGUMENT;
  if (!aligned16(kv_cache) || !aligned16(out_partial) || (workspace && !aligned16(workspace)))
    return DCPMLA_ERR_ALIGNMENT;
  size_t need = 0, dec = 0;
  const int rows = batch * q_len;
  rc = mla_decode_blocks_workspace_size(batch, num_heads, q_len, block_table_stride, block_topk,
                                        num_splits, &need);
  if (rc != DCPMLA_OK) return rc;
  if (!workspace || workspace_bytes < need) return DCPMLA_ERR_WORKSPACE;
  rc = mla_decode_workspace_size(rows, num_heads, num_splits, 0, &dec);
  if (rc != DCPMLA_OK) return rc;
  uint8_t* sel = static_cast<uint8_t*>(workspace) + round256(dec);
  p.out_blocks = out_blocks;
  p.out_table = reinterpret_cast<int*>(sel + layout(rows, num_heads, block_table_stride).total);
  p.out_lens = p.out_table + round256((size_t)rows * block_topk * 4) / 4;
  p.flags = static_cast<int*>(workspace);
  rc = run_select(p, sel, static_cast<cudaStream_t>(stream));
  if (rc != DCPMLA_OK) return rc;
  // the chosen blocks of a query are one request of one shard, in a table of their own
  return mla_decode_partial(q, kv_cache, kv_dtype, num_blocks, block_size, p.out_table, block_topk,
                            p.out_lens, rows, num_heads, 0, 1, nullptr, 0, softmax_scale,
                            out_partial, out_lse, workspace, dec, num_splits, impl, stream);
}

}  // extern "C"
