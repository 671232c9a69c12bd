// Accumulated attention weight of every cached row: for the query tokens of a
// step and the log-sum-exp of their full attention (the merged LSE under DCP),
//
//   mass[b][j] = decay * mass[b][j] + sum_{i, h} exp(scale * q_bih . k_bj - lse_bih)
//
// over this shard's rows j, query i seeing the rows at positions up to
// L_b - q_len + i.  An LSE of -inf (a query that saw nothing) adds nothing.
// Each row is summed by one thread in a fixed order: no atomics, the same bits
// every time.
#include "dcpmla.h"

#include <cmath>
#include <mutex>

#include "common.cuh"
#include "kernels.h"
#include "q_image.cuh"

namespace dcpmla {
namespace {

struct MassParams {
  PartialParams p;       // cache, table, lengths, schedule; q rows of this pass
  const float* lse;      // [batch][rows_o]: this pass's rows first
  float* mass;
  long long mass_stride;
  float decay;
  int kv_dtype;
};

constexpr int kThreads = 256;
constexpr int kKStride = kHeadDim + 1;

__global__ void __launch_bounds__(kThreads) mass_kernel(const MassParams m) {
  extern __shared__ __align__(16) uint8_t smem[];
  float* k = reinterpret_cast<float*>(smem);                                   // [64][577]
  __nv_bfloat16* q = reinterpret_cast<__nv_bfloat16*>(smem + kBlock * kKStride * 4);
  __shared__ float part[4][kBlock];
  __shared__ int warp_sums[32];
  __shared__ Segment list[kThreads];
  __shared__ int list_n;
  const PartialParams& p = m.p;
  const int T = total_tiles(p, warp_sums);
  const int tpc = T > 0 ? (T + p.num_ctas - 1) / p.num_ctas : 0;
  const int lo = blockIdx.x * tpc, hi = min(T, lo + tpc);
  const int hpq = p.heads / p.q_len;
  for_each_dense_segment(p, lo, hi, warp_sums, list, &list_n, [&](const Segment& s) {
    __syncthreads();
    for (int i = threadIdx.x; i < p.heads * kHeadDim; i += kThreads)
      q[i] = p.q[(size_t)s.b * p.rows_q * kHeadDim + i];
    const int last = seq_len_of(p, s.b) - p.q_len;       // position of query 0
    for (int t = s.t0; t < s.t1; ++t) {
      __syncthreads();
      const int blk = tile_block(p, s.b, t);
      if (blk < 0) continue;
      const int n = min(kBlock, s.n_rows - t * kBlock);
      const int rb = m.kv_dtype == kKvBf16 ? kRowBytesBf16 : kRowBytesFp8;
      const uint8_t* rows = p.kv + (size_t)blk * kBlock * rb;
      for (int i = threadIdx.x; i < n * (kHeadDim / 2); i += kThreads) {
        const int r = i / (kHeadDim / 2), d = i % (kHeadDim / 2) * 2;
        const uint8_t* row = rows + (size_t)r * rb;
        float2 v;
        if (m.kv_dtype == kKvFp8 && d < kVDim) {
          const float sc = reinterpret_cast<const float*>(row + 512)[d / 128];
          v = qimg::e4m3x2_to_f32(*reinterpret_cast<const uint16_t*>(row + d));
          v.x *= sc;
          v.y *= sc;
        } else {
          const uint32_t w = *reinterpret_cast<const uint32_t*>(
              row + (m.kv_dtype == kKvFp8 ? 528 + 2 * (d - kVDim) : 2 * d));
          v = make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
        }
        k[r * kKStride + d] = v.x;
        k[r * kKStride + d + 1] = v.y;
      }
      __syncthreads();
      const int r = threadIdx.x & 63, quarter = threadIdx.x >> 6;
      const int pos = (t * kBlock + r) * p.nshards + p.shard;
      float sum = 0.f;
      if (r < n)
        for (int h = quarter; h < p.heads; h += 4) {
          const float lse = m.lse[(size_t)s.b * p.rows_o + h];
          if (pos > last + h / hpq || lse == -INFINITY) continue;
          float dot = 0.f;
          for (int d = 0; d < kHeadDim; ++d)
            dot = fmaf(__bfloat162float(q[h * kHeadDim + d]), k[r * kKStride + d], dot);
          sum += expf(p.scale * dot - lse);
        }
      part[quarter][r] = sum;
      __syncthreads();
      if (threadIdx.x < n && (long long)t * kBlock + threadIdx.x >= m.mass_stride) {
        if (p.flags) atomicOr(p.flags, kFlagBadLength);
      } else if (threadIdx.x < n) {
        float* o = m.mass + (size_t)s.b * m.mass_stride + t * kBlock + threadIdx.x;
        const float add = (part[0][threadIdx.x] + part[1][threadIdx.x]) +
                          (part[2][threadIdx.x] + part[3][threadIdx.x]);
        *o = m.decay == 0.f ? add : fmaf(m.decay, *o, add);
      }
    }
  });
}

bool aligned16(const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0; }
size_t round256(size_t x) { return (x + 255) & ~(size_t)255; }

std::mutex g_mutex;
bool g_done[kMaxDevicesConfigured] = {};

size_t mass_bytes(int batch) { return kWsHeader + round256((size_t)batch * kQImageBytes); }

int check_sizes(int batch, int heads, int q_len) {
  if (batch < 0 || heads < 1 || q_len < 1 || q_len > kMaxQueryLen) return DCPMLA_ERR_INVALID_ARGUMENT;
  return heads > kMaxHeads ? DCPMLA_ERR_UNSUPPORTED : DCPMLA_OK;
}

}  // namespace
}  // namespace dcpmla

using namespace dcpmla;

extern "C" {

int mla_attention_mass_workspace_size(int batch, int num_heads, int q_len, size_t* bytes) {
  if (!bytes) return DCPMLA_ERR_INVALID_ARGUMENT;
  const int rc = check_sizes(batch, num_heads, q_len);
  if (rc != DCPMLA_OK) return rc;
  *bytes = mass_bytes(batch);
  return DCPMLA_OK;
}

int mla_attention_mass(const void* q, const void* kv_cache, int kv_dtype, int64_t num_blocks,
                       int block_size, const int32_t* block_table, int block_table_stride,
                       const int32_t* seq_lens, int batch, int num_heads, int q_len, int shard_id,
                       int num_shards, float softmax_scale, const float* lse, float decay,
                       float* mass, int64_t mass_stride, void* workspace, size_t workspace_bytes,
                       int num_splits, void* stream) {
  if (block_table_stride < 1 || num_shards < 1 || shard_id < 0 || shard_id >= num_shards ||
      num_blocks < 1 || block_size < 1 || num_splits < 0 || mass_stride < 1 ||
      !std::isfinite(softmax_scale) || !std::isfinite(decay) || decay < 0.f)
    return DCPMLA_ERR_INVALID_ARGUMENT;
  int rc = check_sizes(batch, num_heads, q_len);
  if (rc != DCPMLA_OK) return rc;
  if (kv_dtype != DCPMLA_KV_BF16 && kv_dtype != DCPMLA_KV_FP8) return DCPMLA_ERR_INVALID_ARGUMENT;
  if (block_size != kBlock) return DCPMLA_ERR_UNSUPPORTED;
  if (batch == 0) return DCPMLA_OK;
  if (!q || !kv_cache || !block_table || !seq_lens || !lse || !mass)
    return DCPMLA_ERR_INVALID_ARGUMENT;
  if (!aligned16(q) || !aligned16(kv_cache) || (workspace && !aligned16(workspace)))
    return DCPMLA_ERR_ALIGNMENT;
  if (!workspace || workspace_bytes < mass_bytes(batch)) return DCPMLA_ERR_WORKSPACE;
  int dev = 0, ctas = num_splits;
  if (ctas == 0) {
    rc = dcpmla_device_sm_count(&ctas);
    if (rc != DCPMLA_OK) return rc;
  }
  if (cudaGetDevice(&dev) != cudaSuccess) return DCPMLA_ERR_CUDA;
  if (dev < 0 || dev >= kMaxDevicesConfigured) return DCPMLA_ERR_UNSUPPORTED;
  const int smem = kBlock * kKStride * 4 + kMaxHeads * kHeadDim * 2;
  {
    std::lock_guard<std::mutex> lock(g_mutex);
    if (!g_done[dev]) {
      if (cudaFuncSetAttribute(mass_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) !=
          cudaSuccess)
        return DCPMLA_ERR_CUDA;
      g_done[dev] = true;
    }
  }
  MassParams m{};
  PartialParams& p = m.p;
  p.kv = static_cast<const uint8_t*>(kv_cache);
  p.num_blocks = num_blocks;
  p.block_table = block_table;
  p.bt_stride = block_table_stride;
  p.seq_lens = seq_lens;
  p.batch = batch;
  p.shard = shard_id;
  p.nshards = num_shards;
  p.scale = softmax_scale;
  p.rows_q = p.rows_o = num_heads * q_len;
  p.flags = static_cast<int*>(workspace);
  p.num_ctas = ctas;
  m.mass = mass;
  m.mass_stride = mass_stride;
  m.kv_dtype = kv_dtype;
  // As many whole queries as fit 64 rows in a pass over the cache, in order
  // on the stream.  The last queries come first: they see every row, so that
  // their pass is the one that applies the decay.
  const int per = kMaxHeads / num_heads;
  for (int k1 = q_len; k1 > 0; k1 -= per) {
    const int k0 = k1 > per ? k1 - per : 0, n = k1 - k0;
    p.q = static_cast<const __nv_bfloat16*>(q) + (size_t)k0 * num_heads * kHeadDim;
    p.heads = n * num_heads;
    p.q_len = n;
    p.len_delta = q_len - k1;
    m.lse = lse + (size_t)k0 * num_heads;
    m.decay = k1 == q_len ? decay : 1.f;
    mass_kernel<<<ctas, kThreads, smem, static_cast<cudaStream_t>(stream)>>>(m);
    if (cudaGetLastError() != cudaSuccess) return DCPMLA_ERR_CUDA;
  }
  return DCPMLA_OK;
}

}  // extern "C"
