// Block summaries: for every 64-row cache block of a request, the mean of its
// rows (all 576 values, rope included) as int8 codes with one fp32 scale per
// group of 128 latent values and one for the 64 rope values.
//
//   m_d = (1/n) sum_r k_rd over the block's n rows of the request,
//   scale_g = max_{d in g} |m_d| * fp32(1/127) (1 if that is 0),
//   code_d = rint(m_d / scale_g).
//
// Sums are fp32 (a row's value is its code times its scale, fused into the
// add).  A mean that is not finite counts as 0, so that one bad value cannot
// take a whole block's code range.
//
// HBM bounds it: every row is read once and 608 bytes of 42 or 74 KB written.  64
// requests of 779,084 fp8 rows take 93 us (5.5 TB/s), 32 of 1,024 bf16 rows 9.6 us;
// per further row 5.2 TB/s (fp8) and 6.2 (bf16).  Turning e4m3 codes into values is
// next: 63 % of the issue slots at fp8.
#include "dcpmla.h"

#include <algorithm>
#include <mutex>

#include "common.cuh"
#include "kernels.h"
#include "q_image.cuh"
#include "tc_ptx.cuh"

namespace dcpmla {
namespace {

// One group of threads per resident block: it waits for the block's rows in
// its own stage of shared memory, sums them in four phases of every fourth
// row, and adds the phases up; the next block's rows land while the sums are
// turned into codes.
//   fp8:  warps 0-3 take the 512 codes (16 a lane) of phase = warp, warp 4 the
//         rope (8 lanes of 8 values a phase).
//   bf16: 72 lanes of 8 values a phase, 9 warps.
template <int kDtype>
struct Shape;
template <>
struct Shape<kKvFp8> {
  static constexpr int kRowBytes = kRowBytesFp8, kStages = 4, kGroupThreads = 160;
};
template <>
struct Shape<kKvBf16> {
  static constexpr int kRowBytes = kRowBytesBf16, kStages = 2, kGroupThreads = 288;
};

constexpr int kChunk = 1024;      // requests looked at together
constexpr int kPhases = 4;

struct SummaryParams {
  const uint8_t* kv;
  long long num_blocks;
  const int* block_table;
  int bt_stride;
  const int* seq_lens;
  const int* first_positions;     // nullptr: every block
  int batch, shard, nshards;
  uint8_t* summaries;
  int* flags;
};

// First block of request b to summarise and the blocks from there to its end.
__device__ __forceinline__ int units_of(const SummaryParams& p, int b, int* first, int* rows) {
  int L = __ldg(p.seq_lens + b);
  bool bad = L < 0;
  if (bad) L = 0;
  int n = local_len(L, p.shard, p.nshards);
  int nb = n > 0 ? (n - 1) / kBlock + 1 : 0;
  if (nb > p.bt_stride) {
    bad = true;
    nb = p.bt_stride;
    n = nb * kBlock;
  }
  int k0 = 0;
  if (p.first_positions) {
    const int t = max(0, __ldg(p.first_positions + b));
    k0 = local_len(t, p.shard, p.nshards) / kBlock;
    if (local_len(t, p.shard, p.nshards) >= n) k0 = nb;      // nothing new on this shard
  }
  if (bad && p.flags) atomicOr(p.flags, kFlagBadLength);
  *first = k0;
  *rows = n;
  return max(0, nb - k0);
}

template <int kDtype>
__global__ void __launch_bounds__(Shape<kDtype>::kStages* Shape<kDtype>::kGroupThreads, 1)
    summary_kernel(const SummaryParams p) {
  using S = Shape<kDtype>;
  constexpr uint32_t kStageBytes = kBlock * S::kRowBytes;
  constexpr int kThreads = S::kStages * S::kGroupThreads;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int s_end[kChunk];           // units up to and including request i of the chunk
  __shared__ int s_first[kChunk], s_rows[kChunk];
  __shared__ int warp_sums[32];
  __shared__ uint64_t full[S::kStages];
  __shared__ int s_abort;
  const int group = threadIdx.x / S::kGroupThreads, t = threadIdx.x % S::kGroupThreads;
  const int warp = t >> 5, lane = t & 31;
  uint8_t* stage = smem + group * kStageBytes;
  float* part = reinterpret_cast<float*>(smem + S::kStages * kStageBytes) + group * kPhases * kHeadDim;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; ++s) ptx::mbar_init(&full[s], 1);
    s_abort = 0;
    ptx::fence_mbar_init();
  }
  uint32_t loads = 0;
  for (int b0 = 0; b0 < p.batch; b0 += kChunk) {
    __syncthreads();
    if (s_abort) break;
    int total = 0;
    for (int i0 = 0; i0 < kChunk; i0 += kThreads) {
      const int i = i0 + threadIdx.x;
      int first = 0, rows = 0, u = 0;
      if (i < kChunk && b0 + i < p.batch) u = units_of(p, b0 + i, &first, &rows);
      int tot;
      const int ex = block_exclusive_scan(u, warp_sums, &tot);
      if (i < kChunk) {
        s_end[i] = total + ex + u;
        s_first[i] = first;
        s_rows[i] = rows;
      }
      total += tot;
    }
    __syncthreads();
    const int step = gridDim.x * S::kStages;
    // block of unit u: its place in the pool (-1: bad table entry) and rows
    auto locate = [&](int u, int* rows) {
      int lo = 0, hi = kChunk - 1;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (s_end[mid] > u) hi = mid; else lo = mid + 1;
      }
      const int k = s_first[lo] + u - (lo > 0 ? s_end[lo - 1] : 0);
      *rows = min(kBlock, s_rows[lo] - k * kBlock);
      const int blk = __ldg(p.block_table + (size_t)(b0 + lo) * p.bt_stride + k);
      if (blk < 0 || (long long)blk >= p.num_blocks) {
        if (p.flags) atomicOr(p.flags, kFlagBadBlock);
        return -1;
      }
      return blk;
    };
    int u = blockIdx.x + gridDim.x * group, rows = 0, blk = -1;
    auto fetch = [&]() {
      if (blk >= 0) {
        if (t == 0) {
          ptx::mbar_arrive_expect_tx(&full[group], rows * S::kRowBytes);
          ptx::bulk_g2s(ptx::smem_addr(stage), p.kv + (size_t)blk * kStageBytes, rows * S::kRowBytes,
                        &full[group]);
        }
      }
    };
    if (u < total) {
      blk = locate(u, &rows);
      fetch();
    }
    while (u < total) {
      const int cur = blk, n = rows;
      if (cur >= 0) {
        if (!ptx::mbar_wait(&full[group], loads & 1, &s_abort)) break;
        ++loads;
        float acc[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[i] = 0.f;
        if constexpr (kDtype == kKvFp8) {
          if (warp < kPhases) {
#pragma unroll 4
            for (int r = warp; r < n; r += kPhases) {
              const uint8_t* row = stage + r * S::kRowBytes;
              const uint4 c = *reinterpret_cast<const uint4*>(row + 16 * lane);
              const float s = *reinterpret_cast<const float*>(row + 512 + 4 * (lane >> 3));
              const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float2 a = qimg::e4m3x2_to_f32(w[e] & 0xFFFFu);
                const float2 b = qimg::e4m3x2_to_f32(w[e] >> 16);
                acc[4 * e] = fmaf(a.x, s, acc[4 * e]);
                acc[4 * e + 1] = fmaf(a.y, s, acc[4 * e + 1]);
                acc[4 * e + 2] = fmaf(b.x, s, acc[4 * e + 2]);
                acc[4 * e + 3] = fmaf(b.y, s, acc[4 * e + 3]);
              }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
              *reinterpret_cast<float4*>(part + warp * kHeadDim + 16 * lane + 4 * e) =
                  make_float4(acc[4 * e], acc[4 * e + 1], acc[4 * e + 2], acc[4 * e + 3]);
          } else {
            const int ph = lane >> 3, un = lane & 7;
#pragma unroll 4
            for (int r = ph; r < n; r += kPhases) {
              const uint4 c = *reinterpret_cast<const uint4*>(stage + r * S::kRowBytes + 528 + 16 * un);
              const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                acc[2 * e] += __uint_as_float(w[e] << 16);
                acc[2 * e + 1] += __uint_as_float(w[e] & 0xFFFF0000u);
              }
            }
            float* o = part + ph * kHeadDim + kVDim + 8 * un;
            *reinterpret_cast<float4*>(o) = make_float4(acc[0], acc[1], acc[2], acc[3]);
            *reinterpret_cast<float4*>(o + 4) = make_float4(acc[4], acc[5], acc[6], acc[7]);
          }
        } else {
          const int ph = t / 72, un = t % 72;
#pragma unroll 4
          for (int r = ph; r < n; r += kPhases) {
            const uint4 c = *reinterpret_cast<const uint4*>(stage + r * S::kRowBytes + 16 * un);
            const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              acc[2 * e] += __uint_as_float(w[e] << 16);
              acc[2 * e + 1] += __uint_as_float(w[e] & 0xFFFF0000u);
            }
          }
          float* o = part + ph * kHeadDim + 8 * un;
          *reinterpret_cast<float4*>(o) = make_float4(acc[0], acc[1], acc[2], acc[3]);
          *reinterpret_cast<float4*>(o + 4) = make_float4(acc[4], acc[5], acc[6], acc[7]);
        }
      }
      ptx::named_bar(1 + group, S::kGroupThreads);       // stage read, phases written
      u += step;
      blk = -1;
      if (u < total) {
        blk = locate(u, &rows);
        fetch();
      }
      if (cur >= 0 && warp < 5) {
        // warp g: latent group g, four values a lane; warp 4: the rope, two
        const int v = warp < 4 ? 4 : 2, d = warp < 4 ? 128 * warp + 4 * lane : kVDim + 2 * lane;
        float m[4] = {0.f, 0.f, 0.f, 0.f};
        for (int ph = 0; ph < kPhases; ++ph)
          for (int e = 0; e < v; ++e) m[e] += part[ph * kHeadDim + d + e];
        float amax = 0.f;
        const float cnt = (float)n;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          m[e] = __fdiv_rn(m[e], cnt);
          if (!(fabsf(m[e]) <= 3.4028234663852886e38f)) m[e] = 0.f;
          amax = fmaxf(amax, fabsf(m[e]));
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        const float up = __fmul_rn(amax, kInv127), sc = up > 0.f ? up : 1.f;
        uint32_t code = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int q = min(127, max(-127, __float2int_rn(__fdiv_rn(m[e], sc))));
          code |= ((uint32_t)q & 0xFFu) << (8 * e);
        }
        uint8_t* o = p.summaries + (size_t)cur * kSummaryBytes;
        if (warp < 4)
          *reinterpret_cast<uint32_t*>(o + d) = code;
        else
          *reinterpret_cast<uint16_t*>(o + d) = (uint16_t)code;
        if (lane == 0) reinterpret_cast<float*>(o + kHeadDim)[warp] = sc;
        if (warp == 4 && lane < 3) reinterpret_cast<uint32_t*>(o + kHeadDim + 20)[lane] = 0u;
      }
      ptx::named_bar(1 + group, S::kGroupThreads);       // phases read
    }
  }
  __syncthreads();
  if (s_abort && threadIdx.x == 0 && p.flags) atomicOr(p.flags, DCPMLA_FLAG_TIMEOUT);
}

std::mutex g_mutex;
bool g_done[2][kMaxDevicesConfigured] = {};

template <int kDtype>
cudaError_t launch_summary(const SummaryParams& p, int ctas, int dev, cudaStream_t st) {
  using S = Shape<kDtype>;
  const int smem = S::kStages * (kBlock * S::kRowBytes + kPhases * kHeadDim * 4);
  {
    std::lock_guard<std::mutex> lock(g_mutex);
    if (!g_done[kDtype][dev]) {
      cudaError_t e = cudaFuncSetAttribute(summary_kernel<kDtype>,
                                           cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (e != cudaSuccess) return e;
      g_done[kDtype][dev] = true;
    }
  }
  summary_kernel<kDtype><<<ctas, S::kStages * S::kGroupThreads, smem, st>>>(p);
  return cudaGetLastError();
}

bool aligned16(const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0; }

}  // namespace
}  // namespace dcpmla

using namespace dcpmla;

extern "C" int mla_block_summary(const void* kv_cache, int kv_dtype, int64_t num_blocks,
                                 int block_size, const int32_t* block_table, int block_table_stride,
                                 const int32_t* seq_lens, const int32_t* first_positions, int batch,
                                 int shard_id, int num_shards, void* summaries, int32_t* flags,
                                 void* stream) {
  if (batch < 0 || block_table_stride < 1 || num_shards < 1 || shard_id < 0 ||
      shard_id >= num_shards || num_blocks < 1 || block_size < 1)
    return DCPMLA_ERR_INVALID_ARGUMENT;
  if (kv_dtype != DCPMLA_KV_BF16 && kv_dtype != DCPMLA_KV_FP8) return DCPMLA_ERR_INVALID_ARGUMENT;
  if (block_size != kBlock) return DCPMLA_ERR_UNSUPPORTED;
  if (batch == 0) return DCPMLA_OK;
  if (!kv_cache || !block_table || !seq_lens || !summaries) return DCPMLA_ERR_INVALID_ARGUMENT;
  if (!aligned16(kv_cache) || !aligned16(summaries)) return DCPMLA_ERR_ALIGNMENT;
  int ctas = 0, dev = 0;
  int rc = dcpmla_device_sm_count(&ctas);
  if (rc != DCPMLA_OK) return rc;
  if (cudaGetDevice(&dev) != cudaSuccess) return DCPMLA_ERR_CUDA;
  SummaryParams p{};
  p.kv = static_cast<const uint8_t*>(kv_cache);
  p.num_blocks = num_blocks;
  p.block_table = block_table;
  p.bt_stride = block_table_stride;
  p.seq_lens = seq_lens;
  p.first_positions = first_positions;
  p.batch = batch;
  p.shard = shard_id;
  p.nshards = num_shards;
  p.summaries = static_cast<uint8_t*>(summaries);
  p.flags = flags;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = kv_dtype == DCPMLA_KV_FP8 ? launch_summary<kKvFp8>(p, ctas, dev, st)
                                                  : launch_summary<kKvBf16>(p, ctas, dev, st);
  return e == cudaSuccess ? DCPMLA_OK : DCPMLA_ERR_CUDA;
}
