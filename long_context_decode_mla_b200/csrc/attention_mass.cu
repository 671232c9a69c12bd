// Accumulated attention weight of every cached row, on the tensor cores
// (tcgen05 / TMEM / TMA, sm_100a): for the query tokens of a step and the
// log-sum-exp of their full attention (the merged LSE under DCP),
//
//   mass[b][j] = decay * mass[b][j] + sum_{i, h} exp(scale * q_bih . k_bj - lse_bih)
//
// over this shard's rows j, query i seeing the rows at positions up to
// L_b - q_len + i.  An LSE of -inf (a query that saw nothing) adds nothing.
//
// With the LSE given there is no softmax to carry from row to row: a row's
// weight needs its own scores only.  So the scores are computed transposed to
// the decode kernels', D = K Q^T with the 64 rows of a cache block as M and the
// (query, head) rows as N: a TMEM lane then holds one cached row for 32 heads,
// a row's fp32 scales are one thread's registers, and the sum over heads stays
// in a thread but for one exchange between the two lane halves.  Rows past a
// request's end only ever reach their own lanes, so nothing is cleared.
//
//  * fp8 rows: the e4m3 codes are the A operand as they are; Q comes as the
//    decode kernel's operand image (two e4m3 terms in one power-of-two frame,
//    q_image.cuh).  Every 128-value scale group has an accumulator of its own,
//    scaled in fp32, and the bf16 rope a fifth.
//  * bf16 rows and queries multiply as they are (exact products).
//
// A tile is one cache block, loaded by TMA into a stage of its own (fp8: three
// stages of 41 KB; bf16: two of 72 KB), prefetched into L2 six tiles ahead.
// Warps 0-3 and 4-7 turn alternate tiles into weights; warp 8 loads; warp 9
// issues the MMAs (36 a tile).  Tiles are dealt to the CTAs as in decode.  Each
// row is summed by the same threads in the same order whatever the number of
// CTAs: no atomics, the same bits every time.  Every wait is bounded.
#include "dcpmla.h"

#include <cuda.h>

#include <cmath>
#include <mutex>

#include "common.cuh"
#include "kernels.h"
#include "q_image.cuh"
#include "schedule.cuh"
#include "tc_ptx.cuh"

namespace dcpmla {
namespace {

struct MassParams {
  PartialParams p;       // cache, table, lengths, schedule; q rows of this pass
  const float* lse;      // [batch][rows_o]: this pass's rows first
  float* mass;
  long long mass_stride;
  float decay;
  CUtensorMap rows;      // [blocks][64][row bytes] u8, box 128 x 64, 128-byte swizzle
  CUtensorMap scales;    // fp8: the same, box 16 x 64 (the four fp32 scales)
  CUtensorMap q;         // bf16: [batch][rows][1152] u8, box 128 x 64, rows past the pass zero
};

constexpr int kThreads = 320;
constexpr int kLoadWarp = 8, kMmaWarp = 9;
constexpr int kGroupThreads = 128;
constexpr uint32_t kChunk = 8192;                  // 64 rows x 128 bytes
constexpr int kBufs = 3;                           // TMEM accumulator sets
constexpr uint32_t kTmemCols = 512;
constexpr int kPrefetchTiles = 6;
constexpr int kMaxSeg = 64;
constexpr float kLog2e = 1.4426950408889634f;

template <int kDtype>
struct Shape;
template <>
struct Shape<kKvFp8> {
  static constexpr int kRowBytes = kRowBytesFp8, kStages = 3, kChunks = 5, kParts = 5;
  static constexpr uint32_t kStageBytes = 5 * kChunk + 1024, kScales = 5 * kChunk;
  static constexpr uint32_t kQBytes = 9 * kChunk;   // hi, lo, rope
};
template <>
struct Shape<kKvBf16> {
  static constexpr int kRowBytes = kRowBytesBf16, kStages = 2, kChunks = 9, kParts = 1;
  static constexpr uint32_t kStageBytes = 9 * kChunk, kScales = 0;
  static constexpr uint32_t kQBytes = 9 * kChunk;
};

struct Ctl {
  uint64_t full[3], empty[3];          // per stage: bytes landed / MMAs and reads done
  uint64_t d_full[kBufs], d_empty[kBufs];
  uint64_t q_full, q_empty;
  alignas(16) float2 head[2][64];      // per weight group: 2^-a scale log2(e), lse log2(e)
  float half[2][2][64];                // [group][parity]: the other lane half's sums
  int nv[3];                           // rows of the stage's tile that take part
  uint32_t tmem_base;
  int abort;
  int sel_count;
  int warp_sums[16];
  Segment seg[kMaxSeg];
};

template <int kDtype>
constexpr size_t smem_bytes() {
  return Shape<kDtype>::kQBytes + (size_t)Shape<kDtype>::kStages * Shape<kDtype>::kStageBytes +
         sizeof(Ctl) + 1024;
}
static_assert(smem_bytes<kKvFp8>() <= 232448 && smem_bytes<kKvBf16>() <= 232448, "shared memory");

__device__ __forceinline__ uint64_t dplus(uint64_t d, uint32_t byte_off) {
  return d + (uint64_t)(byte_off >> 4);
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

struct Counts {
  uint32_t tau = 0, sigma = 0;     // tiles and requests handled so far
};

// TMA loads of every tile, and of each request's Q once the previous
// request's MMAs are done with it.
template <int kDtype>
__device__ __forceinline__ void load_role(const MassParams& m, Ctl& c, uint8_t* base, int nseg,
                                          Counts& n) {
  using S = Shape<kDtype>;
  const PartialParams& p = m.p;
  TileCursor cur, pf;
  if (!cur.start(p, c, nseg)) return;
  pf = cur;
  bool pf_ok = true;
  constexpr uint32_t kTile = 64 * S::kRowBytes;
  auto prefetch = [&]() {
    if (!pf_ok) return;
    const int blk = tile_block(p, pf.v.b, (pf.v.row_begin >> 6) + pf.t);
    if (blk >= 0) ptx::prefetch_l2(p.kv + (size_t)blk * kTile, kTile);
    pf_ok = pf.next(p, c);
  };
  for (int i = 0; i < kPrefetchTiles; ++i) prefetch();
  while (true) {
    const uint32_t s = n.tau % S::kStages;
    if (n.tau >= (uint32_t)S::kStages &&
        !ptx::mbar_wait(&c.empty[s], ((n.tau / S::kStages) + 1) & 1, &c.abort))
      return;
    const int blk = tile_block(p, cur.v.b, (cur.v.row_begin >> 6) + cur.t);
    const int z = blk >= 0 ? blk : 0;        // a bad entry: a stand-in block, no rows
    c.nv[s] = blk >= 0 ? cur.tile_valid_rows() : 0;
    const uint32_t dst = ptx::smem_addr(base + S::kQBytes + s * S::kStageBytes);
    ptx::mbar_arrive_expect_tx(&c.full[s], kTile);
#pragma unroll
    for (int k = 0; k < S::kChunks; ++k)
      ptx::tma_load_3d(dst + k * kChunk, &m.rows, kDtype == kKvFp8 && k == 4 ? 528 : 128 * k, 0, z,
                       &c.full[s]);
    if constexpr (kDtype == kKvFp8)
      ptx::tma_load_3d(dst + S::kScales, &m.scales, 512, 0, z, &c.full[s]);
    if (cur.t == 0) {
      if (n.sigma > 0 && !ptx::mbar_wait(&c.q_empty, (n.sigma - 1) & 1, &c.abort)) return;
      const uint32_t dq = ptx::smem_addr(base);
      ptx::mbar_arrive_expect_tx(&c.q_full, S::kQBytes);
      if constexpr (kDtype == kKvFp8) {
        ptx::bulk_g2s(dq, p.q_image + (size_t)cur.v.b * kQImageBytes, S::kQBytes, &c.q_full);
      } else {
#pragma unroll
        for (int k = 0; k < 9; ++k)
          ptx::tma_load_3d(dq + k * kChunk, &m.q, 128 * k, 0, cur.v.b, &c.q_full);
      }
      ++n.sigma;
    }
    ++n.tau;
    prefetch();
    if (!cur.next(p, c)) break;
  }
}

// D = K Q^T of every tile (weight-stationary M = 64 rows, N = 64 heads, 32
// TMEM columns a part).
template <int kDtype>
__device__ __forceinline__ void mma_role(const MassParams& m, Ctl& c, uint8_t* base, int nseg,
                                         Counts& n) {
  using S = Shape<kDtype>;
  constexpr uint32_t kIdF8 = ptx::idesc_make(64, 64, 0, false, false);
  constexpr uint32_t kIdBf = ptx::idesc_make(64, 64, 1, false, false);
  const uint64_t dq = ptx::sdesc(ptx::smem_addr(base), 16, 1024, ptx::kSwizzle128B);
  const uint64_t dk0 = ptx::sdesc(ptx::smem_addr(base + S::kQBytes), 16, 1024, ptx::kSwizzle128B);
  TileCursor cur;
  if (!cur.start(m.p, c, nseg)) return;
  while (true) {
    const uint32_t s = n.tau % S::kStages, buf = n.tau % kBufs;
    if (cur.t == 0) {
      if (!ptx::mbar_wait(&c.q_full, n.sigma & 1, &c.abort)) return;
      ++n.sigma;
    }
    if (n.tau >= (uint32_t)kBufs &&
        !ptx::mbar_wait(&c.d_empty[buf], ((n.tau / kBufs) + 1) & 1, &c.abort))
      return;
    if (!ptx::mbar_wait(&c.full[s], (n.tau / S::kStages) & 1, &c.abort)) return;
    ptx::tc_fence_after();
    const uint64_t dk = dplus(dk0, s * S::kStageBytes);
    const uint32_t d = c.tmem_base + buf * (32 * S::kParts);
    if constexpr (kDtype == kKvFp8) {
#pragma unroll 1
      for (int g = 0; g < 4; ++g)
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          const uint32_t off = g * kChunk + ks * 32;
          ptx::mma_ws_f8(d + 32 * g, dplus(dk, off), dplus(dq, off), kIdF8, ks > 0);
          ptx::mma_ws_f8(d + 32 * g, dplus(dk, off), dplus(dq, 4 * kChunk + off), kIdF8, 1u);
        }
#pragma unroll
      for (int ks = 0; ks < 4; ++ks)
        ptx::mma_ws_f16(d + 128, dplus(dk, 4 * kChunk + ks * 32), dplus(dq, 8 * kChunk + ks * 32),
                        kIdBf, ks > 0);
    } else {
#pragma unroll 1
      for (int k = 0; k < 9; ++k)
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          ptx::mma_ws_f16(d, dplus(dk, k * kChunk + ks * 32), dplus(dq, k * kChunk + ks * 32),
                          kIdBf, (k | ks) != 0);
    }
    ptx::mma_commit(&c.empty[s]);
    ptx::mma_commit(&c.d_full[buf]);
    if (cur.last_of_segment()) ptx::mma_commit(&c.q_empty);
    ++n.tau;
    if (!cur.next(m.p, c)) break;
  }
}

// Weights of every other tile (tau % 2 == group): thread (q, i) of the group
// holds cached row (32 q + i) % 64 for 32 of the heads.
template <int kDtype>
__device__ __forceinline__ void weight_role(const MassParams& m, Ctl& c, uint8_t* base, int nseg,
                                            uint32_t& tau, uint32_t& mine) {
  using S = Shape<kDtype>;
  const PartialParams& p = m.p;
  const int group = threadIdx.x >> 7, t = threadIdx.x & 127;
  const int row = t & 63, hh = t >> 6, lane = t & 31;
  const uint32_t lane_base = c.tmem_base + ((uint32_t)((t >> 5) * 32) << 16);
  const int hpq = p.heads / p.q_len;
  const float sl2 = p.scale * kLog2e;
  int seg = -1;
  TileCursor cur;
  if (!cur.start(p, c, nseg)) return;
  while (true) {
    if ((int)(tau & 1) == group) {
      const uint32_t s = tau % S::kStages, buf = tau % kBufs;
      const int b = cur.v.b;
      if (cur.k != seg) {
        // the readers of the old factors passed the group's last barrier
        seg = cur.k;
        if (t < 64) {
          float2 f = make_float2(0.f, INFINITY);     // rows past the pass weigh nothing
          if (t < p.heads) {
            f.x = sl2;
            if constexpr (kDtype == kKvFp8)
              f.x *= __ldg(reinterpret_cast<const float*>(p.q_image + (size_t)b * kQImageBytes +
                                                          S::kQBytes) + t);
            const float l = __ldg(m.lse + (size_t)b * p.rows_o + t);
            f.y = l == -INFINITY ? INFINITY : l * kLog2e;
          }
          c.head[group][t] = f;
        }
        ptx::named_bar(1 + group, kGroupThreads);
      }
      const long long j = (long long)(cur.v.row_begin + cur.t * kTileRows) + row;
      const int last = seq_len_of(p, b) - p.q_len;         // position of query 0
      if (!ptx::mbar_wait(&c.full[s], (tau / S::kStages) & 1, &c.abort)) return;
      const int nv = c.nv[s];
      const bool live = row < nv && j < m.mass_stride;
      float* o = m.mass + (size_t)b * m.mass_stride + j;
      float old = 0.f;
      if (hh == 0 && live && m.decay != 0.f) old = *o;
      float sc[4] = {0.f, 0.f, 0.f, 0.f};
      if constexpr (kDtype == kKvFp8) {
        const float4 v = *reinterpret_cast<const float4*>(base + S::kQBytes + s * S::kStageBytes +
                                                          S::kScales + row * 16);
        sc[0] = v.x;
        sc[1] = v.y;
        sc[2] = v.z;
        sc[3] = v.w;
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&c.empty[s]);
      if (!ptx::mbar_wait(&c.d_full[buf], (tau / kBufs) & 1, &c.abort)) return;
      __syncwarp();
      ptx::tc_fence_after();
      // heads below `from` belong to queries that do not see the row
      const int pos = (int)j * p.nshards + p.shard;
      const int from = p.q_len > 1 && row < nv ? max(0, pos - last) * hpq : 0;
      const bool masked = __any_sync(0xffffffffu, from > 0);
      float sum = 0.f;
#pragma unroll
      for (int piece = 0; piece < 2; ++piece) {
        const int h0 = 32 * hh + 16 * piece;
        uint32_t x[S::kParts][16];
#pragma unroll
        for (int k = 0; k < S::kParts; ++k)
          ptx::tmem_ld16(lane_base + buf * (32 * S::kParts) + 32 * k + 16 * piece, x[k]);
        ptx::tmem_wait_ld();
        if (piece == 1) {
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&c.d_empty[buf]);
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float2 f = c.head[group][h0 + e];
          float y;
          if constexpr (kDtype == kKvFp8) {
            float v = sc[0] * __uint_as_float(x[0][e]);
            v = fmaf(sc[1], __uint_as_float(x[1][e]), v);
            v = fmaf(sc[2], __uint_as_float(x[2][e]), v);
            v = fmaf(sc[3], __uint_as_float(x[3][e]), v);
            y = fmaf(f.x, v, fmaf(sl2, __uint_as_float(x[4][e]), -f.y));
          } else {
            y = fmaf(f.x, __uint_as_float(x[0][e]), -f.y);
          }
          float w = ex2(y);
          if (masked && h0 + e < from) w = 0.f;
          sum += w;
        }
      }
      float* half = c.half[group][mine & 1];
      if (hh == 1) half[row] = sum;
      ptx::named_bar(1 + group, kGroupThreads);
      if (hh == 0) {
        const float add = sum + half[row];
        if (live) *o = m.decay == 0.f ? add : fmaf(m.decay, old, add);
        if (row < nv && !live && p.flags) atomicOr(p.flags, kFlagBadLength);
      }
      ++mine;
    }
    ++tau;
    if (!cur.next(p, c)) break;
  }
}

template <int kDtype>
__global__ void __launch_bounds__(kThreads, 1) mass_kernel(const __grid_constant__ MassParams m) {
  using S = Shape<kDtype>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  Ctl& c = *reinterpret_cast<Ctl*>(base + S::kQBytes + S::kStages * S::kStageBytes);
  const PartialParams& p = m.p;
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      ptx::mbar_init(&c.full[s], 1);
      // the MMAs' commit and the four warps that read the row count and scales
      ptx::mbar_init(&c.empty[s], 5);
    }
    for (int k = 0; k < kBufs; ++k) {
      ptx::mbar_init(&c.d_full[k], 1);
      ptx::mbar_init(&c.d_empty[k], 4);
    }
    ptx::mbar_init(&c.q_full, 1);
    ptx::mbar_init(&c.q_empty, 1);
    c.abort = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 0) ptx::tmem_alloc(&c.tmem_base, kTmemCols);
  ptx::fence_proxy_async();
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const int T = total_tiles(p, c.warp_sums);
  const int tpc = T > 0 ? (T + p.num_ctas - 1) / p.num_ctas : 0;
  const int lo = blockIdx.x * tpc, hi = min(T, lo + tpc);
  Counts n;
  uint32_t tau = 0, mine = 0;
  int first = 0;
  while (lo < hi) {
    const int total = collect_segments_n(p, lo, hi, first, kMaxSeg, c);
    const int nseg = min(kMaxSeg, total - first);
    if (nseg <= 0) break;
    if (warp < kLoadWarp) {
      weight_role<kDtype>(m, c, base, nseg, tau, mine);
    } else if (warp == kLoadWarp) {
      if ((threadIdx.x & 31) == 0) load_role<kDtype>(m, c, base, nseg, n);
    } else {
      if ((threadIdx.x & 31) == 0) mma_role<kDtype>(m, c, base, nseg, n);
    }
    __syncthreads();
    if (c.abort) break;
    first += kMaxSeg;
    if (total <= first) break;
  }
  // Drain: every asynchronous arrival lands before the CTA exits.  The waits
  // are for the latest phase of each barrier (after a timeout: bounded).
  if (threadIdx.x == kMmaWarp * 32) {
    for (uint32_t s = 0; s < (uint32_t)S::kStages; ++s) {
      const uint32_t u = n.tau > s ? (n.tau - s + S::kStages - 1) / S::kStages : 0;
      if (u > 0) ptx::mbar_wait(&c.empty[s], (u - 1) & 1, &c.abort);
    }
    for (uint32_t k = 0; k < (uint32_t)kBufs; ++k) {
      const uint32_t u = n.tau > k ? (n.tau - k + kBufs - 1) / kBufs : 0;
      if (u > 0) ptx::mbar_wait(&c.d_full[k], (u - 1) & 1, &c.abort);
    }
  }
  if (threadIdx.x == kLoadWarp * 32) {
    for (uint32_t s = 0; s < (uint32_t)S::kStages; ++s) {
      const uint32_t u = n.tau > s ? (n.tau - s + S::kStages - 1) / S::kStages : 0;
      if (u > 0) ptx::mbar_wait(&c.full[s], (u - 1) & 1, &c.abort);
    }
    if (n.sigma > 0) {
      ptx::mbar_wait(&c.q_full, (n.sigma - 1) & 1, &c.abort);
      ptx::mbar_wait(&c.q_empty, (n.sigma - 1) & 1, &c.abort);
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (c.abort && threadIdx.x == 0 && p.flags) atomicOr(p.flags, DCPMLA_FLAG_TIMEOUT);
  if (warp == 0) ptx::tmem_dealloc(c.tmem_base, kTmemCols);
}

// ---------------------------------------------------------------- host -----

// Tensor map over [z][y][x] bytes with 128-byte-swizzled boxes of 128 x 64, or
// unswizzled ones of `box` x 64.
bool encode(CUtensorMap* map, const void* base, uint64_t x, uint64_t y, uint64_t z, uint64_t pitch,
            uint64_t plane, uint32_t box) {
  EncodeTiledFn enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[3] = {x, y, z}, strides[2] = {pitch, plane};
  const cuuint32_t boxes[3] = {box, 64, 1}, es[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, boxes,
             es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             box == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

std::mutex g_mutex;
bool g_done[2][kMaxDevicesConfigured] = {};

template <int kDtype>
cudaError_t launch_mass(MassParams& m, int dev, cudaStream_t st) {
  const PartialParams& p = m.p;
  constexpr uint64_t rb = Shape<kDtype>::kRowBytes;
  if (!encode(&m.rows, p.kv, rb, kBlock, p.num_blocks, rb, rb * kBlock, 128))
    return cudaErrorInvalidValue;
  if (kDtype == kKvFp8 && !encode(&m.scales, p.kv, rb, kBlock, p.num_blocks, rb, rb * kBlock, 16))
    return cudaErrorInvalidValue;
  if (kDtype == kKvBf16 && !encode(&m.q, p.q, kRowBytesBf16, p.heads, p.batch, kRowBytesBf16,
                                   (uint64_t)p.rows_q * kRowBytesBf16, 128))
    return cudaErrorInvalidValue;
  constexpr int smem = (int)smem_bytes<kDtype>();
  {
    std::lock_guard<std::mutex> lock(g_mutex);
    if (!g_done[kDtype][dev]) {
      const cudaError_t e = cudaFuncSetAttribute(
          mass_kernel<kDtype>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (e != cudaSuccess) return e;
      g_done[kDtype][dev] = true;
    }
  }
  if (kDtype == kKvFp8) {
    const cudaError_t e = launch_q_image(p, st);
    if (e != cudaSuccess) return e;
  }
  mass_kernel<kDtype><<<p.num_ctas, kThreads, smem, st>>>(m);
  return cudaGetLastError();
}

bool aligned16(const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0; }
size_t round256(size_t x) { return (x + 255) & ~(size_t)255; }

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
  p.q_image = static_cast<uint8_t*>(workspace) + kWsHeader;
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
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = kv_dtype == DCPMLA_KV_FP8 ? launch_mass<kKvFp8>(m, dev, st)
                                                    : launch_mass<kKvBf16>(m, dev, st);
    if (e != cudaSuccess) return DCPMLA_ERR_CUDA;
  }
  return DCPMLA_OK;
}

}  // extern "C"
