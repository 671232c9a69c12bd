// Tensor-core decode (tcgen05 / TMEM / TMA, sm_100a) over bf16 rows as they
// are, for the chosen blocks of a block-sparse decode: the softmax over a
// request's rows of scale * <q_h, k_t> (576 values) applied to the first 512
// values of the rows, with LSE = ln sum_t exp(score).
//
// Against the fp16-operand kernel, whose warps load, convert and store every
// row, the rows go from the cache to the tensor core by TMA: queries and rows
// multiply as bf16 (exact products), and P, in [0, 2^8], is two bf16 terms (hi,
// and what hi leaves, within 2^-17 of it), so that the second product is as
// exact.  A tile is one cache block.  Scores S = Q K^T: 36 weight-stationary
// MMAs (M = 64 heads, N = 64 rows, K = 16), issued for tile t + 1 before the PV
// of tile t; O += P_hi V + P_lo V: 16 (N = 256 values), V being the tile's own
// chunks read MN-major; O stays in TMEM for the request.
//
// Shared memory is what shapes it: Q 72 KB, two tiles of 72 KB, and only 8 KB
// left: P_hi takes the tile's rope chunk, which the scores no longer need, and
// P_lo the 8 KB, one tile's at a time.  Rows past a request's end hold anything:
// their scores are masked and, since 0 times NaN is NaN, the softmax warps clear
// their values before the PV.
//
// Roles (6 warps): 0-3 softmax and epilogue (one TMEM lane a thread: head lane %
// 64, rows 0-31 or 32-63 of the tile), 4 issues the MMAs, 5 loads.  Every wait is
// bounded.
#include <math_constants.h>

#include <mutex>

#include "common.cuh"
#include "kernels.h"
#include "schedule.cuh"
#include "tc_ptx.cuh"

namespace dcpmla {
namespace {

constexpr int kThreads = 192;
constexpr int kMmaWarp = 4, kLoadWarp = 5;
constexpr int kBarSoft = 1, kSoftThreads = 128;
constexpr uint32_t kSlot = 8192;                  // 64 rows x 128 bytes
constexpr int kSlots = 9, kRopeSlot = 8;          // of a tile: 8 latent chunks, the rope (then P_hi)
constexpr uint32_t kTile = kSlots * kSlot;
constexpr uint32_t kOffStage = kTile;             // after Q
constexpr uint32_t kOffPlo = kOffStage + 2 * kTile;
constexpr uint32_t kOffCtl = kOffPlo + kSlot;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 256;                   // scores: [256, 288) and [288, 320); O: [0, 256)
constexpr int kPrefetchTiles = 2;
constexpr int kMaxSegBf = 16;
constexpr int kHalf0 = 4;                         // chunks of a tile's first half (the rest: 5)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleLog2 = 8.f;               // lazy max: O is rescaled when it grows by > 2^8
constexpr int kFlagTimeout = 4;

struct BfParams {
  PartialParams p;
  CUtensorMap rows;      // [blocks][64][1152] u8, box 128 x 64, 128-byte swizzle
  CUtensorMap q;         // [batch][heads][1152] u8, the same box (rows past the heads: zeros)
};

struct BfCtl {
  uint64_t full[2][2];       // per stage and half: bytes landed
  uint64_t empty[2][2];      // per stage and half: PV done (commit)
  uint64_t s_full[2];        // scores ready (commit)
  uint64_t p_full[2];        // P written (softmax arrivals)
  uint64_t o_full;           // a request's last PV done (commit)
  uint64_t q_full, q_empty;  // Q landed / a request's last scores done (commit)
  int nv[2];                 // rows of the stage's tile that take part
  uint32_t tmem_base;
  int abort;
  int sel_count;
  int warp_sums[16];
  float red[2][2][64];
  float lred[2][64];
  Segment seg[kMaxSegBf];
};

constexpr size_t kSmemBytes = kOffCtl + sizeof(BfCtl);
static_assert(kSmemBytes <= 232448, "shared memory budget");

__device__ __forceinline__ uint32_t swz(int row, int unit) {
  return (uint32_t)((row >> 3) * 1024 + (row & 7) * 128 + ((unit ^ (row & 7)) << 4));
}
__device__ __forceinline__ uint64_t dplus(uint64_t d, uint32_t byte_off) {
  return d + (uint64_t)(byte_off >> 4);
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// two fp32 -> two bf16, the first in the low half
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// TMA loads of every tile by halves, each once the PV of the tile two back is
// done with it, and of each request's Q.
__device__ __forceinline__ void load_role(const BfParams& B, BfCtl& c, uint8_t* base, int nseg,
                                          uint32_t& tau, uint32_t& sigma) {
  const PartialParams& p = B.p;
  TileCursor cur, pf;
  if (!cur.start(p, c, nseg)) return;
  pf = cur;
  bool pf_ok = pf.next(p, c);
  int due = kPrefetchTiles;
  while (true) {
    const int st = tau & 1;
    const uint32_t eph = ((tau >> 1) + 1) & 1;
    const uint32_t dst = ptx::smem_addr(base + kOffStage + st * kTile);
    const int blk = tile_block(p, cur.v.b, (cur.v.row_begin >> 6) + cur.t);
    const int z = blk >= 0 ? blk : 0;          // a bad entry: a stand-in block, no rows
    if (tau >= 2 && !ptx::mbar_wait(&c.empty[st][0], eph, &c.abort)) return;
    ptx::mbar_arrive_expect_tx(&c.full[st][0], kHalf0 * kSlot);
#pragma unroll
    for (int k = 0; k < kHalf0; ++k)
      ptx::tma_load_3d(dst + k * kSlot, &B.rows, 128 * k, 0, z, &c.full[st][0]);
    if (cur.t == 0) {
      if (sigma > 0 && !ptx::mbar_wait(&c.q_empty, (sigma - 1) & 1, &c.abort)) return;
      const uint32_t dq = ptx::smem_addr(base);
      ptx::mbar_arrive_expect_tx(&c.q_full, kTile);
#pragma unroll 1
      for (int k = 0; k < kSlots; ++k)
        ptx::tma_load_3d(dq + k * kSlot, &B.q, 128 * k, 0, cur.v.b, &c.q_full);
      ++sigma;
    }
    if (tau >= 2 && !ptx::mbar_wait(&c.empty[st][1], eph, &c.abort)) return;
    c.nv[st] = blk >= 0 ? cur.tile_valid_rows() : 0;
    ptx::mbar_arrive_expect_tx(&c.full[st][1], (kSlots - kHalf0) * kSlot);
#pragma unroll
    for (int k = kHalf0; k < kSlots; ++k)
      ptx::tma_load_3d(dst + k * kSlot, &B.rows, 128 * k, 0, z, &c.full[st][1]);
    ++tau;
    if (!cur.next(p, c)) break;
    for (; pf_ok && due > 0; --due) {
      const int pb = tile_block(p, pf.v.b, (pf.v.row_begin >> 6) + pf.t);
      if (pb >= 0) ptx::prefetch_l2(p.kv + (size_t)pb * kTile, kTile);
      pf_ok = pf.next(p, c);
    }
    due = 1;
  }
}

struct Descs {
  uint64_t q, k, p_hi, p_lo, v;     // of stage 0; stage 1 is kTile further
};

// S[tau & 1] = Q K^T of tile tau.
__device__ __forceinline__ bool issue_qk(BfCtl& c, const Descs& d, uint32_t tau) {
  constexpr uint32_t kId = ptx::idesc_make(64, 64, 1, false, false);
  const uint32_t st = tau & 1, ph = (tau >> 1) & 1;
  const uint64_t kd = dplus(d.k, st * kTile);
  const uint32_t dst = c.tmem_base + kColS + 32 * st;
#pragma unroll 1
  for (int half = 0; half < 2; ++half) {
    if (!ptx::mbar_wait(&c.full[st][half], ph, &c.abort)) return false;
    ptx::tc_fence_after();
#pragma unroll 1
    for (int k = half ? kHalf0 : 0; k < (half ? kSlots : kHalf0); ++k)
#pragma unroll
      for (int ks = 0; ks < 4; ++ks)
        ptx::mma_ws_f16(dst, dplus(d.q, k * kSlot + ks * 32), dplus(kd, k * kSlot + ks * 32), kId,
                        (k | ks) != 0);
  }
  ptx::mma_commit(&c.s_full[st]);
  return true;
}

// O (+)= P V of tile tau; frees its stage by halves.
__device__ __forceinline__ void issue_pv(BfCtl& c, const Descs& d, uint32_t tau, bool first_tile) {
  constexpr uint32_t kId = ptx::idesc_make(64, 256, 1, false, true);
  const uint32_t st = tau & 1;
#pragma unroll 1
  for (int half = 0; half < 2; ++half) {
    const uint64_t vd = dplus(d.v, st * kTile + half * 4 * kSlot);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      ptx::mma_ws_f16(c.tmem_base + half * 128, dplus(d.p_hi, st * kTile + kk * 32),
                      dplus(vd, kk * 2048), kId, !first_tile || kk > 0);
      ptx::mma_ws_f16(c.tmem_base + half * 128, dplus(d.p_lo, kk * 32), dplus(vd, kk * 2048), kId,
                      1u);
    }
    ptx::mma_commit(&c.empty[st][half]);
  }
}

// Issues every MMA: the scores of the next tile before the PV of this one.
__device__ __forceinline__ void mma_role(const PartialParams& p, BfCtl& c, uint8_t* base, int nseg,
                                         uint32_t& tau, uint32_t& sigma, uint32_t (&uses)[2]) {
  Descs d;
  const uint32_t s0 = ptx::smem_addr(base + kOffStage);
  d.q = ptx::sdesc_sw128(ptx::smem_addr(base), 16, 1024);
  d.k = ptx::sdesc_sw128(s0, 16, 1024);
  d.p_hi = ptx::sdesc_sw128(s0 + kRopeSlot * kSlot, 16, 1024);
  d.p_lo = ptx::sdesc_sw128(ptx::smem_addr(base + kOffPlo), 16, 1024);
  d.v = ptx::sdesc_sw128(s0, kSlot, 1024);
  TileCursor cur, ahead;
  if (!cur.start(p, c, nseg)) return;
  ahead = cur;
  if (!ptx::mbar_wait(&c.q_full, sigma & 1, &c.abort)) return;
  if (!issue_qk(c, d, tau)) return;
  if (ahead.last_of_segment()) ptx::mma_commit(&c.q_empty);
  uint32_t sigma_ahead = sigma;
  while (true) {
    const bool seg_end = ahead.last_of_segment();
    if (ahead.next(p, c)) {
      if (seg_end) {
        ++sigma_ahead;
        if (!ptx::mbar_wait(&c.q_full, sigma_ahead & 1, &c.abort)) return;
      }
      if (!issue_qk(c, d, tau + 1)) return;
      if (ahead.last_of_segment()) ptx::mma_commit(&c.q_empty);
    }
    const int st = tau & 1;
    if (!ptx::mbar_wait(&c.p_full[st], (tau >> 1) & 1, &c.abort)) return;
    ptx::tc_fence_after();
    issue_pv(c, d, tau, cur.t == 0);
    ++uses[st];
    if (cur.last_of_segment()) {
      ptx::mma_commit(&c.o_full);
      ++sigma;
    }
    ++tau;
    if (!cur.next(p, c)) break;
  }
}

// Online softmax, P and the epilogue (128 threads, one TMEM lane each).
__device__ __forceinline__ void softmax_role(const PartialParams& p, BfCtl& c, uint8_t* base,
                                             int nseg, uint32_t& tau, uint32_t& sigma) {
  const int L = threadIdx.x;                 // 0..127
  const int h = L & 63, half = L >> 6, lane = L & 31;
  const uint32_t lane_base = c.tmem_base + ((uint32_t)((L >> 5) * 32) << 16);
  const float sl2 = p.scale * kLog2e;
  TileCursor cur;
  if (!cur.start(p, c, nseg)) return;
  float m_used = -CUDART_INF_F, l = 0.f;
  while (true) {
    const int st = tau & 1;
    const uint32_t ph = (tau >> 1) & 1;
    if (!ptx::mbar_wait3(&c.s_full[st], ph, &c.full[st][1], ph, &c.full[st][0], ph, &c.abort)) return;
    __syncwarp();
    ptx::tc_fence_after();
    uint32_t sr[32];
    ptx::tmem_ld32(lane_base + kColS + 32 * st, sr);
    ptx::tmem_wait_ld();
    const int nv = c.nv[st];
    uint8_t* stage = base + kOffStage + st * kTile;
    if (nv < kTileRows) {
      // absent rows: zeros over their values (the scores have been computed)
      for (int k = L; k < (kTileRows - nv) * 64; k += kSoftThreads) {
        const int r = nv + (k >> 6), u = k & 63;
        *reinterpret_cast<uint4*>(stage + (u >> 3) * kSlot + swz(r, u & 7)) = make_uint4(0, 0, 0, 0);
      }
    }
    const int left = nv - half * 32;         // rows of this thread's half that take part
    float x[32];
    float mloc = -CUDART_INF_F;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      x[j] = j < left ? __uint_as_float(sr[j]) * sl2 : -CUDART_INF_F;
      mloc = fmaxf(mloc, x[j]);
    }
    c.red[st][half][h] = mloc;
    ptx::named_bar(kBarSoft, kSoftThreads);
    const float mnew = fmaxf(mloc, c.red[st][half ^ 1][h]);
    // Lazy rescale, decided per warp (the loads and stores of O are
    // warp-collective); the partner warp holds the same heads and decides alike.
    const bool first = m_used == -CUDART_INF_F;
    const bool any_need = __any_sync(0xffffffffu, !first && mnew > m_used + kRescaleLog2);
    float alpha = 1.f;
    if (first) {
      m_used = mnew;
    } else if (any_need) {
      const float m2 = fmaxf(m_used, mnew);
      alpha = ex2(m_used - m2);
      m_used = m2;
      l *= alpha;
    }
    const float mu = m_used == -CUDART_INF_F ? 0.f : m_used;   // all masked: x = -inf -> p = 0
    float sum = 0.f;
    uint32_t hi[16], lo[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float p0 = ex2(x[2 * j] - mu), p1 = ex2(x[2 * j + 1] - mu);
      sum += p0 + p1;
      hi[j] = bf16x2(p0, p1);
      lo[j] = bf16x2(p0 - __uint_as_float(hi[j] << 16), p1 - __uint_as_float(hi[j] & 0xFFFF0000u));
    }
    l += sum;
    // P_lo's buffer and O are free once the PV of the previous tile is done: its
    // last MMA released the second half of its stage.  That phase is pending or
    // complete here (the next PV needs this thread's P), so the parity is
    // unambiguous.
    if (tau > 0 && !ptx::mbar_wait(&c.empty[st ^ 1][1], ((tau - 1) >> 1) & 1, &c.abort)) return;
    uint8_t* phi = stage + kRopeSlot * kSlot;
    uint8_t* plo = base + kOffPlo;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      *reinterpret_cast<uint4*>(phi + swz(h, 4 * half + u)) =
          make_uint4(hi[4 * u], hi[4 * u + 1], hi[4 * u + 2], hi[4 * u + 3]);
      *reinterpret_cast<uint4*>(plo + swz(h, 4 * half + u)) =
          make_uint4(lo[4 * u], lo[4 * u + 1], lo[4 * u + 2], lo[4 * u + 3]);
    }
    if (any_need) {
      __syncwarp();
      ptx::tc_fence_after();
#pragma unroll 1
      for (int q = 0; q < 8; ++q) {
        uint32_t r[32];
        const uint32_t addr = lane_base + 32 * q;
        ptx::tmem_ld32(addr, r);
        ptx::tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * alpha);
        ptx::tmem_st32(addr, r);
      }
      ptx::tmem_wait_st();
    }
    ptx::fence_proxy_async();
    ptx::tc_fence_before();
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(&c.p_full[st]);
    // ---- epilogue after the request's last tile
    if (cur.last_of_segment()) {
      const SegView& v = cur.v;
      const size_t slot = seg_slot(p, v);
      const size_t row = slot * (v.whole ? p.rows_o : p.heads) + h;
      float* l_base = (v.whole ? p.out_lse : p.ws_lse) + row;
      // o_full completes once per request, after its last PV; the next phase
      // needs this thread's P, so the parity is unambiguous
      if (!ptx::mbar_wait(&c.o_full, sigma & 1, &c.abort)) return;
      __syncwarp();
      ptx::tc_fence_after();
      c.lred[half][h] = l;
      ptx::named_bar(kBarSoft, kSoftThreads);
      const float ltot = l + c.lred[half ^ 1][h];
      const float inv = ltot > 0.f ? 1.f / ltot : 0.f;
      // A lane holds 32 values of its head's row per load; eight lanes exchange
      // them (an 8 x 8 transpose of 16-byte pieces in three butterfly steps), so
      // that a row's pieces leave together as a whole 128-byte line.
      const int i8 = L & 7, row8 = L & 24;
      float* o_rows = (v.whole ? p.out : p.ws_o) + (row - h + (h & ~31) + row8) * kVDim;
#pragma unroll 1
      for (int q = 0; q < 8; ++q) {
        uint32_t r[32];
        ptx::tmem_ld32(lane_base + 32 * q, r);
        ptx::tmem_wait_ld();
        float4 piece[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
          piece[e] = make_float4(__uint_as_float(r[4 * e]) * inv, __uint_as_float(r[4 * e + 1]) * inv,
                                 __uint_as_float(r[4 * e + 2]) * inv,
                                 __uint_as_float(r[4 * e + 3]) * inv);
#pragma unroll
        for (int m = 4; m >= 1; m >>= 1) {
          const bool upper = (i8 & m) != 0;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (e & m) continue;
            const float4 send = upper ? piece[e] : piece[e | m];
            float4 got;
            got.x = __shfl_xor_sync(0xffffffffu, send.x, m);
            got.y = __shfl_xor_sync(0xffffffffu, send.y, m);
            got.z = __shfl_xor_sync(0xffffffffu, send.z, m);
            got.w = __shfl_xor_sync(0xffffffffu, send.w, m);
            if (upper) piece[e] = got; else piece[e | m] = got;
          }
        }
        // piece[k] is now piece i8 of the row of lane row8 + k
        const int col = (q >> 2) * 256 + half * 128 + (q & 3) * 32 + 4 * i8;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if ((h & ~31) + row8 + k < p.heads)
            *reinterpret_cast<float4*>(o_rows + (size_t)k * kVDim + col) = piece[k];
      }
      if (h < p.heads && half == 0)
        *l_base = ltot > 0.f ? (m_used + log2f(ltot)) * kLn2 : -CUDART_INF_F;
      ptx::tc_fence_before();
      ptx::named_bar(kBarSoft, kSoftThreads);
      ++sigma;
      m_used = -CUDART_INF_F;
      l = 0.f;
    }
    ++tau;
    if (!cur.next(p, c)) break;
  }
}

__global__ void __launch_bounds__(kThreads, 1) partial_bf16_kernel(const __grid_constant__ BfParams B) {
  extern __shared__ __align__(1024) uint8_t base[];
  PartialParams p = B.p;
  p.sparse_idx = nullptr;
  BfCtl& c = *reinterpret_cast<BfCtl*>(base + kOffCtl);
  const int warp = threadIdx.x >> 5;
  // swizzled operands need 1024-byte alignment; there is no room to round up
  if (ptx::smem_addr(base) & 1023u) {
    if (threadIdx.x == 0 && p.flags) atomicOr(p.flags, kFlagTimeout);
    return;
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      for (int k = 0; k < 2; ++k) {
        ptx::mbar_init(&c.full[s][k], 1);
        ptx::mbar_init(&c.empty[s][k], 1);
      }
      ptx::mbar_init(&c.s_full[s], 1);
      ptx::mbar_init(&c.p_full[s], kSoftThreads / 32);
    }
    ptx::mbar_init(&c.o_full, 1);
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
  const int lo = (int)min((long long)T, (long long)blockIdx.x * tpc), hi = min(T, lo + tpc);
  uint32_t tau = 0, sigma = 0;
  uint32_t uses[2] = {0, 0};
  int first = 0;
  while (lo < hi) {
    const int total = collect_segments_n(p, lo, hi, first, kMaxSegBf, c);
    const int nseg = min(kMaxSegBf, total - first);
    if (nseg <= 0) break;
    if (warp < 4) {
      softmax_role(p, c, base, nseg, tau, sigma);
    } else if (warp == kMmaWarp) {
      if ((threadIdx.x & 31) == 0) mma_role(p, c, base, nseg, tau, sigma, uses);
    } else {
      if ((threadIdx.x & 31) == 0) load_role(B, c, base, nseg, tau, sigma);
    }
    __syncthreads();
    if (c.abort) break;
    first += kMaxSegBf;
    if (total <= first) break;
  }
  // Drain: every asynchronous arrival lands before the CTA exits.  Normally only
  // the last stage releases and the last Q release are unconsumed; after a
  // timeout any may be (these waits are bounded too).
  if (threadIdx.x == kMmaWarp * 32) {
    for (int s = 0; s < 2; ++s)
      if (uses[s] > 0)
        for (int k = 0; k < 2; ++k) ptx::mbar_wait(&c.empty[s][k], (uses[s] - 1) & 1, &c.abort);
    if (sigma > 0) ptx::mbar_wait(&c.q_empty, (sigma - 1) & 1, &c.abort);
  }
  if (threadIdx.x == kLoadWarp * 32) {
    for (uint32_t s = 0; s < 2; ++s) {
      const uint32_t n = tau > s ? (tau - s + 1) / 2 : 0;
      if (n > 0)
        for (int k = 0; k < 2; ++k) ptx::mbar_wait(&c.full[s][k], (n - 1) & 1, &c.abort);
    }
    if (sigma > 0) ptx::mbar_wait(&c.q_full, (sigma - 1) & 1, &c.abort);
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (c.abort && threadIdx.x == 0 && p.flags) atomicOr(p.flags, kFlagTimeout);
  if (warp == 0) ptx::tmem_dealloc(c.tmem_base, kTmemCols);
}

std::mutex g_mutex;
bool g_done[kMaxDevicesConfigured] = {};

}  // namespace

bool bf16_supports(const PartialParams& p, int kv_dtype) {
  return kv_dtype == kKvBf16 && p.q_len == 1 && p.heads >= 1 && p.heads <= kMaxHeads &&
         p.sparse_idx == nullptr && tensor_map_encoder() != nullptr;
}

cudaError_t launch_partial_bf16(const PartialParams& p, cudaStream_t st) {
  BfParams b;
  b.p = p;
  EncodeTiledFn enc = tensor_map_encoder();
  if (!enc) return cudaErrorInvalidValue;
  const cuuint32_t box[3] = {128, 64, 1}, es[3] = {1, 1, 1};
  auto encode = [&](CUtensorMap* m, const void* at, cuuint64_t rows, cuuint64_t planes,
                    cuuint64_t plane_bytes) {
    const cuuint64_t dims[3] = {(cuuint64_t)kRowBytesBf16, rows, planes};
    const cuuint64_t strides[2] = {(cuuint64_t)kRowBytesBf16, plane_bytes};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(at), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  if (!encode(&b.rows, p.kv, kBlock, p.num_blocks, (cuuint64_t)kRowBytesBf16 * kBlock) ||
      !encode(&b.q, p.q, p.heads, p.batch, (cuuint64_t)p.rows_q * kRowBytesBf16))
    return cudaErrorInvalidValue;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevicesConfigured) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lock(g_mutex);
    if (!g_done[dev]) {
      e = cudaFuncSetAttribute(partial_bf16_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               (int)kSmemBytes);
      if (e != cudaSuccess) return e;
      g_done[dev] = true;
    }
  }
  partial_bf16_kernel<<<p.num_ctas, kThreads, kSmemBytes, st>>>(b);
  return cudaGetLastError();
}

}  // namespace dcpmla
