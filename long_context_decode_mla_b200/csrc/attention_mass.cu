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
// the decode kernels', D = K Q^T with the cached rows as M and the (query, head)
// rows as N: a TMEM lane then holds one cached row for all heads, a row's fp32
// scales are one thread's registers, and the sum over heads stays in a thread
// but for one exchange between two.  Rows past a
// request's end only ever reach their own lanes, so nothing is cleared.
//
//  * fp8 rows: the e4m3 codes are the A operand as they are; Q comes as two e4m3
//    terms in one power-of-two frame (q_image.cuh), 128 rows of one operand with an
//    accumulator each, the second times 2^4: in one accumulator, and so in one
//    frame, the format's smallest step left 1e-6 to 6e-6 of a query's weights as
//    error, a head's own, which no sum over rows averages away.  Every 128-value
//    scale group is a part, scaled in fp32, and the bf16 rope a fifth.
//  * bf16 rows and queries multiply as they are (exact products), in nine parts of
//    64 values that are added in fp32: the tensor core cuts low bits at each of its
//    additions.  One query of 8 heads over 512 rows: 36 additions in one accumulator
//    leave a relative error of 2.3e-6, three parts 0.63e-6, five 0.44e-6, nine
//    0.32e-6, at the same time (58 us for 32 requests of 8,191 rows).
//
// A tile is two cache blocks (M = 128: a weight-stationary M = 64 MMA takes as
// long, and 36 of them more than a block's share of HBM time).  Its rows go
// through a ring of eight 16 KB slots, 128 bytes of every row each, loaded by
// TMA and given back slot by slot, with whole blocks prefetched into L2 ahead.
// Warp 8 loads; warps 9 and 10 issue the MMAs (a tile of bf16 rows 36, of fp8 rows
// 20: both terms of a group are one operand); warps 0-3 and 4-7 add each part into the
// scores of 32 heads a thread, so that a part's accumulator is free again as soon as
// it is read, and exchange the sums of their halves.
// Tiles are dealt to the CTAs as in decode.  Each row is summed by the same
// threads in the same order whatever the number of CTAs: no atomics, the same
// bits every time.  Every wait is bounded.
//
// HBM bounds bf16 rows (per further row 6.9 TB/s; 32 requests of 8,191 rows 58 us
// with some 15 us of start and ends), the MMAs' issue and HBM together fp8 rows
// (779,084 rows 115 us; 130 to 138 once back-to-back calls have brought the device to
// its power limit).
#include "dcpmla.h"

#include <cuda.h>

#include <algorithm>
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
  float scale2, scale2_err;   // softmax scale * log2(e) in fp32, and its relative rounding
  CUtensorMap rows;      // [blocks][64][row bytes] u8, box 128 x 64, 128-byte swizzle
  CUtensorMap scales;    // fp8: the same, box 16 x 64 (the four fp32 scales)
  CUtensorMap q;         // bf16: [batch][rows][1152] u8, box 128 x 64, rows past the pass zero
};

constexpr int kThreads = 352;
constexpr int kLoadWarp = 8, kMmaWarp = 9, kIssuers = 2;
constexpr int kWeightThreads = 256;
constexpr uint32_t kHalf = 8192;                   // 64 rows x 128 bytes
constexpr uint32_t kSlot = 2 * kHalf;              // of a tile's two blocks
constexpr int kSlots = 8;
constexpr uint32_t kTmemCols = 512;
constexpr int kMaxBufs = 8;
constexpr int kLoBits = 4;                         // Q's second e4m3 term is times 2^4
constexpr uint32_t kQBytes = 9 * kHalf;            // fp8: hi, lo, rope; bf16: nine chunks
constexpr int kPrefetchTiles = 1;                  // more crowd the L2: 61 us at 1, 86 at 4
constexpr int kMaxSeg = 64;
constexpr int kTileMass = 128;                     // rows of a tile
constexpr float kLog2e = 1.4426950408889634f, kLog2eLo = 1.4426950408889634 - (double)kLog2e;

template <int kDtype>
struct Shape;
template <>
struct Shape<kKvFp8> {
  static constexpr int kRowBytes = kRowBytesFp8, kChunks = 5, kBufs = 4;    // 128 columns
};
template <>
struct Shape<kKvBf16> {
  static constexpr int kRowBytes = kRowBytesBf16, kChunks = 9, kBufs = 8;   // 64 columns
};
// Tiles between their load and their weights: when tile t's first chunk is loaded,
// the slots and accumulators have let the weights past the rows and scales of tile
// t - 4 (fp8: 1.6 and 0.8 tiles; bf16: 0.9 and 0.9).
constexpr int kMeta = 4;
constexpr uint32_t kScaleBytes = kTileMass * 16;   // fp8: four fp32 scales a row

struct Ctl {
  uint64_t full[kSlots], empty[kSlots];      // a slot's bytes landed / its MMAs done
  uint64_t d_full[kMaxBufs], d_empty[kMaxBufs];    // an accumulator done / read
  uint64_t meta[kMeta];                      // a tile's row counts written and scales landed
  uint64_t q_full, q_empty;
  // fp8: 2^-a; lse log2(e) in fp32; a factor for the weights that makes up for what
  // the rounding of that and of the scale left, at the weights that matter; -inf for a
  // row of Q that weighs nothing whatever its score (fminf prefers it to a NaN), else NaN
  alignas(16) float4 head[64];
  float half[2][kTileMass];                  // [tile parity]: the other half's sums
  int nv[kMeta][2];                          // rows of each block that take part
  uint32_t tmem_base;
  int abort;
  int sel_count;
  int warp_sums[16];
  Segment seg[kMaxSeg];
};

template <int kDtype>
constexpr uint32_t ctl_offset() {
  return kQBytes + kSlots * kSlot + (kDtype == kKvFp8 ? kMeta * kScaleBytes : 0);
}
template <int kDtype>
constexpr size_t smem_bytes() {
  return ctl_offset<kDtype>() + sizeof(Ctl) + 1024;
}
static_assert(smem_bytes<kKvFp8>() <= 232448 && smem_bytes<kKvBf16>() <= 232448, "shared memory");
constexpr uint32_t kOffSlot = kQBytes, kOffScale = kQBytes + kSlots * kSlot;

__device__ __forceinline__ uint64_t dplus(uint64_t d, uint32_t byte_off) {
  return d + (uint64_t)(byte_off >> 4);
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Walks the CTA's tiles: two blocks of one segment each.
struct PairCursor {
  int k, t, nseg, nt;
  SegView v;
  __device__ __forceinline__ bool open(const PartialParams& p, const Ctl& c) {
    for (; k < nseg; ++k) {
      v = seg_view(p, c, k);
      nt = (v.nrows + kTileMass - 1) / kTileMass;
      if (nt > 0) return true;
    }
    return false;
  }
  __device__ __forceinline__ bool start(const PartialParams& p, const Ctl& c, int n) {
    nseg = n;
    k = t = 0;
    return open(p, c);
  }
  __device__ __forceinline__ bool next(const PartialParams& p, const Ctl& c) {
    if (++t < nt) return true;
    t = 0;
    ++k;
    return open(p, c);
  }
  __device__ __forceinline__ bool last_of_segment() const { return t == nt - 1; }
  // rows of block half `i` of the tile that lie in the segment (0: no block)
  __device__ __forceinline__ int rows(int i) const {
    return max(0, min(kBlock, v.nrows - t * kTileMass - i * kBlock));
  }
  __device__ __forceinline__ int block(int i) const { return (v.row_begin >> 6) + 2 * t + i; }
};

// Counters of one thread's way through the tiles, kept across segment batches.
struct Counts {
  uint32_t tau = 0, chunk = 0, part = 0, sigma = 0;
};

// TMA loads of every tile, slot by slot, and of each request's Q once the
// previous request's MMAs are done with it.
template <int kDtype>
__device__ __forceinline__ void load_role(const MassParams& m, Ctl& c, uint8_t* base, int nseg,
                                          Counts& n) {
  using S = Shape<kDtype>;
  const PartialParams& p = m.p;
  PairCursor cur, pf;
  if (!cur.start(p, c, nseg)) return;
  pf = cur;
  bool pf_ok = true;
  constexpr uint32_t kBlockBytes = 64 * S::kRowBytes;
  auto prefetch = [&]() {
    if (!pf_ok) return;
    for (int i = 0; i < 2; ++i)
      if (pf.rows(i) > 0) {
        const int blk = tile_block(p, pf.v.b, pf.block(i));
        if (blk >= 0) ptx::prefetch_l2(p.kv + (size_t)blk * kBlockBytes, kBlockBytes);
      }
    pf_ok = pf.next(p, c);
  };
  // the first tile's own loads come before any prefetch: its table entries and
  // the prefetch instructions would hold them up by 2,000 cycles
  int ahead = kPrefetchTiles;
  pf_ok = pf.next(p, c);
  while (true) {
    // a bad table entry: a stand-in block, no rows; a missing second block: nothing
    int blk[2], halves = 1;
    const uint32_t meta = n.tau % kMeta;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int rows = cur.rows(i);
      blk[i] = rows > 0 ? tile_block(p, cur.v.b, cur.block(i)) : -1;
      if (i == 1 && rows > 0) halves = 2;
    }
#pragma unroll 1
    for (int k = 0; k < S::kChunks; ++k) {
      const uint32_t s = n.chunk % kSlots;
      if (n.chunk >= (uint32_t)kSlots &&
          !ptx::mbar_wait(&c.empty[s], ((n.chunk / kSlots) + 1) & 1, &c.abort))
        return;
      if (k == 0) {
        // the tile kMeta before this one has been turned into weights by now
        // (kMeta): its row counts and scales can go
        c.nv[meta][0] = blk[0] >= 0 ? cur.rows(0) : 0;
        c.nv[meta][1] = blk[1] >= 0 ? cur.rows(1) : 0;
        if constexpr (kDtype == kKvFp8) {
          ptx::mbar_arrive_expect_tx(&c.meta[meta], halves * 1024);
          for (int i = 0; i < halves; ++i)
            ptx::tma_load_3d(ptx::smem_addr(base + kOffScale + meta * kScaleBytes + i * 1024),
                             &m.scales, 512, 0, max(blk[i], 0), &c.meta[meta]);
        } else {
          ptx::mbar_arrive(&c.meta[meta]);
        }
      }
      const uint32_t dst = ptx::smem_addr(base + kOffSlot + s * kSlot);
      ptx::mbar_arrive_expect_tx(&c.full[s], halves * kHalf);
      for (int i = 0; i < halves; ++i)
        ptx::tma_load_3d(dst + i * kHalf, &m.rows, kDtype == kKvFp8 && k == 4 ? 528 : 128 * k, 0,
                         max(blk[i], 0), &c.full[s]);
      ++n.chunk;
      if (k == 0 && cur.t == 0) {
        if (n.sigma > 0 && !ptx::mbar_wait(&c.q_empty, (n.sigma - 1) & 1, &c.abort)) return;
        const uint32_t dq = ptx::smem_addr(base);
        ptx::mbar_arrive_expect_tx(&c.q_full, kQBytes);
        if constexpr (kDtype == kKvFp8) {
          ptx::wait_primary();       // the images' kernel
          // the two terms of a group one after the other: 128 rows of one operand
          const uint8_t* image = p.q_image + (size_t)cur.v.b * kQImageBytes;
#pragma unroll 1
          for (int j = 0; j < 9; ++j)
            ptx::bulk_g2s(dq + (j < 4 ? 2 * j : j < 8 ? 2 * j - 7 : 8) * kHalf, image + j * kHalf,
                          kHalf, &c.q_full);
        } else {
#pragma unroll 1
          for (int j = 0; j < 9; ++j)
            ptx::tma_load_3d(dq + j * kHalf, &m.q, 128 * j, 0, cur.v.b, &c.q_full);
        }
        ++n.sigma;
      }
    }
    ++n.tau;
    for (; ahead > 0; --ahead) prefetch();
    ahead = 1;
    if (!cur.next(p, c)) break;
  }
}

// D = K Q^T (M = 128 rows, N = 64 heads, or 128: both terms of 64).  A wait costs an
// issuing thread some 600 cycles while the tensor core streams its operands, as much
// as eight MMAs take, so the parts alternate between two issuers (bf16 rows with one
// issuer and five parts: 62 us for 58).
template <int kDtype>
__device__ __forceinline__ void mma_role(const MassParams& m, Ctl& c, uint8_t* base, int nseg,
                                         uint32_t side, Counts& n) {
  using S = Shape<kDtype>;
  constexpr uint32_t kIdF8 = ptx::idesc_make(128, 128, 0, false, false);    // both terms of Q
  constexpr uint32_t kIdBf = ptx::idesc_make(128, 64, 1, false, false);
  const uint64_t dq = ptx::sdesc(ptx::smem_addr(base), 16, 1024, ptx::kSwizzle128B);
  const uint64_t dk0 = ptx::sdesc(ptx::smem_addr(base + kOffSlot), 16, 1024, ptx::kSwizzle128B);
  PairCursor cur;
  if (!cur.start(m.p, c, nseg)) return;
  while (true) {
    if (cur.t == 0) {
      if (!ptx::mbar_wait(&c.q_full, n.sigma & 1, &c.abort)) return;
      ++n.sigma;
    }
#pragma unroll 1
    for (int k = 0; k < S::kChunks; ++k, ++n.chunk, ++n.part) {
      if ((n.chunk & 1) != side) continue;
      const uint32_t s = n.chunk % kSlots, buf = n.part % S::kBufs;
      uint64_t* reuse = n.part >= (uint32_t)S::kBufs ? &c.d_empty[buf] : &c.full[s];
      const uint32_t parity = (n.chunk / kSlots) & 1;
      if (!ptx::mbar_wait3(&c.full[s], parity, reuse,
                           n.part >= (uint32_t)S::kBufs ? ((n.part / S::kBufs) + 1) & 1 : parity,
                           &c.full[s], parity, &c.abort))
        return;
      ptx::tc_fence_after();
      const uint64_t dk = dplus(dk0, s * kSlot);
      const uint32_t d = c.tmem_base + kTmemCols / S::kBufs * buf;
      if (kDtype == kKvFp8 && k < 4) {
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          ptx::mma_f8(d, dplus(dk, ks * 32), dplus(dq, 2 * k * kHalf + ks * 32), kIdF8, ks > 0);
      } else {
        const uint32_t q = (kDtype == kKvFp8 ? 8 : k) * kHalf;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          ptx::mma_f16(d, dplus(dk, ks * 32), dplus(dq, q + ks * 32), kIdBf, ks > 0);
      }
      ptx::mma_commit(&c.empty[s]);
      ptx::mma_commit(&c.d_full[buf]);
    }
    if (cur.last_of_segment()) ptx::mma_commit(&c.q_empty);
    ++n.tau;
    if (!cur.next(m.p, c)) break;
  }
}

// Weights: thread (hh, row) sums heads [32 hh, 32 hh + 32) of the tile's row.
template <int kDtype>
__device__ __forceinline__ void weight_role(const MassParams& m, Ctl& c, uint8_t* base, int nseg,
                                            Counts& n) {
  using S = Shape<kDtype>;
  const PartialParams& p = m.p;
  const int hh = threadIdx.x >> 7, row = threadIdx.x & 127, lane = threadIdx.x & 31;
  const uint32_t lane_base =
      c.tmem_base + ((uint32_t)((row >> 5) * 32) << 16) + 32 * hh;
  const int hpq = p.heads / p.q_len;
  const float sl2 = m.scale2;
  PairCursor cur;
  if (!cur.start(p, c, nseg)) return;
  while (true) {
    const int b = cur.v.b;
    if (cur.t == 0) {
      // the readers of the old factors passed the last tile's barrier
      if (threadIdx.x < 64) {
        const int h = threadIdx.x;
        float4 f = make_float4(0.f, 0.f, 1.f, -INFINITY);     // rows past the pass weigh nothing
        if (h < p.heads) {
          f.x = 1.f;
          if constexpr (kDtype == kKvFp8) {
            ptx::wait_primary();
            f.x = __ldcg(reinterpret_cast<const float*>(p.q_image + (size_t)b * kQImageBytes +
                                                         kQBytes) + h);
          }
          const float l = __ldg(m.lse + (size_t)b * p.rows_o + h);
          if (l != -INFINITY) {
            f.y = l * kLog2e;
            f.w = NAN;
            // A weight near 1 has scale s = lse, and sl2 s - f.y is then off by what both
            // constants' roundings are: lse log2(e) (1 + err) - f.y, the same for all rows.
            // At an LSE of 2^22 and more, where fp32 scores are worse than that, it is
            // held to one: far beyond, an infinite factor would meet weights of zero.
            if (isfinite(f.y)) {
              const float off = fmaf(l, kLog2e, -f.y) + l * kLog2eLo + f.y * m.scale2_err;
              f.z = exp2f(fminf(1.f, fmaxf(-1.f, -off)));
            }
          }
        }
        c.head[h] = f;
      }
      ptx::named_bar(1, kWeightThreads);
    }
    const long long j = (long long)(cur.v.row_begin + cur.t * kTileMass) + row;
    const int last = seq_len_of(p, b) - p.q_len;         // position of query 0
    const uint32_t meta = n.tau % kMeta;
    if (!ptx::mbar_wait(&c.meta[meta], (n.tau / kMeta) & 1, &c.abort)) return;
    const bool in = (row & 63) < c.nv[meta][row >> 6];
    const bool live = in && j < m.mass_stride;
    float* o = m.mass + (size_t)b * m.mass_stride + j;
    float old = 0.f;
    if (hh == 0 && live && m.decay != 0.f) old = *o;
    float sc[4] = {0.f, 0.f, 0.f, 0.f};
    if constexpr (kDtype == kKvFp8) {
      const float4 v =
          *reinterpret_cast<const float4*>(base + kOffScale + meta * kScaleBytes + row * 16);
      sc[0] = v.x;
      sc[1] = v.y;
      sc[2] = v.z;
      sc[3] = v.w;
    }
    // heads below `from` belong to queries that do not see the row
    const int pos = (int)j * p.nshards + p.shard;
    const int from = p.q_len > 1 && in ? max(0, pos - last) * hpq : 0;
    const bool masked = __any_sync(0xffffffffu, from > 0);
    float v[32], sum = 0.f;
#pragma unroll
    for (int k = 0; k < S::kChunks; ++k) {
      const uint32_t buf = n.part % S::kBufs, at = lane_base + kTmemCols / S::kBufs * buf;
      const bool two = kDtype == kKvFp8 && k < S::kChunks - 1;     // accumulators
      if (!ptx::mbar_wait(&c.d_full[buf], (n.part / S::kBufs) & 1, &c.abort)) return;
      __syncwarp();
      ptx::tc_fence_after();
      uint32_t x[32], lo[32];
      ptx::tmem_ld32(at, x);
      if (two) ptx::tmem_ld32(at + 64, lo);
      ptx::tmem_wait_ld();
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&c.d_empty[buf]);
      ++n.part;
      if (k < S::kChunks - 1) {
#pragma unroll
        for (int e = 0; e < 32; ++e)
          if constexpr (kDtype == kKvFp8) {
            const float s = fmaf(__uint_as_float(lo[e]), 1.f / (1 << kLoBits), __uint_as_float(x[e]));
            v[e] = k == 0 ? sc[0] * s : fmaf(sc[k & 3], s, v[e]);
          } else {
            v[e] = k == 0 ? __uint_as_float(x[e]) : v[e] + __uint_as_float(x[e]);
          }
      } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const float4 f = c.head[32 * hh + e];
          const float z = __uint_as_float(x[e]);       // the rope
          const float s = kDtype == kKvFp8 ? fmaf(f.x, v[e], z) : v[e] + z;
          float w = ex2(fminf(fmaf(sl2, s, -f.y), f.w));
          if (masked && 32 * hh + e < from) w = 0.f;
          sum = fmaf(f.z, w, sum);
        }
      }
    }
    float* half = c.half[n.tau & 1];
    if (hh == 1) half[row] = sum;
    ptx::named_bar(1, kWeightThreads);
    if (hh == 0) {
      const float add = sum + half[row];
      if (live) *o = m.decay == 0.f ? add : fmaf(m.decay, old, add);
      if (in && !live && p.flags) atomicOr(p.flags, kFlagBadLength);
    }
    ++n.tau;
    if (!cur.next(p, c)) break;
  }
}

// Uses of ring entry i after n uses in all of a ring of `size`, and a wait for
// the last of them.
__device__ __forceinline__ void drain(uint64_t* ring, int size, uint32_t n, Ctl& c) {
  for (uint32_t i = 0; i < (uint32_t)size; ++i) {
    const uint32_t u = n > i ? (n - i + size - 1) / size : 0;
    if (u > 0) ptx::mbar_wait(&ring[i], (u - 1) & 1, &c.abort);
  }
}

template <int kDtype>
__global__ void __launch_bounds__(kThreads, 1) mass_kernel(const __grid_constant__ MassParams m) {
  using S = Shape<kDtype>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  Ctl& c = *reinterpret_cast<Ctl*>(base + ctl_offset<kDtype>());
  const PartialParams& p = m.p;
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kSlots; ++s) {
      ptx::mbar_init(&c.full[s], 1);
      ptx::mbar_init(&c.empty[s], 1);
    }
    for (int k = 0; k < S::kBufs; ++k) {
      ptx::mbar_init(&c.d_full[k], 1);
      ptx::mbar_init(&c.d_empty[k], kWeightThreads / 32);
    }
    for (int k = 0; k < kMeta; ++k) ptx::mbar_init(&c.meta[k], 1);
    ptx::mbar_init(&c.q_full, 1);
    ptx::mbar_init(&c.q_empty, kIssuers);
    c.abort = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 0) ptx::tmem_alloc(&c.tmem_base, kTmemCols);
  ptx::fence_proxy_async();
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const int T = total_tiles(p, c.warp_sums);
  // an even number of blocks a CTA, so that few tiles are half empty
  int tpc = T > 0 ? (T - 1) / p.num_ctas + 1 : 0;
  tpc += tpc & 1;
  const int lo = min((long long)T, (long long)blockIdx.x * tpc), hi = min(T, lo + tpc);
  Counts n;
  int first = 0;
  while (lo < hi) {
    const int total = collect_segments_n(p, lo, hi, first, kMaxSeg, c);
    const int nseg = min(kMaxSeg, total - first);
    if (nseg <= 0) break;
    if (warp < kLoadWarp) {
      weight_role<kDtype>(m, c, base, nseg, n);
    } else if (warp == kLoadWarp) {
      if ((threadIdx.x & 31) == 0) load_role<kDtype>(m, c, base, nseg, n);
    } else {
      if ((threadIdx.x & 31) == 0 && warp < kMmaWarp + kIssuers)
        mma_role<kDtype>(m, c, base, nseg, warp - kMmaWarp, n);
    }
    __syncthreads();
    if (c.abort) break;
    first += kMaxSeg;
    if (total <= first) break;
  }
  // a CTA without tiles waits too: this kernel's end implies the images' kernel's
  ptx::wait_primary();
  // Drain: every asynchronous arrival lands before the CTA exits (after a
  // timeout these waits are bounded too).
  if ((threadIdx.x & 31) == 0 && warp >= kMmaWarp && warp < kMmaWarp + kIssuers) {
    drain(c.empty, kSlots, n.chunk, c);
    drain(c.d_full, S::kBufs, n.part, c);
    if (n.sigma > 0) ptx::mbar_wait(&c.q_empty, (n.sigma - 1) & 1, &c.abort);
  }
  if (threadIdx.x == kLoadWarp * 32) {
    drain(c.full, kSlots, n.chunk, c);
    drain(c.meta, kMeta, n.tau, c);
    if (n.sigma > 0) ptx::mbar_wait(&c.q_full, (n.sigma - 1) & 1, &c.abort);
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (c.abort && threadIdx.x == 0 && p.flags) atomicOr(p.flags, DCPMLA_FLAG_TIMEOUT);
  if (warp == 0) ptx::tmem_dealloc(c.tmem_base, kTmemCols);
}

// Q operand images of every request (q_image.cuh), the second term times 2^kLoBits.
// Grid (batch, 2): each CTA covers 32 head rows with 8 threads per head.
__global__ void __launch_bounds__(256) mass_q_image_kernel(const PartialParams p, uint8_t* image) {
  ptx::launch_dependents();
  qimg::build_q_image_row<kLoBits>(p.q, p.rows_q, p.heads, blockIdx.x,
                                   blockIdx.y * 32 + (threadIdx.x >> 3), threadIdx.x & 7, image);
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
    mass_q_image_kernel<<<dim3(p.batch, 2), 256, 0, st>>>(p, p.q_image);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return launch_kernel(mass_kernel<kDtype>, dim3(p.num_ctas), kThreads, smem, st, 0,
                       kDtype == kKvFp8, m);
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
  // no more CTAs than the tables have blocks: any number may be asked for, and
  // rounding up by more than the tiles there are must not leave the int range
  ctas = (int)std::min<long long>(ctas, (long long)batch * block_table_stride);
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
    const double scale2 = (double)softmax_scale * 1.4426950408889634;
    m.scale2 = (float)scale2;
    m.scale2_err = scale2 != 0. ? (float)(m.scale2 / scale2 - 1.) : 0.f;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = kv_dtype == DCPMLA_KV_FP8 ? launch_mass<kKvFp8>(m, dev, st)
                                                    : launch_mass<kKvBf16>(m, dev, st);
    if (e != cudaSuccess) return DCPMLA_ERR_CUDA;
  }
  return DCPMLA_OK;
}

}  // extern "C"
