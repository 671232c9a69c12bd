// Choice of the cache blocks that a query token reads, from the block
// summaries (int8 codes of the mean key and their scales), and the decode over
// the chosen blocks.
//
//   q codes: per head and scale group, step = max|q| * fp32(1/127) (1 if 0), code
//            = rint(q / step)                               (values not finite: 0;
//            a decode with a negative softmax scale: the codes of -q)
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

#include <algorithm>
#include <climits>
#include <cmath>
#include <mutex>

#include "common.cuh"
#include "kernels.h"
#include "q_image.cuh"
#include "select_topk.cuh"
#include "tc_ptx.cuh"

namespace dcpmla {
namespace {

constexpr int kGroups = 5;
constexpr int kTile = 128;                          // blocks per scoring tile
constexpr uint32_t kChunk = 8192;                   // 64 query rows x 128 bytes
// Query image of a row: the int8 codes of 64 heads (zeros past the call's) in
// the scoring kernel's shared-memory order, a 128-byte-swizzled chunk per
// group (the rope's is half used), then the steps [group][head], 2 KB reserved.
constexpr int kQCodes = kGroups * kChunk;
constexpr int kQBytes = kQCodes + 2048;

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
  uint8_t* q_image;            // the e4m3 decode kernel's Q images, or nullptr
  int negate;                  // 1: rank by -q (a negative softmax scale)
  int num_ctas;                // SMs
  float* scores;               // [rows][tiles][heads][kTile]
  uint32_t* row_max;           // [rows][64] the heads' best scores, as ordered keys
  uint32_t* keys;              // [rows][bt_stride] ranks, or nullptr: the chooser's own
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
  if (bad && p.flags) atomicOr(p.flags, kFlagBadLength);
  *blocks = nb;
  return n;
}

// Query images of four heads of one row: half a warp per head and scale group, eight
// values a lane (its issue slots are what bounds it: 64 queries of 64 heads 7.2 us,
// with four values a lane 7.9, with 72 9; 48 of 16 heads 4.7 and 6.3).  With an
// e4m3 cache the decode kernel's Q image (its layout and rules: q_image.cuh) is built
// from the same loads.
constexpr int kCodeHeads = 4, kCodeThreads = kCodeHeads / 2 * kGroups * 32;
__global__ void __launch_bounds__(kCodeThreads) q_codes_kernel(const SelectParams p) {
  ptx::launch_dependents();
  __shared__ uint32_t top[kCodeHeads][4];        // latent: largest |q| bits of each group
  const int r = blockIdx.x, warp = threadIdx.x >> 5, l = threadIdx.x & 15;
  const uint32_t lanes = (threadIdx.x & 16) ? 0xFFFF0000u : 0xFFFFu;     // of this head
  const int hh = warp / kGroups * 2 + ((threadIdx.x >> 4) & 1), g = warp % kGroups;
  const int h = blockIdx.y * kCodeHeads + hh;
  const bool live = h < p.heads;
  const __nv_bfloat16* q =
      p.q + ((size_t)r * p.heads + (live ? h : 0)) * kHeadDim + 128 * g;
  const int d = (g < 4 ? 8 : 4) * l;             // first of the lane's values
  uint4 w = make_uint4(0, 0, 0, 0);
  if (live) {
    if (g < 4) {
      w = __ldg(reinterpret_cast<const uint4*>(q + d));
    } else {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(q + d));
      w.x = v.x;
      w.y = v.y;
    }
  }
  const uint32_t words[4] = {w.x, w.y, w.z, w.w};
  float x[8];
  uint32_t finite = 0, any = 0;         // largest magnitudes, as bits: finite ones, all but NaN
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t u = e & 1 ? words[e >> 1] & 0xFFFF0000u : words[e >> 1] << 16;
    const uint32_t m = u & 0x7FFFFFFFu;
    if (m <= 0x7F800000u) any = max(any, m);
    if (m < 0x7F800000u) finite = max(finite, m);
    x[e] = m < 0x7F800000u ? __uint_as_float(u) : 0.f;
  }
  finite = __reduce_max_sync(lanes, finite);
  const float amax = __uint_as_float(finite);
  const float up = __fmul_rn(amax, kInv127), step = up > 0.f ? up : 1.f;
  const float by = p.negate ? -step : step;
  const float inv = __frcp_rn(by);
  uint32_t code[2] = {0, 0};
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    // x / by, to the nearest: the product with the reciprocal is within 2^-16 of the
    // quotient (magnitudes up to 127); near a half, or where the reciprocal overflowed,
    // the division decides
    float c = rintf(__fmul_rn(x[e], inv));
    if (!(fabsf(__fsub_rn(__fmul_rn(x[e], inv), c)) < 0.4999f)) c = rintf(__fdiv_rn(x[e], by));
    code[e >> 2] |= ((uint32_t)min(127, max(-127, (int)c)) & 0xFFu) << (8 * (e & 3));
  }
  uint8_t* out = p.q_codes + (size_t)r * kQBytes;
  const uint32_t at = g * kChunk + qimg::sw128(h, d >> 4) + (d & 15);
  if (g < 4)
    *reinterpret_cast<uint2*>(out + at) = make_uint2(code[0], code[1]);
  else
    *reinterpret_cast<uint32_t*>(out + at) = code[0];
  if (l == 0) {
    reinterpret_cast<float*>(out + kQCodes)[g * 64 + h] = step;
    if (g == 0) p.row_max[(size_t)r * 64 + h] = 0u;      // below every score's key
  }
  if (!p.q_image) return;
  any = __reduce_max_sync(lanes, any);
  if (l == 0 && g < 4) top[hh][g] = any;
  __syncthreads();
  uint8_t* img = p.q_image + (size_t)r * kQImageBytes;
  if (g == 4) {
    *reinterpret_cast<uint2*>(img + qimg::kRope + qimg::sw128(h, d >> 3) + 2 * (d & 7)) =
        make_uint2(w.x, w.y);
    return;
  }
  const uint32_t m = max(max(top[hh][0], top[hh][1]), max(top[hh][2], top[hh][3]));
  const int a = m > 0 ? min(120, max(-120, 7 - ((int)(m >> 23) - 127))) : 0;
  const float fa = __uint_as_float((uint32_t)(127 + a) << 23);
  uint2 hi, lo;
  qimg::split_q4(w.x, w.y, fa, hi.x, lo.x);
  qimg::split_q4(w.z, w.w, fa, hi.y, lo.y);
  *reinterpret_cast<uint2*>(img + qimg::kHi + at) = hi;
  *reinterpret_cast<uint2*>(img + qimg::kLo + at) = lo;
  if (l == 0 && g == 0)
    reinterpret_cast<float*>(img + qimg::kFrame)[h] = __uint_as_float((uint32_t)(127 - a) << 23);
}

// ----------------------------------------------------------- scoring ----
//
// Scores of tiles of 128 blocks on the tensor cores (tcgen05, kind::i8): the
// summaries' codes are A (M = 128 blocks), the query's B (N = 64 heads), each
// scale group an int32 accumulator of its own, so that a TMEM lane holds one
// block for all heads.  Summaries are scattered over the pool: seven warps bring
// them into swizzled chunks (two tiles); warps 0-3 and 4-7 add each group's product, scaled, into the scores of 32 heads a
// thread, which are written [head][block], and keep each head's best of a row
// until its end.  The tiles of all rows, end to end, are dealt to the CTAs in
// contiguous ranges, so that a CTA rarely changes query.
//
// What bounds it is the copying, some 9,000 cycles a tile of 78 KB (64 queries of
// 1,024 blocks 24 us, of 4,096 blocks 66 us: 2.4 TB/s of summaries), then scoring
// and the int8 MMAs, 5,000 and 4,000.
// Sixteen warps: eight score, seven copy, one issues the MMAs; the launch gives a
// thread 128 registers, of which the scoring warpgroups take from the others.
constexpr int kScoreThreads = 512;
constexpr int kCopyBase = 256, kCopyThreads = 224, kMmaWarp = 15;
constexpr int kBarCopy = 1;
constexpr int kLaunchRegs = 128, kScoreRegs = 152, kCopyRegs = 104;
static_assert(256 * (kScoreRegs + kCopyRegs) == kScoreThreads * kLaunchRegs,
              "the register split must add up to what the launch holds");
constexpr int kUnits = kSummaryBytes / 16;         // 16-byte pieces of a summary
constexpr int kLoadWarps = 5;                      // of the copying threads: first these,
constexpr int kGatherBase = 32 * kLoadWarps, kAheadBase = kGatherBase + 32;   // then a warp each
static_assert(4 * kUnits <= kGatherBase && kAheadBase + 32 == kCopyThreads, "copy roles");
constexpr int kCopyBatch = 8;                      // pieces of a batch, two of them in flight
constexpr int kGatherRows = 32, kLoadRows = kTile - kGatherRows;   // of a tile's blocks
constexpr int kLoads = kLoadRows / 4, kCopyBatches = (kLoads + kCopyBatch - 1) / kCopyBatch;
static_assert(kGatherRows % 8 == 0 && kCopyBatch % 4 == 0 && kCopyBatches >= 2, "copy split");
constexpr int kScoreStages = 2, kBufs = 8;
constexpr uint32_t kSlot = 2 * kChunk;             // 128 blocks x 128 bytes
// A stage: the four latent chunks, then bytes 480 to 607 of every summary: the rope's
// codes 32 bytes into it, the scales at its end.
constexpr int kRopeX = kSummaryBytes - 128;
constexpr uint32_t kRopeAt = 512 - kRopeX;
constexpr uint32_t kStageBytes = kGroups * kSlot;
constexpr uint32_t kTmemCols = 64 * kBufs;
constexpr int kRowChunk = kScoreThreads; // rows looked at together

struct ScoreCtl {
  uint64_t full[kScoreStages], empty[kScoreStages];
  uint64_t d_full[kBufs], d_empty[kBufs];
  uint64_t q_full, q_empty;
  alignas(16) int ids[2][4][kTile / 4];  // the blocks of a tile, by tile parity and row % 4
  uint32_t tmem_base;
  int abort;
  int copies_end;                        // a copying thread's wait gave up
  int warp_sums[16];
  int end[kRowChunk];                    // tiles up to and including each row of the chunk
  int blocks[kRowChunk];
};
constexpr uint32_t kOffStage = kQCodes + 2048;     // after the query image
constexpr uint32_t kOffCtl = kOffStage + kScoreStages * kStageBytes;
constexpr size_t kScoreSmem = kOffCtl + sizeof(ScoreCtl) + 1024;
static_assert(kQBytes == kQCodes + 2048 && kOffStage % 1024 == 0 && kStageBytes % 1024 == 0 &&
                  kScoreSmem <= 232448,
              "shared memory layout");

__device__ __forceinline__ uint64_t dplus(uint64_t d, uint32_t byte_off) {
  return d + (uint64_t)(byte_off >> 4);
}

// Tile u of a chunk of rows: its row and place in the row.
struct TileWalk {
  int u, hi, row, tile, nb;
  __device__ __forceinline__ void locate(const ScoreCtl& c, int row_lo) {
    int a = row_lo, b = kRowChunk - 1;
    while (a < b) {
      const int mid = (a + b) >> 1;
      if (c.end[mid] > u) b = mid; else a = mid + 1;
    }
    row = a;
    tile = u - (a > 0 ? c.end[a - 1] : 0);
    nb = c.blocks[a];
  }
  __device__ __forceinline__ bool start(const ScoreCtl& c, int lo, int hi_) {
    u = lo;
    hi = hi_;
    if (u >= hi) return false;
    locate(c, 0);
    return true;
  }
  __device__ __forceinline__ bool last_of_row() const {
    return (tile + 1) * kTile >= nb || u + 1 >= hi;
  }
  __device__ __forceinline__ bool next(const ScoreCtl& c) {
    if (++u >= hi) return false;
    if ((tile + 1) * kTile < nb) {
      ++tile;
      return true;
    }
    locate(c, row + 1);
    return true;
  }
};

// fp32 of a whole number below 2^22 in magnitude (a group's products stay below
// 2^21): added to the bits of 1.5 * 2^23 it lands in the mantissa.  Two plain
// operations; the conversion instruction runs at a quarter of their rate.
__device__ __forceinline__ float small_int(uint32_t x) {
  return __fsub_rn(__uint_as_float(0x4B400000u + x), 12582912.f);
}

// Copies of every tile and of each row's query image, by both ways from memory to
// shared memory.  Five warps load the first 96 blocks through registers: thread
// (rr, un) of 152 has piece un of the rows 4 i + rr, so that a warp reads 512 bytes
// that mostly follow one another and a thread's addresses are sums of constants.
// A sixth issues four-row TMA gathers of the last 32, and the seventh walks a tile
// ahead: it looks up the blocks and sends their lines on their way to L2.  64
// queries of 4,096 blocks: 96 us with all blocks through registers, their pieces
// dealt to 224 threads in order, 89 as dealt here, and with 16, 24, 32, 48, 64 and 96
// of them by gathers 82, 69, 66, 66, 81 and 98 (a gather takes some 65 cycles to
// issue; the loads wait for one another's lines in L1, even where L2 has them all).
__device__ __forceinline__ void copy_role(const SelectParams& p, const CUtensorMap& map, ScoreCtl& c,
                                          uint8_t* base, int r0, int lo, int hi, uint32_t& tau,
                                          uint32_t& sigma) {
  const int t = threadIdx.x - kCopyBase;
  TileWalk w;
  if (!w.start(c, lo, hi)) return;
  bool fresh = true;
  // the blocks of the walk's tile; a bad entry: a stand-in, flagged
  auto look_up = [&](uint32_t parity) {
    const int* table = p.block_table + (size_t)((r0 + w.row) / p.q_len) * p.bt_stride;
    int blk[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int k = w.tile * kTile + t - kAheadBase + 32 * e;
      blk[e] = k < w.nb ? __ldg(table + k) : -1;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int row = t - kAheadBase + 32 * e;
      const bool live = w.tile * kTile + row < w.nb;
      if (blk[e] < 0 || (long long)blk[e] >= p.num_blocks) {
        if (live && p.flags) atomicOr(p.flags, kFlagBadBlock);
        blk[e] = 0;
      }
      c.ids[parity][row & 3][row >> 2] = blk[e];
      if (live) {
        const uint8_t* src = p.summaries + (size_t)blk[e] * kSummaryBytes;
#pragma unroll
        for (int i = 0; i < 5; ++i) ptx::prefetch_line_l2(src + 128 * i);
      }
    }
  };
  const bool ahead = t >= kAheadBase;
  const int rr = min(t / kUnits, 3), un = t - rr * kUnits;       // un past the end: no piece
  const uint8_t* from = p.summaries + un * 16;
  // places of the thread's rows 0 and 4 i + rr, i = 1; two rows further: + 1024
  const int chunk = un < 32 ? un >> 3 : 4, unit = un < 32 ? un & 7 : un - kRopeX / 16;
  const uint32_t to0 = chunk * kSlot + qimg::sw128(rr, unit & 7);
  const uint32_t to1 = chunk * kSlot + qimg::sw128(rr + 4, unit & 7);
  if (ahead) look_up(tau & 1);
  ptx::named_bar(kBarCopy, kCopyThreads);
  while (true) {
    const uint32_t s = tau % kScoreStages;
    const int r = r0 + w.row;
    // rows past the tile's end are left as they are (they only reach their own lanes)
    const int blocks = min(kTile, w.nb - w.tile * kTile);
    const bool row_ends = w.last_of_row();
    const bool more = w.next(c);
    uint8_t* stage = base + kOffStage + s * kStageBytes;
    if (ahead) {
      if (more) look_up((tau + 1) & 1);
    } else if (t >= kGatherBase) {
      const int lane = t - kGatherBase;
      // groups of four blocks (past the tile's end: stand-ins, block 0)
      const int groups = max(blocks - kLoadRows + 3, 0) / 4;
      if (tau >= (uint32_t)kScoreStages &&
          !__all_sync(0xffffffffu,
                      ptx::mbar_wait(&c.empty[s], ((tau / kScoreStages) + 1) & 1, &c.abort))) {
        c.copies_end = 1;              // seen by all at the barrier below
      } else {
        if (lane == 0) ptx::mbar_arrive_expect_tx(&c.full[s], groups * 4 * kGroups * 128);
        __syncwarp();
        for (int u = lane; u < groups * kGroups; u += 32) {
          const int q = u / kGroups, g = u - q * kGroups, row = kLoadRows + 4 * q;
          const int (*ids)[kTile / 4] = c.ids[tau & 1];
          const int4 rows = make_int4(ids[0][row >> 2], ids[1][row >> 2], ids[2][row >> 2],
                                      ids[3][row >> 2]);
          ptx::tma_gather4(ptx::smem_addr(stage + g * kSlot + row * 128), &map,
                           g < 4 ? g * 128 : kRopeX, rows, &c.full[s]);
        }
      }
    } else {
      const int rows = un < kUnits ? min(blocks, kLoadRows) - rr : 0;
      const int* ids = c.ids[tau & 1][rr];
      uint4 v[2][kCopyBatch];
      auto load = [&](int b) {
#pragma unroll
        for (int i = 0; i < kCopyBatch; i += 4) {
          const int4 id = *reinterpret_cast<const int4*>(ids + b * kCopyBatch + i);
          const int blk[4] = {id.x, id.y, id.z, id.w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (b * kCopyBatch + i + e < kLoads && 4 * (b * kCopyBatch + i + e) < rows)
              v[b & 1][i + e] =
                  __ldg(reinterpret_cast<const uint4*>(from + (size_t)blk[e] * kSummaryBytes));
        }
      };
      load(0);
      load(1);
      if (tau >= (uint32_t)kScoreStages &&
          !__all_sync(0xffffffffu,
                      ptx::mbar_wait(&c.empty[s], ((tau / kScoreStages) + 1) & 1, &c.abort)))
        c.copies_end = 1;              // seen by all at the barrier below
#pragma unroll
      for (int b = 0; b < kCopyBatches; ++b) {
        if (b > 0 && b + 1 < kCopyBatches) load(b + 1);
#pragma unroll
        for (int i = 0; i < kCopyBatch; ++i) {
          const int k = b * kCopyBatch + i;
          if (k < kLoads && 4 * k < rows)
            *reinterpret_cast<uint4*>(stage + ((k & 1) ? to1 : to0) + (k >> 1) * 1024) = v[b & 1][i];
        }
      }
      ptx::fence_proxy_async();          // the MMAs read through the async proxy
      __syncwarp();
      if ((t & 31) == 0) ptx::mbar_arrive(&c.full[s]);
    }
    if (fresh) {
      if (t == 0) {
        if (sigma > 0 && !ptx::mbar_wait(&c.q_empty, (sigma - 1) & 1, &c.abort)) {
          c.copies_end = 1;
        } else {
          ptx::wait_primary();     // the query images' kernel
          // the scorers read the old steps through the generic proxy
          ptx::fence_proxy_async();
          ptx::mbar_arrive_expect_tx(&c.q_full, kQBytes);
          ptx::bulk_g2s(ptx::smem_addr(base), p.q_codes + (size_t)r * kQBytes, kQBytes, &c.q_full);
        }
      }
      ++sigma;
    }
    fresh = row_ends;
    ++tau;
    if (!more) break;
    ptx::named_bar(kBarCopy, kCopyThreads);
    if (c.copies_end) return;
  }
}

__device__ __forceinline__ void score_mma_role(ScoreCtl& c, uint8_t* base, int lo, int hi,
                                               uint32_t& tau, uint32_t& sigma, uint32_t& part) {
  constexpr uint32_t kId = ptx::idesc_i8(128, 64);
  const uint64_t dq = ptx::sdesc(ptx::smem_addr(base), 16, 1024, ptx::kSwizzle128B);
  const uint64_t dk0 = ptx::sdesc(ptx::smem_addr(base + kOffStage), 16, 1024, ptx::kSwizzle128B);
  TileWalk w;
  if (!w.start(c, lo, hi)) return;
  bool fresh = true;
  while (true) {
    const uint32_t s = tau % kScoreStages;
    if (fresh) ++sigma;
    uint64_t* full = &c.full[s];
    const uint32_t pf = (tau / kScoreStages) & 1;
    const uint64_t dk = dplus(dk0, s * kStageBytes);
    // one round trip tests the barriers of parts 0-1 with the tile's, then of 2-4
#pragma unroll 1
    for (int g0 = 0; g0 < kGroups; g0 += g0 == 0 ? 2 : 3) {
      const int n = g0 == 0 ? 2 : 3;
      uint64_t* bars[4];
      uint32_t pars[4];
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        const uint32_t pi = part + (i < n ? i : 0);
        const bool reuse = pi >= (uint32_t)kBufs;
        bars[i] = reuse ? &c.d_empty[pi % kBufs] : full;
        pars[i] = reuse ? ((pi / kBufs) + 1) & 1 : pf;
      }
      if (g0 == 0) {
        bars[2] = &c.q_full;
        pars[2] = (sigma - 1) & 1;
      }
      bars[3] = full;
      pars[3] = pf;
      if (!ptx::mbar_wait4(bars, pars, &c.abort)) return;
      ptx::tc_fence_after();
#pragma unroll 1
      for (int g = g0; g < g0 + n; ++g, ++part) {
        const uint32_t d = c.tmem_base + 64 * (part % kBufs);
        for (int ks = 0; ks < (g < 4 ? 4 : 2); ++ks)
          ptx::mma_i8(d, dplus(dk, g * kSlot + (g < 4 ? 0 : kRopeAt) + ks * 32), dplus(dq, g * kChunk + ks * 32), kId,
                      ks > 0);
        ptx::mma_commit(&c.d_full[part % kBufs]);
      }
    }
    ptx::mma_commit(&c.empty[s]);
    fresh = w.last_of_row();
    if (fresh) ptx::mma_commit(&c.q_empty);
    ++tau;
    if (!w.next(c)) break;
  }
}

// Scores: thread (hh, row) has heads [32 hh, 32 hh + 32) of the tile's block.
__device__ __forceinline__ void score_role(const SelectParams& p, ScoreCtl& c, uint8_t* base, int r0,
                                           int lo, int hi, uint32_t& tau, uint32_t& sigma,
                                           uint32_t& part) {
  const int hh = threadIdx.x >> 7, row = threadIdx.x & 127, lane = threadIdx.x & 31;
  const uint32_t lane_base = c.tmem_base + ((uint32_t)((row >> 5) * 32) << 16) + 32 * hh;
  const float* steps = reinterpret_cast<const float*>(base + kQCodes) + 32 * hh;
  const int heads = min(32, p.heads - 32 * hh);      // of this thread (may be <= 0)
  TileWalk w;
  if (!w.start(c, lo, hi)) return;
  bool fresh = true;
  float best[32];
  while (true) {
    if (fresh) {
      if (!ptx::mbar_wait(&c.q_full, sigma & 1, &c.abort)) return;
      ++sigma;
#pragma unroll
      for (int e = 0; e < 32; ++e) best[e] = -INFINITY;
    }
    fresh = w.last_of_row();
    const uint32_t s = tau % kScoreStages;
    const int r = r0 + w.row, k = w.tile * kTile + row;
    bool live = k < w.nb;
    if (live) {
      const int blk = __ldg(p.block_table + (size_t)(r / p.q_len) * p.bt_stride + k);
      live = blk >= 0 && (long long)blk < p.num_blocks;
    }
    if (!ptx::mbar_wait(&c.full[s], (tau / kScoreStages) & 1, &c.abort)) return;
    const uint8_t* sp = base + kOffStage + s * kStageBytes + (kGroups - 1) * kSlot;
    const float4 s4 = *reinterpret_cast<const float4*>(sp + qimg::sw128(row, 6));
    const float sc[kGroups] = {s4.x, s4.y, s4.z, s4.w,
                               *reinterpret_cast<const float*>(sp + qimg::sw128(row, 7))};
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(&c.empty[s]);
    float v[32];
#pragma unroll
    for (int g = 0; g < kGroups; ++g, ++part) {
      const uint32_t buf = part % kBufs;
      if (!ptx::mbar_wait(&c.d_full[buf], (part / kBufs) & 1, &c.abort)) return;
      __syncwarp();
      ptx::tc_fence_after();
      uint32_t x[32];
      ptx::tmem_ld32(lane_base + 64 * buf, x);
      ptx::tmem_wait_ld();
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&c.d_empty[buf]);
#pragma unroll
      for (int e4 = 0; e4 < 8; ++e4) {
        const float4 q4 = *reinterpret_cast<const float4*>(steps + g * 64 + 4 * e4);
        const float qs[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int e = 4 * e4 + i;
          const float term = __fmul_rn(small_int(x[e]), __fmul_rn(qs[i], sc[g]));
          v[e] = g == 0 ? term : __fadd_rn(v[e], term);
        }
      }
    }
    float* out = p.scores + (((size_t)r * p.tiles + w.tile) * p.heads + 32 * hh) * kTile + row;
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      if (!live) v[e] = -INFINITY;
      best[e] = fmaxf(best[e], v[e]);
      if (e < heads) out[e * kTile] = v[e];
    }
    if (fresh) {
      // the row's image is done with here; its heads' best go to the row
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&c.q_empty);
      uint32_t mine = 0;
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        const uint32_t m = __reduce_max_sync(0xffffffffu, topk::key_of(best[e]));
        if (lane == e) mine = m;
      }
      if (lane < heads) atomicMax(p.row_max + (size_t)r * 64 + 32 * hh + lane, mine);
    }
    ++tau;
    if (!w.next(c)) break;
  }
}

// Barrier over the whole block, written out so that the two sides of the register
// split can both use it.
__device__ __forceinline__ void block_bar() { ptx::named_bar(2, kScoreThreads); }

// The chunks of rows, on one side of the register split: kScorers the scoring
// warps, else the copies and the MMAs and, at the end, the drains.  Both take the
// same block barriers.
template <bool kScorers>
__device__ __forceinline__ void run_scores(const SelectParams& p, const CUtensorMap& map, ScoreCtl& c, uint8_t* base) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rows = p.batch * p.q_len;
  uint32_t tau = 0, sigma = 0, part = 0;
  for (int r0 = 0; r0 < rows; r0 += kRowChunk) {
    // a row a thread (kRowChunk = kScoreThreads): tiles, and their running sum
    int nb = 0;
    if (r0 + (int)threadIdx.x < rows) rows_of(p, r0 + threadIdx.x, &nb);
    const int nt = nb > p.topk ? (nb + kTile - 1) / kTile : 0;     // else all are taken
    int x = nt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) c.warp_sums[warp] = x;
    block_bar();
    int total = 0;
#pragma unroll
    for (int k = 0; k < kScoreThreads / 32; ++k) {
      if (k < warp) x += c.warp_sums[k];
      total += c.warp_sums[k];
    }
    c.end[threadIdx.x] = x;
    c.blocks[threadIdx.x] = nb;
    block_bar();
    const int lo = (int)((long long)blockIdx.x * total / gridDim.x);
    const int hi = (int)((long long)(blockIdx.x + 1) * total / gridDim.x);
    if constexpr (kScorers) {
      score_role(p, c, base, r0, lo, hi, tau, sigma, part);
    } else {
      if (warp < kMmaWarp)
        copy_role(p, map, c, base, r0, lo, hi, tau, sigma);
      else if (lane == 0)
        score_mma_role(c, base, lo, hi, tau, sigma, part);
    }
    block_bar();
    if (c.abort) break;
  }
  if constexpr (!kScorers) {
    // Drain: every asynchronous arrival and copy lands before the CTA exits.
    if (threadIdx.x == kMmaWarp * 32) {
      for (uint32_t s = 0; s < (uint32_t)kScoreStages; ++s) {
        const uint32_t u = tau > s ? (tau - s + kScoreStages - 1) / kScoreStages : 0;
        if (u > 0) ptx::mbar_wait(&c.empty[s], (u - 1) & 1, &c.abort);
      }
      for (uint32_t k = 0; k < (uint32_t)kBufs; ++k) {
        const uint32_t u = part > k ? (part - k + kBufs - 1) / kBufs : 0;
        if (u > 0) ptx::mbar_wait(&c.d_full[k], (u - 1) & 1, &c.abort);
      }
      if (sigma > 0) ptx::mbar_wait(&c.q_empty, (sigma - 1) & 1, &c.abort);
    }
    if (threadIdx.x == kCopyBase && sigma > 0)
      ptx::mbar_wait(&c.q_full, (sigma - 1) & 1, &c.abort);
    if (threadIdx.x == kCopyBase + kGatherBase)
      for (uint32_t s = 0; s < (uint32_t)kScoreStages; ++s) {
        const uint32_t u = tau > s ? (tau - s + kScoreStages - 1) / kScoreStages : 0;
        if (u > 0) ptx::mbar_wait(&c.full[s], (u - 1) & 1, &c.abort);
      }
  }
}

__global__ void __launch_bounds__(kScoreThreads, 1) score_kernel(const SelectParams p, const __grid_constant__ CUtensorMap map) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  ScoreCtl& c = *reinterpret_cast<ScoreCtl*>(base + kOffCtl);
  const int warp = threadIdx.x >> 5;
  ptx::launch_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kScoreStages; ++s) {
      ptx::mbar_init(&c.full[s], kLoadWarps + 1);
      ptx::mbar_init(&c.empty[s], 1 + 8);    // the MMAs' commit, eight warps' scale reads
    }
    for (int k = 0; k < kBufs; ++k) {
      ptx::mbar_init(&c.d_full[k], 1);
      ptx::mbar_init(&c.d_empty[k], 8);
    }
    ptx::mbar_init(&c.q_full, 1);
    ptx::mbar_init(&c.q_empty, 1 + 8);       // the MMAs' commit, eight warps' step reads
    c.abort = 0;
    c.copies_end = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 0) ptx::tmem_alloc(&c.tmem_base, kTmemCols);
  ptx::fence_proxy_async();
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  // every warpgroup adjusts its registers here, before any role can return
  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kScoreRegs));
    run_scores<true>(p, map, c, base);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kCopyRegs));
    run_scores<false>(p, map, c, base);
  }
  // a CTA without tiles waits too: this kernel's end implies the previous one's
  ptx::wait_primary();
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (c.abort && threadIdx.x == 0 && p.flags) atomicOr(p.flags, DCPMLA_FLAG_TIMEOUT);
  if (warp == 0) ptx::tmem_dealloc(c.tmem_base, kTmemCols);
}

// Key of block k of a row: its rank, or the largest key where it is taken anyway.
__device__ __forceinline__ uint32_t rank_key(const SelectParams& p, const float* hmax, int r, int k,
                                             int nb) {
  if (nb <= p.topk || k < p.sink || k >= nb - p.recent) return 0xFFFFFFFFu;
  const float* s = p.scores + ((size_t)r * p.tiles + k / kTile) * p.heads * kTile + k % kTile;
  float rank = -INFINITY;
  auto add = [&](float v, int h) {
    // equal infinities: no distance
    rank = fmaxf(rank, v == hmax[h] ? 0.f : __fsub_rn(v, hmax[h]));
  };
  int h = 0;
  for (; h + 16 <= p.heads; h += 16) {
    float v[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] = __ldcg(s + (h + e) * kTile);
#pragma unroll
    for (int e = 0; e < 16; ++e) add(v[e], h + e);
  }
  for (; h < p.heads; ++h) add(__ldcg(s + h * kTile), h);
  return topk::key_of(rank);
}

// Ranks of long rows, all over the device (a row's scores are 256 bytes a block
// and head set: read by its cluster alone, 16,384 blocks took 20 us).
constexpr int kRankThreads = 256;
__global__ void __launch_bounds__(kRankThreads) rank_kernel(const SelectParams p) {
  __shared__ float hmax[64];
  ptx::launch_dependents();
  const int r = blockIdx.y, k = blockIdx.x * kRankThreads + threadIdx.x;
  int nb;
  rows_of(p, r, &nb);
  ptx::wait_primary();
  if (blockIdx.x * kRankThreads >= nb) return;
  if (threadIdx.x < 64) hmax[threadIdx.x] = topk::value_of(__ldcg(p.row_max + r * 64 + threadIdx.x));
  __syncthreads();
  if (k < nb) p.keys[(size_t)r * p.bt_stride + k] = rank_key(p, hmax, r, k, nb);
}

// Ranks (unless there) and the choice of one row: one cluster.
__global__ void __launch_bounds__(topk::kThreads) choose_kernel(const SelectParams p, int bit_words) {
  extern __shared__ __align__(16) uint32_t dyn[];
  __shared__ topk::Ctl c;
  __shared__ float hmax[64];
  topk::cg::cluster_group cl = topk::cg::this_cluster();
  const int r = blockIdx.y, b = r / p.q_len;
  int nb;
  const int n = rows_of(p, r, &nb);
  uint32_t* bits = dyn;
  uint32_t* keys = dyn + bit_words;
  int lo, hi;
  topk::slice(nb, cl.block_rank(), cl.num_blocks(), &lo, &hi);
  const int want = min(nb, p.topk);
  ptx::wait_primary();
  if (threadIdx.x < 64) hmax[threadIdx.x] = topk::value_of(__ldcg(p.row_max + r * 64 + threadIdx.x));
  __syncthreads();
  for (int k = lo + threadIdx.x; k < hi; k += topk::kThreads)
    keys[k - lo] = p.keys ? __ldcg(p.keys + (size_t)r * p.bt_stride + k) : rank_key(p, hmax, r, k, nb);
  __syncthreads();
  if (want > 0)
    topk::mark(cl, c, lo, hi, want, bits, [&](int i) { return keys[i - lo]; },
               [](int, uint32_t k, bool) { return k; });
  // places of this slice's blocks in the list
  int pos[1] = {0};
  if (cl.num_blocks() > 1) {
    int mine = 0, tot;
    for (int w = threadIdx.x; w < (hi - lo + 31) / 32; w += topk::kThreads) mine += __popc(bits[w]);
    block_exclusive_scan(mine, c.warp_sums, &tot);
    if (threadIdx.x == 0) c.share[0] = tot;
    topk::sync(cl);
    pos[0] = topk::before(cl, c, 0);
    topk::sync(cl);          // shared memory stays until every CTA has read it
  }
  topk::emit<1>(c, lo, hi, pos, [&](int, int w) { return bits[w]; }, [&](int, int k, int at) {
    if (p.out_blocks) p.out_blocks[(size_t)r * p.topk + at] = k;
    const int blk = __ldg(p.block_table + (size_t)b * p.bt_stride + k);
    if ((blk < 0 || (long long)blk >= p.num_blocks) && p.flags) atomicOr(p.flags, kFlagBadBlock);
    p.out_table[(size_t)r * p.topk + at] = blk;
  });
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

// Rows of more blocks than this are ranked by a kernel of its own.
constexpr int kRankStride = 4096;

// Workspace: 256-byte header (flag word), q codes, scores, the heads' best, keys.
struct SelectLayout {
  size_t q_codes, scores, row_max, keys, total;
};
SelectLayout layout(int rows, int heads, int stride) {
  const size_t tiles = ((size_t)stride + kTile - 1) / kTile;
  SelectLayout l;
  l.q_codes = kWsHeader;
  l.scores = l.q_codes + round256((size_t)rows * kQBytes);
  l.row_max = l.scores + round256((size_t)rows * tiles * heads * kTile * 4);
  l.keys = l.row_max + (size_t)rows * 256;
  l.total = l.keys + (stride > kRankStride ? round256((size_t)rows * stride * 4) : 0);
  return l;
}

// Largest table stride: a row's keys and bits fit one cluster's shared memory.
constexpr int kMaxKeys = 49152;            // of a CTA
constexpr int kMaxStride = topk::kMaxCluster * kMaxKeys;

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
  // the register split assumes exactly kLaunchRegs a thread at launch: with fewer the
  // scoring warpgroups' increase could never be granted.  A kernel that moves registers
  // is launched with as many as its launch bounds leave a thread (65,536 / 512),
  // whatever its code needs; this check is for a compiler that does otherwise
  cudaFuncAttributes fa;
  e = cudaFuncGetAttributes(&fa, score_kernel);
  if (e != cudaSuccess) return e;
  if (fa.numRegs != kLaunchRegs) return cudaErrorInvalidDeviceFunction;
  e = cudaFuncSetAttribute(score_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)kScoreSmem);
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

// The summaries as [num_blocks][608] bytes, boxes of 128 bytes of one row (gathers).
bool summary_map(const SelectParams& p, CUtensorMap* map) {
  EncodeTiledFn enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)kSummaryBytes, (cuuint64_t)std::min<long long>(p.num_blocks, INT_MAX)};
  const cuuint64_t strides[1] = {(cuuint64_t)kSummaryBytes};
  const cuuint32_t box[2] = {128, 1}, es[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(p.summaries), dims, strides,
             box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_select(const SelectParams& p, cudaStream_t st) {
  const int rows = p.batch * p.q_len;
  q_codes_kernel<<<dim3(rows, kMaxHeads / kCodeHeads), kCodeThreads, 0, st>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  CUtensorMap map;
  if (!summary_map(p, &map)) return cudaErrorNotSupported;
  e = launch_kernel(score_kernel, dim3((unsigned)std::min<long long>(p.num_ctas, (long long)rows * p.tiles)),
                    kScoreThreads, kScoreSmem, st, 0, true, p, map);
  if (e != cudaSuccess) return e;
  if (p.keys) {
    e = launch_kernel(rank_kernel, dim3((p.bt_stride + kRankThreads - 1) / kRankThreads, rows),
                      kRankThreads, 0, st, 0, true, p);
    if (e != cudaSuccess) return e;
  }
  int size = topk::cluster_size(p.bt_stride, rows, p.num_ctas);
  while ((long long)size * kMaxKeys < p.bt_stride) size *= 2;      // keys and bits in shared memory
  const int words = topk::slice_words(p.bt_stride, size);
  return launch_kernel(choose_kernel, dim3(size, rows), topk::kThreads, (size_t)words * 33 * 4, st,
                       size, true, p, words);
}

// The choice on a workspace part `ws` (laid out by layout()).
int run_select(SelectParams& p, uint8_t* ws, cudaStream_t st) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return DCPMLA_ERR_CUDA;
  if (dev < 0 || dev >= kMaxDevicesConfigured) return DCPMLA_ERR_UNSUPPORTED;
  if (prepare_device(dev) != cudaSuccess) return DCPMLA_ERR_CUDA;
  int rc = dcpmla_device_sm_count(&p.num_ctas);
  if (rc != DCPMLA_OK) return rc;
  const SelectLayout l = layout(p.batch * p.q_len, p.heads, p.bt_stride);
  p.q_codes = ws + l.q_codes;
  p.scores = reinterpret_cast<float*>(ws + l.scores);
  p.row_max = reinterpret_cast<uint32_t*>(ws + l.row_max);
  p.keys = p.bt_stride > kRankStride ? reinterpret_cast<uint32_t*>(ws + l.keys) : nullptr;
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
  // With fewer chosen blocks than CTAs a CTA takes two of them, down to sixteen
  // pieces a query: half the pieces to combine (one request of 64 blocks: 79 us
  // with 64 pieces, 74 with 32, 76 with 16; the workspace has room for more).
  // With more, a whole number of CTAs a query, if that leaves few SMs out: no CTA
  // then starts a second query (64 queries of 32 blocks: 116 us on 128 CTAs, 121 on
  // 148).
  int splits = num_splits;
  if (splits == 0) {
    int sms = 0;
    rc = dcpmla_device_sm_count(&sms);
    if (rc != DCPMLA_OK) return rc;
    const long long tiles = (long long)rows * block_topk;
    splits = (int)std::min<long long>(
        sms, std::max<long long>((long long)rows * std::min(block_topk, 16), (tiles + 1) / 2));
    if (splits == sms && rows <= sms && (sms - sms % rows) * 7 >= sms * 6) splits = sms - sms % rows;
  }
  p.out_blocks = out_blocks;
  p.out_table = reinterpret_cast<int*>(sel + layout(rows, num_heads, block_table_stride).total);
  p.out_lens = p.out_table + round256((size_t)rows * block_topk * 4) / 4;
  p.flags = static_cast<int*>(workspace);
  p.negate = softmax_scale < 0.f;
  p.q_image = decode_chosen_q_image(kv_dtype, rows, num_heads, splits, impl, workspace);
  rc = run_select(p, sel, static_cast<cudaStream_t>(stream));
  if (rc != DCPMLA_OK) return rc;
  // the chosen blocks of a query are one request of one shard, in a table of their own
  return decode_chosen_blocks(q, kv_cache, kv_dtype, num_blocks, p.out_table, block_topk,
                              p.out_lens, rows, num_heads, softmax_scale, out_partial, out_lse,
                              workspace, dec, splits, impl, stream);
}

}  // extern "C"
