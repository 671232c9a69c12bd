// Selection of the `want` largest of n 32-bit keys by one thread-block
// cluster, ties to the lowest index.
//
// The CTAs of the cluster own consecutive slices of the index range.  A radix
// descent of 8 bits a pass finds the key T of the last one taken: every CTA
// counts its slice's digits among the keys that match the prefix so far, the
// histograms are summed over distributed shared memory, and the digit in
// which the want-th key falls extends the prefix.  The keys above T are taken
// and, of those equal to T, the first ones.  The result is a bit per index in
// the owning CTA's shared memory, independent of the cluster's size.
//
// What bounds it for all but the longest inputs is the number of barriers, not
// the keys: a pass has two (counts complete; digit known), one warp scans the
// 256 bins, and slices of up to kHeld keys a thread stay in registers.
#pragma once

#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace dcpmla {
namespace topk {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kBins = 256;
constexpr int kHeld = 16;        // keys a thread holds in registers
constexpr int kMaxCluster = 8;   // the largest portable cluster
constexpr int kPasses = 4;

struct Ctl {
  alignas(16) uint32_t hist[kPasses][kBins];   // this CTA's digit counts
  alignas(16) uint32_t total[kBins];           // the cluster's, of the current pass
  int warp_sums[kThreads / 32];
  int digit, above, equal;         // chosen digit, keys above it and in it (whole cluster)
  int share[2];                    // what the other CTAs of the cluster read of this one
  int offs[2][kThreads];           // emit(): entries before each word of a batch
};

// fp32 -> a key in the same order; NaN below everything, -0 equal to 0.
__device__ __forceinline__ uint32_t key_of(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// The value of a key that is not NaN's.
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? key & 0x7FFFFFFFu : ~key);
}

// Barrier over the cluster (over the block if that is the cluster).
__device__ __forceinline__ void sync(cg::cluster_group& cl) {
  if (cl.num_blocks() == 1)
    __syncthreads();
  else
    cl.sync();
}

// Sum of `share[which]` over the CTAs before this one (call between cluster
// barriers that order the writes and the next reuse).
__device__ __forceinline__ int before(cg::cluster_group& cl, Ctl& c, int which) {
  const unsigned r = threadIdx.x & 31;        // a lane a CTA: the reads are in flight together
  const int v = r < cl.block_rank() ? cl.map_shared_rank(c.share, r)[which] : 0;
  return (int)__reduce_add_sync(0xffffffffu, (unsigned)v);
}

// mark() for slices whose keys are read again in every pass (kPer 0), or of at
// most kPer keys a thread, held in registers.
template <int kPer, class LoadFn, class KeyFn>
__device__ __forceinline__ void mark_keys(cg::cluster_group& cl, Ctl& c, int lo, int hi, int want,
                                          uint32_t* bits, LoadFn&& load, KeyFn&& key) {
  using Raw = decltype(load(0));
  const int tid = threadIdx.x, lane = tid & 31;
  constexpr int kRegs = kPer > 0 ? kPer : 1;
  uint32_t held[kRegs];
  if constexpr (kPer > 0) {
    Raw raw[kRegs];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int i = lo + j * kThreads + tid;
      if (i < hi) raw[j] = load(i);
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int i = lo + j * kThreads + tid;
      held[j] = i < hi ? key(i, raw[j], true) : 0u;
    }
  }
  // f(index, key, inside) for this thread's keys, in rounds of kThreads; all
  // threads take part in every round
  bool first = true;
  auto rounds = [&](auto&& f) {
    if constexpr (kPer > 0) {
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (lo + j * kThreads < hi) {
          const int i = lo + j * kThreads + tid;
          f(i, held[j], i < hi);
        }
    } else {
      for (int base = lo; base < hi; base += 8 * kThreads) {
        uint32_t k[8];
        Raw raw[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int i = base + j * kThreads + tid;
          if (i < hi) raw[j] = load(i);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int i = base + j * kThreads + tid;
          k[j] = i < hi ? key(i, raw[j], first) : 0u;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (base + j * kThreads < hi) {
            const int i = base + j * kThreads + tid;
            f(i, k[j], i < hi);
          }
      }
      first = false;
    }
  };
  for (int b = tid; b < kPasses * kBins; b += kThreads) (&c.hist[0][0])[b] = 0;
  __syncthreads();
  uint32_t prefix = 0, mask = 0;
  int left = want, pass = 0;
  // once all keys of the chosen digit are taken the lower digits do not matter
  // (distinct keys: two or three passes of the four)
  bool all = false;
#pragma unroll
  for (; pass < kPasses && !all; ++pass) {
    const int shift = 24 - 8 * pass;
    uint32_t* h = c.hist[pass];
    // plain increments without a result: the hardware merges a warp's equal digits
    rounds([&](int, uint32_t k, bool in) {
      if (in && (k & mask) == prefix) atomicAdd(&h[(k >> shift) & 255u], 1u);
    });
    sync(cl);
    if (cl.num_blocks() > 1) {
      if (tid < kBins / 4) {
        uint4 v[kMaxCluster];
        uint4 s = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (unsigned r = 0; r < (unsigned)kMaxCluster; ++r)
          v[r] = r < cl.num_blocks() ? reinterpret_cast<const uint4*>(cl.map_shared_rank(h, r))[tid]
                                     : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) {
          s.x += v[r].x;
          s.y += v[r].y;
          s.z += v[r].z;
          s.w += v[r].w;
        }
        reinterpret_cast<uint4*>(c.total)[tid] = s;
      }
      __syncthreads();
      h = c.total;
    }
    if (tid < 32) {
      // lane l: bins 255 - 8 l .. 248 - 8 l, from the largest digit down
      int v[8], sum = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[e] = (int)h[kBins - 1 - 8 * lane - e];
        sum += v[e];
      }
      int ex = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, ex, o);
        if (lane >= o) ex += y;
      }
      ex -= sum;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (ex < left && left <= ex + v[e]) {
          c.digit = kBins - 1 - 8 * lane - e;
          c.above = ex;
          c.equal = v[e];
        }
        ex += v[e];
      }
    }
    __syncthreads();
    left -= c.above;
    prefix |= (uint32_t)c.digit << shift;
    mask |= 255u << shift;
    all = left == c.equal;
  }
  // Unless all are taken, the last pass's histogram counts the keys equal to T and
  // their order decides.
  int seen = 0;
  if (!all) {
    if (tid == 0) c.share[0] = (int)c.hist[kPasses - 1][c.digit];
    sync(cl);
    seen = before(cl, c, 0);
  }
  if (all) {
    rounds([&](int i, uint32_t k, bool in) {
      const uint32_t word = __ballot_sync(0xffffffffu, in && k >= prefix);
      if (lane == 0 && in) bits[(i - lo) >> 5] = word;
    });
  } else {
    // first the keys above T and, beside them, those equal to it; then the equal
    // ones up to the `left`-th, a batch of words at a time
    rounds([&](int i, uint32_t k, bool in) {
      const uint32_t word = __ballot_sync(0xffffffffu, in && k > prefix);
      const uint32_t same = __ballot_sync(0xffffffffu, in && k == prefix);
      if (lane == 0 && in) {
        bits[(i - lo) >> 5] = word;
        if constexpr (kPer > 0) c.offs[0][(i - lo) >> 5] = (int)same;   // all in one batch
      }
    });
    const int words = (hi - lo + 31) / 32;
    static_assert(kPer * kThreads / 32 <= kThreads, "held keys make one batch of words");
    for (int w0 = 0; w0 < words; w0 += kThreads) {
      for (int j = tid >> 5; kPer == 0 && j < kThreads && w0 + j < words; j += kThreads / 32) {
        const int i = lo + 32 * (w0 + j) + lane;
        const uint32_t word = __ballot_sync(0xffffffffu, i < hi && key(i, load(i), false) == prefix);
        if (lane == 0) c.offs[0][j] = (int)word;
      }
      __syncthreads();
      const uint32_t eq = w0 + tid < words ? (uint32_t)c.offs[0][tid] : 0u;
      int tot;
      const int before_w = seen + block_exclusive_scan(__popc(eq), c.warp_sums, &tot);
      seen += tot;
      const int room = left - before_w;        // equal keys still taken in this word
      if (eq && room > 0) {
        uint32_t keep = eq;
        for (int over = __popc(eq) - room; over > 0; --over) keep &= ~(0x80000000u >> __clz(keep));
        bits[w0 + tid] |= keep;
      }
      __syncthreads();
    }
  }
  sync(cl);      // `bits` complete; the shared fields may be written again
}

// Marks the taken indices of this CTA's slice [lo, hi) in `bits` (bit i - lo;
// room for ceil((hi - lo) / 32) words).  load(i) reads what the key of index i is
// made of, key(i, raw, first) makes it: for every index with `first` once, possibly
// again without.  A thread's loads come before its key() calls, which may write.  All threads of all CTAs of the cluster call
// it with the same n and 1 <= want <= n.
template <class LoadFn, class KeyFn>
__device__ __forceinline__ void mark(cg::cluster_group& cl, Ctl& c, int lo, int hi, int want,
                                     uint32_t* bits, LoadFn&& load, KeyFn&& key) {
  const int n = hi - lo;
  if (n <= 2 * kThreads)
    mark_keys<2>(cl, c, lo, hi, want, bits, load, key);
  else if (n <= 8 * kThreads)
    mark_keys<8>(cl, c, lo, hi, want, bits, load, key);
  else if (n <= kHeld * kThreads)
    mark_keys<kHeld>(cl, c, lo, hi, want, bits, load, key);
  else
    mark_keys<0>(cl, c, lo, hi, want, bits, load, key);
}

// Numbers the set bits of kLists masks of the slice in index order:
// f(list, index, place) for each.  word(list, w) gives the mask of word w;
// places start at base[list], counted over the CTAs before this one.  totals
// of the slice come back in base.
template <int kLists, class WordFn, class F>
__device__ __forceinline__ void emit(Ctl& c, int lo, int hi, int (&base)[kLists], WordFn&& word,
                                     F&& f) {
  const int words = (hi - lo + 31) / 32, lane = threadIdx.x & 31;
  for (int w0 = 0; w0 < words; w0 += kThreads) {
    // a batch's counts fit 16 bits each: one scan for both lists
    static_assert(kLists <= 2 && 32 * kThreads < (1 << 15), "packed counts");
    const int w = w0 + threadIdx.x;
    int n = 0, tot;
    if (w < words)
#pragma unroll
      for (int l = 0; l < kLists; ++l) n += __popc(word(l, w)) << (16 * l);
    const int ex = block_exclusive_scan(n, c.warp_sums, &tot);
#pragma unroll
    for (int l = 0; l < kLists; ++l) {
      c.offs[l][threadIdx.x] = base[l] + ((ex >> (16 * l)) & 0xFFFF);
      base[l] += (tot >> (16 * l)) & 0xFFFF;
    }
    __syncthreads();
    for (int k = threadIdx.x >> 5; k < kThreads && w0 + k < words; k += kThreads / 32)
#pragma unroll
      for (int l = 0; l < kLists; ++l) {
        const uint32_t m = word(l, w0 + k);
        if ((m >> lane) & 1u)
          f(l, lo + 32 * (w0 + k) + lane, c.offs[l][k] + __popc(m & ((1u << lane) - 1u)));
      }
    __syncthreads();
  }
}

// Slice of CTA `rank` of `size` over n indices, in multiples of 32.
__device__ __forceinline__ void slice(int n, unsigned rank, unsigned size, int* lo, int* hi) {
  const int per = (int)((((long long)n + size - 1) / size + 31) / 32 * 32);
  *lo = (int)min((long long)n, (long long)rank * per);
  *hi = (int)min((long long)n, (long long)*lo + per);
}
inline int slice_words(long long n, int size) {
  return (int)(((n + size - 1) / size + 31) / 32);
}

// CTAs a cluster takes for rows of up to n keys.  A cluster's barriers cost 2 to
// 3 us over a block's, so one CTA works alone up to 4,096 keys (one row of 1,024:
// 4.2 us alone, 6.6 by two; of 4,096: 7.7 and 9.7); past that as many as leave
// 2,048 keys each (16 rows of 16,384: 33.0, 14.9, 11.1 and 10.7 us by 1, 2, 4 and 8)
// while the clusters fill the device no more than twice (64 rows of 16,384: 14.1 us
// by 4, 22.8 by 8).
inline int cluster_size(long long n, int rows, int sms) {
  int size = 1;
  if (n <= 4096) return size;
  while (size < kMaxCluster && n > 2048ll * size && (long long)rows * size <= sms) size *= 2;
  return size;
}

}  // namespace topk
}  // namespace dcpmla
