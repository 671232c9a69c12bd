// Selection of the `want` largest of n 32-bit keys by one thread-block
// cluster, ties to the lowest index.
//
// The CTAs of the cluster own consecutive slices of the index range.  A radix
// descent of 8 bits a pass finds the key T of the last one taken: every CTA
// counts its slice's digits among the keys that match the prefix so far, the
// histograms are summed over distributed shared memory, and the digit in
// which the want-th key falls extends the prefix.  The keys above T are taken
// and, of those equal to T, the first `ties`.  The result is a bit per index
// in the owning CTA's shared memory, independent of the cluster's size.
#pragma once

#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace dcpmla {
namespace topk {

namespace cg = cooperative_groups;

constexpr int kThreads = 1024;
constexpr int kBins = 256;

struct Ctl {
  uint32_t hist[2][kBins];    // this CTA's digit counts, by pass parity
  uint32_t total[kBins];      // the cluster's
  int warp_sums[kThreads / 32];
  int digit, above;           // chosen digit and the keys above it
  int share[2];               // what the other CTAs of the cluster read of this one
};

// fp32 -> a key in the same order; NaN below everything.
__device__ __forceinline__ uint32_t key_of(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);    // -0 equals 0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// The value of a key that is not NaN's.
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? key & 0x7FFFFFFFu : ~key);
}

// Sum of `share[which]` over the CTAs before this one (call between cluster
// barriers that order the writes and the next reuse).
__device__ __forceinline__ int before(cg::cluster_group& cl, Ctl& c, int which) {
  int s = 0;
  for (unsigned r = 0; r < cl.block_rank(); ++r) s += cl.map_shared_rank(c.share, r)[which];
  return s;
}

// Marks the taken indices of this CTA's slice [lo, hi) in `bits` (bit i - lo;
// room for ceil((hi - lo) / 32) words).  key(i) is called for indices of the
// slice, several times.  All threads of all CTAs of the cluster call it with
// the same n and 1 <= want <= n.
template <class KeyFn>
__device__ void mark(cg::cluster_group& cl, Ctl& c, int lo, int hi, int want, uint32_t* bits,
                     KeyFn&& key) {
  const int tid = threadIdx.x;
  uint32_t prefix = 0, mask = 0;
  int left = want, eq_here = 0;
  for (int pass = 0; pass < 4; ++pass) {
    const int shift = 24 - 8 * pass;
    uint32_t* h = c.hist[pass & 1];
    if (tid < kBins) h[tid] = 0;
    __syncthreads();
    for (int i = lo + tid; i < hi; i += kThreads) {
      const uint32_t k = key(i);
      if ((k & mask) == prefix) atomicAdd(&h[(k >> shift) & 255u], 1u);
    }
    cl.sync();
    int v = 0;
    if (tid < kBins) {
      // bin 255 - tid, so that a running sum goes from the largest digit down
      for (unsigned r = 0; r < cl.num_blocks(); ++r)
        v += (int)cl.map_shared_rank(h, r)[kBins - 1 - tid];
    }
    int tot;
    const int ex = block_exclusive_scan(v, c.warp_sums, &tot);
    if (tid < kBins && ex < left && left <= ex + v) {
      c.digit = kBins - 1 - tid;
      c.above = ex;
    }
    __syncthreads();
    left -= c.above;
    prefix |= (uint32_t)c.digit << shift;
    mask |= 255u << shift;
    eq_here = (int)h[c.digit];
  }
  // the last pass's histogram counts the keys equal to T
  if (tid == 0) c.share[0] = eq_here;
  cl.sync();
  int seen = before(cl, c, 0);
  for (int base = lo; base < hi; base += kThreads) {
    const int i = base + tid;
    const uint32_t k = i < hi ? key(i) : 0u;
    const bool eq = i < hi && k == prefix;
    int tot;
    const int rank = seen + block_exclusive_scan(eq ? 1 : 0, c.warp_sums, &tot);
    seen += tot;
    const bool take = i < hi && (k > prefix || (eq && rank < left));
    const uint32_t word = __ballot_sync(0xffffffffu, take);
    if ((tid & 31) == 0 && i < hi) bits[(i - lo) >> 5] = word;
  }
  cl.sync();      // `bits` complete; share may be written again
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

// Launches `kernel` with `rows` clusters of `size` CTAs (grid x = cluster rank).
template <class... Args>
cudaError_t launch(void (*kernel)(Args...), int rows, int size, size_t smem, cudaStream_t st,
                   Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(size, rows);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = size;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace topk
}  // namespace dcpmla
