// The LSE-weighted merge of one (request, head) row, shared by the cross-shard
// DCP merges (stacked buffers or one pointer per shard) and the split-KV
// combine inside a shard.
//
// With M = max_i LSE_i and w_i = exp(LSE_i - M):
//   O = sum_i w_i O_i / sum_i w_i,   LSE = M + ln sum_i w_i,
// and pieces with LSE = -inf weigh exactly zero; if all are -inf the result
// is (0, -inf).  "GLM-5.2 vLLM Decode Context Parallelism", sections "See why
// vLLM 0.26.0 fails" (partials combined with the softmax normalisation via
// LSE) and "Separate the backend merge from stable" (the neutral (0, -inf)
// pair of an empty shard drops out of the merge).
#pragma once

#include <math_constants.h>

#include "common.cuh"

namespace dcpmla {

// Pieces laid out with a fixed stride: piece k of the row is entry
// first + k * stride of lse, with its 512 outputs at that entry of o.
struct StridedPieces {
  const float* __restrict__ o;
  const float* __restrict__ lse;
  size_t first, stride;
  __device__ __forceinline__ float lse_of(int k) const { return __ldg(lse + first + k * stride); }
  __device__ __forceinline__ const float4* row(int k) const {
    return reinterpret_cast<const float4*>(o + (first + k * stride) * kVDim);
  }
};

// One buffer per piece: piece k of the row is entry `entry` of lse[k], with
// its 512 outputs at that entry of o[k].  The pointer tables live in shared
// memory; the buffers may be another device's memory mapped into this one.
struct TablePieces {
  const float* const* o;
  const float* const* lse;
  size_t entry;
  __device__ __forceinline__ float lse_of(int k) const { return __ldg(lse[k] + entry); }
  __device__ __forceinline__ const float4* row(int k) const {
    return reinterpret_cast<const float4*>(o[k] + entry * kVDim);
  }
};

// One warp merges `count` pieces of one row into out_o (512 floats, 16-byte
// aligned) and *out_lse (if not null): all of it, or columns [128 part, 128
// part + 128) with kParts = 4 (part 0 writes the LSE).  The pieces are added in
// order whatever the batch, each lane working out the weights of its own pieces:
// this runs once from cold instruction caches, and its length is what it costs (one
// request's 64 heads and 32 pieces: 10.5 us with an expf per piece and lane, 6.6 so,
// by 8, 16 or 32 loads in flight; 42 us one piece after the other).  For whole rows
// the registers of four pieces cost more than they give (a dense step of 32 requests
// and 8 shards 195 us, one by one 191 us).
template <int kParts = 1, class Pieces>
__device__ __forceinline__ void merge_warp(const Pieces& pc, int count, float* __restrict__ out_o,
                                           float* __restrict__ out_lse, int part = 0) {
  constexpr int kVec = 4 / kParts;               // float4 per lane
  constexpr int kBatch = kParts == 1 ? 1 : 8;    // pieces with loads in flight
  const int lane = threadIdx.x & 31;
  const int col = part * 32 + lane;
  float M = -CUDART_INF_F;
  for (int k = lane; k < count; k += 32) M = fmaxf(M, pc.lse_of(k));
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, s));
  float4 acc[kVec];
#pragma unroll
  for (int i = 0; i < kVec; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  if (M == -CUDART_INF_F) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) reinterpret_cast<float4*>(out_o)[i * 32 + col] = acc[i];
    if (lane == 0 && out_lse && part == 0) *out_lse = -CUDART_INF_F;
    return;
  }
  float wsum = 0.f;
  for (int k0 = 0; k0 < count; k0 += 32) {
    const float mine = k0 + lane < count ? pc.lse_of(k0 + lane) : -CUDART_INF_F;
    const int n = min(32, count - k0);
    // a lane each: the piece's weight (0 past the end), and whether it has one
    const float weight = expf(mine - M);
    const unsigned live = __ballot_sync(0xffffffffu, mine != -CUDART_INF_F);
    for (int j0 = 0; j0 < n; j0 += kBatch) {
      float4 v[kBatch][kVec];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        if (!(live >> (j0 + j) & 1u)) continue;
        const float4* src = pc.row(k0 + j0 + j);
#pragma unroll
        for (int i = 0; i < kVec; ++i) v[j][i] = __ldg(src + i * 32 + col);
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        if (!(live >> (j0 + j) & 1u)) continue;
        const float w = __shfl_sync(0xffffffffu, weight, j0 + j);
        wsum += w;
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          acc[i].x = fmaf(w, v[j][i].x, acc[i].x);
          acc[i].y = fmaf(w, v[j][i].y, acc[i].y);
          acc[i].z = fmaf(w, v[j][i].z, acc[i].z);
          acc[i].w = fmaf(w, v[j][i].w, acc[i].w);
        }
      }
    }
  }
  const float inv = 1.f / wsum;
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    float4 v = acc[i];
    v.x *= inv; v.y *= inv; v.z *= inv; v.w *= inv;
    reinterpret_cast<float4*>(out_o)[i * 32 + col] = v;
  }
  if (lane == 0 && out_lse && part == 0) *out_lse = M + logf(wsum);
}

}  // namespace dcpmla
