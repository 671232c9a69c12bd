// Internal launch entry points shared between the kernel files and the C ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "common.cuh"

namespace dcpmla {

// Launch with an optional cluster size (0: none) along x; `dependent`: the kernel
// may start before the stream's previous one is complete and waits for it itself
// (griddepcontrol).
template <class... KArgs, class... Args>
cudaError_t launch_kernel(void (*kernel)(KArgs...), dim3 grid, int threads, size_t smem,
                          cudaStream_t st, int cluster, bool dependent, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  int n = 0;
  if (cluster > 0) {
    at[n].id = cudaLaunchAttributeClusterDimension;
    at[n].val.clusterDim.x = cluster;
    at[n].val.clusterDim.y = 1;
    at[n].val.clusterDim.z = 1;
    ++n;
  }
  if (dependent) {
    at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cfg.attrs = at;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// cuTensorMapEncodeTiled of the driver, nullptr if it has none.
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn tensor_map_encoder();

cudaError_t launch_partial_simt(const PartialParams& p, int kv_dtype, cudaStream_t st);
cudaError_t launch_partial_tc(const PartialParams& p, int kv_dtype, cudaStream_t st);
bool tc_supports(const PartialParams& p, int kv_dtype);
cudaError_t launch_partial_f8(const PartialParams& p, cudaStream_t st);
bool f8_supports(const PartialParams& p, int kv_dtype);
cudaError_t launch_partial_bf16(const PartialParams& p, cudaStream_t st);   // chosen blocks
bool bf16_supports(const PartialParams& p, int kv_dtype);
cudaError_t launch_split_combine(const PartialParams& p, cudaStream_t st);
cudaError_t launch_dcp_merge(const float* partials, const float* lses, int num_shards, int batch,
                             int heads, float* out, float* out_lse, cudaStream_t st);
// mla_decode_partial over `rows` requests of one shard, each its own table of
// chosen blocks, with P rounded (PartialParams::round_p): the few thousand rows
// of a choice average less of P's rounding away than a long dense context.
int decode_chosen_blocks(const void* q, const void* kv_cache, int kv_dtype, int64_t num_blocks,
                         const int32_t* table, int stride, const int32_t* lens, int rows,
                         int num_heads, float softmax_scale, float* out, float* out_lse,
                         void* workspace, size_t workspace_bytes, int num_splits, int impl,
                         void* stream);
// Where that call, on this workspace, keeps the e4m3 kernel's Q images: written
// by the caller before it if `q_image_ready` is passed on; nullptr if the call
// will not run that kernel.
uint8_t* decode_chosen_q_image(int kv_dtype, int rows, int num_heads, int num_splits, int impl,
                               void* workspace);
int simt_sparse_chunk_max();
cudaError_t launch_sparse_gather(const PartialParams& p, int row_bytes, int maxblk,
                                 uint8_t* gathered, int* counts, cudaStream_t st);
cudaError_t launch_sparse_rows(const PartialParams& p, int maxblk, int* rows, int* counts,
                               uint8_t* q_image, cudaStream_t st);

}  // namespace dcpmla
