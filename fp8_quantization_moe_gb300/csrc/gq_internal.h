// gq_internal.h -- host-side declarations shared by the translation units of
// libgqfp8 (not part of the public ABI).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "gq_fp8.h"

namespace gq {

// Per-device facts and handles, filled once per device.
struct DeviceInfo {
  int device = -1;
  int sm_count = 0;
  unsigned* err_word = nullptr;  // device address of the error word
  int colwise_ctas_per_sm = 0;
  int rowwise_ctas_per_sm = 0;
  int mx_ctas_per_sm = 0;
  int rows_ctas_per_sm = 0;
  int sort_cluster = 0;  // most blocks of the token sort
  int mm_pairs = 0;      // block pairs of a grouped product resident at once
  int mm_split[4] = {};  // its clusters of 1, 2, 4, 8 blocks that split a contraction
};

// Launch-time knobs (test hooks).
struct DebugKnobs {
  int skip_arrival = 0;
  int no_split = 0;  // rowwise_t: never split units across blocks
  uint64_t timeout_ns = 1000000000ull;
  int32_t lag[2] = {0, 0};  // per kind; 0 = automatic
};

// Encodes a 2-D tiled tensor map (row-major, dim0 innermost).
gq_status encode_tiled_2d(CUtensorMap* map, CUtensorMapDataType dtype,
                          void* base, uint64_t dim0, uint64_t dim1,
                          uint64_t row_stride_bytes, uint32_t box0,
                          uint32_t box1, CUtensorMapSwizzle swizzle);

// Encodes a 3-D tiled tensor map.
gq_status encode_tiled_3d(CUtensorMap* map, CUtensorMapDataType dtype,
                          void* base, uint64_t dim0, uint64_t dim1, uint64_t dim2,
                          uint64_t stride1_bytes, uint64_t stride2_bytes, uint32_t box0,
                          uint32_t box1, CUtensorMapSwizzle swizzle, uint32_t box2 = 1);

// Records a message for gq_last_error() and returns `st`.
gq_status fail(gq_status st, const char* fmt, ...);

// Returns GQ_ERR_CUDA with the runtime's message if `e` is an error.
gq_status check_cuda(cudaError_t e, const char* what);

// Launches a kernel that begins with grid_wait: it may be brought up while the
// kernel before it in the stream still runs, which hides the launch (a sort
// and the dispatch after it: 16,381 tokens, 33.6 -> 28.6 us in a stream).  `cluster` blocks
// form a cluster.
template <typename... P, typename... A>
gq_status launch_chained(const char* what, void (*kernel)(P...), dim3 grid, unsigned threads,
                         size_t smem, cudaStream_t stream, unsigned cluster, A... args) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  if (e != cudaSuccess) (void)cudaGetLastError();  // reported here, once
  return check_cuda(e, what);
}

// Colwise workspace layout: a 256-byte header (work counters), one counter
// per (group, 128-column slab) strip, then the (G, K) amax words.  Offsets
// in bytes; every region starts on a 256-byte boundary.  Every launch
// leaves all of it zero.
struct WorkspaceLayout {
  size_t counters = 0;  // start of the strip counters
  size_t amax = 0;      // start of the amax words
  size_t total = 0;
};
WorkspaceLayout colwise_workspace(int64_t K, int64_t G);

namespace colwise {
constexpr int kW = 128;  // columns per slab
gq_status setup(DeviceInfo& info);
// offs == nullptr: G groups of `uniform` rows each.
gq_status launch(const DeviceInfo& info, const DebugKnobs& dbg, const void* x,
                 int32_t M, int32_t K, const int32_t* offs, int32_t uniform, int32_t G,
                 void* out, float* scales, uint32_t flags, void* ws, cudaStream_t stream);
}  // namespace colwise

namespace rowwise {
constexpr int kTn = 64;  // rows of A per window: one row band
constexpr int kTm = 64;  // token columns per window
constexpr size_t kHeaderBytes = 256;  // unit counter, finished-blocks counter, padded
constexpr int kSplitWords = 68;        // per split unit: kTn amax words, a counter, padding
// Workspace of a call: the header, then kSplitWords words for every
// (row band, group) unit that may be split (groups of 4090 tokens or more).
size_t workspace_bytes(int64_t N, int64_t Mg, int64_t G);
gq_status setup(DeviceInfo& info);
gq_status launch(const DeviceInfo& info, const DebugKnobs& dbg, const void* a,
                 int32_t N, int32_t Mg, const int32_t* offs, int32_t G,
                 void* out_t, float* scales, uint32_t flags, void* ws, cudaStream_t stream);
}  // namespace rowwise

namespace mx {
gq_status setup(DeviceInfo& info);
gq_status launch(const DeviceInfo& info, const void* x, int64_t M, int64_t K, void* out,
                 uint8_t* scales, int mode, cudaStream_t stream);
}  // namespace mx

namespace rows {
gq_status setup(DeviceInfo& info);
gq_status launch(const DeviceInfo& info, const void* w, int64_t rows, int64_t K, void* out,
                 float* scales, bool pow2, cudaStream_t stream);
}  // namespace rows

namespace wgrad {
gq_status setup(DeviceInfo& info);
gq_status launch(const DeviceInfo& info, const DebugKnobs& dbg, const void* qa_t, const float* sa,
                 const void* qx, const float* sx, int32_t T, int32_t N, int32_t K,
                 const int32_t* offs, int32_t G, void* out, cudaStream_t stream);
}  // namespace wgrad

namespace block {
gq_status launch_rows(const void* x, bool f32, int64_t rows, int64_t K,
                      int64_t ld, const int32_t* pos, int32_t top_k, int64_t out_rows, void* out,
                      float* scales, bool pow2, cudaStream_t stream);
gq_status launch_tiles(const void* w, bool f32, int64_t E, int64_t N, int64_t K, void* out,
                       float* scales, bool pow2, cudaStream_t stream);
}  // namespace block

namespace moe {
gq_status setup(DeviceInfo& info);
gq_status launch_sort(const DeviceInfo& info, const void* ids, bool i64, int64_t tokens, int32_t top_k, int32_t experts,
                      int32_t* offs, int32_t* pos, int32_t* token, cudaStream_t stream);
gq_status launch_dispatch(const void* x, int64_t tokens, int64_t row_bytes, int64_t ld_bytes,
                          const int32_t* pos, int32_t top_k, int64_t out_rows, void* out,
                          cudaStream_t stream);
gq_status launch_combine(const void* y, bool f32, int64_t rows, int64_t H, const int32_t* pos,
                         const float* weights, int64_t tokens, int32_t top_k, void* out,
                         cudaStream_t stream);
gq_status launch_combine_backward(const void* g, const void* y, bool f32, int64_t rows, int64_t H,
                                  const int32_t* pos, const float* weights, int64_t tokens,
                                  int32_t top_k, void* dy, float* dweights, cudaStream_t stream);
}  // namespace moe

namespace gmm {
gq_status setup(DeviceInfo& info);
gq_status launch(const DeviceInfo& info, const DebugKnobs& dbg, const void* qa, const float* sa,
                 int64_t M, const void* qb, const float* sb, int32_t N, int32_t K, bool transposed,
                 const int32_t* offs, int32_t E, void* out, cudaStream_t stream);
gq_status launch_gated(const DeviceInfo& info, const DebugKnobs& dbg, const void* qa,
                       const float* sa, int64_t M, const void* qb, const float* sb, int32_t N,
                       int32_t K, int activation, const int32_t* offs, int32_t E, void* out,
                       void* q, float* scales, void* pre, bool pow2, cudaStream_t stream);
gq_status launch_gated_grad(const DeviceInfo& info, const DebugKnobs& dbg, const void* qd,
                            const float* sd, int64_t M, const void* qb, const float* sb, int32_t N,
                            int32_t K, const int32_t* offs, int32_t E, void* out,
                            cudaStream_t stream);
}  // namespace gmm

namespace gated {
gq_status launch_backward(const void* g, const void* pre, bool f32, int64_t rows, int64_t N,
                          int64_t ld, int activation, void* out, void* q, float* scales, bool pow2,
                          cudaStream_t stream);
}  // namespace gated

namespace clip {
size_t workspace_bytes(const int64_t* sizes, const int32_t* dtypes, int32_t count);
gq_status check_overlap(const void* const* in, void* const* out, const int64_t* sizes,
                        const int32_t* dtypes, int32_t count, const float* given,
                        const float* norm);
// The norm of the tensors, unless `given`, to `norm`, unless nullptr; with
// `write` the tensors scaled to `most`, into `out` or in place.
gq_status launch(const DeviceInfo& info, const void* const* in, void* const* out, bool write,
                 const int64_t* sizes, const int32_t* dtypes, int32_t count, float most,
                 const float* given, void* workspace, float* norm, cudaStream_t stream);
}  // namespace clip

// Writes the scale of an empty group -- 448 / 1e-12 (fp32), or its power
// of two below with GQ_SCALE_POW2 -- into n scales: every group is empty
// when the token extent is 0.
gq_status launch_fill_empty_scales(float* scales, int64_t n, uint32_t flags,
                                   cudaStream_t stream);

}  // namespace gq
