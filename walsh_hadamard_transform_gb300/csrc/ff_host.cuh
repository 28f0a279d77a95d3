// Host helpers of the feed-forward launchers: tensor maps and per-device set-up.
#pragma once

#include <atomic>
#include <cstdint>

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include "feed_forward.cuh"

namespace fwt {

// The driver's tensor-map encoder, resolved once at run time (nullptr if absent).
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();
// Whether kernels are launched with programmatic stream serialisation (fwt_set_pdl).
int pdl_mode();
// A line of the plan log (FWT_LOG), and the events of fwt_trace_events around a launch.
void log_kernel(const char* format, ...) __attribute__((format(printf, 1, 2)));
cudaError_t trace_begin(cudaStream_t stream, bool& traced);
cudaError_t trace_end(cudaStream_t stream);

namespace ff {

// rows x cols, 128-byte boxes of `box_rows` rows with 128-byte swizzle; zero outside.
inline bool swizzled_map(CUtensorMap* out, const void* p, int bytes, CUtensorMapDataType type,
                         int64_t rows, int64_t cols, int64_t ld, int box_rows) {
  const PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
  if (!encode) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)(ld * bytes)};
  const cuuint32_t box[2] = {(cuuint32_t)(128 / bytes), (cuuint32_t)box_rows};
  const cuuint32_t steps[2] = {1, 1};
  return encode(out, type, 2, const_cast<void*>(p), dims, strides, box, steps,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Multiprocessors of the current device, asked once for each device; at least two, as many as a pair
// of CTAs takes (also where no device answers: the launch then says so).
inline int multiprocessors() {
  static std::atomic<int> known[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 2;
  int n = dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
  if (!n) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 2) return 2;
    if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

// Launches `kernel` in clusters of `cluster` CTAs.  On grids of up to 2048 CTAs it may be
// scheduled while the previous kernel on the stream finishes: every kernel launched here
// waits for that one (pdl_begin) before it touches global memory.
template <typename... KArgs, typename... Args>
cudaError_t launch_overlapped(void (*kernel)(KArgs...), unsigned grid, unsigned threads, size_t smem,
                              unsigned cluster, cudaStream_t st, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  cfg.attrs = attr;
  if (cluster > 1) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim.x = cluster;
    attr[cfg.numAttrs].val.clusterDim.y = attr[cfg.numAttrs].val.clusterDim.z = 1;
    ++cfg.numAttrs;
  }
  if (pdl_mode() && grid <= 2048) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
    ++cfg.numAttrs;
  }
  bool traced;
  cudaError_t err = trace_begin(st, traced);
  if (err == cudaSuccess) err = cudaLaunchKernelEx(&cfg, kernel, args...);
  return err == cudaSuccess && traced ? trace_end(st) : err;
}

// The same for kernels with dynamic shared memory, whose limit the first launch on each
// device raises.
template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kernel)(KArgs...), std::atomic<uint64_t>& ready, unsigned grid,
                           unsigned threads, size_t smem, unsigned cluster, cudaStream_t st,
                           const Args&... args) {
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  const uint64_t bit = dev < 64 ? uint64_t{1} << dev : 0;
  if (!(ready.load(std::memory_order_acquire) & bit) || !bit) {
    err = cudaFuncSetAttribute((const void*)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               (int)smem);
    if (err != cudaSuccess) return err;
    ready.fetch_or(bit, std::memory_order_release);
  }
  return launch_overlapped(kernel, grid, threads, smem, cluster, st, args...);
}

}  // namespace ff
}  // namespace fwt
