// internal.h -- what the library's translation units share beside the C ABI:
// error text, launch counting, device properties, the driver's tensor-map
// encoder and the launch switches.  Defined in conv3d_api.cu.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "conv3d.h"

namespace conv3d_internal {

// Properties of the current device; CONV3D_ERR_UNSUPPORTED unless it is sm_100.
struct Device {
  int num_sms;
  int max_smem_optin;
  int* status;      // device status word (conv3d_poll_status)
};
conv3d_status_t current_device(Device& out);

// Sets the text that conv3d_last_error returns on this thread.
void set_error(const char* fmt, ...);
conv3d_status_t cuda_fail(cudaError_t e, const char* what);

// The status of the launch just enqueued, which it also counts.
cudaError_t launched();

// cuTensorMapEncodeTiled of a row-major [rows][cols] matrix with `pitch_bytes`
// between rows, in boxes of box_rows x box_cols elements.
conv3d_status_t encode_matrix(CUtensorMap& map, CUtensorMapDataType type, const void* base,
                              unsigned long long cols, unsigned long long rows,
                              unsigned long long pitch_bytes, unsigned box_cols, unsigned box_rows,
                              CUtensorMapSwizzle swizzle, const char* what);

bool pdl_enabled();     // programmatic dependent launches (CONV3D_PDL=0 turns them off)
bool plan_log();        // CONV3D_LOG=1
bool take_stall(unsigned long long& timeout_ns);   // failure-detection test hook
unsigned long long wait_limit_ns();                // limit of every device-side wait

inline bool aligned(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Whether [a, a + na) and [b, b + nb) share a byte (false for a null pointer).
inline bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  if (a == nullptr || b == nullptr || na == 0 || nb == 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a0 < b0 + nb && b0 < a0 + na;
}

// Bytes of an 8-bit checkpoint's codes and exponent bytes for [rows, C].
inline size_t act8_code_bytes(long long rows, int C) {
  return static_cast<size_t>(rows) * ((C + 31) / 32) * 32;
}
inline size_t act8_scale_bytes(long long rows, int C) {
  return static_cast<size_t>(rows) * ((C + 31) / 32);
}

// Launches `kern` with an optional cluster width, as a programmatic dependent
// of the kernel before it on the stream where that is enabled (the kernel
// waits for it, griddepcontrol.wait, before it touches global memory).
template <typename... KArgs, typename... Args>
cudaError_t launch(void (*kern)(KArgs...), unsigned blocks, unsigned threads, size_t smem,
                   unsigned cluster, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  unsigned n = 0;
  cfg.gridDim = dim3(blocks, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  if (cluster > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = cluster;
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    ++n;
  }
  if (pdl_enabled()) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
  if (e != cudaSuccess) return e;
  return launched();
}

}  // namespace conv3d_internal
