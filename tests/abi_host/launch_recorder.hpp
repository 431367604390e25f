// Stand-in for the part of the HIP runtime that host code of a .hip file calls to launch
// kernels: every launch and every attribute set is recorded, nothing runs.  For host-only
// builds (hipcc --offload-host-only) linked without the runtime.
#pragma once

#include <hip/hip_runtime_api.h>

#include <map>
#include <string>
#include <vector>

struct Launch {
  std::string kernel;
  dim3 grid, block;
  size_t lds;
  size_t lds_bound;  // as set by hipFuncSetAttribute before; 0: not set
};
inline std::vector<Launch> launches;
inline std::vector<std::pair<std::string, int>> bounds_set;  // kernel, bytes, in order
inline std::map<const void*, std::string> kernel_names;
inline std::map<const void*, int> lds_bounds;
inline int fail_launch = -1;  // the launch that is rejected; -1: none

namespace recorder {
inline dim3 grid, block;
inline size_t lds;
inline hipStream_t stream;
inline hipError_t error = hipSuccess;
}  // namespace recorder

extern "C" {
void** __hipRegisterFatBinary(const void*) {
  static void* handle;
  return &handle;
}
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterFunction(void**, const void* host, char*, const char* name, unsigned, void*, void*, void*, void*, int*) {
  kernel_names[host] = name;
}
hipError_t __hipPushCallConfiguration(dim3 g, dim3 b, size_t lds, hipStream_t s) {
  recorder::grid = g, recorder::block = b, recorder::lds = lds, recorder::stream = s;
  return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3* g, dim3* b, size_t* lds, hipStream_t* s) {
  *g = recorder::grid, *b = recorder::block, *lds = recorder::lds, *s = recorder::stream;
  return hipSuccess;
}
hipError_t hipLaunchKernel(const void* f, dim3 g, dim3 b, void**, size_t lds, hipStream_t) {
  if ((int)launches.size() == fail_launch) return recorder::error = hipErrorLaunchFailure;
  Launch l = {kernel_names.count(f) ? kernel_names[f] : "?", g, b, lds, lds_bounds.count(f) ? (size_t)lds_bounds[f] : 0};
  launches.push_back(l);
  return hipSuccess;
}
hipError_t hipFuncSetAttribute(const void* f, hipFuncAttribute, int bytes) {
  lds_bounds[f] = bytes;
  bounds_set.emplace_back(kernel_names.count(f) ? kernel_names[f] : "?", bytes);
  return hipSuccess;
}
hipError_t hipGetLastError() {
  const hipError_t e = recorder::error;
  recorder::error = hipSuccess;
  return e;
}
}
