// vsa_launch.h -- what the serving calls' host sides share: ranges that must not meet, and
// launches that may start up while their predecessor ends.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "vsa_host.h"

namespace vsa {

// Byte ranges of a call's buffers: an output may overlap nothing else.
struct Range {
  const void* p;
  size_t n;
};
inline bool meets(const Range& x, const Range& y) {
  if (!x.p || !y.p || !x.n || !y.n) return false;
  const uintptr_t a = reinterpret_cast<uintptr_t>(x.p), b = reinterpret_cast<uintptr_t>(y.p);
  return a < b + y.n && b < a + x.n;
}
template <int NO, int NI>
bool outputs_clear(const Range (&out)[NO], const Range (&in)[NI]) {
  for (int o = 0; o < NO; ++o) {
    for (int i = 0; i < NI; ++i)
      if (meets(out[o], in[i])) return false;
    for (int p = o + 1; p < NO; ++p)
      if (meets(out[o], out[p])) return false;
  }
  return true;
}

// One launch; the kernel may start up while its predecessor in the stream ends (each begins
// with after_predecessor()).  `cluster` CTAs form a cluster.
template <typename... P, typename... A>
vsa_status launch(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s,
                  int cluster, A... args) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 0 ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, kern, P(args)...) != cudaSuccess) {
    cudaGetLastError();
    return VSA_ERR_CUDA;
  }
  host_set_launches(1);
  return VSA_OK;
}

}  // namespace vsa
