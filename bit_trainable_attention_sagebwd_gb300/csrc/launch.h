// Host-side kernel launch with programmatic stream serialization: the kernel may begin
// while its predecessor on the stream drains, and waits for it with griddepcontrol.wait
// (pdl_wait) before it reads or writes anything the predecessor touches.  One exception: packed_dq, which reads nothing of
// packed_dkv and takes from it the word that packed_pre is complete (pdl_wait_unless).
#pragma once

#include <cuda_runtime.h>

#include <utility>

namespace sage {

template <class... KArgs, class... Args>
inline cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                              Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

}  // namespace sage
