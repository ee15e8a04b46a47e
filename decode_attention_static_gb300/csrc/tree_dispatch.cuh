// Launch of one instance of the tree attention (one translation unit for each query type).
#pragma once

#include <atomic>

#include "tree_attn.cuh"

namespace da {

template <typename T, int D, bool EIGHT>
cudaError_t launch_tree_instance(const TreeLaunch& l, int ctas, const TreeSpace& space, cudaStream_t stream) {
  using Shape = TreeShape<D, EIGHT>;
  auto* fn = tree_kernel<T, D, EIGHT>;
  static std::atomic<bool> ready[64];  // per device: the shared-memory opt-in is applied
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  if (device < 0 || device >= 64) return cudaErrorInvalidDevice;
  if (!ready[device].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape::kSmem);
    if (e != cudaSuccess) return e;
    ready[device].store(true, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(Shape::kThreads);
  cfg.dynamicSmemBytes = Shape::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, l, space.arrived, space.meets, space.partials);
}

template <typename T>
cudaError_t launch_tree_as(const TreeLaunch& l, int head_dim, bool e4m3, int ctas, const TreeSpace& space,
                           cudaStream_t stream) {
  if (head_dim == 128)
    return e4m3 ? launch_tree_instance<T, 128, true>(l, ctas, space, stream)
                : launch_tree_instance<T, 128, false>(l, ctas, space, stream);
  return e4m3 ? launch_tree_instance<T, 64, true>(l, ctas, space, stream)
              : launch_tree_instance<T, 64, false>(l, ctas, space, stream);
}

}  // namespace da
