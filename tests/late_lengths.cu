// Test helper: a kernel that lets the next one start and writes lengths late.
// Every CTA first reads the lengths as they are, as kernels of an earlier step
// would have; the last one then writes the new ones after a bounded delay.
#include <cuda_runtime.h>
#include <stdint.h>

__global__ void late_kernel(int32_t* kv_len, const int32_t* next, int n, int32_t* seen, unsigned long long ns) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int32_t sum = 0;
  for (int i = threadIdx.x; i < n; i += blockDim.x) sum += kv_len[i];
  if (sum == INT32_MIN) *seen = sum;  // (keeps the reads)
  if (blockIdx.x + 1 < gridDim.x) return;
  unsigned long long begin, now;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(begin));
  for (int turn = 0; turn < 1000000; ++turn) {
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(now));
    if (now - begin >= ns) break;
    __nanosleep(200);
  }
  for (int i = threadIdx.x; i < n; i += blockDim.x) kv_len[i] = next[i];
}

extern "C" int late_lengths(int32_t* kv_len, const int32_t* next, int n, int32_t* seen, unsigned long long ns,
                            void* stream) {
  late_kernel<<<16, 128, 0, static_cast<cudaStream_t>(stream)>>>(kv_len, next, n, seen, ns);
  return (int)cudaGetLastError();
}
