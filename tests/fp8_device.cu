// Device helpers of the 8-bit operators' tests: the library's own silu on an array, and a kernel that lets its dependents start
// at once and then runs on.
#include "fp8.cuh"

__global__ void silu_kernel(const float* a, float* y, int n) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i < n) y[i] = awq::fp8_silu(a[i]);
}

extern "C" int silu_of(const float* a, float* y, int n, void* stream) {
  silu_kernel<<<(n + 255) / 256, 256, 0, static_cast<cudaStream_t>(stream)>>>(a, y, n);
  return (int)cudaGetLastError();
}

// Lets the next kernel start, then sleeps until `ns` have passed (at most 10^7 sleeps of up to 2 us).
__global__ void early_kernel(unsigned long long ns) {
  awq::pdl_launch_dependents();
  const unsigned long long t0 = awq::globaltimer_ns();
  for (int i = 0; i < 10000000 && awq::globaltimer_ns() - t0 < ns; ++i) __nanosleep(1000);
}

extern "C" int signal_then_run(unsigned long long ns, void* stream) {
  early_kernel<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>(ns);
  return (int)cudaGetLastError();
}
