// Device helpers of the 8-bit operators' tests: the library's own silu on an array.
#include "fp8.cuh"

__global__ void silu_kernel(const float* a, float* y, int n) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i < n) y[i] = awq::fp8_silu(a[i]);
}

extern "C" int silu_of(const float* a, float* y, int n, void* stream) {
  silu_kernel<<<(n + 255) / 256, 256, 0, static_cast<cudaStream_t>(stream)>>>(a, y, n);
  return (int)cudaGetLastError();
}
