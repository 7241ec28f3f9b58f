// A kernel that lets its dependents be launched at once and writes their inputs
// late: what a caller's own kernel in front of a decode may do.  Compiled by
// test_gpu_late_inputs.py.
#include <cuda_runtime.h>

struct Copies {
  const int* src[4];
  int* dst[4];
  int words[4];
};

__global__ void late_writer(Copies c, long long cycles) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const long long start = clock64();
  for (int i = 0; i < 1000000 && clock64() - start < cycles; ++i) {
  }
  for (int k = 0; k < 4; ++k)
    for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < c.words[k]; i += gridDim.x * blockDim.x)
      c.dst[k][i] = c.src[k][i];
}

// Copies `words` 32-bit words each from src to dst, `cycles` after its start.
extern "C" int late_write(const int* const* src, int* const* dst, const int* words, long long cycles, void* stream) {
  Copies c;
  for (int k = 0; k < 4; ++k) {
    c.src[k] = src[k];
    c.dst[k] = dst[k];
    c.words[k] = words[k];
  }
  late_writer<<<4, 256, 0, static_cast<cudaStream_t>(stream)>>>(c, cycles);
  return static_cast<int>(cudaGetLastError());
}
