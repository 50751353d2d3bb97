// node_device.hpp -- device functions that several of node_*.hip use.
#pragma once

#include <hip/hip_runtime.h>

namespace tpconv {

template <class T>
struct alignas(16) Pack {  // one 16-byte piece
  T v[16 / sizeof(T)];
};

// Orders a wavefront's own LDS accesses: what its lanes wrote before is seen by
// all of them after, and what they read before is read before it is written
// again.  No instruction comes of it (a wavefront's LDS operations run in
// order); it binds the compiler.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

// ------------------------------------------------------------ matrix cores
// D[i][j] += sum_k A[i][k] B[k][j], 16 x 16 x 4: lane holds A[lane % 16]
// [lane / 16], B[lane / 16][lane % 16] and the four D[row(lane / 16, r)][lane % 16].
template <class T>
struct Mfma;
template <>
struct Mfma<float> {
  typedef float Acc __attribute__((ext_vector_type(4)));
  static __device__ __forceinline__ Acc step(float a, float b, Acc c) {
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ int row(int g, int r) { return 4 * g + r; }
};
template <>
struct Mfma<double> {
  typedef double Acc __attribute__((ext_vector_type(4)));
  static __device__ __forceinline__ Acc step(double a, double b, Acc c) {
    return __builtin_amdgcn_mfma_f64_16x16x4f64(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ int row(int g, int r) { return 4 * r + g; }
};

}  // namespace tpconv
