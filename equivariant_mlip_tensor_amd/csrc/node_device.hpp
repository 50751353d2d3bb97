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

}  // namespace tpconv
