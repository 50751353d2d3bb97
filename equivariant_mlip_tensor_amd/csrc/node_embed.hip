// node_embed.hip -- species embedding: out = scale * table[type], and the
// table's gradient.
#include <hip/hip_runtime.h>

#include "node_internal.hpp"

namespace tpconv {
namespace {

int blocks_for(int64_t n, int block) {
  const int64_t g = (n + block - 1) / block;
  return static_cast<int>(g < 1 ? 1 : (g > 65536 ? 65536 : g));
}

template <class T>
__global__ void k_embed(EmbedArgs a, const T* __restrict__ table, T* __restrict__ out) {
  const T scale = static_cast<T>(a.scale);
  const int64_t total = a.n_rows * a.dim, step = int64_t(gridDim.x) * blockDim.x;
  for (int64_t q = blockIdx.x * int64_t(blockDim.x) + threadIdx.x; q < total; q += step) {
    const int64_t i = q / a.dim, c = q - i * a.dim;
    const int64_t t = a.types[i];
    out[i * a.stride + c] = t >= 0 && t < a.n_types ? scale * table[t * a.dim + c] : T(0);
  }
}

// One block per type walks all rows in order, a thread per column.
template <class T>
__global__ void k_embed_grad(EmbedArgs a, const T* __restrict__ grad, T* __restrict__ grad_table) {
  for (int64_t t = blockIdx.x; t < a.n_types; t += gridDim.x)
    for (int64_t c = threadIdx.x; c < a.dim; c += blockDim.x) {
      T s = 0;
      for (int64_t i = 0; i < a.n_rows; ++i)
        if (a.types[i] == t) s += grad[i * a.stride + c];
      grad_table[t * a.dim + c] = static_cast<T>(a.scale) * s;
    }
}

}  // namespace

size_t embed_workspace(bool, int64_t, int64_t, int64_t) { return 256; }

hipError_t launch_embed_forward(bool f64, const EmbedArgs& a, const void* table, void* out, hipStream_t s) {
  const dim3 grid(blocks_for(a.n_rows * a.dim, 256));
  if (f64)
    hipLaunchKernelGGL(k_embed<double>, grid, dim3(256), 0, s, a, static_cast<const double*>(table),
                       static_cast<double*>(out));
  else
    hipLaunchKernelGGL(k_embed<float>, grid, dim3(256), 0, s, a, static_cast<const float*>(table),
                       static_cast<float*>(out));
  return hipGetLastError();
}

hipError_t launch_embed_backward(bool f64, const EmbedArgs& a, const void* grad, void* grad_table, void*,
                                 hipStream_t s) {
  const dim3 grid(blocks_for(a.n_types, 1));
  if (f64)
    hipLaunchKernelGGL(k_embed_grad<double>, grid, dim3(256), 0, s, a, static_cast<const double*>(grad),
                       static_cast<double*>(grad_table));
  else
    hipLaunchKernelGGL(k_embed_grad<float>, grid, dim3(256), 0, s, a, static_cast<const float*>(grad),
                       static_cast<float*>(grad_table));
  return hipGetLastError();
}

}  // namespace tpconv
