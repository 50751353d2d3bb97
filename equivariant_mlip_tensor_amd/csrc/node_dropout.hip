// node_dropout.hip -- dropout on irreps rows from a counter-based generator.
#include <hip/hip_runtime.h>

#include "node_internal.hpp"

namespace tpconv {
namespace {

// Philox4x32-10 (Salmon et al., "Parallel random numbers: as easy as 1, 2, 3",
// 2011): ten rounds of two 32x32->64 bit products, the key stepped by Weyl
// constants.  Word w of the block with counter (block, offset).
struct Words {
  uint32_t w[4];
};

__device__ __forceinline__ Words philox(uint64_t block, uint64_t offset, uint64_t seed) {
  uint32_t c0 = uint32_t(block), c1 = uint32_t(block >> 32), c2 = uint32_t(offset), c3 = uint32_t(offset >> 32);
  uint32_t k0 = uint32_t(seed), k1 = uint32_t(seed >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = uint64_t(c0) * 0xD2511F53u, b = uint64_t(c2) * 0xCD9E8D57u;
    c0 = uint32_t(b >> 32) ^ c1 ^ k0;
    c1 = uint32_t(b);
    c2 = uint32_t(a >> 32) ^ c3 ^ k1;
    c3 = uint32_t(a);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return Words{{c0, c1, c2, c3}};
}

// One thread per element.
template <class T>
__global__ void k_dropout(DropArgs a, const T* x, const T* residual, T* out) {
  const T scale = static_cast<T>(a.scale);
  const int64_t total = a.n_rows * a.dim, step = int64_t(gridDim.x) * blockDim.x;
  for (int64_t q = blockIdx.x * int64_t(blockDim.x) + threadIdx.x; q < total; q += step) {
    const int64_t i = q / a.dim;
    const int32_t col = static_cast<int32_t>(q - i * a.dim);
    int s = 0;
    while (col >= a.seg[s].end) ++s;
    const int64_t ch = i * a.channels + a.seg[s].channel + (col - a.seg[s].off) / a.seg[s].d;
    const Words w = philox(uint64_t(ch) >> 2, a.offset, a.seed);
    const T base = residual != nullptr ? residual[q] : T(0);
    out[q] = w.w[ch & 3] >= a.threshold ? base + scale * x[q] : base;
  }
}

}  // namespace

hipError_t launch_dropout(bool f64, const DropArgs& a, const void* x, const void* residual, void* out,
                          hipStream_t s) {
  const int64_t g = (a.n_rows * a.dim + 255) / 256;
  const dim3 grid(static_cast<unsigned>(g > 65536 ? 65536 : g));
  if (f64)
    hipLaunchKernelGGL(k_dropout<double>, grid, dim3(256), 0, s, a, static_cast<const double*>(x),
                       static_cast<const double*>(residual), static_cast<double*>(out));
  else
    hipLaunchKernelGGL(k_dropout<float>, grid, dim3(256), 0, s, a, static_cast<const float*>(x),
                       static_cast<const float*>(residual), static_cast<float*>(out));
  return hipGetLastError();
}

}  // namespace tpconv
