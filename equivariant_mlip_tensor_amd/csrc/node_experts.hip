// node_experts.hip -- the experts' equivariant maps on irreps rows and their
// gradients.
#include <hip/hip_runtime.h>

#include "node_internal.hpp"

namespace tpconv {
namespace {

int blocks_for(int64_t n, int block) {
  const int64_t g = (n + block - 1) / block;
  return static_cast<int>(g < 1 ? 1 : (g > 65536 ? 65536 : g));
}

struct MapArgs {
  int64_t n_rows, dim_in, dim_out, weight_numel;
  int32_t X, k;
  ExpertMap m;
};

template <class T>
__global__ void k_zero_columns(int64_t n_rows, int64_t dim, int32_t off, int32_t len, T* __restrict__ out) {
  const int64_t total = n_rows * len, step = int64_t(gridDim.x) * blockDim.x;
  for (int64_t q = blockIdx.x * int64_t(blockDim.x) + threadIdx.x; q < total; q += step)
    out[(q / len) * dim + off + q % len] = T(0);
}

// rows of out (ADJ: of grad_x) for one map, a thread per element
template <class T, bool ADJ>
__global__ void k_rows(MapArgs a, const T* __restrict__ x, const T* __restrict__ weights,
                       const int32_t* __restrict__ experts, const T* __restrict__ gates, T* __restrict__ out) {
  const int d = a.m.d, K = ADJ ? a.m.mul_out : a.m.mul_in, N = ADJ ? a.m.mul_in : a.m.mul_out;
  const int64_t ldx = ADJ ? a.dim_out : a.dim_in, ldo = ADJ ? a.dim_in : a.dim_out;
  const int xo = ADJ ? a.m.out_off : a.m.in_off, oo = ADJ ? a.m.in_off : a.m.out_off;
  const int64_t len = int64_t(N) * d, total = a.n_rows * len, step = int64_t(gridDim.x) * blockDim.x;
  for (int64_t q = blockIdx.x * int64_t(blockDim.x) + threadIdx.x; q < total; q += step) {
    const int64_t i = q / len;
    const int col = int(q - i * len), v = col / d, mm = col - v * d;
    T s = 0;
    for (int j = 0; j < a.k; ++j) {
      const int e = experts[i * a.k + j];
      if (e < 0 || e >= a.X) continue;
      const T* M = weights + e * a.weight_numel + a.m.woff;
      const T* xr = x + i * ldx + xo + mm;
      T t = 0;
      for (int u = 0; u < K; ++u) t += xr[u * d] * M[ADJ ? v * a.m.mul_out + u : u * a.m.mul_out + v];
      s += gates[i * a.k + j] * t;
    }
    out[i * ldo + oo + col] = s;
  }
}

// gradient of one map's weights, a thread per weight over all rows
template <class T>
__global__ void k_wgrad(MapArgs a, const T* __restrict__ x, const int32_t* __restrict__ experts,
                        const T* __restrict__ gates, const T* __restrict__ grad, T* __restrict__ out) {
  const int d = a.m.d;
  const int64_t per = int64_t(a.m.mul_in) * a.m.mul_out, total = a.X * per, step = int64_t(gridDim.x) * blockDim.x;
  for (int64_t q = blockIdx.x * int64_t(blockDim.x) + threadIdx.x; q < total; q += step) {
    const int e = int(q / per), r = int(q - e * per), u = r / a.m.mul_out, v = r - u * a.m.mul_out;
    T s = 0;
    for (int64_t i = 0; i < a.n_rows; ++i)
      for (int j = 0; j < a.k; ++j) {
        if (experts[i * a.k + j] != e) continue;
        const T* xr = x + i * a.dim_in + a.m.in_off + u * d;
        const T* gr = grad + i * a.dim_out + a.m.out_off + v * d;
        T t = 0;
        for (int m = 0; m < d; ++m) t += xr[m] * gr[m];
        s += gates[i * a.k + j] * t;
      }
    out[e * a.weight_numel + a.m.woff + r] = s;
  }
}

// gradient of the gates, a wavefront per entry; the maps after the first add
template <class T>
__global__ void k_ggrad(MapArgs a, bool add, const T* __restrict__ x, const T* __restrict__ weights,
                        const int32_t* __restrict__ experts, const T* __restrict__ grad, T* __restrict__ out) {
  const int lane = threadIdx.x & 63, d = a.m.d, V = a.m.mul_out;
  const int64_t total = a.n_rows * a.k, step = int64_t(gridDim.x) * (blockDim.x >> 6);
  for (int64_t q = blockIdx.x * int64_t(blockDim.x >> 6) + (threadIdx.x >> 6); q < total; q += step) {
    const int64_t i = q / a.k;
    const int e = experts[q];
    T s = 0;
    if (e >= 0 && e < a.X) {
      const T* M = weights + e * a.weight_numel + a.m.woff;
      const T* xr = x + i * a.dim_in + a.m.in_off;
      const T* gr = grad + i * a.dim_out + a.m.out_off;
      for (int v = lane; v < V; v += 64)
        for (int u = 0; u < a.m.mul_in; ++u) {
          T t = 0;
          for (int m = 0; m < d; ++m) t += xr[u * d + m] * gr[v * d + m];
          s += t * M[u * V + v];
        }
    }
    for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o, 64);
    if (lane == 0) out[q] = add ? out[q] + s : s;
  }
}

__global__ void k_load(int64_t total, int X, const int32_t* __restrict__ experts, int32_t* __restrict__ load) {
  const int e = blockIdx.x;
  int c = 0;
  for (int64_t q = threadIdx.x; q < total; q += blockDim.x) c += experts[q] == e;
  for (int o = 32; o > 0; o >>= 1) c += __shfl_xor(c, o, 64);
  if (threadIdx.x == 0) load[e] = c;
}

MapArgs args_of(const Experts& p, int64_t n_rows, const ExpertMap& m) {
  return MapArgs{n_rows, p.dim_in, p.dim_out, p.weight_numel, p.n_experts, p.top_k, m};
}

template <class T, bool ADJ>
void rows(const Experts& p, int64_t n, const T* x, const T* weights, const int32_t* experts, const T* gates, T* out,
          hipStream_t s) {
  for (const ColumnRun& r : ADJ ? p.bare_in : p.bare_out)
    hipLaunchKernelGGL(k_zero_columns<T>, dim3(blocks_for(n * r.len, 256)), dim3(256), 0, s, n,
                       ADJ ? p.dim_in : p.dim_out, r.off, r.len, out);
  for (const ExpertMap& m : p.maps)
    hipLaunchKernelGGL((k_rows<T, ADJ>), dim3(blocks_for(n * (ADJ ? m.mul_in : m.mul_out) * m.d, 256)), dim3(256), 0,
                       s, args_of(p, n, m), x, weights, experts, gates, out);
}

template <class T>
void backward(const Experts& p, int64_t n, const T* x, const T* weights, const int32_t* experts, const T* gates,
              const T* grad, T* gx, T* gw, T* gg, hipStream_t s) {
  if (gx != nullptr && n > 0) rows<T, true>(p, n, grad, weights, experts, gates, gx, s);
  for (size_t q = 0; q < p.maps.size(); ++q) {
    const MapArgs a = args_of(p, n, p.maps[q]);
    if (gw != nullptr)
      hipLaunchKernelGGL(k_wgrad<T>, dim3(blocks_for(int64_t(a.X) * a.m.mul_in * a.m.mul_out, 256)), dim3(256), 0, s,
                         a, x, experts, gates, grad, gw);
    if (gg != nullptr && n > 0)
      hipLaunchKernelGGL(k_ggrad<T>, dim3(blocks_for(n * a.k, 4)), dim3(256), 0, s, a, q > 0, x, weights, experts,
                         grad, gg);
  }
}

}  // namespace

size_t experts_layout_bytes(const Experts&, int64_t) { return 256; }
size_t experts_workspace(const Experts&, int64_t) { return 256; }

hipError_t launch_experts_layout(const Experts& p, int64_t n, const int32_t* experts, void*, int32_t* load,
                                 hipStream_t s) {
  if (load != nullptr)
    hipLaunchKernelGGL(k_load, dim3(p.n_experts), dim3(64), 0, s, n * p.top_k, p.n_experts, experts, load);
  return hipGetLastError();
}

hipError_t launch_experts_forward(const Experts& p, int64_t n, const void* x, const void* weights,
                                  const int32_t* experts, const void* gates, const void*, void* out, hipStream_t s) {
  if (p.f64)
    rows<double, false>(p, n, static_cast<const double*>(x), static_cast<const double*>(weights), experts,
                        static_cast<const double*>(gates), static_cast<double*>(out), s);
  else
    rows<float, false>(p, n, static_cast<const float*>(x), static_cast<const float*>(weights), experts,
                       static_cast<const float*>(gates), static_cast<float*>(out), s);
  return hipGetLastError();
}

hipError_t launch_experts_backward(const Experts& p, int64_t n, const void* x, const void* weights,
                                   const int32_t* experts, const void* gates, const void*, const void* grad_out,
                                   void* grad_x, void* grad_weights, void* grad_gates, void*, hipStream_t s) {
  if (p.f64)
    backward(p, n, static_cast<const double*>(x), static_cast<const double*>(weights), experts,
             static_cast<const double*>(gates), static_cast<const double*>(grad_out), static_cast<double*>(grad_x),
             static_cast<double*>(grad_weights), static_cast<double*>(grad_gates), s);
  else
    backward(p, n, static_cast<const float*>(x), static_cast<const float*>(weights), experts,
             static_cast<const float*>(gates), static_cast<const float*>(grad_out), static_cast<float*>(grad_x),
             static_cast<float*>(grad_weights), static_cast<float*>(grad_gates), s);
  return hipGetLastError();
}

}  // namespace tpconv
