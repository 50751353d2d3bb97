// node_route.hip -- routing of rows to experts: scores, groups, top_k, gates,
// and the gradient of the gates with respect to the logits.
#include <hip/hip_runtime.h>

#include "node_internal.hpp"

namespace tpconv {
namespace {

template <class T>
__device__ __forceinline__ T inf() {
  return static_cast<T>(__builtin_huge_val());
}

// log sigmoid(z), without overflow at either end
template <class T>
__device__ __forceinline__ T log_sigmoid(T z) {
  return (z < T(0) ? z : T(0)) - log1p(exp(z < T(0) ? z : -z));
}

template <class T>
__device__ __forceinline__ T sigmoid(T z) {
  const T e = exp(z < T(0) ? z : -z);
  return (z < T(0) ? e : T(1)) / (T(1) + e);
}

// maximum and sum of exponentials of a row's softmax (masked entries add nothing; 0 for a row all masked)
template <class T>
__device__ __forceinline__ void softmax_stats(const T* z, int X, T& top, T& sum) {
  top = -inf<T>();
  for (int e = 0; e < X; ++e) top = z[e] > top ? z[e] : top;
  sum = 0;
  for (int e = 0; e < X; ++e)
    if (!(z[e] == -inf<T>())) sum += exp(z[e] - top);
}

template <class T>
__device__ __forceinline__ T key_of(const RouteArgs& a, const T* z, const T* bias, int e, T top, T sum) {
  if (z[e] == -inf<T>()) return -inf<T>();
  T s = a.sigmoid ? sigmoid(z[e]) : exp(z[e] - top) / sum;
  if (bias != nullptr) s += bias[e];
  const T lowest = sizeof(T) == 4 ? T(-3.402823466e38f) : T(-1.7976931348623157e308);
  return s >= lowest ? s : lowest;  // NaN (and -inf from the bias) last of the unmasked
}

// One thread per row, the keys recomputed as they are needed.
template <class T>
__global__ void k_route(RouteArgs a, const T* __restrict__ logits, const T* __restrict__ bias,
                        int32_t* __restrict__ experts, T* __restrict__ gates) {
  const int64_t i = blockIdx.x * int64_t(blockDim.x) + threadIdx.x;
  if (i >= a.n_rows) return;
  const T* z = logits + i * a.X;
  T top = 0, sum = 1;
  if (!a.sigmoid) softmax_stats(z, a.X, top, sum);
  const int per = a.X / a.groups;
  uint64_t in = ~uint64_t(0);
  if (a.top_groups < a.groups) {
    in = 0;
    for (int r = 0; r < a.top_groups; ++r) {
      int best = -1;
      T best_key = -inf<T>();
      for (int g = 0; g < a.groups; ++g) {
        if ((in >> g) & 1) continue;
        T k1 = -inf<T>(), k2 = -inf<T>();
        for (int e = g * per; e < (g + 1) * per; ++e) {
          const T k = key_of(a, z, bias, e, top, sum);
          if (k > k1) {
            k2 = k1;
            k1 = k;
          } else if (k > k2) {
            k2 = k;
          }
        }
        const T score = k2 > -inf<T>() ? k1 + k2 : k1;
        if (score > best_key) {
          best_key = score;
          best = g;
        }
      }
      if (best >= 0) in |= uint64_t(1) << best;
    }
  }
  int pick[TPCONV_MAX_TOP_K];
  T last_key = inf<T>();
  int last = -1, n = 0;
  for (; n < a.k; ++n) {  // the next in the order (key descending, index ascending)
    int best = -1;
    T best_key = -inf<T>();
    for (int e = 0; e < a.X; ++e) {
      if (!((in >> (e / per)) & 1)) continue;
      const T k = key_of(a, z, bias, e, top, sum);
      if (k < last_key || (k == last_key && e > last))
        if (k > best_key) {
          best_key = k;
          best = e;
        }
    }
    if (best < 0) break;
    pick[n] = last = best;
    last_key = best_key;
  }
  // gates, the renormalised ones from the logits of the chosen
  T m = -inf<T>(), total = 0;
  if (a.renorm) {
    for (int j = 0; j < n; ++j) {
      const T l = a.sigmoid ? log_sigmoid(z[pick[j]]) : z[pick[j]];
      m = l > m ? l : m;
    }
    for (int j = 0; j < n; ++j) total += exp((a.sigmoid ? log_sigmoid(z[pick[j]]) : z[pick[j]]) - m);
    if (!a.sigmoid) total += sum - sum;  // a NaN row stays NaN
  }
  for (int j = 0; j < a.k; ++j) {
    T w = 0;
    if (j < n) {
      const T zj = z[pick[j]];
      if (a.renorm)
        w = exp((a.sigmoid ? log_sigmoid(zj) : zj) - m) / total;
      else
        w = a.sigmoid ? sigmoid(zj) : exp(zj - top) / sum;
      w *= static_cast<T>(a.scale);
    }
    experts[i * a.k + j] = j < n ? pick[j] : -1;
    gates[i * a.k + j] = w;
  }
}

template <class T>
__global__ void k_route_grad(RouteArgs a, const T* __restrict__ logits, const int32_t* __restrict__ experts,
                             const T* __restrict__ grad, T* __restrict__ out) {
  const int64_t i = blockIdx.x * int64_t(blockDim.x) + threadIdx.x;
  if (i >= a.n_rows) return;
  const T* z = logits + i * a.X;
  T* dz = out + i * a.X;
  const T scale = static_cast<T>(a.scale);
  int pick[TPCONV_MAX_TOP_K];
  T g[TPCONV_MAX_TOP_K], w[TPCONV_MAX_TOP_K];
  for (int j = 0; j < a.k; ++j) {
    const int e = experts[i * a.k + j];
    pick[j] = e >= 0 && e < a.X ? e : -1;
    g[j] = pick[j] >= 0 ? grad[i * a.k + j] : T(0);
  }
  T top = 0, sum = 1, m = -inf<T>(), total = 0;
  if (a.renorm) {
    for (int j = 0; j < a.k; ++j)
      if (pick[j] >= 0) {
        const T l = a.sigmoid ? log_sigmoid(z[pick[j]]) : z[pick[j]];
        m = l > m ? l : m;
      }
    for (int j = 0; j < a.k; ++j)
      if (pick[j] >= 0) total += exp((a.sigmoid ? log_sigmoid(z[pick[j]]) : z[pick[j]]) - m);
  } else if (!a.sigmoid) {
    softmax_stats(z, a.X, top, sum);
  }
  T inner = 0;  // sum of gate gradient times gate / scale
  for (int j = 0; j < a.k; ++j) {
    w[j] = 0;
    if (pick[j] < 0) continue;
    const T zj = z[pick[j]];
    w[j] = a.renorm ? exp((a.sigmoid ? log_sigmoid(zj) : zj) - m) / total
                    : (a.sigmoid ? sigmoid(zj) : exp(zj - top) / sum);
    inner += g[j] * w[j];
  }
  for (int e = 0; e < a.X; ++e) {
    T d = 0;
    for (int j = 0; j < a.k; ++j) {
      if (pick[j] != e) continue;
      T t = a.renorm ? w[j] * (g[j] - inner) : w[j] * g[j];
      if (a.sigmoid) t *= sigmoid(-z[e]);
      d += t;
    }
    if (!a.renorm && !a.sigmoid && !(z[e] == -inf<T>())) d -= exp(z[e] - top) / sum * inner;
    dz[e] = scale * d;
  }
}

}  // namespace

hipError_t launch_route_forward(bool f64, const RouteArgs& a, const void* logits, const void* bias, int32_t* experts,
                                void* gates, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>((a.n_rows + 255) / 256));
  if (f64)
    hipLaunchKernelGGL(k_route<double>, grid, dim3(256), 0, s, a, static_cast<const double*>(logits),
                       static_cast<const double*>(bias), experts, static_cast<double*>(gates));
  else
    hipLaunchKernelGGL(k_route<float>, grid, dim3(256), 0, s, a, static_cast<const float*>(logits),
                       static_cast<const float*>(bias), experts, static_cast<float*>(gates));
  return hipGetLastError();
}

hipError_t launch_route_backward(bool f64, const RouteArgs& a, const void* logits, const int32_t* experts,
                                 const void* grad_gates, void* grad_logits, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>((a.n_rows + 255) / 256));
  if (f64)
    hipLaunchKernelGGL(k_route_grad<double>, grid, dim3(256), 0, s, a, static_cast<const double*>(logits), experts,
                       static_cast<const double*>(grad_gates), static_cast<double*>(grad_logits));
  else
    hipLaunchKernelGGL(k_route_grad<float>, grid, dim3(256), 0, s, a, static_cast<const float*>(logits), experts,
                       static_cast<const float*>(grad_gates), static_cast<float*>(grad_logits));
  return hipGetLastError();
}

}  // namespace tpconv
