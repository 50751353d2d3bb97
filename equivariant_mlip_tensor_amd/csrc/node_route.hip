// node_route.hip -- routing of rows to experts: scores, groups, top_k, gates,
// and the gradient of the gates with respect to the logits.
//
// 2^LG lanes hold a row, VPL logits each (expert v * 2^LG + lane), so a row
// is read once, coalesced, and several short rows share a wavefront.  The
// reductions over a row run on the vector units (DPP and lane swaps); one
// round of the selection is a maximum over the row, a ballot of the lanes that
// hold it, and the lowest of them: no sort, and ties are settled exactly.
#include <hip/hip_runtime.h>

#include "node_internal.hpp"

namespace tpconv {
namespace {

template <class T>
__device__ __forceinline__ T inf() {
  return static_cast<T>(__builtin_huge_val());
}
__device__ __forceinline__ float lowest(float) { return -3.402823466e38f; }
__device__ __forceinline__ double lowest(double) { return -1.7976931348623157e308; }

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

// ------------------------------------------------- reductions over 2^LG lanes
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, 0xF, 0xF, false));
}
// v of the lane across: by 1, 2, 4, 8 (the last two mirror, which is the same
// once the lanes below agree), 16, 32
template <int STEP>
__device__ __forceinline__ uint32_t across(uint32_t v) {
  if constexpr (STEP == 0) return dpp<0xB1>(v);
  if constexpr (STEP == 1) return dpp<0x4E>(v);
  if constexpr (STEP == 2) return dpp<0x141>(v);
  if constexpr (STEP == 3) return dpp<0x140>(v);
  return static_cast<uint32_t>(__shfl_xor(static_cast<int>(v), 1 << STEP, 64));
}
template <int STEP>
__device__ __forceinline__ float across(float v) {
  return __uint_as_float(across<STEP>(__float_as_uint(v)));
}
template <int STEP>
__device__ __forceinline__ double across(double v) {
  return __hiloint2double(static_cast<int>(across<STEP>(static_cast<uint32_t>(__double2hiint(v)))),
                          static_cast<int>(across<STEP>(static_cast<uint32_t>(__double2loint(v)))));
}

struct Max {
  template <class T>
  __device__ __forceinline__ T operator()(T a, T b) const {
    return a > b ? a : b;  // no NaN reaches it
  }
};
struct Sum {
  template <class T>
  __device__ __forceinline__ T operator()(T a, T b) const {
    return a + b;
  }
};
template <int LG, class Op, class T>
__device__ __forceinline__ T reduce(T v, Op op) {
  if constexpr (LG > 0) v = op(v, across<0>(v));
  if constexpr (LG > 1) v = op(v, across<1>(v));
  if constexpr (LG > 2) v = op(v, across<2>(v));
  if constexpr (LG > 3) v = op(v, across<3>(v));
  if constexpr (LG > 4) v = op(v, across<4>(v));
  if constexpr (LG > 5) v = op(v, across<5>(v));
  return v;
}

// lanes of this row for which `on` holds, the row's first lane at bit 0
template <int LG>
__device__ __forceinline__ uint64_t row_ballot(bool on) {
  const uint64_t m = __ballot(on);
  if constexpr (LG == 6) return m;
  return (m >> (threadIdx.x & 63 & ~((1 << LG) - 1))) & ((uint64_t(1) << (1 << LG)) - 1);
}

// maximum and sum of exponentials of a row's softmax (masked entries add
// nothing; a row all masked has sum 0).  NaN is passed over by the maximum and
// makes the sum NaN.
template <class T, int LG, int VPL>
__device__ __forceinline__ void softmax_stats(const T (&z)[VPL], T& top, T& sum) {
  T m = -inf<T>();
#pragma unroll
  for (int v = 0; v < VPL; ++v) m = z[v] > m ? z[v] : m;
  top = reduce<LG>(m, Max{});
  T s = 0;
#pragma unroll
  for (int v = 0; v < VPL; ++v) s += z[v] == -inf<T>() ? T(0) : exp(z[v] - top);
  sum = reduce<LG>(s, Sum{});
}

// Gates of the chosen, lane j of the row holding the j-th (z of it, `has`):
// over 8 lanes at most, since top_k is at most 8.
template <class T, int LG>
__device__ __forceinline__ T gate_of(const RouteArgs& a, T z, bool has, T top, T sum) {
  constexpr int L = LG < 3 ? LG : 3;
  if (a.renorm) {
    const T l = a.sigmoid ? log_sigmoid(z) : z;
    const bool number = has && l == l;
    const T m = reduce<L>(number ? l : -inf<T>(), Max{});
    const T e = has ? exp(l - m) : T(0);
    const T total = reduce<L>(e, Sum{});
    return has ? e / total : T(0);
  }
  return has ? (a.sigmoid ? sigmoid(z) : exp(z - top) / sum) : T(0);
}

constexpr int kThreads = 256;

// Rows of a wavefront: 64 >> LG.  BY_SCORE: the keys are scores (there is a
// bias, or a group's two best are summed); otherwise the logits themselves,
// which have the same order.
template <class T, int LG, int VPL, bool BY_SCORE>
__global__ __launch_bounds__(kThreads) void k_route(RouteArgs a, const T* __restrict__ logits,
                                                    const T* __restrict__ bias, int32_t* __restrict__ experts,
                                                    T* __restrict__ gates) {
  constexpr int P = 1 << LG, kRows = kThreads / P;
  __shared__ T keys[BY_SCORE ? kRows * P * VPL : 1];  // rows' keys, for the groups
  __shared__ T best[BY_SCORE ? kRows * P : 1];
  const int sub = threadIdx.x & (P - 1), in_block = threadIdx.x >> LG;
  const int64_t step = int64_t(gridDim.x) * kRows;
  for (int64_t i0 = int64_t(blockIdx.x) * kRows; i0 < a.n_rows; i0 += step) {
    const int64_t i = min(i0 + in_block, a.n_rows - 1);  // lanes past the end redo the last row and write nothing
    const bool live = i0 + in_block < a.n_rows;
    const T* const zr = logits + i * a.X;
    T z[VPL], key[VPL];
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      const int e = v * P + sub;
      z[v] = e < a.X ? zr[e] : -inf<T>();
    }
    T top = 0, sum = 1;
    if (!a.sigmoid) softmax_stats<T, LG>(z, top, sum);
    const T inv = T(1) / sum;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      const int e = v * P + sub;
      T s = z[v];
      if (BY_SCORE) {
        s = a.sigmoid ? sigmoid(z[v]) : exp(z[v] - top) * inv;
        if (bias != nullptr) s += bias[e < a.X ? e : 0];
      } else if (!a.sigmoid && sum != sum) {
        s = sum;  // a NaN row orders by index
      }
      const T low = lowest(T(0));
      s = s >= low ? s : low;  // NaN (and -inf from the bias) last of the unmasked
      key[v] = z[v] == -inf<T>() ? -inf<T>() : s;
    }
    if (BY_SCORE && a.top_groups < a.groups) {
      T* const row = keys + in_block * (P * VPL);
      T* const score = best + in_block * P;
      __syncthreads();
#pragma unroll
      for (int v = 0; v < VPL; ++v) row[v * P + sub] = key[v];
      __syncthreads();
      const int per = a.X / a.groups;
      T k1 = -inf<T>(), k2 = -inf<T>();
      if (sub < a.groups)
        for (int e = sub * per; e < (sub + 1) * per; ++e) {
          const T k = row[e];
          k2 = k > k1 ? k1 : (k > k2 ? k : k2);
          k1 = k > k1 ? k : k1;
        }
      const T mine = k2 > -inf<T>() ? k1 + k2 : k1;
      score[sub] = mine;
      __syncthreads();
      int rank = 0;
      for (int g = 0; g < a.groups; ++g) {
        const T other = score[g];
        rank += other > mine || (other == mine && g < sub);
      }
      const uint64_t inside = row_ballot<LG>(sub < a.groups && rank < a.top_groups && mine > -inf<T>());
#pragma unroll
      for (int v = 0; v < VPL; ++v)
        if (!((inside >> ((v * P + sub) / per & 63)) & 1)) key[v] = -inf<T>();
    }
    // the next in the order (key descending, index ascending), top_k times
    int pick = -1;
    for (int j = 0; j < a.k; ++j) {
      T m = key[0];
#pragma unroll
      for (int v = 1; v < VPL; ++v) m = key[v] > m ? key[v] : m;
      m = reduce<LG>(m, Max{});
      int e = -1;
#pragma unroll
      for (int v = VPL - 1; v >= 0; --v) {
        const uint64_t have = row_ballot<LG>(key[v] == m && m > -inf<T>());
        if (have != 0) e = v * P + __ffsll(static_cast<unsigned long long>(have)) - 1;
      }
#pragma unroll
      for (int v = 0; v < VPL; ++v)
        if (e == v * P + sub) key[v] = -inf<T>();
      if (sub == j) pick = e;
    }
    const bool has = sub < a.k && pick >= 0;
    T w = gate_of<T, LG>(a, has ? zr[pick] : T(0), has, top, sum);
    if (!a.sigmoid && has && sum != sum) w = sum;  // NaN in, NaN out
    if (live && sub < a.k) {
      experts[i * a.k + sub] = pick;
      gates[i * a.k + sub] = static_cast<T>(a.scale) * w;
    }
  }
}

template <class T, int LG, int VPL>
__global__ __launch_bounds__(kThreads) void k_route_grad(RouteArgs a, const T* __restrict__ logits,
                                                         const int32_t* __restrict__ experts,
                                                         const T* __restrict__ grad, T* __restrict__ out) {
  constexpr int P = 1 << LG, kRows = kThreads / P, L = LG < 3 ? LG : 3;
  const int sub = threadIdx.x & (P - 1), in_block = threadIdx.x >> LG;
  const int first = threadIdx.x & 63 & ~(P - 1);  // the row's first lane
  const int64_t step = int64_t(gridDim.x) * kRows;
  const T scale = static_cast<T>(a.scale);
  for (int64_t i0 = int64_t(blockIdx.x) * kRows; i0 < a.n_rows; i0 += step) {
    const int64_t i = min(i0 + in_block, a.n_rows - 1);
    const bool live = i0 + in_block < a.n_rows;
    const T* const zr = logits + i * a.X;
    // lane j: the j-th chosen expert, its logit and the gradient of its gate.
    int pick = -1;
    T g = 0, zp = 0;
    if (sub < a.k) {
      const int e = experts[i * a.k + sub];
      if (e >= 0 && e < a.X) {
        pick = e;
        g = grad[i * a.k + sub];
        zp = zr[e];
      }
    }
    T top = 0, sum = 1;
    T z[VPL];
    if (!a.renorm && !a.sigmoid) {
#pragma unroll
      for (int v = 0; v < VPL; ++v) z[v] = v * P + sub < a.X ? zr[v * P + sub] : -inf<T>();
      softmax_stats<T, LG>(z, top, sum);
    }
    const T w = gate_of<T, LG>(a, zp, pick >= 0, top, sum);
    const T inner = reduce<L>(g * w, Sum{});
    // what lane j's expert gets
    T d = a.renorm ? w * (g - __shfl(inner, first, 64)) : w * g;
    if (a.sigmoid) d *= sigmoid(-zp);
    T dz[VPL];
#pragma unroll
    for (int v = 0; v < VPL; ++v) dz[v] = T(0);
    for (int j = 0; j < a.k; ++j) {
      const int e = __shfl(pick, first + j, 64);
      const T t = __shfl(d, first + j, 64);
#pragma unroll
      for (int v = 0; v < VPL; ++v)
        if (e == v * P + sub) dz[v] += t;
    }
    if (!a.renorm && !a.sigmoid) {
      const T all = __shfl(inner, first, 64), inv = T(1) / sum;
#pragma unroll
      for (int v = 0; v < VPL; ++v)
        if (!(z[v] == -inf<T>())) dz[v] -= exp(z[v] - top) * inv * all;
    }
    if (live)
#pragma unroll
      for (int v = 0; v < VPL; ++v)
        if (v * P + sub < a.X) out[i * a.X + v * P + sub] = scale * dz[v];
  }
}

template <int LG_, int VPL_>
struct Shape {
  static constexpr int LG = LG_, VPL = VPL_;
};

// the lanes and values of a row of X logits
template <class F>
hipError_t with_shape(int X, F f) {
  if (X <= 8) return f(Shape<3, 1>{});  // 8 lanes at least: a place for each of top_k
  if (X <= 16) return f(Shape<4, 1>{});
  if (X <= 32) return f(Shape<5, 1>{});
  if (X <= 64) return f(Shape<6, 1>{});
  if (X <= 128) return f(Shape<6, 2>{});
  return f(Shape<6, 4>{});
}

dim3 grid_of(int64_t n_rows, int lg) {
  const int64_t rows = kThreads >> lg, g = (n_rows + rows - 1) / rows;
  return dim3(static_cast<unsigned>(g < 4096 ? g : 4096));  // 16 blocks' wavefronts a SIMD, then rows in turn
}

template <class T>
hipError_t forward(const RouteArgs& a, const T* logits, const T* bias, int32_t* experts, T* gates, hipStream_t s) {
  return with_shape(a.X, [&](auto shape) {
    constexpr int LG = decltype(shape)::LG, VPL = decltype(shape)::VPL;
    if (bias != nullptr || a.top_groups < a.groups)
      hipLaunchKernelGGL((k_route<T, LG, VPL, true>), grid_of(a.n_rows, LG), dim3(kThreads), 0, s, a, logits, bias,
                         experts, gates);
    else
      hipLaunchKernelGGL((k_route<T, LG, VPL, false>), grid_of(a.n_rows, LG), dim3(kThreads), 0, s, a, logits, bias,
                         experts, gates);
    return hipGetLastError();
  });
}

template <class T>
hipError_t backward(const RouteArgs& a, const T* logits, const int32_t* experts, const T* grad, T* out,
                    hipStream_t s) {
  return with_shape(a.X, [&](auto shape) {
    constexpr int LG = decltype(shape)::LG, VPL = decltype(shape)::VPL;
    hipLaunchKernelGGL((k_route_grad<T, LG, VPL>), grid_of(a.n_rows, LG), dim3(kThreads), 0, s, a, logits, experts,
                       grad, out);
    return hipGetLastError();
  });
}

}  // namespace

hipError_t launch_route_forward(bool f64, const RouteArgs& a, const void* logits, const void* bias, int32_t* experts,
                                void* gates, hipStream_t s) {
  return f64 ? forward(a, static_cast<const double*>(logits), static_cast<const double*>(bias), experts,
                       static_cast<double*>(gates), s)
             : forward(a, static_cast<const float*>(logits), static_cast<const float*>(bias), experts,
                       static_cast<float*>(gates), s);
}

hipError_t launch_route_backward(bool f64, const RouteArgs& a, const void* logits, const int32_t* experts,
                                 const void* grad_gates, void* grad_logits, hipStream_t s) {
  return f64 ? backward(a, static_cast<const double*>(logits), experts, static_cast<const double*>(grad_gates),
                        static_cast<double*>(grad_logits), s)
             : backward(a, static_cast<const float*>(logits), experts, static_cast<const float*>(grad_gates),
                        static_cast<float*>(grad_logits), s);
}

}  // namespace tpconv
