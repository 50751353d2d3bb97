// node_route.hip -- routing of rows to experts: scores, groups, top_k, gates,
// and the gradient of the gates with respect to the logits.
//
// 8 or 16 lanes hold a row, VPL logits each (expert v * lanes + lane), so a row
// is read once and 8 or 4 rows share a wavefront.  (A whole wavefront to a row
// of 128 took 125 us for 131072 rows: the steps across lanes, the group
// search and the gates then serve one row.)  The reductions over a row run on
// the vector units (DPP); one round of the selection is a maximum over the
// row's keys, as ordered whole numbers, and a minimum over the indices that
// hold it: no sort, and ties are settled exactly.  The forward is bound by its
// vector instructions, the gradient by its reads of single logits and gates,
// each of which waits for the expert's number: 131072 fp32 rows of 128 experts
// in 8 groups, 6 chosen, take 55 us (1050 instructions for four rows, a fourth
// of them in the groups' search and a fourth in the rounds; the vector units are
// busy in 95 % of the cycles) and 22 us; 67 MB of logits read and 67 MB of their
// gradient written are 13 us each at the rate of a copy.  28000 rows of 16
// experts take 4.4 us and 5.4 us.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "node_device.hpp"
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

// a / b for 1 <= b: the reciprocal instruction is good to a unit in the last
// place, a tenth of a division's cost
__device__ __forceinline__ float over(float a, float b) { return a * __builtin_amdgcn_rcpf(b); }
__device__ __forceinline__ double over(double a, double b) { return a / b; }

template <class T>
__device__ __forceinline__ T sigmoid(T z) {
  const T e = exp(z < T(0) ? z : -z);
  return over(z < T(0) ? e : T(1), T(1) + e);
}

// ------------------------------------------------- reductions over 2^LG lanes
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, 0xF, 0xF, true));
}
// v of the lane across: by 1, 2, 4, 8 (the last two mirror, which is the same
// once the lanes below agree)
template <int STEP>
__device__ __forceinline__ uint32_t across(uint32_t v) {
  if constexpr (STEP == 0) return dpp<0xB1>(v);
  if constexpr (STEP == 1) return dpp<0x4E>(v);
  if constexpr (STEP == 2) return dpp<0x141>(v);
  return dpp<0x140>(v);
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

template <int STEP>
__device__ __forceinline__ uint64_t across(uint64_t v) {
  return uint64_t(across<STEP>(static_cast<uint32_t>(v >> 32))) << 32 | across<STEP>(static_cast<uint32_t>(v));
}

// v of the lane before (0 in lanes 0, 16, 32, 48)
__device__ __forceinline__ uint32_t lane_before(uint32_t v) { return dpp<0x111>(v); }
__device__ __forceinline__ uint64_t lane_before(uint64_t v) {
  return uint64_t(dpp<0x111>(static_cast<uint32_t>(v >> 32))) << 32 | dpp<0x111>(static_cast<uint32_t>(v));
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
  static_assert(LG <= 4, "rows of 16 lanes at most");
  if constexpr (LG > 0) v = op(v, across<0>(v));
  if constexpr (LG > 1) v = op(v, across<1>(v));
  if constexpr (LG > 2) v = op(v, across<2>(v));
  if constexpr (LG > 3) v = op(v, across<3>(v));
  return v;
}

// v of lane `from` of this row
template <int LG, class T>
__device__ __forceinline__ T of_lane(T v, int from) {
  return __shfl(v, (threadIdx.x & 63 & ~((1 << LG) - 1)) + from, 64);
}

// Scores as whole numbers in the same order; 0 (none) and 1 (NaN) are below
// every score.
__device__ __forceinline__ uint32_t ordered(float s) {
  const uint32_t b = __float_as_uint(s + 0.0f);  // one zero
  return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ uint64_t ordered(double s) {
  const uint64_t b = static_cast<uint64_t>(__double_as_longlong(s + 0.0));
  return b ^ (static_cast<uint64_t>(static_cast<int64_t>(b) >> 63) | 0x8000000000000000ull);
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
    T e = 0;
    // sigmoids far from underflow are divided as they are, others through their logarithms: by rows, so that a row's
    // gates do not depend on the others of its wavefront
    uint64_t low = ~uint64_t(0);  // lanes with a score that is not far from it
    if (a.sigmoid) {
      e = has ? sigmoid(z) : T(0);
      low = __ballot(has && !(e > T(1e-30)));
    }
    if (low != 0) {
      const bool plain = ((low >> (threadIdx.x & 63 & ~((1 << LG) - 1))) & ((1u << (1 << LG)) - 1)) == 0;
      const T l = a.sigmoid ? log_sigmoid(z) : z;
      const bool number = has && l == l;
      const T m = reduce<L>(number ? l : -inf<T>(), Max{});
      e = plain ? e : (has ? exp(l - m) : T(0));
    }
    const T total = reduce<L>(e, Sum{});
    return has ? e / total : T(0);
  }
  return has ? (a.sigmoid ? sigmoid(z) : exp(z - top) / sum) : T(0);
}

constexpr int kThreads = 256;

// BY_SCORE: scores are formed (there is a bias to add, or a group's two best are
// summed); 28000 rows of 16 take 4.6 us without, 5.4 with.  Without a bias the
// keys are the logits, which have the scores' order and tell apart scores that
// round to one number (0 or 1); with one, equal keys go by the logits, so that a
// bias of zeros chooses the same.  Rows of up to 128 are held to the registers of
// five wavefronts a SIMD (fp64: three): 131072 rows of 128 in groups in 55 us,
// with two registers more and four wavefronts in 59; 65536 fp64 rows in 57 us,
// with two wavefronts in 67.
template <class T, int LG, int VPL, bool BY_SCORE>
__global__ __launch_bounds__(kThreads, VPL <= 8 ? (sizeof(T) == 4 ? 5 : 3) : 1) void k_route(
    RouteArgs a, const T* __restrict__ logits, const T* __restrict__ bias, int32_t* __restrict__ experts,
    T* __restrict__ gates) {
  constexpr int P = 1 << LG, kRows = kThreads / P, X_MAX = P * VPL;
  using Key = decltype(ordered(T(0)));
  constexpr Key kNaN = 1;
  __shared__ T rows[kRows][X_MAX + 4];  // a row's scores, then its logits; rows start 4 banks apart
  __shared__ T groups[BY_SCORE ? kRows : 1][BY_SCORE ? 136 : 1];  // a row's groups' scores, then 1 for the chosen; 8 banks apart
  const int sub = threadIdx.x & (P - 1), in_block = threadIdx.x >> LG;
  T* const row = rows[in_block];
  T* const group = groups[BY_SCORE ? in_block : 0];
  const int per = a.X / a.groups;
  const bool by_bias = BY_SCORE && bias != nullptr;
  const int64_t step = int64_t(gridDim.x) * kRows;
  T ahead[VPL];  // the next row's logits
  auto load = [&](int64_t i0) {
    const T* const zr = logits + min(i0 + in_block, a.n_rows - 1) * a.X;
#pragma unroll
    for (int v = 0; v < VPL; ++v) ahead[v] = zr[min(v * P + sub, a.X - 1)];
  };
  load(int64_t(blockIdx.x) * kRows);
  T shift[BY_SCORE ? VPL : 1];     // the experts' biases
  uint32_t group_of[(VPL + 3) / 4] = {};  // a byte for each expert
  if (BY_SCORE)
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      const int e = min(v * P + sub, a.X - 1);
      shift[v] = bias != nullptr ? bias[e] : T(0);
      group_of[v / 4] |= static_cast<uint32_t>(e / per) << (v % 4 * 8);
    }
  for (int64_t i0 = int64_t(blockIdx.x) * kRows; i0 < a.n_rows; i0 += step) {
    const int64_t i = min(i0 + in_block, a.n_rows - 1);  // lanes past the end redo the last row and write nothing
    const bool live = i0 + in_block < a.n_rows;
    T z[VPL], score[VPL];
#pragma unroll
    for (int v = 0; v < VPL; ++v) z[v] = v * P + sub < a.X ? ahead[v] : -inf<T>();
    load(i0 + step);
    T top = 0, sum = 1;
    if (!a.sigmoid) softmax_stats<T, LG>(z, top, sum);
    const T inv = T(1) / sum;
    bool odd = false;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      T s = z[v];
      if (BY_SCORE) {
        s = (a.sigmoid ? sigmoid(z[v]) : exp(z[v] - top) * inv) + shift[BY_SCORE ? v : 0];
      } else if (!a.sigmoid && sum != sum) {
        s = sum;  // a NaN row orders by index
      }
      const bool masked = z[v] == -inf<T>() || (BY_SCORE && shift[BY_SCORE ? v : 0] == -inf<T>());
      score[v] = masked ? -inf<T>() : s;
      odd |= score[v] != score[v];
    }
    odd = __any(odd);  // NaN among the wavefront's scores: rare
    uint32_t out_of_group = 0;  // bit v: the group of expert v * P + sub is not chosen
    if (BY_SCORE && a.top_groups < a.groups) {
      wave_sync();
#pragma unroll
      for (int v = 0; v < VPL; ++v) row[v * P + sub] = score[v];
      if (odd)
#pragma unroll
        for (int v = 0; v < VPL; ++v)
          if (score[v] != score[v]) row[v * P + sub] = lowest(T(0));
      wave_sync();
      for (int g = sub; g < a.groups; g += P) {
        T k1 = -inf<T>(), k2 = -inf<T>();
        for (int e = g * per; e < (g + 1) * per; ++e) {
          const T k = row[e];
          k2 = fmax(k2, fmin(k1, k));
          k1 = fmax(k1, k);
        }
        // NaN (here the lowest value) and the two keys' sum stay numbers: the group is not one that is all masked
        const T least = lowest(T(0)) / 2;
        group[g] = k1 == -inf<T>() ? k1 : fmax(k1, least) + (k2 == -inf<T>() ? T(0) : fmax(k2, least));
      }
      wave_sync();
      for (int g = sub; g < a.groups; g += P) {
        const T mine = group[g];
        int rank = 0;
        for (int o = 0; o < a.groups; ++o) {
          const T other = group[o];
          rank += other > mine || (other == mine && o < g);
        }
        group[64 + g] = rank < a.top_groups && mine > -inf<T>() ? T(1) : T(0);
      }
      wave_sync();
#pragma unroll
      for (int v = 0; v < VPL; ++v)
        if (group[64 + ((group_of[v / 4] >> (v % 4 * 8)) & 255)] == T(0)) out_of_group |= 1u << v;
    }
    Key key[VPL];
    auto make_keys = [&](const T (&by)[VPL]) {
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
        const Key number = ordered(by[v]);
        key[v] = score[v] == -inf<T>() || ((out_of_group >> v) & 1) != 0 ? Key(0) : number;
      }
    };
    if (by_bias)
      make_keys(score);
    else
      make_keys(z);
    if (odd)
#pragma unroll
      for (int v = 0; v < VPL; ++v)
        if (score[v] != score[v] && ((out_of_group >> v) & 1) == 0) key[v] = kNaN;
    wave_sync();
#pragma unroll
    for (int v = 0; v < VPL; ++v) row[v * P + sub] = z[v];  // out of the registers during the rounds
    wave_sync();
    // the next in the order (key descending, then index ascending or, with LOGITS, logit descending and index
    // ascending), top_k times; lane j keeps the j-th and its key
    int pick = -1;
    Key picked = 0, last = 0;
    auto choose = [&](auto LOGITS) {
      for (int j = 0; j < a.k; ++j) {
        Key most = key[0];
#pragma unroll
        for (int v = 1; v < VPL; ++v) most = key[v] > most ? key[v] : most;
        const Key m = reduce<LG>(most, [](Key x, Key y) { return x > y ? x : y; });
        T best = -inf<T>();
        if constexpr (LOGITS) {
#pragma unroll
          for (int v = 0; v < VPL; ++v) {
            const T l = row[v * P + sub];
            best = key[v] == m && l > best ? l : best;
          }
          best = reduce<LG>(best, Max{});
        }
        uint32_t at = X_MAX;
#pragma unroll
        for (int v = VPL - 1; v >= 0; --v)
          at = key[v] == m && (!LOGITS || m <= kNaN || row[v * P + sub] == best) ? v * P + sub : at;
        const int e = static_cast<int>(reduce<LG>(at, [](uint32_t x, uint32_t y) { return x < y ? x : y; }));
#pragma unroll
        for (int v = 0; v < VPL; ++v)
          if (e == v * P + sub) key[v] = 0;
        pick = sub == j ? e : pick;
        picked = sub == j ? m : picked;
        last = m;
      }
    };
    choose(std::false_type{});
    if (by_bias) {
      // equal keys, rare, stand side by side, the last chosen's perhaps among those left: then the rounds are made
      // again with the logits (131072 rows of 128 in groups: 55 us; with a check in each round 59-60)
      bool equal = sub > 0 && picked > kNaN && picked == lane_before(picked);
#pragma unroll
      for (int v = 0; v < VPL; ++v) equal |= key[v] == last && last > kNaN;
      if (__any(equal)) {
        for (int j = 0; j < a.k; ++j) {
          const int e = of_lane<LG>(pick, j);
          const Key m = of_lane<LG>(picked, j);
#pragma unroll
          for (int v = 0; v < VPL; ++v)
            if (e == v * P + sub) key[v] = m;
        }
        choose(std::true_type{});
      }
    }
    pick = picked != 0 ? pick : -1;  // nothing was left
    const bool has = pick >= 0;
    T w = gate_of<T, LG>(a, has ? row[pick] : T(0), has, top, sum);
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
  const int64_t step = int64_t(gridDim.x) * kRows;
  const T scale = static_cast<T>(a.scale);
  // lane j: the j-th chosen expert, its logit and the gradient of its gate,
  // the expert two rows ahead and the others one
  auto row_at = [&](int64_t i0) { return min(i0 + in_block, a.n_rows - 1); };
  auto expert = [&](int64_t i0) {
    const int e = experts[row_at(i0) * a.k + min(sub, a.k - 1)];
    return sub < a.k && e >= 0 && e < a.X ? e : -1;
  };
  const int64_t begin = int64_t(blockIdx.x) * kRows;
  int pick1 = expert(begin), pick2 = expert(begin + step);
  T g1, z1;
  auto load = [&](int64_t i0, int pick) {
    const int64_t i = row_at(i0);
    g1 = grad[i * a.k + min(sub, a.k - 1)];
    z1 = logits[i * a.X + max(pick, 0)];
  };
  load(begin, pick1);
  for (int64_t i0 = begin; i0 < a.n_rows; i0 += step) {
    const int64_t i = row_at(i0);
    const bool live = i0 + in_block < a.n_rows;
    const T* const zr = logits + i * a.X;
    const int pick = pick1;
    const T g = pick >= 0 ? g1 : T(0), zp = pick >= 0 ? z1 : T(0);
    pick1 = pick2;
    load(i0 + step, pick1);
    pick2 = expert(i0 + 2 * step);
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
    const T all = of_lane<LG>(inner, 0);
    T d = a.renorm ? w * (g - all) : w * g;
    if (a.sigmoid) d *= sigmoid(-zp);
    T dz[VPL];
#pragma unroll
    for (int v = 0; v < VPL; ++v) dz[v] = T(0);
    for (int j = 0; j < a.k; ++j) {
      const int e = of_lane<LG>(pick, j);
      const T t = of_lane<LG>(d, j);
#pragma unroll
      for (int v = 0; v < VPL; ++v)
        if (e == v * P + sub) dz[v] += t;
    }
    if (!a.renorm && !a.sigmoid) {
      const T inv = T(1) / sum;
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

// the lanes and values of a row of X logits, the fewest that hold them: 28000 rows of 16 in 4.6 us, with places for 32
// 5.0; 16 fp64 rows of 8 in 2.3 us and 2.5
template <class F>
hipError_t with_shape(int X, F f) {
  if (X <= 8) return f(Shape<3, 1>{});  // 8 lanes at least: a place for each of top_k
  if (X <= 16) return f(Shape<4, 1>{});
  if (X <= 32) return f(Shape<4, 2>{});
  if (X <= 64) return f(Shape<4, 4>{});
  if (X <= 128) return f(Shape<4, 8>{});
  return f(Shape<4, 16>{});
}

dim3 grid_of(int64_t n_rows, int lg) {
  const int64_t rows = kThreads >> lg, g = (n_rows + rows - 1) / rows;
  return dim3(static_cast<unsigned>(g < 4096 ? g : 4096));  // 16 wavefronts for each SIMD, then rows in turn
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
