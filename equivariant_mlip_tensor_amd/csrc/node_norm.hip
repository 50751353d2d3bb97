// node_norm.hip -- the root-mean-square norm of irreps rows, its gradients, and
// rows in 8 bits.  With h = x + residual, ms the mean square of what is
// normalised together (a segment, or the row's segments counted alike):
//   r = (ms + eps)^(-1/2),  y = gamma r h,
//   grad_h_j = r (w_j - k_j u_j sum_i w_i u_i) + grad_sum_j,  u = r h, w = gamma g,
//   grad_gamma_c = sum over rows and components of g u,
// k_j the weight of h_j^2 in ms.
//
// Bound by memory: every row is read once, held in registers until its sums are
// known, and written once.  The lanes of a row keep the same columns for all
// the rows they take, so a column's segment and channel are found once, gamma
// stays in registers, and grad_gamma is summed in registers down the rows.
// Rows of up to 256 pieces (16 bytes, or single elements where a segment does
// not start at a multiple of one) are held by 1 to 64 lanes of a wavefront, and
// longer ones by a block.
// Sums run in 64 bits for both types: squares of any fp32 value fit, and the
// gradient's difference keeps what fp32 would cancel in a segment of one or two
// columns.
#include <hip/hip_runtime.h>

#include "node_device.hpp"
#include "node_internal.hpp"

namespace tpconv {
namespace {

constexpr int kThreads = 256;
constexpr int kMostBlocks = 1024;      // 4 blocks for each CU
constexpr int kMostGradBlocks = 768;

// What a lane keeps of its pieces' columns.
template <class T, int PER, int NP>
struct Columns {
  int col[NP];     // first column of a piece, -1: none
  int seg[NP];
  double share[NP];  // weight of a square in the mean
  T gamma[NP][PER];

  __device__ __forceinline__ void find(const NormArgs& a, int lane, int lanes, const T* from) {
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      const int c = (lane + j * lanes) * PER;
      col[j] = c < a.dim ? c : -1;
      int s = 0;
      if (c < a.dim)
        while (c >= a.seg[s].end) ++s;
      seg[j] = s;
      share[j] = 1.0 / (double(a.seg[s].end - a.seg[s].off) * (a.row_scope ? a.n_segs : 1));
#pragma unroll
      for (int e = 0; e < PER; ++e)
        gamma[j][e] = from != nullptr && c < a.dim ? from[a.seg[s].channel + (c + e - a.seg[s].off) / a.seg[s].d] : T(1);
    }
  }
};

template <class T, int PER, int NP>
__device__ __forceinline__ void load_row(T (&v)[NP][PER], const T* row, const int (&col)[NP]) {
  struct alignas(PER * sizeof(T)) Piece {
    T v[PER];
  };
#pragma unroll
  for (int j = 0; j < NP; ++j) {
    Piece p = {};
    if (col[j] >= 0) p = *reinterpret_cast<const Piece*>(row + col[j]);
#pragma unroll
    for (int e = 0; e < PER; ++e) v[j][e] = p.v[e];
  }
}

template <class T, int PER, int NP>
__device__ __forceinline__ void store_row(const T (&v)[NP][PER], T* row, const int (&col)[NP]) {
  struct alignas(PER * sizeof(T)) Piece {
    T v[PER];
  };
#pragma unroll
  for (int j = 0; j < NP; ++j)
    if (col[j] >= 0) {
      Piece p;
#pragma unroll
      for (int e = 0; e < PER; ++e) p.v[e] = v[j][e];
      *reinterpret_cast<Piece*>(row + col[j]) = p;
    }
}

// Reductions over a row's lanes; every lane gets the result.  ALL: the row is
// a block's (sums by wavefront pass through LDS, added in order), else `lanes`
// neighbours' of a wavefront.
template <bool ALL>
struct Team {
  int lanes;
  double* lds;  // ALL: two sets of 32 segments' sums of each wavefront

  template <class V, class F>
  __device__ __forceinline__ V wave(V v, F&& f) const {
    if (ALL) {
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) v = f(v, __shfl_xor(v, o, 64));
    } else {
      for (int o = 1; o < lanes; o <<= 1) v = f(v, __shfl_xor(v, o, 64));
    }
    return v;
  }
  __device__ __forceinline__ double sum(double v) const {
    return wave(v, [](double p, double q) { return p + q; });
  }
};

// r of a segment's or row's mean square: the root's error is a few units of 64
// bits, so r itself is next to exact in fp32 and within 3 units in fp64.
__device__ __forceinline__ double inverse_root(double ms, double eps) { return 1.0 / sqrt(ms + eps); }

__device__ __forceinline__ uint32_t max_bits(uint32_t a, uint32_t b) { return a > b ? a : b; }

// Sums over what is normalised together of up to N values of each piece; for
// each piece, its segment's or row's sums.
template <bool ALL, int NP, int N>
__device__ __forceinline__ void together(const Team<ALL>& team, const NormArgs& a, const int (&seg)[NP],
                                         const double (&v)[N][NP], double (&total)[N][NP]) {
  const int groups = a.row_scope ? 1 : a.n_segs;
  const int w = threadIdx.x >> 6, nw = blockDim.x >> 6;
  if (ALL) __syncthreads();  // the last sums are read
  for (int s = 0; s < groups; ++s) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      double p = 0;
#pragma unroll
      for (int j = 0; j < NP; ++j) p += a.row_scope || seg[j] == s ? v[i][j] : 0.0;
      p = team.sum(p);
      if (ALL) {
        if ((threadIdx.x & 63) == 0) team.lds[(i * kMaxNormSegs + s) * nw + w] = p;
      } else {
#pragma unroll
        for (int j = 0; j < NP; ++j)
          if (a.row_scope || seg[j] == s) total[i][j] = p;
      }
    }
  }
  if (ALL) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        const double* const part = team.lds + (i * kMaxNormSegs + (a.row_scope ? 0 : seg[j])) * nw;
        double p = 0;
        for (int q = 0; q < nw; ++q) p += part[q];
        total[i][j] = p;
      }
  }
}

// ---------------------------------------------------------------- 8 bits
// Codes are e4m3 (OCP).  The conversion's two results go to the low or high
// half of a register.
__device__ __forceinline__ uint32_t codes4(const float (&v)[4]) {
  int r = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
  return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], r, true));
}

template <bool ALL, int PER, int NP>
__device__ __forceinline__ void write_codes(const Team<ALL>& team, const NormArgs& a,
                                            const Columns<float, PER, NP>& cols, const float (&y)[NP][PER],
                                            uint8_t* codes, float* scales) {
  // magnitudes are compared as whole numbers: NaN is above infinity, so it is not lost
  uint32_t mine[NP], top[NP];
#pragma unroll
  for (int j = 0; j < NP; ++j) {
    mine[j] = 0;
#pragma unroll
    for (int e = 0; e < PER; ++e) mine[j] = max_bits(mine[j], __float_as_uint(y[j][e]) & 0x7FFFFFFFu);
    top[j] = 0;
  }
  const int w = threadIdx.x >> 6, nw = blockDim.x >> 6;
  uint32_t* const lds = reinterpret_cast<uint32_t*>(team.lds);
  if (ALL) __syncthreads();
  for (int s = 0; s < a.n_segs; ++s) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < NP; ++j) m = cols.seg[j] == s && cols.col[j] >= 0 ? max_bits(m, mine[j]) : m;
    m = team.wave(m, max_bits);
    if (ALL) {
      if ((threadIdx.x & 63) == 0) lds[s * nw + w] = m;
    } else {
#pragma unroll
      for (int j = 0; j < NP; ++j) top[j] = cols.seg[j] == s ? m : top[j];
    }
  }
  if (ALL) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NP; ++j)
      for (int q = 0; q < nw; ++q) top[j] = max_bits(top[j], lds[cols.seg[j] * nw + q]);
  }
#pragma unroll
  for (int j = 0; j < NP; ++j) {
    if (cols.col[j] < 0) continue;
    float scale = __uint_as_float(top[j]) * static_cast<float>(1.0 / 448.0);
    scale = scale < 0x1p-126f ? 0x1p-126f : scale;  // false for NaN, which stays
    const float inv = 1.0f / scale;
    if (cols.col[j] == a.seg[cols.seg[j]].off) scales[cols.seg[j]] = scale;
    if constexpr (PER == 4) {
      const float v[4] = {y[j][0] * inv, y[j][1] * inv, y[j][2] * inv, y[j][3] * inv};
      *reinterpret_cast<uint32_t*>(codes + cols.col[j]) = codes4(v);
    } else {
#pragma unroll
      for (int e = 0; e < PER; ++e)
        codes[cols.col[j] + e] =
            static_cast<uint8_t>(__builtin_amdgcn_cvt_pk_fp8_f32(y[j][e] * inv, 0.0f, 0, false) & 0xFF);
    }
  }
}

// ------------------------------------------------------------------ forward
// NORM: y is the norm of h; without it, h itself (rows into 8 bits alone).
template <class T, int PER, int NP, bool ALL, int THREADS, bool NORM>
__global__ __launch_bounds__(THREADS) void k_norm(NormArgs a, const T* x, const T* residual, const T* gamma, T* sum,
                                                  T* out, uint8_t* codes, float* scales) {
  __shared__ double lds[ALL ? kMaxNormSegs * (THREADS / 64) : 1];
  const int lanes = ALL ? THREADS : a.lanes;
  const int lane = ALL ? threadIdx.x : threadIdx.x & (lanes - 1);
  const Team<ALL> team{lanes, lds};
  Columns<T, PER, NP> cols;
  cols.find(a, lane, lanes, gamma);
  const int64_t teams = int64_t(gridDim.x) * (THREADS / lanes);
  for (int64_t row = int64_t(blockIdx.x) * (THREADS / lanes) + threadIdx.x / lanes; row < a.n_rows; row += teams) {
    const int64_t at = row * a.dim;
    T h[NP][PER];
    load_row(h, x + at, cols.col);
    if (residual != nullptr) {
      T more[NP][PER];
      load_row(more, residual + at, cols.col);
#pragma unroll
      for (int j = 0; j < NP; ++j)
#pragma unroll
        for (int e = 0; e < PER; ++e) h[j][e] += more[j][e];
    }
    if (sum != nullptr) store_row(h, sum + at, cols.col);
    if constexpr (NORM) {
      double square[1][NP], total[1][NP];
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        double q = 0;
#pragma unroll
        for (int e = 0; e < PER; ++e) q = fma(double(h[j][e]), double(h[j][e]), q);
        square[0][j] = cols.col[j] >= 0 ? q * cols.share[j] : 0.0;
        total[0][j] = 0;
      }
      together<ALL, NP, 1>(team, a, cols.seg, square, total);
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        const double r = inverse_root(total[0][j], a.eps);
#pragma unroll
        for (int e = 0; e < PER; ++e) h[j][e] = static_cast<T>(double(h[j][e]) * r) * cols.gamma[j][e];
      }
      if (out != nullptr) store_row(h, out + at, cols.col);
    }
    if constexpr (sizeof(T) == 4)
      if (codes != nullptr) write_codes<ALL, PER, NP>(team, a, cols, h, codes + at, scales + row * a.n_segs);
  }
}

// --------------------------------------------------------------- gradients
// part: a row of column sums for each block, or, where there is one block of
// wavefronts' rows, nothing: it writes grad_gamma itself.
template <class T, int PER, int NP, bool ALL, int THREADS>
__global__ __launch_bounds__(THREADS) void k_norm_grad(NormArgs a, const T* h_rows, const T* gamma, const T* grad_out,
                                                       const T* grad_sum, T* grad_x, T* grad_gamma, T* part) {
  __shared__ double lds[ALL ? 2 * kMaxNormSegs * (THREADS / 64) : 1];
  extern __shared__ char dynamic[];  // column sums, where wavefronts hold rows
  const int lanes = ALL ? THREADS : a.lanes;
  const int lane = ALL ? threadIdx.x : threadIdx.x & (lanes - 1);
  const Team<ALL> team{lanes, lds};
  Columns<T, PER, NP> cols;
  cols.find(a, lane, lanes, gamma);
  T mine[NP][PER];
#pragma unroll
  for (int j = 0; j < NP; ++j)
#pragma unroll
    for (int e = 0; e < PER; ++e) mine[j][e] = 0;
  const int64_t teams = int64_t(gridDim.x) * (THREADS / lanes);
  for (int64_t row = int64_t(blockIdx.x) * (THREADS / lanes) + threadIdx.x / lanes; row < a.n_rows; row += teams) {
    const int64_t at = row * a.dim;
    T h[NP][PER], g[NP][PER], more[NP][PER];
    load_row(h, h_rows + at, cols.col);
    load_row(g, grad_out + at, cols.col);
    if (grad_sum != nullptr) load_row(more, grad_sum + at, cols.col);
    double v[2][NP], total[2][NP];
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      double q = 0, p = 0;
#pragma unroll
      for (int e = 0; e < PER; ++e) {
        const double he = h[j][e];
        q = fma(he, he, q);
        p = fma(he, double(g[j][e]) * double(cols.gamma[j][e]), p);
      }
      v[0][j] = cols.col[j] >= 0 ? q * cols.share[j] : 0.0;
      v[1][j] = cols.col[j] >= 0 ? p : 0.0;
      total[0][j] = total[1][j] = 0;
    }
    together<ALL, NP, 2>(team, a, cols.seg, v, total);
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      const double r = inverse_root(total[0][j], a.eps);
      const double c = total[1][j] * r * r * cols.share[j];
#pragma unroll
      for (int e = 0; e < PER; ++e) {
        const double he = h[j][e], ge = g[j][e];
        mine[j][e] += static_cast<T>(ge * (he * r));
        h[j][e] = static_cast<T>(r * (ge * double(cols.gamma[j][e]) - he * c));
        if (grad_sum != nullptr) h[j][e] += more[j][e];
      }
    }
    if (grad_x != nullptr) store_row(h, grad_x + at, cols.col);
  }
  if (grad_gamma == nullptr) return;
  if (ALL) {
    store_row(mine, part + int64_t(blockIdx.x) * a.dim, cols.col);
    return;
  }
  // the wavefront's groups of lanes, then the block's wavefronts, in order
  T* const sums = reinterpret_cast<T*>(dynamic);
  const int w = threadIdx.x >> 6;
#pragma unroll
  for (int j = 0; j < NP; ++j)
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      T s = mine[j][e];
      for (int o = lanes; o < 64; o <<= 1) s += __shfl_xor(s, o, 64);
      if ((threadIdx.x & 63) < lanes && cols.col[j] >= 0) sums[w * a.dim + cols.col[j] + e] = s;
    }
  __syncthreads();
  const bool alone = part == nullptr;
  T* const to = alone ? sums : part + int64_t(blockIdx.x) * a.dim;
  for (int c = threadIdx.x; c < a.dim; c += THREADS) {
    T s = sums[c];
    for (int q = 1; q < THREADS / 64; ++q) s += sums[q * a.dim + c];
    to[c] = s;
  }
  if (!alone) return;
  __syncthreads();
  for (int s = 0; s < a.n_segs; ++s) {
    const NormSeg& g = a.seg[s];
    const int mul = (g.end - g.off) / g.d;
    for (int u = threadIdx.x; u < mul; u += THREADS) {
      T v = 0;
      for (int m = 0; m < g.d; ++m) v += sums[g.off + u * g.d + m];
      grad_gamma[g.channel + u] = v;
    }
  }
}

// The blocks' column sums, added in order: a block takes as many whole channels
// of a segment as 64 columns hold, its wavefronts every 16th row of sums.
template <class T>
__global__ __launch_bounds__(1024) void k_norm_join(NormArgs a, int blocks, const T* __restrict__ part,
                                                    T* __restrict__ grad_gamma) {
  __shared__ double sums[16][64];
  int s = 0, b = blockIdx.x;
  for (; s < a.n_segs; ++s) {
    const int per = 64 / a.seg[s].d, mul = (a.seg[s].end - a.seg[s].off) / a.seg[s].d, n = (mul + per - 1) / per;
    if (b < n) break;
    b -= n;
  }
  const NormSeg g = a.seg[s];
  const int per = 64 / g.d, u0 = b * per, mul = (g.end - g.off) / g.d;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int c = g.off + u0 * g.d + lane;
  double v = 0;
  if (lane < per * g.d && c < g.end) {
#pragma unroll 8
    for (int q = w; q < blocks; q += 16) v += double(part[int64_t(q) * a.dim + c]);
  }
  sums[w][lane] = v;
  __syncthreads();
  if (w == 0) {
    v = 0;
#pragma unroll
    for (int q = 0; q < 16; ++q) v += sums[q][lane];
    sums[0][lane] = v;
  }
  __syncthreads();
  if (threadIdx.x < per && u0 + int(threadIdx.x) < mul) {
    v = 0;
    for (int m = 0; m < g.d; ++m) v += sums[0][threadIdx.x * g.d + m];
    grad_gamma[g.channel + u0 + threadIdx.x] = static_cast<T>(v);
  }
}

// ---------------------------------------------------------------- from 8 bits
// Memory bound: five bytes an element.
template <int PER, int NP, int THREADS>
__global__ __launch_bounds__(THREADS) void k_unpack8(NormArgs a, const uint8_t* __restrict__ codes,
                                                     const float* __restrict__ scales, float* __restrict__ x) {
  const int lanes = a.lanes, lane = threadIdx.x & (lanes - 1);
  Columns<float, PER, NP> cols;
  cols.find(a, lane, lanes, nullptr);
  const int64_t teams = int64_t(gridDim.x) * (THREADS / lanes);
  for (int64_t row = int64_t(blockIdx.x) * (THREADS / lanes) + threadIdx.x / lanes; row < a.n_rows; row += teams) {
    const int64_t at = row * a.dim;
    float v[NP][PER];
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      const bool in = cols.col[j] >= 0;
      const float scale = scales[row * a.n_segs + cols.seg[j]];
      int code = 0;
      if constexpr (PER == 4)
        code = in ? *reinterpret_cast<const int*>(codes + at + cols.col[j]) : 0;
      else
        code = in ? codes[at + cols.col[j]] : 0;
      v[j][0] = __builtin_amdgcn_cvt_f32_fp8(code, 0) * scale;
      if constexpr (PER == 4) {
        v[j][1] = __builtin_amdgcn_cvt_f32_fp8(code, 1) * scale;
        v[j][2] = __builtin_amdgcn_cvt_f32_fp8(code, 2) * scale;
        v[j][3] = __builtin_amdgcn_cvt_f32_fp8(code, 3) * scale;
      }
    }
    store_row(v, x + at, cols.col);
  }
}

// -------------------------------------------------------------------- host
// Whether rows are taken in pieces of 16 bytes.
template <class T>
bool in_pieces(const NormArgs& a) {
  constexpr int per = 16 / sizeof(T);
  bool ok = a.dim % per == 0;
  for (int s = 0; s < a.n_segs; ++s) ok = ok && a.seg[s].off % per == 0;
  return ok;
}

// How a row's pieces are spread: lanes of a wavefront (a power of two), or a
// block's threads, and pieces a lane.
struct Spread {
  int lanes, np;
  bool all;
};
Spread spread(int pieces) {
  if (pieces <= 64) {
    int l = 1;
    while (l < pieces) l *= 2;
    return {l, 1, false};
  }
  if (pieces <= 256) return {64, pieces <= 128 ? 2 : 4, false};
  if (pieces <= 2048) return {256, pieces <= 1024 ? 4 : 8, true};
  return {1024, 8, true};
}

int64_t blocks_of(const Spread& sp, int64_t n_rows, int most) {
  const int64_t per = sp.all ? 1 : kThreads / sp.lanes;
  const int64_t b = (n_rows + per - 1) / per;
  return b < 1 ? 1 : (b > most ? most : b);
}

// f(pieces of 16 bytes?, NP, ALL, THREADS) as constants
template <class T, class F>
hipError_t dispatch(bool vec, const Spread& sp, F&& f) {
  using std::integral_constant;
  auto at = [&](auto per) -> hipError_t {
    auto go = [&](auto np, auto all, auto threads) { return f(per, np, all, threads); };
    using I = integral_constant<int, 256>;
    if (!sp.all) {
      if (sp.np == 1) return go(integral_constant<int, 1>{}, std::false_type{}, I{});
      if (sp.np == 2) return go(integral_constant<int, 2>{}, std::false_type{}, I{});
      return go(integral_constant<int, 4>{}, std::false_type{}, I{});
    }
    if (sp.lanes == 1024) return go(integral_constant<int, 8>{}, std::true_type{}, integral_constant<int, 1024>{});
    if (sp.np == 4) return go(integral_constant<int, 4>{}, std::true_type{}, I{});
    return go(integral_constant<int, 8>{}, std::true_type{}, I{});
  };
  if (vec) return at(integral_constant<int, 16 / sizeof(T)>{});
  return at(integral_constant<int, 1>{});
}

bool all_aligned(std::initializer_list<const void*> ptrs) {
  for (const void* p : ptrs)
    if (!aligned16(p)) return false;
  return true;
}

template <class T, bool NORM>
hipError_t forward(NormArgs a, const T* x, const T* residual, const T* gamma, T* sum, T* out, uint8_t* codes,
                   float* scales, hipStream_t s) {
  const bool vec = in_pieces<T>(a) && all_aligned({x, residual, sum, out}) &&
                   reinterpret_cast<uintptr_t>(codes) % 4 == 0;
  const Spread sp = spread(vec ? a.dim * int(sizeof(T)) / 16 : a.dim);
  a.lanes = sp.lanes;
  return dispatch<T>(vec, sp, [&](auto per, auto np, auto all, auto threads) {
    hipLaunchKernelGGL((k_norm<T, per.value, np.value, all.value, threads.value, NORM>),
                       dim3(static_cast<unsigned>(blocks_of(sp, a.n_rows, kMostBlocks))), dim3(threads.value), 0, s, a,
                       x, residual, gamma, sum, out, codes, scales);
    return hipGetLastError();
  });
}

template <class T>
hipError_t backward(NormArgs a, const T* h, const T* gamma, const T* grad_out, const T* grad_sum, T* grad_x,
                    T* grad_gamma, T* part, hipStream_t s) {
  const bool vec = in_pieces<T>(a) && all_aligned({h, grad_out, grad_sum, grad_x});
  const Spread sp = spread(vec ? a.dim * int(sizeof(T)) / 16 : a.dim);
  a.lanes = sp.lanes;
  const int64_t blocks = blocks_of(sp, a.n_rows, kMostGradBlocks);
  if (blocks == 1 && !sp.all) part = nullptr;
  const hipError_t he = dispatch<T>(vec, sp, [&](auto per, auto np, auto all, auto threads) {
    const size_t lds = all.value || grad_gamma == nullptr ? 0 : sizeof(T) * (threads.value / 64) * a.dim;
    hipLaunchKernelGGL((k_norm_grad<T, per.value, np.value, all.value, threads.value>),
                       dim3(static_cast<unsigned>(blocks)), dim3(threads.value), lds, s, a, h, gamma, grad_out,
                       grad_sum, grad_x, grad_gamma, part);
    return hipGetLastError();
  });
  if (he != hipSuccess || grad_gamma == nullptr || part == nullptr) return he;
  int join = 0;
  for (int i = 0; i < a.n_segs; ++i) {
    const int per = 64 / a.seg[i].d, mul = (a.seg[i].end - a.seg[i].off) / a.seg[i].d;
    join += (mul + per - 1) / per;
  }
  hipLaunchKernelGGL(k_norm_join<T>, dim3(static_cast<unsigned>(join)), dim3(1024), 0, s, a,
                     static_cast<int>(blocks), part, grad_gamma);
  return hipGetLastError();
}

}  // namespace

size_t norm_workspace(bool f64, const NormArgs& a, int64_t n_rows) {
  // rows of column sums for the most blocks that any spread of the row takes: one team a block at least
  const int64_t blocks = n_rows < 1 ? 1 : (n_rows > kMostGradBlocks ? kMostGradBlocks : n_rows);
  return align_up((f64 ? 8 : 4) * static_cast<size_t>(blocks) * a.dim);
}

hipError_t launch_norm_forward(bool f64, const NormArgs& a, const void* x, const void* residual, const void* gamma,
                               void* sum, void* out, uint8_t* codes, float* scales, hipStream_t s) {
  if (f64)
    return forward<double, true>(a, static_cast<const double*>(x), static_cast<const double*>(residual),
                                 static_cast<const double*>(gamma), static_cast<double*>(sum),
                                 static_cast<double*>(out), nullptr, nullptr, s);
  return forward<float, true>(a, static_cast<const float*>(x), static_cast<const float*>(residual),
                              static_cast<const float*>(gamma), static_cast<float*>(sum), static_cast<float*>(out),
                              codes, scales, s);
}

hipError_t launch_norm_backward(bool f64, const NormArgs& a, const void* h, const void* gamma, const void* grad_out,
                                const void* grad_sum, void* grad_x, void* grad_gamma, void* ws, hipStream_t s) {
  if (f64)
    return backward<double>(a, static_cast<const double*>(h), static_cast<const double*>(gamma),
                            static_cast<const double*>(grad_out), static_cast<const double*>(grad_sum),
                            static_cast<double*>(grad_x), static_cast<double*>(grad_gamma), static_cast<double*>(ws),
                            s);
  return backward<float>(a, static_cast<const float*>(h), static_cast<const float*>(gamma),
                         static_cast<const float*>(grad_out), static_cast<const float*>(grad_sum),
                         static_cast<float*>(grad_x), static_cast<float*>(grad_gamma), static_cast<float*>(ws), s);
}

hipError_t launch_pack8(const NormArgs& a, const float* x, uint8_t* codes, float* scales, hipStream_t s) {
  return forward<float, false>(a, x, nullptr, nullptr, nullptr, nullptr, codes, scales, s);
}

hipError_t launch_unpack8(NormArgs a, const uint8_t* codes, const float* scales, float* x, hipStream_t s) {
  const bool vec = in_pieces<float>(a) && aligned16(x) && reinterpret_cast<uintptr_t>(codes) % 4 == 0;
  const Spread sp = spread(vec ? a.dim / 4 : a.dim);
  a.lanes = sp.lanes;
  return dispatch<float>(vec, sp, [&](auto per, auto np, auto, auto threads) {
    hipLaunchKernelGGL((k_unpack8<per.value, np.value, threads.value>),
                       dim3(static_cast<unsigned>(blocks_of(sp, a.n_rows, 2 * kMostBlocks))), dim3(threads.value), 0, s,
                       a, codes, scales, x);
    return hipGetLastError();
  });
}

}  // namespace tpconv
