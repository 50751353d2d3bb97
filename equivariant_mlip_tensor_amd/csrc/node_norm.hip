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
// not start at a multiple of one; the gradient: 128) are held by 1 to 64 lanes
// of a wavefront, and longer ones by a block.
// Sums, and the factors formed of them, run in 64 bits for both types, so that
// squares of any fp32 value fit.
// 28000 fp32 rows of 1024 with a residual: 78 us (459 MB, 5.9 TB/s); the gradient
// 111 us (459 MB, 4.1 TB/s), joining grad_gamma's parts 10; into 8 bits 38 us (143
// MB, latency of the maxima), back 24 us (6.0 TB/s).  4096 rows of 512 with codes:
// 12 us.  16 fp64 rows of 16: 2.5 and 4.4 us (latency).
#include <hip/hip_runtime.h>

#include "node_device.hpp"
#include "node_internal.hpp"

namespace tpconv {
namespace {

constexpr int kThreads = 256;
constexpr int kMostBlocks = 1024;      // 4 blocks for each CU
constexpr int kMostGradBlocks = 2048;

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

// A column's place in a row (bytes) that the compiler takes for new: the row's
// start stays in scalar registers and the place beside it, where pointers of
// every piece of every array, carried from row to row, took 64 registers (and
// gamma's pieces, loaded ahead of the loop, spilled).
template <class T>
__device__ __forceinline__ uint32_t place_of(int col) {
  uint32_t at = static_cast<uint32_t>(col) * sizeof(T);
  asm volatile("" : "+v"(at));
  return at;
}

template <class T, int PER, int NP>
__device__ __forceinline__ void load_row(T (&v)[NP][PER], const T* row, const int (&col)[NP]) {
  struct alignas(PER * sizeof(T)) Piece {
    T v[PER];
  };
#pragma unroll
  for (int j = 0; j < NP; ++j) {
    Piece p = {};
    if (col[j] >= 0) p = *reinterpret_cast<const Piece*>(reinterpret_cast<const char*>(row) + place_of<T>(col[j]));
#pragma unroll
    for (int e = 0; e < PER; ++e) v[j][e] = p.v[e];
  }
}

// A piece of a row in LDS.
template <class T, int PER>
__device__ __forceinline__ void load_piece(T (&v)[PER], const T* row, int col) {
  struct alignas(PER * sizeof(T)) Piece {
    T v[PER];
  };
  const Piece p = *reinterpret_cast<const Piece*>(reinterpret_cast<const char*>(row) + place_of<T>(col < 0 ? 0 : col));
#pragma unroll
  for (int e = 0; e < PER; ++e) v[e] = p.v[e];
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
      *reinterpret_cast<Piece*>(reinterpret_cast<char*>(row) + place_of<T>(col[j])) = p;
    }
}

// Sums over the 16 lanes of a row of lanes by moves on the vector units: with
// the lane next to it, the pair, the four and the eight beside it.
template <int CTRL>
__device__ __forceinline__ double moved(double v) {
  return __hiloint2double(__builtin_amdgcn_update_dpp(0, __double2hiint(v), CTRL, 0xF, 0xF, true),
                          __builtin_amdgcn_update_dpp(0, __double2loint(v), CTRL, 0xF, 0xF, true));
}
template <int CTRL>
__device__ __forceinline__ uint32_t moved(uint32_t v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xF, 0xF, true);
}

// Reductions over a row's lanes; every lane gets the result.  ALL: the row is
// a block's (sums by wavefront pass through LDS, added in order), else `lanes`
// neighbours' of a wavefront.
template <bool ALL, bool FULL>  // FULL: of whole wavefronts
struct Team {
  int lanes;
  double* lds;  // ALL: two sets of 32 segments' sums of each wavefront

  template <class V, class F>
  __device__ __forceinline__ V wave(V v, F&& f) const {
    if constexpr (FULL) {
      v = f(v, moved<0xB1>(v));
      v = f(v, moved<0x4E>(v));
      v = f(v, moved<0x141>(v));
      v = f(v, moved<0x140>(v));
      v = f(v, __shfl_xor(v, 16, 64));
      v = f(v, __shfl_xor(v, 32, 64));
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
__device__ __forceinline__ double inverse_root(double ms, double eps) { return rsqrt(ms + eps); }

__device__ __forceinline__ uint32_t max_bits(uint32_t a, uint32_t b) { return a > b ? a : b; }

// Sums over what is normalised together of up to N values of each piece; for
// each piece, its segment's or row's sums.
template <bool ALL, int NP, int N>
__device__ __forceinline__ void together(const Team<ALL, (NP > 1)>& team, const NormArgs& a, const int (&seg)[NP],
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
__device__ __forceinline__ void write_codes(const Team<ALL, (NP > 1)>& team, const NormArgs& a,
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

// The first row of this thread's lanes and, with more than one piece a lane
// (a wavefront's or block's lanes all have it), the same for all of them.
template <int NP>
__device__ __forceinline__ int first_row(int rows_of_block, int lanes) {
  const int row = static_cast<int>(blockIdx.x) * rows_of_block + static_cast<int>(threadIdx.x) / lanes;
  return NP > 1 ? __builtin_amdgcn_readfirstlane(row) : row;
}

// ------------------------------------------------------------------ forward
// NORM: y is the norm of h; without it, h itself (rows into 8 bits alone).
template <class T, int PER, int NP, bool ALL, int THREADS, bool NORM>
__global__ __launch_bounds__(THREADS) void k_norm(NormArgs a, const T* x, const T* residual, const T* gamma, T* sum,
                                                  T* out, uint8_t* codes, float* scales) {
  __shared__ double lds[ALL ? kMaxNormSegs * (THREADS / 64) : 1];
  const int lanes = ALL ? THREADS : (NP > 1 ? 64 : a.lanes);
  const int lane = ALL ? threadIdx.x : threadIdx.x & (lanes - 1);
  const Team<ALL, (NP > 1)> team{lanes, lds};
  Columns<T, PER, NP> cols;
  cols.find(a, lane, lanes, gamma);
  const int teams = static_cast<int>(gridDim.x) * (THREADS / lanes);
  for (int64_t row = first_row<NP>(THREADS / lanes, lanes); row < a.n_rows; row += teams) {
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
        for (int e = 0; e < PER; ++e) h[j][e] = static_cast<T>(double(h[j][e]) * r * double(cols.gamma[j][e]));
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
  extern __shared__ char dynamic[];  // gamma by column (in registers it takes a fifth of them); then column sums,
                                     // where wavefronts hold rows
  const int lanes = ALL ? THREADS : (NP > 1 ? 64 : a.lanes);
  const int lane = ALL ? threadIdx.x : threadIdx.x & (lanes - 1);
  const Team<ALL, (NP > 1)> team{lanes, lds};
  Columns<T, PER, NP> cols;
  cols.find(a, lane, lanes, nullptr);
  T* const weight = reinterpret_cast<T*>(dynamic);
  for (int s = 0; s < a.n_segs; ++s)
    for (int c = a.seg[s].off + threadIdx.x; c < a.seg[s].end; c += THREADS)
      weight[c] = gamma != nullptr ? gamma[a.seg[s].channel + (c - a.seg[s].off) / a.seg[s].d] : T(1);
  __syncthreads();
  T mine[NP][PER];
#pragma unroll
  for (int j = 0; j < NP; ++j)
#pragma unroll
    for (int e = 0; e < PER; ++e) mine[j][e] = 0;
  const int teams = static_cast<int>(gridDim.x) * (THREADS / lanes);
  for (int64_t row = first_row<NP>(THREADS / lanes, lanes); row < a.n_rows; row += teams) {
    const int64_t at = row * a.dim;
    T h[NP][PER], g[NP][PER], more[NP][PER];
    load_row(h, h_rows + at, cols.col);
    load_row(g, grad_out + at, cols.col);
    double v[2][NP], total[2][NP];
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      double q = 0, p = 0;
      T gamma[PER];
      load_piece(gamma, weight, cols.col[j]);
#pragma unroll
      for (int e = 0; e < PER; ++e) {
        const double he = h[j][e];
        q = fma(he, he, q);
        p = fma(he, double(g[j][e]) * double(gamma[e]), p);
      }
      v[0][j] = cols.col[j] >= 0 ? q * cols.share[j] : 0.0;
      v[1][j] = cols.col[j] >= 0 ? p : 0.0;
      total[0][j] = total[1][j] = 0;
    }
    together<ALL, NP, 2>(team, a, cols.seg, v, total);
    if (grad_sum != nullptr) load_row(more, grad_sum + at, cols.col);
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      const double r = inverse_root(total[0][j], a.eps);
      const double pull = total[1][j] * r * cols.share[j];
      T gamma[PER];
      load_piece(gamma, weight, cols.col[j]);
#pragma unroll
      for (int e = 0; e < PER; ++e) {
        const double ge = g[j][e], u = double(h[j][e]) * r;
        mine[j][e] = fma(g[j][e], static_cast<T>(u), mine[j][e]);
        // rounded once: in a segment of one column the difference is what eps leaves of its terms
        const double grad = r * fma(-u, pull, ge * double(gamma[e]));
        h[j][e] = static_cast<T>(grad_sum != nullptr ? grad + double(more[j][e]) : grad);
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
  __syncthreads();  // gamma is read
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
// of a segment as 16 columns hold, a row of 16 lanes every 64th row of sums.
template <class T>
__global__ __launch_bounds__(1024) void k_norm_join(NormArgs a, int blocks, const T* __restrict__ part,
                                                    T* __restrict__ grad_gamma) {
  __shared__ double sums[64][16];
  int s = 0, b = blockIdx.x;
  for (; s < a.n_segs; ++s) {
    const int per = 16 / a.seg[s].d, mul = (a.seg[s].end - a.seg[s].off) / a.seg[s].d, n = (mul + per - 1) / per;
    if (b < n) break;
    b -= n;
  }
  const NormSeg g = a.seg[s];
  const int per = 16 / g.d, u0 = b * per, mul = (g.end - g.off) / g.d;
  const int lane = threadIdx.x & 15, w = threadIdx.x >> 4;
  const int c = g.off + u0 * g.d + lane;
  double v = 0;
  if (lane < per * g.d && c < g.end) {
#pragma unroll 8
    for (int q = w; q < blocks; q += 64) v += double(part[int64_t(q) * a.dim + c]);
  }
  sums[w][lane] = v;
  __syncthreads();
  if (w < 4) {  // 4 rows of lanes take 16 sums each
    v = 0;
#pragma unroll
    for (int q = 0; q < 16; ++q) v += sums[16 * w + q][lane];
    v += __shfl_xor(v, 16, 64);
    v += __shfl_xor(v, 32, 64);
    sums[w][lane] = v;
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
  const int teams = static_cast<int>(gridDim.x) * (THREADS / lanes);
  for (int64_t row = first_row<NP>(THREADS / lanes, lanes); row < a.n_rows; row += teams) {
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
// block's threads, and pieces a lane (two, as far as 1024 threads reach).
struct Spread {
  int lanes, np;
  bool all;
};
Spread spread(int pieces, bool grad) {
  if (pieces <= 64) {
    int l = 1;
    while (l < pieces) l *= 2;
    return {l, 1, false};
  }
  if (pieces <= 128) return {64, 2, false};
  // the gradient holds three rows: a wavefront's registers do not (28000 rows of 1024: 170 us, 112 by two wavefronts;
  // the norm itself 78)
  if (pieces <= 256 && !grad) return {64, 4, false};
  int threads = 128;
  while (threads < 1024 && 2 * threads < pieces) threads *= 2;
  return {threads, pieces <= 2048 ? 2 : (pieces <= 4096 ? 4 : 8), true};
}

int64_t blocks_of(const Spread& sp, int64_t n_rows, int most) {
  const int64_t per = sp.all ? 1 : kThreads / sp.lanes;
  const int64_t b = (n_rows + per - 1) / per;
  return b < 1 ? 1 : (b > most ? most : b);
}

// f(elements of a piece, NP, ALL, THREADS) as constants
template <class T, bool GRAD, class F>
hipError_t dispatch(bool vec, const Spread& sp, F&& f) {
  auto at = [&](auto per) -> hipError_t {
    constexpr int kMost = TPCONV_MAX_NORM_DIM / decltype(per)::value;  // pieces
    auto go = [&](auto np, auto all, auto threads) { return f(per, np, all, threads); };
    using std::integral_constant;
    using N2 = integral_constant<int, 2>;
    using N4 = integral_constant<int, 4>;
    using Wave = std::false_type;
    using Block = std::true_type;
    using Quarter = integral_constant<int, kThreads>;
    if (!sp.all) {
      if (sp.np == 1) return go(integral_constant<int, 1>{}, Wave{}, Quarter{});
      if constexpr (!GRAD)
        if (sp.np == 4) return go(N4{}, Wave{}, Quarter{});
      return go(N2{}, Wave{}, Quarter{});
    }
    if constexpr (kMost > 4096)
      if (sp.np == 8) return go(integral_constant<int, 8>{}, Block{}, integral_constant<int, 1024>{});
    if constexpr (kMost > 2048)
      if (sp.np == 4) return go(N4{}, Block{}, integral_constant<int, 1024>{});
    if constexpr (GRAD)
      if (sp.lanes == 128) return go(N2{}, Block{}, integral_constant<int, 128>{});
    if (sp.lanes == 256) return go(N2{}, Block{}, Quarter{});
    if (sp.lanes == 512) return go(N2{}, Block{}, integral_constant<int, 512>{});
    return go(N2{}, Block{}, integral_constant<int, 1024>{});
  };
  if (vec) return at(std::integral_constant<int, 16 / sizeof(T)>{});
  return at(std::integral_constant<int, 1>{});
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
  const Spread sp = spread(vec ? a.dim * int(sizeof(T)) / 16 : a.dim, false);
  a.lanes = sp.lanes;
  return dispatch<T, false>(vec, sp, [&](auto per, auto np, auto all, auto threads) {
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
  const Spread sp = spread(vec ? a.dim * int(sizeof(T)) / 16 : a.dim, true);
  a.lanes = sp.lanes;
  const int64_t blocks = blocks_of(sp, a.n_rows, kMostGradBlocks);
  if (blocks == 1 && !sp.all) part = nullptr;
  const hipError_t he = dispatch<T, true>(vec, sp, [&](auto per, auto np, auto all, auto threads) {
    const size_t lds = sizeof(T) * (all.value ? 1 : threads.value / 64) * a.dim;
    hipLaunchKernelGGL((k_norm_grad<T, per.value, np.value, all.value, threads.value>),
                       dim3(static_cast<unsigned>(blocks)), dim3(threads.value), lds, s, a, h, gamma, grad_out,
                       grad_sum, grad_x, grad_gamma, part);
    return hipGetLastError();
  });
  if (he != hipSuccess || grad_gamma == nullptr || part == nullptr) return he;
  int join = 0;
  for (int i = 0; i < a.n_segs; ++i) {
    const int per = 16 / a.seg[i].d, mul = (a.seg[i].end - a.seg[i].off) / a.seg[i].d;
    join += (mul + per - 1) / per;
  }
  hipLaunchKernelGGL(k_norm_join<T>, dim3(static_cast<unsigned>(join)), dim3(1024), 0, s, a,
                     static_cast<int>(blocks), part, grad_gamma);
  return hipGetLastError();
}

}  // namespace

size_t norm_workspace(bool f64, const NormArgs& a, int64_t n_rows) {
  // none where one block has all rows, whichever way they are spread (by single elements over the most lanes); else rows
  // of column sums for the most blocks: a row each
  const Spread sp = spread(a.dim, true);
  if (!sp.all && n_rows <= kThreads / sp.lanes) return 0;
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
  const Spread sp = spread(vec ? a.dim / 4 : a.dim, false);
  a.lanes = sp.lanes;
  return dispatch<float, false>(vec, sp, [&](auto per, auto np, auto, auto threads) {
    hipLaunchKernelGGL((k_unpack8<per.value, np.value, threads.value>),
                       dim3(static_cast<unsigned>(blocks_of(sp, a.n_rows, 2 * kMostBlocks))), dim3(threads.value), 0, s,
                       a, codes, scales, x);
    return hipGetLastError();
  });
}

}  // namespace tpconv
