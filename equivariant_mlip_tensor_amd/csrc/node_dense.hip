// node_dense.hip -- equivariant products of irreps rows with one set of maps,
// and what stands around them: the linear map with bias, activation and
// residual, the gated feed-forward product, and their gradients.
//   u_s[i][v][m] = sum_u M_s[u][v] x_s[i][u][m]           (a map of segment s)
//   z[i][c]      = sum_u Wg[u][c] x_0e[i][u] + b[c]       (gated: its gates)
//   linear: out = residual + a(u + bias);  gated: out[s][v][m] = a(z[c(s, v)]) u_s[v][m]
// A map's 2l+1 components all see the same matrix, so it is a matrix product
// whose rows are (component, atom); it runs on the matrix cores
// (v_mfma_f32_16x16x4f32, v_mfma_f64_16x16x4f64: the library's data types).
// A matrix instruction's 16 rows are 16 atoms at one component, so a lane ends
// up with all 2l+1 components of its (atom, channel) pairs, and with their gate:
// activation, product, their derivatives and the gate gradient's sum over
// components need no exchange between lanes.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "node_device.hpp"
#include "node_internal.hpp"

namespace tpconv {
namespace {

// -------------------------------------------------------------- activations
template <class T>
__device__ __forceinline__ T normal_below(T z) {  // Phi(z)
  return T(0.5) * erfc(z * T(-0.70710678118654752440));
}

template <class T>
__device__ __forceinline__ T activated(int kind, T z) {
  switch (kind) {
    case TPCONV_ACT_SILU: return z / (T(1) + exp(-z));
    case TPCONV_ACT_SIGMOID: return T(1) / (T(1) + exp(-z));
    case TPCONV_ACT_TANH: return tanh(z);
    case TPCONV_ACT_GELU: return z * normal_below(z);
    default: return z;
  }
}

// The activation and its slope, the slope in forms that do not cancel where it
// saturates: 1 - s as the sigmoid of -z, 1 - tanh^2 by exponentials.
template <class T>
__device__ __forceinline__ void activated_with_slope(int kind, T z, T& value, T& slope) {
  switch (kind) {
    case TPCONV_ACT_SILU: {
      const T s = T(1) / (T(1) + exp(-z)), t = T(1) / (T(1) + exp(z));
      value = z / (T(1) + exp(-z));
      slope = s + z * s * t;
      return;
    }
    case TPCONV_ACT_SIGMOID: {
      value = T(1) / (T(1) + exp(-z));
      slope = value / (T(1) + exp(z));
      return;
    }
    case TPCONV_ACT_TANH: {
      value = tanh(z);
      const T e = exp(T(-2) * fabs(z)), q = T(1) / (T(1) + e);
      slope = T(4) * e * q * q;
      return;
    }
    case TPCONV_ACT_GELU: {
      const T below = normal_below(z);
      value = z * below;
      slope = below + z * exp(T(-0.5) * z * z) * T(0.39894228040143267794);
      return;
    }
    default:
      value = z;
      slope = T(1);
  }
}

// ------------------------------------------------------------------ staging
// Rows of a segment on their way to LDS: `len` elements of each of `rows` rows,
// element c of row s at lds[s * pitch + c], in pieces of PER, kBatch of a
// thread's in flight.
constexpr int kBatch = 8;

// (row, piece) of number q of rows of `pieces` pieces; q stays below 2^16, so
// the rounded product is exact
__device__ __forceinline__ void split(int q, int pieces, float inv, int& row, int& piece) {
  row = static_cast<int>((static_cast<float>(q) + 0.5f) * inv);
  piece = q - row * pieces;
}

template <class T, int PER>
__device__ __forceinline__ void stage_rows(T* lds, int pitch, const T* from, int64_t ld, int rows, int len, int tid,
                                           int threads) {
  struct alignas(PER * sizeof(T)) Piece {
    T v[PER];
  };
  const int pieces = len / PER, total = rows * pieces;
  const float inv = 1.0f / static_cast<float>(pieces);
  for (int q0 = tid; q0 < total; q0 += kBatch * threads) {
    Piece p[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      int s, c;
      split(min(q0 + j * threads, total - 1), pieces, inv, s, c);
      p[j] = *reinterpret_cast<const Piece*>(from + s * ld + c * PER);
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      int s, c;
      split(min(q0 + j * threads, total - 1), pieces, inv, s, c);
      if (q0 + j * threads < total) *reinterpret_cast<Piece*>(lds + s * pitch + c * PER) = p[j];
    }
  }
}

// The same from 8 bits: codes of a row and segment times its scale.
template <int PER>
__device__ __forceinline__ void stage_codes(float* lds, int pitch, const uint8_t* from, int64_t ld,
                                            const float* scales, int64_t ld_scales, int rows, int len, int tid,
                                            int threads) {
  const int pieces = len / PER, total = rows * pieces;
  const float inv = 1.0f / static_cast<float>(pieces);
  for (int q0 = tid; q0 < total; q0 += kBatch * threads) {
    int code[kBatch];
    float scale[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      int s, c;
      split(min(q0 + j * threads, total - 1), pieces, inv, s, c);
      const uint8_t* const at = from + s * ld + c * PER;
      if constexpr (PER == 4)
        code[j] = *reinterpret_cast<const int*>(at);
      else
        code[j] = *at;
      scale[j] = scales[s * ld_scales];
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      int s, c;
      split(min(q0 + j * threads, total - 1), pieces, inv, s, c);
      if (q0 + j * threads >= total) continue;
      float* const to = lds + s * pitch + c * PER;
      to[0] = __builtin_amdgcn_cvt_f32_fp8(code[j], 0) * scale[j];
      if constexpr (PER == 4) {
        to[1] = __builtin_amdgcn_cvt_f32_fp8(code[j], 1) * scale[j];
        to[2] = __builtin_amdgcn_cvt_f32_fp8(code[j], 2) * scale[j];
        to[3] = __builtin_amdgcn_cvt_f32_fp8(code[j], 3) * scale[j];
      }
    }
  }
}

// A segment of rows to stage from.
struct RowSource {
  const void* rows;      // T, or codes where `scales`
  const float* scales;   // of the segment in row 0
  int64_t ld, ld_scales; // elements of a row; scales of a row
  int32_t off;           // the segment's first column
  int32_t K;             // its channels
  int32_t packed;        // pieces of 16 bytes (codes: of 4)
};

// `count` channels of d components from channel k0 on, of rows base ..
template <class T>
__device__ __forceinline__ void stage_source(const RowSource& a, T* lds, int pitch, int64_t base, int rows, int k0,
                                             int count, int d, int tid, int threads) {
  const int64_t at = base * a.ld + a.off + k0 * d;
  const int len = count * d;
  if (sizeof(T) == 4 && a.scales != nullptr) {
    const uint8_t* const from = static_cast<const uint8_t*>(a.rows) + at;
    float* const to = reinterpret_cast<float*>(lds);
    if (a.packed)
      stage_codes<4>(to, pitch, from, a.ld, a.scales + base * a.ld_scales, a.ld_scales, rows, len, tid, threads);
    else
      stage_codes<1>(to, pitch, from, a.ld, a.scales + base * a.ld_scales, a.ld_scales, rows, len, tid, threads);
    return;
  }
  const T* const from = static_cast<const T*>(a.rows) + at;
  if (a.packed)
    stage_rows<T, 16 / sizeof(T)>(lds, pitch, from, a.ld, rows, len, tid, threads);
  else
    stage_rows<T, 1>(lds, pitch, from, a.ld, rows, len, tid, threads);
}

// ------------------------------------------------------------------- products
// A block takes a tile of atoms, one map and up to 64 (fp64: 32) of its output
// channels, 16 to a wavefront.  The atoms' segment goes to LDS as it lies in
// memory; a row's pitch is 4 more (fp64: 2) than a multiple of 64 (32) banks, so
// 16 atoms times 4 channels fall into as many banks, whatever 2l+1 (it is odd).
// The weights go straight to registers.  Results pass through LDS on their way
// out, so that rows are written (and a residual or grad_out is read) in whole
// pieces.
enum Mode { kLinear, kGated, kLinearGrad, kGatedGrad, kTransposed };

constexpr int atoms_of(int d) { return d == 1 ? 64 : (d == 3 ? 32 : 16); }

// One product's operands: rows and weights W[k * ldw + n], or, transposed,
// W[n * ldw + k].
struct Term {
  RowSource src;
  const void* weights;
  int32_t ldw;
  int32_t transposed_packed;  // transposed: 16-byte pieces along k
};

struct DenseJob {
  Term main;       // components d
  Term gate;       // kGated, kGatedGrad: the gates' (rows of 0e); kTransposed: the second term of 0e, K = 0 without
  int32_t d, N;
  int32_t out_off; // first column in a row of out (kLinearGrad: of dz)
  int32_t g_off;   // first column in a row of grad_out
  int32_t bias;    // first bias of the job, -1: none
  int32_t gate0;   // first gate
  int32_t act;
  int32_t packed_out, packed_g;
  int32_t first;   // first share (a block of output channels) of this job
};

struct DenseArgs {
  int64_t n_rows;
  int64_t ld_out, ld_g, n_gates;
  void* out;
  const void* extra;  // kLinear: residual, kLinearGrad, kGatedGrad: grad_out
  const void* bias;
  void* dz;           // kGatedGrad: [n_rows][n_gates]
  int64_t groups;     // of atoms, a block's
  int32_t group;      // atoms of one: 16, 32 or 64
  int32_t n_jobs, shares, waves;
  int64_t block0;
  DenseJob job[kMaxMaps];
};

// acc[t][m] += rows of tile t, component m
template <class T, int D, int KS, bool ADJ, int MT>
__device__ __forceinline__ void accumulate(const Term& t, T* lds, int64_t base, int rows, int col,
                                           typename Mfma<T>::Acc (&acc)[MT][D]) {
  constexpr int CH = 4 * KS, P = CH * D + 16 / int(sizeof(T));
  const int tid = threadIdx.x, lane = tid & 63, i16 = lane & 15, g4 = lane >> 4;
  const T* const W = static_cast<const T*>(t.weights);
  for (int k0 = 0; k0 < t.src.K; k0 += CH) {
    const int count = min(CH, t.src.K - k0);
    T b[KS];
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const int k = 4 * s + g4;
      const int64_t kc = k0 + min(k, count - 1);
      const T v = ADJ ? W[int64_t(col) * t.ldw + kc] : W[kc * t.ldw + col];
      b[s] = k < count ? v : T(0);
    }
    __syncthreads();  // what was in LDS is read
    stage_source(t.src, lds, P, base, rows, k0, count, D, tid, blockDim.x);
    if (count < CH)  // no NaN from channels that are not there
      for (int q = tid; q < rows * (CH - count) * D; q += blockDim.x) {
        const int s = q / ((CH - count) * D);
        lds[s * P + count * D + (q - s * (CH - count) * D)] = T(0);
      }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      if (16 * i >= rows) break;
      const T* const ap = lds + (16 * i + i16) * P + g4 * D;
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int m = 0; m < D; ++m) acc[i][m] = Mfma<T>::step(ap[4 * s * D + m], b[s], acc[i][m]);
    }
  }
}

template <class T, int D, int KS, int MODE>
__device__ __forceinline__ void dense_tile(const DenseArgs& a, const DenseJob& j, int64_t base, int rows, int n0,
                                           T* lds) {
  constexpr int TA = atoms_of(D), MT = TA / 16;
  constexpr bool ADJ = MODE == kTransposed;
  using Acc = typename Mfma<T>::Acc;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, i16 = lane & 15, g4 = lane >> 4;
  const int wide = 16 * a.waves, n_here = min(wide, j.N - n0), c = 16 * w + i16;
  const int col = min(n0 + c, j.N - 1);  // past the last channel: a column that is not written

  Acc u[MT][D];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int m = 0; m < D; ++m) u[i][m] = Acc{0, 0, 0, 0};
  accumulate<T, D, KS, ADJ, MT>(j.main, lds, base, rows, col, u);

  Acc z[MT][1];
  if constexpr (MODE == kGated || MODE == kGatedGrad) {
#pragma unroll
    for (int i = 0; i < MT; ++i) z[i][0] = Acc{0, 0, 0, 0};
    accumulate<T, 1, KS, false, MT>(j.gate, lds, base, rows, j.gate0 + col, z);
  }
  if constexpr (MODE == kTransposed && D == 1)
    if (j.gate.src.K > 0) accumulate<T, 1, KS, true, MT>(j.gate, lds, base, rows, col, u);

  const int pitch = wide * D + 16 / int(sizeof(T));
  const T bias = MODE != kTransposed && j.bias >= 0 ? static_cast<const T*>(a.bias)[j.bias + col] : T(0);
  __syncthreads();
  if constexpr (MODE == kLinearGrad || MODE == kGatedGrad) {
    const RowSource g{a.extra, nullptr, a.ld_g, 0, j.g_off, j.N, j.packed_g};
    stage_source(g, lds, pitch, base, rows, n0, n_here, D, tid, blockDim.x);
    __syncthreads();
  }
  if (c < n_here) {
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      if (16 * i >= rows) break;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int s = 16 * i + Mfma<T>::row(g4, q);
        T* const at = lds + s * pitch + c * D;
        if constexpr (MODE == kGated) {
          const T gate = activated(j.act, z[i][0][q] + bias);
#pragma unroll
          for (int m = 0; m < D; ++m) at[m] = gate * u[i][m][q];
        } else if constexpr (MODE == kGatedGrad) {
          T gate, slope, dot = 0;
          activated_with_slope(j.act, z[i][0][q] + bias, gate, slope);
#pragma unroll
          for (int m = 0; m < D; ++m) {
            const T g = at[m];
            dot = fma(g, u[i][m][q], dot);
            at[m] = g * gate;
          }
          if (s < rows) static_cast<T*>(a.dz)[(base + s) * a.n_gates + j.gate0 + n0 + c] = dot * slope;
        } else if constexpr (MODE == kLinearGrad) {
          T value, slope;
          activated_with_slope(j.act, u[i][0][q] + bias, value, slope);
          at[0] *= slope;
        } else if constexpr (MODE == kLinear && D == 1) {
          at[0] = activated(j.act, u[i][0][q] + bias);
        } else {
#pragma unroll
          for (int m = 0; m < D; ++m) at[m] = u[i][m][q];
        }
      }
    }
  }
  __syncthreads();
  // out, in whole pieces where rows allow it
  T* const out = static_cast<T*>(a.out) + base * a.ld_out + j.out_off + n0 * D;
  const T* const res = MODE == kLinear && a.extra != nullptr
                           ? static_cast<const T*>(a.extra) + base * a.ld_out + j.out_off + n0 * D
                           : nullptr;
  auto write = [&](auto per) {
    constexpr int PER = decltype(per)::value;
    struct alignas(PER * sizeof(T)) Piece {
      T v[PER];
    };
    const int pieces = n_here * D / PER, total = rows * pieces;
    const float inv = 1.0f / static_cast<float>(pieces);
    for (int q0 = tid; q0 < total; q0 += kBatch * blockDim.x) {
      Piece r[kBatch] = {};
      if (MODE == kLinear && res != nullptr)
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          int s, e;
          split(min(q0 + k * int(blockDim.x), total - 1), pieces, inv, s, e);
          r[k] = *reinterpret_cast<const Piece*>(res + s * a.ld_out + e * PER);
        }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        if (q0 + k * int(blockDim.x) >= total) break;
        int s, e;
        split(q0 + k * blockDim.x, pieces, inv, s, e);
        Piece p = *reinterpret_cast<const Piece*>(lds + s * pitch + e * PER);
        if (MODE == kLinear && res != nullptr)
#pragma unroll
          for (int x = 0; x < PER; ++x) p.v[x] += r[k].v[x];
        *reinterpret_cast<Piece*>(out + s * a.ld_out + e * PER) = p;
      }
    }
  };
  if (j.packed_out)
    write(std::integral_constant<int, 16 / sizeof(T)>{});
  else
    write(std::integral_constant<int, 1>{});
}

template <class T, int KS, int MODE>
__global__ __launch_bounds__(256) void k_dense(DenseArgs a) {
  extern __shared__ char lds[];
  // a group's shares run on one XCD (blocks go round them), so its rows of 0e are fetched once there
  const int64_t block = a.block0 + blockIdx.x, eight = block / (8 * a.shares);
  const int in = static_cast<int>(block - eight * 8 * a.shares), share = in >> 3;
  const int64_t group = eight * 8 + (in & 7);
  if (group >= a.groups) return;
  int ji = 0;
  while (ji + 1 < a.n_jobs && share >= a.job[ji + 1].first) ++ji;
  const DenseJob& j = a.job[ji];
  const int n0 = (share - j.first) * 16 * a.waves;
  T* const mem = reinterpret_cast<T*>(lds);
  const int64_t from = group * a.group;
  const int atoms = static_cast<int>(min<int64_t>(a.group, a.n_rows - from));
#define TPCONV_DENSE(D)                                                                                  \
  case D:                                                                                                \
    for (int i = 0; i < atoms; i += atoms_of(D)) {                                                       \
      if (i > 0) __syncthreads();                                                                        \
      dense_tile<T, D, KS, MODE>(a, j, from + i, min(atoms - i, atoms_of(D)), n0, mem);                  \
    }                                                                                                    \
    break;
  if constexpr (MODE == kLinearGrad) {
    dense_tile<T, 1, KS, MODE>(a, j, from, atoms, n0, mem);
  } else {
    switch (j.d) {
      TPCONV_DENSE(1)
      TPCONV_DENSE(3)
      TPCONV_DENSE(5)
      TPCONV_DENSE(7)
      TPCONV_DENSE(9)
      default: break;
    }
  }
#undef TPCONV_DENSE
}

// --------------------------------------------------------- parameters' gradients
// dM[u][v] = sum over atoms and components of x[i][u][m] g[i][v][m]: a matrix
// product whose inner dimension is the (atom, component) pairs.  A block takes
// one S x S tile of a map's matrix and a run of atoms, a few of them at a time
// in LDS as they lie in memory (the pitch makes the next atom's channels go on
// where the 16 of one end, so 4 atoms times 16 channels fall into as many banks);
// its 4 wavefronts share the tile.  Runs' matrices go to the workspace and are
// added in order; one run writes the gradient itself.  The first row of tiles
// also sums its columns of g, for the bias.
struct ParamJob {
  RowSource x, g;
  int32_t d, nu, nv;
  int32_t first;        // first block
  int32_t runs;         // runs of atoms
  int64_t run;          // atoms of a run
  int64_t at;           // the job's first value in a set of parts, its matrix then its column sums
  int32_t column_sums;
  void *matrix, *sums;  // the gradients
};

struct ParamArgs {
  int64_t n_rows;
  void* part;           // NULL: one run each, written to the gradients
  int32_t n_jobs;
  int32_t block0;
  ParamJob job[kMaxMaps + 1];
};

template <class T>
constexpr int tile_side() {
  return sizeof(T) == 4 ? 64 : 32;
}
// atoms of a stage, a multiple of 4
constexpr int stage_atoms(int d) { return d == 1 ? 32 : (d == 3 ? 16 : 8); }

template <class T, int D>
__device__ __forceinline__ void param_tile(const ParamArgs& a, const ParamJob& j, int uv, int run, T* lds) {
  constexpr int S = tile_side<T>(), SA = stage_atoms(D), P = S * D + 16, H = S / 2, F = H / 16;
  using Acc = typename Mfma<T>::Acc;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, i16 = lane & 15, g4 = lane >> 4;
  const int u0 = uv / j.nv * S, v0 = uv % j.nv * S;
  const int nu = min(S, j.x.K - u0), nv = min(S, j.g.K - v0);
  const int64_t from = run * j.run, upto = min(from + j.run, a.n_rows);
  T* const xs = lds;
  T* const gs = lds + SA * P;
  // channels that are not there stay zero
  for (int q = tid; q < 2 * SA * P; q += 256) lds[q] = T(0);
  const int tu = (w >> 1) * H, tv = (w & 1) * H;
  Acc acc[F][F];
#pragma unroll
  for (int i = 0; i < F; ++i)
#pragma unroll
    for (int k = 0; k < F; ++k) acc[i][k] = Acc{0, 0, 0, 0};
  T column = 0;  // of g, where D is 1: thread t sums column t % S of every (256 / S)-th atom
  for (int64_t base = from; base < upto; base += SA) {
    const int rows = static_cast<int>(min<int64_t>(SA, upto - base));
    __syncthreads();
    stage_source(j.x, xs, P, base, rows, u0, nu, D, tid, 256);
    stage_source(j.g, gs, P, base, rows, v0, nv, D, tid, 256);
    for (int q = tid; q < (SA - rows) * P; q += 256) xs[rows * P + q] = gs[rows * P + q] = T(0);
    __syncthreads();
    if (D == 1 && j.column_sums && u0 == 0)
      for (int s = tid / S; s < rows; s += 256 / S) column += gs[s * P + tid % S];
#pragma unroll
    for (int s = 0; s < SA; s += 4) {
      if (s >= rows) break;
      const T* const xp = xs + (s + g4) * P + (tu + i16) * D;
      const T* const gp = gs + (s + g4) * P + (tv + i16) * D;
#pragma unroll
      for (int m = 0; m < D; ++m) {
        T xv[F], gv[F];
#pragma unroll
        for (int i = 0; i < F; ++i) {
          xv[i] = xp[16 * i * D + m];
          gv[i] = gp[16 * i * D + m];
        }
#pragma unroll
        for (int i = 0; i < F; ++i)
#pragma unroll
          for (int k = 0; k < F; ++k) acc[i][k] = Mfma<T>::step(xv[i], gv[k], acc[i][k]);
      }
    }
  }
  const int64_t numel = int64_t(j.x.K) * j.g.K;
  T* const to = a.part == nullptr ? static_cast<T*>(j.matrix)
                                  : static_cast<T*>(a.part) + j.at + run * (numel + (j.column_sums ? j.g.K : 0));
  if (to != nullptr)
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
      for (int k = 0; k < F; ++k)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int u = tu + 16 * i + Mfma<T>::row(g4, q), v = tv + 16 * k + i16;
          if (u < nu && v < nv) to[int64_t(u0 + u) * j.g.K + v0 + v] = acc[i][k][q];
        }
  if (D == 1 && j.column_sums && u0 == 0) {
    __syncthreads();
    lds[tid] = column;
    __syncthreads();
    T* const sums = a.part == nullptr ? static_cast<T*>(j.sums) : to + numel;
    if (tid < nv && sums != nullptr) {
      T s = lds[tid];
#pragma unroll
      for (int q = 1; q < 256 / S; ++q) s += lds[q * S + tid];
      sums[v0 + tid] = s;
    }
  }
}

template <class T>
__global__ __launch_bounds__(256) void k_param(ParamArgs a) {
  extern __shared__ char lds[];
  const int block = a.block0 + static_cast<int>(blockIdx.x);
  int ji = 0;
  while (ji + 1 < a.n_jobs && block >= a.job[ji + 1].first) ++ji;
  const ParamJob& j = a.job[ji];
  const int r = block - j.first, uv = r % (j.nu * j.nv), run = r / (j.nu * j.nv);
  T* const mem = reinterpret_cast<T*>(lds);
  switch (j.d) {
    case 1: param_tile<T, 1>(a, j, uv, run, mem); break;
    case 3: param_tile<T, 3>(a, j, uv, run, mem); break;
    case 5: param_tile<T, 5>(a, j, uv, run, mem); break;
    case 7: param_tile<T, 7>(a, j, uv, run, mem); break;
    case 9: param_tile<T, 9>(a, j, uv, run, mem); break;
    default: break;
  }
}

// The runs' matrices and column sums, added in order in 64 bits: 64 values a
// block, its 16 wavefronts every 16th run.
struct JoinJob {
  int64_t at, numel, sums;  // of a run: first value, matrix, column sums
  int32_t runs, first;
  void *matrix, *columns;
};
struct JoinArgs {
  int32_t n_jobs;
  JoinJob job[kMaxMaps + 1];
};

template <class T>
__global__ __launch_bounds__(1024) void k_param_join(JoinArgs a, const T* __restrict__ part) {
  __shared__ double sums[16][64];
  int ji = 0;
  while (ji + 1 < a.n_jobs && static_cast<int>(blockIdx.x) >= a.job[ji + 1].first) ++ji;
  const JoinJob& j = a.job[ji];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t per = j.numel + j.sums, q = int64_t(static_cast<int>(blockIdx.x) - j.first) * 64 + lane;
  double v = 0;
  if (q < per) {
#pragma unroll 4
    for (int r = w; r < j.runs; r += 16) v += double(part[j.at + r * per + q]);
  }
  sums[w][lane] = v;
  __syncthreads();
  if (w > 0 || q >= per) return;
  v = 0;
#pragma unroll
  for (int r = 0; r < 16; ++r) v += sums[r][lane];
  if (q < j.numel) {
    if (j.matrix != nullptr) static_cast<T*>(j.matrix)[q] = static_cast<T>(v);
  } else if (j.columns != nullptr) {
    static_cast<T*>(j.columns)[q - j.numel] = static_cast<T>(v);
  }
}

template <class T>
__global__ void k_clear_columns(int64_t n_rows, int64_t dim, int32_t off, int32_t len, T* __restrict__ out) {
  const int64_t total = n_rows * len, step = int64_t(gridDim.x) * blockDim.x;
  for (int64_t q = blockIdx.x * int64_t(blockDim.x) + threadIdx.x; q < total; q += step)
    out[(q / len) * dim + off + q % len] = T(0);
}

// -------------------------------------------------------------------- host
template <class T>
bool pieces16(const void* p, int64_t ld, int64_t off, int64_t len) {
  constexpr int per = 16 / sizeof(T);
  return aligned16(p) && ld % per == 0 && off % per == 0 && len % per == 0;
}

// x's segment s_in as a source
template <class T>
RowSource source_of(const Dense& p, const DenseInput& x, int32_t off, int32_t mul, int d, int seg) {
  RowSource r{};
  r.ld = p.dim_in;
  r.off = off;
  r.K = mul;
  if (x.codes != nullptr) {
    r.rows = x.codes;
    r.scales = x.scales + seg;
    r.ld_scales = p.n_segs_in;
    r.packed = reinterpret_cast<uintptr_t>(x.codes) % 4 == 0 && p.dim_in % 4 == 0 && off % 4 == 0 && mul * d % 4 == 0;
  } else {
    r.rows = x.rows;
    r.packed = pieces16<T>(x.rows, p.dim_in, off, int64_t(mul) * d);
  }
  return r;
}

template <class T>
RowSource source_rows(const void* rows, int64_t ld, int32_t off, int32_t mul, int d) {
  RowSource r{};
  r.rows = rows;
  r.ld = ld;
  r.off = off;
  r.K = mul;
  r.packed = pieces16<T>(rows, ld, off, int64_t(mul) * d);
  return r;
}

template <class T>
constexpr int most_waves() {
  return sizeof(T) == 4 ? 4 : 2;
}

// Shares of the jobs, LDS and launch; the jobs' sizes and terms are set.
template <class T, int MODE>
hipError_t run_dense(DenseArgs& a, hipStream_t s) {
  if (a.n_rows == 0 || a.n_jobs == 0) return hipSuccess;
  int widest = 1, deepest = 1;
  for (int i = 0; i < a.n_jobs; ++i) {
    widest = std::max(widest, a.job[i].N);
    deepest = std::max({deepest, a.job[i].main.src.K, a.job[i].gate.src.K});
  }
  a.waves = std::min(most_waves<T>(), (widest + 15) / 16);
  // channels that LDS holds at a time: 64 (fp64: 32), fewer where no map has so many
  const int ks = sizeof(T) == 4 ? (deepest <= 16 ? 4 : (deepest <= 32 ? 8 : 16)) : (deepest <= 16 ? 4 : 8);
  size_t lds = 0;
  a.shares = 0;
  for (int i = 0; i < a.n_jobs; ++i) {
    DenseJob& j = a.job[i];
    j.first = a.shares;
    a.shares += (j.N + 16 * a.waves - 1) / (16 * a.waves);
    const size_t pad = 16 / sizeof(T), wide = std::max(4 * ks, 16 * a.waves);
    lds = std::max(lds, sizeof(T) * atoms_of(j.d) * (wide * j.d + pad));  // 37 KiB at most
  }
  a.group = 64;
  while (a.group > 16 && (a.n_rows + a.group - 1) / a.group * a.shares < 2048) a.group /= 2;
  a.groups = (a.n_rows + a.group - 1) / a.group;
  const int64_t blocks = (a.groups + 7) / 8 * 8 * a.shares;
  auto go = [&](auto* f) -> hipError_t {
    in_launches(blocks, 64 * a.waves, [&](int64_t block0, unsigned n) {
      a.block0 = block0;
      hipLaunchKernelGGL(f, dim3(n), dim3(64 * a.waves), lds, s, a);
    });
    return hipGetLastError();
  };
  if (ks == 4) return go(k_dense<T, 4, MODE>);
  if (ks == 8 || sizeof(T) == 8) return go(k_dense<T, 8, MODE>);
  return go(k_dense<T, sizeof(T) == 4 ? 16 : 8, MODE>);
}

// The jobs of a pass over the maps: rows of x times the maps.
template <class T>
void forward_jobs(const Dense& p, const DenseInput& x, const void* weights, const void* gate_weights,
                  const void* bias, DenseArgs& a, bool scalars_only) {
  a.bias = bias;
  a.n_jobs = 0;
  for (const DenseMap& m : p.maps) {
    if (scalars_only && !m.even) continue;
    DenseJob& j = a.job[a.n_jobs++];
    j.main.src = source_of<T>(p, x, m.in_off, m.mul_in, m.d, m.seg_in);
    j.main.weights = static_cast<const T*>(weights) + m.woff;
    j.main.ldw = m.mul_out;
    j.d = m.d;
    j.N = m.mul_out;
    j.out_off = j.g_off = m.out_off;
    j.act = m.act;
    if (p.gated) {
      j.gate.src = source_of<T>(p, x, p.scalar_off, p.scalar_mul, 1, p.scalar_seg);
      j.gate.weights = gate_weights;
      j.gate.ldw = static_cast<int32_t>(p.n_gates);
      j.gate0 = m.gate;
      j.bias = bias != nullptr ? m.gate : -1;
    } else {
      j.bias = bias != nullptr && m.even ? 0 : -1;
    }
  }
}

template <class T>
hipError_t dense_forward(const Dense& p, int64_t n_rows, const void* x, const void* weights, const void* gate_weights,
                         const void* bias, const void* residual, void* out, hipStream_t s) {
  DenseArgs a{};
  a.n_rows = n_rows;
  a.ld_out = p.dim_out;
  a.n_gates = p.n_gates;
  a.out = out;
  a.extra = residual;
  forward_jobs<T>(p, DenseInput{x, nullptr, nullptr}, weights, gate_weights, bias, a, false);
  for (int i = 0; i < a.n_jobs; ++i) {
    DenseJob& j = a.job[i];
    const int64_t len = int64_t(j.N) * j.d;
    j.packed_out = pieces16<T>(out, p.dim_out, j.out_off, len) && aligned16(residual);
  }
  return p.gated ? run_dense<T, kGated>(a, s) : run_dense<T, kLinear>(a, s);
}

// How the atoms of the parameters' jobs are cut into runs: about kParamBlocks
// blocks of equal work, a run a whole number of stages.
constexpr int kParamBlocks = 1024;

struct ParamShape {
  int n_jobs = 0;
  int32_t U[kMaxMaps + 1], V[kMaxMaps + 1], d[kMaxMaps + 1], nu[kMaxMaps + 1], nv[kMaxMaps + 1], runs[kMaxMaps + 1];
  int64_t run[kMaxMaps + 1], at[kMaxMaps + 1], per[kMaxMaps + 1];
  bool sums[kMaxMaps + 1];
  int64_t total = 0, blocks = 0;
  bool single = true;  // one run each
};

template <class T>
ParamShape param_shape(const Dense& p, int64_t n_rows) {
  ParamShape h;
  constexpr int S = tile_side<T>();
  auto add = [&](int U, int V, int d, bool sums) {
    const int i = h.n_jobs++;
    h.U[i] = U;
    h.V[i] = V;
    h.d[i] = d;
    h.sums[i] = sums;
    h.nu[i] = (U + S - 1) / S;
    h.nv[i] = (V + S - 1) / S;
  };
  for (const DenseMap& m : p.maps) add(m.mul_in, m.mul_out, m.d, !p.gated && m.even);
  if (p.gated) add(p.scalar_mul, static_cast<int>(p.n_gates), 1, true);
  int64_t work = 0;
  for (int i = 0; i < h.n_jobs; ++i) work += int64_t(h.nu[i]) * h.nv[i] * h.d[i];
  for (int i = 0; i < h.n_jobs; ++i) {
    const int sa = stage_atoms(h.d[i]);
    // atoms whose components are a block's part of the work
    const int64_t part = n_rows * work / (int64_t(kParamBlocks) * h.d[i]) + 1;
    h.run[i] = (part + sa - 1) / sa * sa;
    h.runs[i] = static_cast<int32_t>(std::max<int64_t>(1, (n_rows + h.run[i] - 1) / h.run[i]));
    h.per[i] = int64_t(h.U[i]) * h.V[i] + (h.sums[i] ? h.V[i] : 0);
    h.at[i] = h.total;
    h.total += h.per[i] * h.runs[i];
    h.blocks += int64_t(h.nu[i]) * h.nv[i] * h.runs[i];
    h.single = h.single && h.runs[i] == 1;
  }
  return h;
}

struct DenseSpace {
  size_t rows, gates, parts, total;
};

template <class T>
DenseSpace dense_space(const Dense& p, int64_t n_rows) {
  DenseSpace w{};
  const ParamShape h = param_shape<T>(p, n_rows);
  w.rows = 0;
  size_t at = 0;
  if (p.gated) {
    at = align_up(sizeof(T) * static_cast<size_t>(n_rows) * p.dim_out);
    w.gates = at;
    at += align_up(sizeof(T) * static_cast<size_t>(n_rows) * p.n_gates);
  } else if (p.sloped()) {
    at = align_up(sizeof(T) * static_cast<size_t>(n_rows) * p.scalar_out_mul);
  }
  w.parts = at;
  if (!h.single) at += align_up(sizeof(T) * static_cast<size_t>(h.total));
  w.total = at;
  return w;
}

template <class T>
hipError_t dense_backward(const Dense& p, int64_t n_rows, const DenseInput& x, const void* weights,
                          const void* gate_weights, const void* bias, const void* grad_out, void* grad_x,
                          void* grad_weights, void* grad_gate_weights, void* grad_bias, void* ws, hipStream_t s) {
  const DenseSpace space = dense_space<T>(p, n_rows);
  char* const mem = static_cast<char*>(ws);
  // grad_out through the activations: rows (gated), their gates, or the even scalars alone (linear)
  T* const dz = reinterpret_cast<T*>(p.gated ? mem + space.gates : mem);
  const T* du = static_cast<const T*>(grad_out);
  if (p.gated || p.sloped()) {
    DenseArgs a{};
    a.n_rows = n_rows;
    a.ld_g = p.dim_out;
    a.n_gates = p.n_gates;
    a.extra = grad_out;
    forward_jobs<T>(p, x, weights, gate_weights, bias, a, !p.gated);
    if (p.gated) {
      du = reinterpret_cast<T*>(mem);
      a.out = mem;
      a.ld_out = p.dim_out;
      a.dz = dz;
    } else {
      a.out = dz;
      a.ld_out = p.scalar_out_mul;
      a.job[0].out_off = 0;
    }
    for (int i = 0; i < a.n_jobs; ++i) {
      DenseJob& j = a.job[i];
      j.packed_g = pieces16<T>(grad_out, p.dim_out, j.g_off, int64_t(j.N) * j.d);
      j.packed_out = pieces16<T>(a.out, a.ld_out, j.out_off, int64_t(j.N) * j.d);
    }
    const hipError_t he = p.gated ? run_dense<T, kGatedGrad>(a, s) : run_dense<T, kLinearGrad>(a, s);
    if (he != hipSuccess) return he;
  }
  // rows of the gradient that a map's output segment gets
  auto grad_rows = [&](const DenseMap& m) {
    if (!p.gated && p.sloped() && m.even) return source_rows<T>(dz, p.scalar_out_mul, 0, m.mul_out, 1);
    return source_rows<T>(du, p.dim_out, m.out_off, m.mul_out, m.d);
  };
  if (grad_x != nullptr && n_rows > 0) {
    DenseArgs a{};
    a.n_rows = n_rows;
    a.out = grad_x;
    a.ld_out = p.dim_in;
    for (const DenseMap& m : p.maps) {
      DenseJob& j = a.job[a.n_jobs++];
      j.main.src = grad_rows(m);
      j.main.weights = static_cast<const T*>(weights) + m.woff;
      j.main.ldw = m.mul_out;
      j.d = m.d;
      j.N = m.mul_in;
      j.out_off = m.in_off;
      j.bias = -1;
      if (p.gated && m.even) {
        j.gate.src = source_rows<T>(dz, p.n_gates, 0, static_cast<int32_t>(p.n_gates), 1);
        j.gate.weights = gate_weights;
        j.gate.ldw = static_cast<int32_t>(p.n_gates);
      }
      j.packed_out = pieces16<T>(grad_x, p.dim_in, m.in_off, int64_t(m.mul_in) * m.d);
    }
    if (p.gated && !p.even_out) {  // the even scalars reach the gates alone
      DenseJob& j = a.job[a.n_jobs++];
      j.main.src = source_rows<T>(dz, p.n_gates, 0, static_cast<int32_t>(p.n_gates), 1);
      j.main.weights = gate_weights;
      j.main.ldw = static_cast<int32_t>(p.n_gates);
      j.d = 1;
      j.N = p.scalar_mul;
      j.out_off = p.scalar_off;
      j.bias = -1;
      j.packed_out = pieces16<T>(grad_x, p.dim_in, p.scalar_off, p.scalar_mul);
    }
    hipError_t he = run_dense<T, kTransposed>(a, s);
    if (he != hipSuccess) return he;
    for (const ColumnRun& r : p.bare_in) {
      const int64_t b = (n_rows * r.len + 255) / 256;
      hipLaunchKernelGGL(k_clear_columns<T>, dim3(static_cast<unsigned>(b > 65536 ? 65536 : b)), dim3(256), 0, s, n_rows,
                         p.dim_in, r.off, r.len, static_cast<T*>(grad_x));
      he = hipGetLastError();
      if (he != hipSuccess) return he;
    }
  }
  if (grad_weights == nullptr && grad_gate_weights == nullptr && grad_bias == nullptr) return hipSuccess;
  const ParamShape h = param_shape<T>(p, n_rows);
  ParamArgs a{};
  a.n_rows = n_rows;
  a.part = h.single ? nullptr : mem + space.parts;
  JoinArgs join{};
  int64_t blocks = 0;
  int joins = 0;
  size_t lds = 0;
  for (int i = 0; i < h.n_jobs; ++i) {
    const bool gates = i == static_cast<int>(p.maps.size());
    void* const matrix = gates ? grad_gate_weights
                               : (grad_weights != nullptr ? static_cast<T*>(grad_weights) + p.maps[i].woff : nullptr);
    void* const sums = h.sums[i] ? grad_bias : nullptr;
    if (matrix == nullptr && sums == nullptr) continue;
    ParamJob& j = a.job[a.n_jobs];
    if (gates) {
      j.x = source_of<T>(p, x, p.scalar_off, p.scalar_mul, 1, p.scalar_seg);
      j.g = source_rows<T>(dz, p.n_gates, 0, static_cast<int32_t>(p.n_gates), 1);
    } else {
      const DenseMap& m = p.maps[i];
      j.x = source_of<T>(p, x, m.in_off, m.mul_in, m.d, m.seg_in);
      j.g = grad_rows(m);
    }
    j.d = h.d[i];
    j.nu = h.nu[i];
    j.nv = h.nv[i];
    j.first = static_cast<int32_t>(blocks);
    j.runs = h.runs[i];
    j.run = h.run[i];
    j.at = h.at[i];
    j.column_sums = h.sums[i];
    j.matrix = matrix;
    j.sums = sums;
    blocks += int64_t(h.nu[i]) * h.nv[i] * h.runs[i];
    JoinJob& q = join.job[a.n_jobs++];
    q = JoinJob{h.at[i], int64_t(h.U[i]) * h.V[i], h.sums[i] ? h.V[i] : 0, h.runs[i], joins, matrix, sums};
    joins += static_cast<int>((h.per[i] + 63) / 64);
    lds = std::max(lds, sizeof(T) * 2 * stage_atoms(j.d) * (tile_side<T>() * j.d + 16));
  }
  join.n_jobs = a.n_jobs;
  if (a.n_jobs == 0) return hipSuccess;
  in_launches(blocks, 256, [&](int64_t block0, unsigned n) {
    a.block0 = static_cast<int32_t>(block0);
    hipLaunchKernelGGL(k_param<T>, dim3(n), dim3(256), lds, s, a);
  });
  hipError_t he = hipGetLastError();
  if (he != hipSuccess || h.single) return he;
  hipLaunchKernelGGL(k_param_join<T>, dim3(static_cast<unsigned>(joins)), dim3(1024), 0, s, join,
                     static_cast<const T*>(a.part));
  return hipGetLastError();
}

}  // namespace

size_t dense_workspace(const Dense& p, int64_t n_rows) {
  return p.f64 ? dense_space<double>(p, n_rows).total : dense_space<float>(p, n_rows).total;
}

hipError_t launch_dense_forward(const Dense& p, int64_t n_rows, const void* x, const void* weights,
                                const void* gate_weights, const void* bias, const void* residual, void* out,
                                hipStream_t s) {
  return p.f64 ? dense_forward<double>(p, n_rows, x, weights, gate_weights, bias, residual, out, s)
               : dense_forward<float>(p, n_rows, x, weights, gate_weights, bias, residual, out, s);
}

hipError_t launch_dense_backward(const Dense& p, int64_t n_rows, const DenseInput& x, const void* weights,
                                 const void* gate_weights, const void* bias, const void* grad_out, void* grad_x,
                                 void* grad_weights, void* grad_gate_weights, void* grad_bias, void* ws,
                                 hipStream_t s) {
  return p.f64 ? dense_backward<double>(p, n_rows, x, weights, gate_weights, bias, grad_out, grad_x, grad_weights,
                                        grad_gate_weights, grad_bias, ws, s)
               : dense_backward<float>(p, n_rows, x, weights, gate_weights, bias, grad_out, grad_x, grad_weights,
                                       grad_gate_weights, grad_bias, ws, s);
}

}  // namespace tpconv
