// node_dense.hpp -- equivariant products of irreps rows with one set of maps,
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
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>

#include "node_device.hpp"
#include "node_internal.hpp"

namespace tpconv {
namespace dense {

// -------------------------------------------------------------- activations
template <class T>
__device__ __forceinline__ T normal_below(T z) {  // Phi(z)
  return T(0.5) * erfc(z * T(-0.70710678118654752440));
}

// e^v for v <= 0, and 1/v for v in [1, 2]: fp32 by the hardware's 2^t and
// reciprocal (one unit in the last place each).  log2(e) is split into two fp32
// numbers, so what the constant's and the product's rounding leave out of t comes
// back as a factor, and e^v is within 2 units over the whole range, with the first
// number alone by 10 at v = -80.  2^t gives no subnormal numbers, so below 2^-125 it
// is formed of t + 64, which is exact; zero from v = -104 on.  (214648 edges of 64
// scalars, silu and its gradient: 118 us; with the first number and normal results
// alone 114; by the library's functions, with their cases for other arguments, 132.)
__device__ __forceinline__ float exp_below(float v) {
#pragma clang fp contract(off)  // t + 64 is of the rounded t
  constexpr float kLog2e = 0x1.715476p+0f, kRest = 0x1.4ae0cp-26f;
  v = fmaxf(v, -200.0f);  // the parts of an infinite product would give NaN
  const float t = v * kLog2e, rest = fmaf(v, kRest, fmaf(v, kLog2e, -t));
  const bool tiny = t < -125.0f;
  const float e = __builtin_amdgcn_exp2f(tiny ? t + 64.0f : t) * fmaf(rest, 0.69314718055994530942f, 1.0f);
  return tiny ? e * 0x1p-64f : e;
}
__device__ __forceinline__ double exp_below(double v) { return exp(v); }
__device__ __forceinline__ float reciprocal(float v) { return __builtin_amdgcn_rcpf(v); }
__device__ __forceinline__ double reciprocal(double v) { return 1.0 / v; }

// 1/(1 + e^-z) and 1/(1 + e^z), neither by a difference; one exponential and one
// reciprocal for both.
template <class T>
struct Sigmoids {
  T of, other;
  __device__ __forceinline__ explicit Sigmoids(T z) {
    const T e = exp_below(-fabs(z)), q = reciprocal(T(1) + e);
    of = z < T(0) ? e * q : q;
    other = z < T(0) ? q : e * q;
    of = z != z ? z : of;
    other = z != z ? z : other;
  }
};

// The activation and its slope, in forms that do not cancel where they saturate.
template <int KIND, class T>
__device__ __forceinline__ T activated(T z) {
  if constexpr (KIND == TPCONV_ACT_SILU) return z * Sigmoids<T>(z).of;
  if constexpr (KIND == TPCONV_ACT_SIGMOID) return Sigmoids<T>(z).of;
  if constexpr (KIND == TPCONV_ACT_TANH) return tanh(z);
  if constexpr (KIND == TPCONV_ACT_GELU) return z * normal_below(z);
  return z;
}

template <int KIND, class T>
__device__ __forceinline__ T slope_of(T z) {
  if constexpr (KIND == TPCONV_ACT_SILU) {
    const Sigmoids<T> s(z);
    return s.of + z * s.of * s.other;
  }
  if constexpr (KIND == TPCONV_ACT_SIGMOID) {
    const Sigmoids<T> s(z);
    return s.of * s.other;
  }
  if constexpr (KIND == TPCONV_ACT_TANH) {
    const Sigmoids<T> s(T(2) * z);  // 1 - tanh^2
    return T(4) * s.of * s.other;
  }
  if constexpr (KIND == TPCONV_ACT_GELU) return normal_below(z) + z * exp(T(-0.5) * z * z) * T(0.39894228040143267794);
  return T(1);
}

// f(the kind as a constant)
template <class F>
__device__ __forceinline__ void for_activation(int kind, F&& f) {
  switch (kind) {
    case TPCONV_ACT_SILU: return f(std::integral_constant<int, TPCONV_ACT_SILU>{});
    case TPCONV_ACT_SIGMOID: return f(std::integral_constant<int, TPCONV_ACT_SIGMOID>{});
    case TPCONV_ACT_TANH: return f(std::integral_constant<int, TPCONV_ACT_TANH>{});
    case TPCONV_ACT_GELU: return f(std::integral_constant<int, TPCONV_ACT_GELU>{});
    default: return f(std::integral_constant<int, TPCONV_ACT_IDENTITY>{});
  }
}

// ------------------------------------------------------------------ staging
template <class T, int PER>
struct PieceOf {
  typedef T Type __attribute__((ext_vector_type(PER)));
};
template <class T>
struct PieceOf<T, 1> {
  typedef T Type;
};

constexpr int kWaves = 4;  // of a block

// A thread's place in its block; the wavefront's number is uniform.
struct Place {
  int tid, lane, wave;
  __device__ __forceinline__ Place()
      : tid(threadIdx.x), lane(threadIdx.x & 63), wave(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) {}
};

// A segment of rows to stage from.
struct RowSource {
  const void* rows;       // T, or codes where `scales`
  const float* scales;    // of the segment in row 0
  int32_t ld, ld_scales;  // elements of a row; scales of a row
  int32_t off;            // the segment's first column
  int32_t K;              // its channels
  int32_t packed;         // in pieces of 16 bytes (codes: of 4)
};

// ROWS rows of up to MOST elements on their way from memory to LDS (element c of
// row s at lds[s * P + c]), held in registers in between, so that they can be
// issued ahead of the work on the rows before.  A wavefront takes a whole row,
// or several where they are short: a piece's place is a part common to the
// wavefront and one that a lane keeps.  X8: rows in 8 bits, restored on the way.
template <class T, int MOST, int ROWS, int P, bool VEC, bool X8>
struct Mover {
  static constexpr int kPer = VEC ? (X8 ? 4 : 16 / int(sizeof(T))) : 1, kPieces = MOST / kPer;
  static constexpr int lanes() {
    int l = 1;
    while (l < 64 && l < kPieces) l *= 2;
    return l;
  }
  static constexpr int kLanes = lanes(), kRows = 64 / kLanes, kSteps = (kPieces + 63) / 64;
  static constexpr int kTrips = ROWS / (kWaves * kRows);
  static_assert(kTrips * kWaves * kRows == ROWS, "rows are whole trips of the block");
  using Piece = typename PieceOf<T, kPer>::Type;

  Piece v[X8 ? 1 : kTrips][kSteps];
  int code[X8 ? kTrips : 1][kSteps];
  float scale[X8 ? kTrips : 1];

  // rows base .., `count` channels of d components from channel k0 on
  __device__ __forceinline__ void issue(const Place& t, const RowSource& a, int64_t base, int rows, int k0, int count,
                                        int d) {
    const int sub = t.lane / kLanes, e = t.lane % kLanes * kPer, len = count * d;
    const uint32_t mine = sub * a.ld + e;
    const int64_t at = base * a.ld + a.off + k0 * d;
#pragma unroll
    for (int b = 0; b < kTrips; ++b) {
      const int row = (b * kWaves + t.wave) * kRows;
      if constexpr (X8) {
        scale[b] = 0;
        if (row + sub < rows) scale[b] = a.scales[(base + row + sub) * a.ld_scales];
      }
#pragma unroll
      for (int k = 0; k < kSteps; ++k)
        if (row + sub < rows && e + 64 * kPer * k < len) {
          if constexpr (X8) {
            const uint8_t* const from = static_cast<const uint8_t*>(a.rows) + at + int64_t(row) * a.ld + 64 * kPer * k;
            if constexpr (VEC)
              code[b][k] = *reinterpret_cast<const int*>(from + mine);
            else
              code[b][k] = from[mine];
          } else {
            const T* const from = static_cast<const T*>(a.rows) + at + int64_t(row) * a.ld + 64 * kPer * k;
            v[b][k] = *reinterpret_cast<const Piece*>(from + mine);
          }
        }
    }
  }

  __device__ __forceinline__ void land(const Place& t, T* lds, int rows, int len) const {
    const int sub = t.lane / kLanes, e = t.lane % kLanes * kPer;
    T* const to = lds + sub * P + e;
#pragma unroll
    for (int b = 0; b < kTrips; ++b) {
      const int row = (b * kWaves + t.wave) * kRows;
#pragma unroll
      for (int k = 0; k < kSteps; ++k)
        if (row + sub < rows && e + 64 * kPer * k < len) {
          T* const at = to + row * P + 64 * kPer * k;
          if constexpr (X8) {
            at[0] = __builtin_amdgcn_cvt_f32_fp8(code[b][k], 0) * scale[b];
            if constexpr (VEC) {
              at[1] = __builtin_amdgcn_cvt_f32_fp8(code[b][k], 1) * scale[b];
              at[2] = __builtin_amdgcn_cvt_f32_fp8(code[b][k], 2) * scale[b];
              at[3] = __builtin_amdgcn_cvt_f32_fp8(code[b][k], 3) * scale[b];
            }
          } else {
            *reinterpret_cast<Piece*>(at) = v[b][k];
          }
        }
    }
  }
};

// The same at once, some pieces of a thread at a time.
template <class T, int MOST, int ROWS, int P, bool VEC, bool X8>
__device__ __forceinline__ void stage(const Place& t, const RowSource& a, T* lds, int64_t base, int rows, int k0,
                                      int count, int d) {
  constexpr int kAll = Mover<T, MOST, ROWS, P, VEC, X8>::kTrips, kSteps = Mover<T, MOST, ROWS, P, VEC, X8>::kSteps;
  constexpr int kTrips = kAll * kSteps <= 8 ? kAll : (kSteps >= 8 ? 1 : 8 / kSteps), kPart = ROWS / kAll * kTrips;
#pragma unroll 1
  for (int r = 0; r < rows; r += kPart) {
    Mover<T, MOST, kPart, P, VEC, X8> part;
    part.issue(t, a, base + r, rows - r, k0, count, d);
    part.land(t, lds + r * P, rows - r, count * d);
  }
}

// Channels count .. CH of LDS rows become zero, so that no NaN stands beside
// weights that are not there.
template <class T, int D, int CH, int P>
__device__ __forceinline__ void clear_channels(const Place& t, T* lds, int rows, int count) {
  const int len = (CH - count) * D;
  for (int q = t.tid; q < rows * len; q += 64 * kWaves) {
    const int s = q / len;
    lds[s * P + count * D + (q - s * len)] = T(0);
  }
}

// ------------------------------------------------------------------- products
// A block keeps one map and C (16, 32, 64) of its output channels, and goes over
// tiles of atoms; its four wavefronts are C/16 sets of channels times 64/C sets
// of atoms.  A tile's segment goes to LDS as it lies in memory.  The weights are
// a matrix instruction's rows and 16 atoms at one component its columns, and the
// inner index is dealt so that a lane's four channels follow one another, in the
// rows that it reads from LDS (4 (2l+1) neighbouring values, 16 bytes at a time)
// as in those that it ends up with: results, residuals and gradients go between
// registers and memory directly, 16 bytes a lane.  A row's pitch in LDS is 16
// bytes more than a multiple of 64 banks (16 times an odd number), so the 16
// atoms' reads fall into all banks once.  Where a map's channels are read in one
// go, the weights stay in registers and the next tile is on its way while one is
// multiplied.
// 28000 fp32 rows of 64 channels l <= 3: gated 82 us (229 MB, 2.8 TB/s; 4.6
// GFLOP, 56 TFLOP/s), linear with residual 87 us (344 MB, 3.9 TB/s): memory's
// latency, with three blocks a CU; with one tile staged and multiplied in turn
// the gated one took 170.  2048 fp64 rows of 16 channels l <= 4: 15 us, latency
// of a tile's loads, products and stores in turn.
enum Mode { kLinear, kGated, kLinearGrad, kGatedGrad, kTransposed };

constexpr bool has_gates(int mode) { return mode == kGated || mode == kGatedGrad; }
constexpr bool has_grad(int mode) { return mode == kLinearGrad || mode == kGatedGrad; }

// 16-atom tiles of a wavefront: enough products between a weight's uses
template <class T>
constexpr int tiles_of(int d) {
  return sizeof(T) == 8 ? (d == 1 ? 2 : 1) : (d == 1 ? 4 : (d == 3 ? 2 : 1));
}
template <class T>
constexpr int atoms_of(int d, int C) {
  return 16 * tiles_of<T>(d) * (64 / C);
}
template <class T>
constexpr int pitch_of(int d, int C) {
  return C * d + 16 / int(sizeof(T));
}

// One product's operands: rows and weights W[k * ldw + n], or, transposed,
// W[n * ldw + k].
struct Term {
  RowSource src;
  const void* weights;
  int32_t ldw;
  int32_t packed;  // transposed: the weights in pieces of 16 bytes along k
};

struct DenseJob {
  Term main;        // components d
  Term gate;        // the gates' (rows of 0e); kTransposed: the second term of 0e; K = 0: none
  int32_t d, N;
  int32_t out_off;  // first column in a row of out (kLinearGrad: of dz)
  int32_t g_off;    // first column in a row of grad_out
  int32_t bias;     // first bias of the job, -1: none
  int32_t gate0;    // first gate
  int32_t act;
  int32_t packed_out, packed_g, packed_dz;
  int32_t first;    // first block
  int32_t shares;   // blocks of output channels
  int32_t blocks;   // of one share
};

struct DenseArgs {
  int64_t n_rows;
  int32_t ld_out, ld_g, n_gates;
  int32_t n_jobs;
  void* out;
  const void* extra;  // kLinear: residual; kLinearGrad, kGatedGrad: grad_out
  const void* bias;
  void* dz;           // kGatedGrad: [n_rows][n_gates]
  DenseJob job[kMaxMaps];
};

// Step s's channel of the sum in lane group g: four neighbouring ones per group.
constexpr int channel_of(int s, int g) { return s / 4 * 16 + 4 * g + s % 4; }

// A lane's weights of channels k0 .. k0 + count: row `n` of the product.
template <class T, int KS, bool ADJ>
__device__ __forceinline__ void load_weights(const Term& t, int n, int g4, int k0, int count, T (&w)[KS]) {
  constexpr int kPer = 16 / sizeof(T);
  const T* const from = static_cast<const T*>(t.weights) + (ADJ ? int64_t(k0) : int64_t(k0) * t.ldw);
  const uint32_t mine = ADJ ? n * t.ldw + 4 * g4 : 4 * g4 * t.ldw + n;  // a map has at most 2^20 weights
  if (count == 4 * KS && ADJ && t.packed) {
    using Piece = typename PieceOf<T, kPer>::Type;
#pragma unroll
    for (int s = 0; s < KS; s += kPer) {
      const Piece p = *reinterpret_cast<const Piece*>(from + channel_of(s, 0) + mine);
#pragma unroll
      for (int e = 0; e < kPer; ++e) w[s + e] = p[e];
    }
  } else if (count == 4 * KS) {
#pragma unroll
    for (int s = 0; s < KS; ++s) w[s] = (from + (ADJ ? channel_of(s, 0) : channel_of(s, 0) * t.ldw))[mine];
  } else {
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const int k = min(channel_of(s, g4), count - 1);
      const T v = from[ADJ ? uint32_t(n * t.ldw + k) : uint32_t(k * t.ldw + n)];
      w[s] = channel_of(s, g4) < count ? v : T(0);
    }
  }
}

// acc[i][m] += weights times the i-th 16 rows of LDS, component m
template <class T, int D, int KS, int MT, int P>
__device__ __forceinline__ void multiply(const T* lds, int i16, int g4, int rows, const T (&w)[KS],
                                         typename Mfma<T>::Acc (&acc)[MT][D]) {
  constexpr int kPer = 16 / sizeof(T);
  using Piece = typename PieceOf<T, kPer>::Type;
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    if (16 * i >= rows) break;
    const T* const at = lds + (16 * i + i16) * P + 4 * g4 * D;
#pragma unroll
    for (int s = 0; s < KS; s += 4) {
      T x[4 * D];
#pragma unroll
      for (int e = 0; e < 4 * D; e += kPer) {
        const Piece p = *reinterpret_cast<const Piece*>(at + 4 * s * D + e);
#pragma unroll
        for (int q = 0; q < kPer; ++q) x[e + q] = p[q];
      }
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int m = 0; m < D; ++m) acc[i][m] = Mfma<T>::step(w[s + q], x[q * D + m], acc[i][m]);
    }
  }
}

// A lane's four channels, 4 D neighbouring values, from or to memory; in pieces
// of 16 bytes, or one by one (`there` of the channels).
template <class T, int D>
__device__ __forceinline__ void load_run(T (&v)[4 * D], const T* at, bool packed, int there) {
  constexpr int kPer = 16 / sizeof(T);
  using Piece = typename PieceOf<T, kPer>::Type;
  if (packed) {
#pragma unroll
    for (int e = 0; e < 4 * D; e += kPer) {
      const Piece p = *reinterpret_cast<const Piece*>(at + e);
#pragma unroll
      for (int q = 0; q < kPer; ++q) v[e + q] = p[q];
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4 * D; ++e) {
      v[e] = 0;
      if (e / D < there) v[e] = at[e];
    }
  }
}
template <class T, int D>
__device__ __forceinline__ void store_run(const T (&v)[4 * D], T* at, bool packed, int there) {
  constexpr int kPer = 16 / sizeof(T);
  using Piece = typename PieceOf<T, kPer>::Type;
  if (packed) {
#pragma unroll
    for (int e = 0; e < 4 * D; e += kPer) {
      Piece p;
#pragma unroll
      for (int q = 0; q < kPer; ++q) p[q] = v[e + q];
      *reinterpret_cast<Piece*>(at + e) = p;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4 * D; ++e)
      if (e / D < there) at[e] = v[e];
  }
}

// What a lane has to do with: its atom in a tile of 16, its four channels of the
// result, and the row of the weights that it holds.
template <class T, int C>
struct LanePart {
  int i16, g4, wa;  // wa: the wavefront's set of atoms
  int c0, there;    // first channel of four, and how many there are
  int n;            // row of the weights
  T bias[4];

  __device__ __forceinline__ LanePart(const Place& p, int n0, int N, const void* first_bias) {
    i16 = p.lane & 15;
    g4 = p.lane >> 4;
    wa = p.wave / (C / 16);
    const int n16 = n0 + 16 * (p.wave % (C / 16));
    c0 = n16 + 4 * g4;
    there = min(4, N - c0);
    n = min(n16 + (sizeof(T) == 8 ? 4 * (i16 % 4) + i16 / 4 : i16), N - 1);
#pragma unroll
    for (int q = 0; q < 4; ++q) bias[q] = first_bias != nullptr && q < there ? static_cast<const T*>(first_bias)[c0 + q] : T(0);
  }
};

template <class T, int MT, int D>
__device__ __forceinline__ void clear_sums(typename Mfma<T>::Acc (&acc)[MT][D]) {
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int m = 0; m < D; ++m) acc[i][m] = typename Mfma<T>::Acc{0, 0, 0, 0};
}

// Gates' activations (and slopes), before the products, so that they alone stay.
template <class T, int MT, bool SLOPE>
__device__ __forceinline__ void activate_gates(int act, const T (&bias)[4], typename Mfma<T>::Acc (&z)[MT][1],
                                               typename Mfma<T>::Acc (&slope)[SLOPE ? MT : 1]) {
  for_activation(act, [&](auto kind) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const T v = z[i][0][q] + bias[q];
        z[i][0][q] = activated<decltype(kind)::value>(v);
        if constexpr (SLOPE) slope[i][q] = slope_of<decltype(kind)::value>(v);
      }
  });
}

// What stands at the results' places: the residual, or grad_out.
template <class T, int D, int C, int MODE, int MT>
__device__ __forceinline__ void load_extra(const DenseArgs& a, const DenseJob& j, const LanePart<T, C>& l,
                                           int64_t base, int own, T (&v)[MT][4 * D]) {
  constexpr bool kGrad = has_grad(MODE);
#pragma unroll
  for (int i = 0; i < MT; ++i)
    if (16 * i + l.i16 < own && l.there > 0)
      load_run<T, D>(v[i],
                     static_cast<const T*>(a.extra) +
                         (base + 16 * (MT * l.wa + i) + l.i16) * (kGrad ? a.ld_g : a.ld_out) +
                         (kGrad ? j.g_off : j.out_off) + l.c0 * D,
                     kGrad ? j.packed_g : j.packed_out, l.there);
}

// Products to results, and to memory.
template <class T, int D, int C, int MODE, int MT>
__device__ __forceinline__ void finish(const DenseArgs& a, const DenseJob& j, const LanePart<T, C>& l, int64_t base,
                                       int own, bool with_extra, typename Mfma<T>::Acc (&u)[MT][D],
                                       const typename Mfma<T>::Acc (&z)[has_gates(MODE) ? MT : 1][1],
                                       const typename Mfma<T>::Acc (&slope)[MODE == kGatedGrad ? MT : 1],
                                       const T (&extra)[MODE == kLinear || has_grad(MODE) ? MT : 1][4 * D]) {
  if constexpr ((MODE == kLinear && D == 1) || MODE == kLinearGrad)
    for_activation(j.act, [&](auto kind) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const T v = u[i][0][q] + l.bias[q];
          u[i][0][q] = MODE == kLinear ? activated<decltype(kind)::value>(v) : slope_of<decltype(kind)::value>(v);
        }
    });
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    if (16 * i + l.i16 < own && l.there > 0) {
      const int64_t row = base + 16 * (MT * l.wa + i) + l.i16;
      T v[4 * D], dz[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        T dot = 0;
#pragma unroll
        for (int m = 0; m < D; ++m) {
          const T r = u[i][m][q];
          if constexpr (MODE == kGated) {
            v[q * D + m] = z[i][0][q] * r;
          } else if constexpr (MODE == kGatedGrad) {
            const T g = extra[i][q * D + m];
            dot = fma(g, r, dot);
            v[q * D + m] = g * z[i][0][q];
          } else if constexpr (MODE == kLinearGrad) {
            v[q * D + m] = extra[i][q * D + m] * r;
          } else if constexpr (MODE == kLinear) {
            v[q * D + m] = with_extra ? extra[i][q * D + m] + r : r;
          } else {
            v[q * D + m] = r;
          }
        }
        if constexpr (MODE == kGatedGrad) dz[q] = dot * slope[i][q];
      }
      store_run<T, D>(v, static_cast<T*>(a.out) + row * a.ld_out + j.out_off + l.c0 * D, j.packed_out, l.there);
      if constexpr (MODE == kGatedGrad)
        store_run<T, 1>(dz, static_cast<T*>(a.dz) + row * a.n_gates + j.gate0 + l.c0, j.packed_dz, l.there);
    }
  }
}

// A map whose channels (and the gates') are read in one go.
template <class T, int D, int C, int MODE, bool VEC, bool X8>
__device__ __forceinline__ void whole_job(const DenseArgs& a, const DenseJob& j, int n0, int index, T* lds) {
  constexpr int KS = C / 4, MT = tiles_of<T>(D), TA = atoms_of<T>(D, C), P = pitch_of<T>(D, C), P0 = pitch_of<T>(1, C);
  constexpr bool kGates = has_gates(MODE), kExtra = MODE == kLinear || has_grad(MODE);
  using Acc = typename Mfma<T>::Acc;
  const Place p;
  const LanePart<T, C> l(p, n0, j.N, j.bias >= 0 ? static_cast<const T*>(a.bias) + j.bias : nullptr);
  const int64_t n_tiles = (a.n_rows + TA - 1) / TA;
  T* const gate_lds = lds + TA * P;
  const int K = j.main.src.K, K0 = j.gate.src.K;
  const bool same = kGates && D == 1 && j.main.src.off == j.gate.src.off;  // the gates' rows are the map's
  const bool with_extra = has_grad(MODE) || (MODE == kLinear && a.extra != nullptr);
  Mover<T, C * D, TA, P, VEC, X8> main;
  Mover<T, C, TA, P0, VEC, X8> gate;
  T w[KS], wg[kGates ? KS : 1];
  int64_t base = int64_t(index) * TA;
  int rows = static_cast<int>(min<int64_t>(TA, a.n_rows - base));
  main.issue(p, j.main.src, base, rows, 0, K, D);
  if (kGates && !same) gate.issue(p, j.gate.src, base, rows, 0, K0, 1);
  load_weights<T, KS, MODE == kTransposed>(j.main, l.n, l.g4, 0, K, w);
  if constexpr (kGates) load_weights<T, KS, false>(j.gate, j.gate0 + l.n, l.g4, 0, K0, wg);
  if (K < C) clear_channels<T, D, C, P>(p, lds, TA, K);
  if (kGates && !same && K0 < C) clear_channels<T, 1, C, P0>(p, gate_lds, TA, K0);
  const T* const mine = lds + 16 * MT * l.wa * P;
  const T* const mine_gate = gate_lds + 16 * MT * l.wa * P0;
  for (int64_t t = index; t < n_tiles; t += j.blocks) {
    const int own = rows - 16 * MT * l.wa;  // atoms from this wavefront's first on
    const int64_t here = base;
    __syncthreads();                        // the last tile is multiplied
    main.land(p, lds, rows, K * D);
    if (kGates && !same) gate.land(p, gate_lds, rows, K0);
    __syncthreads();
    T extra[kExtra ? MT : 1][4 * D];
    if constexpr (kExtra)
      if (with_extra) load_extra<T, D, C, MODE, MT>(a, j, l, here, own, extra);
    if (t + j.blocks < n_tiles) {
      base = (t + j.blocks) * TA;
      rows = static_cast<int>(min<int64_t>(TA, a.n_rows - base));
      main.issue(p, j.main.src, base, rows, 0, K, D);
      if (kGates && !same) gate.issue(p, j.gate.src, base, rows, 0, K0, 1);
    }
    Acc z[kGates ? MT : 1][1], slope[MODE == kGatedGrad ? MT : 1], u[MT][D];
    if constexpr (kGates) {
      clear_sums<T, MT, 1>(z);
      if (D == 1 && same)
        multiply<T, 1, KS, MT, P>(mine, l.i16, l.g4, own, wg, z);
      else
        multiply<T, 1, KS, MT, P0>(mine_gate, l.i16, l.g4, own, wg, z);
      activate_gates<T, MT, MODE == kGatedGrad>(j.act, l.bias, z, slope);
    }
    clear_sums<T, MT, D>(u);
    multiply<T, D, KS, MT, P>(mine, l.i16, l.g4, own, w, u);
    finish<T, D, C, MODE, MT>(a, j, l, here, own, with_extra, u, z, slope, extra);
  }
}

// acc += a term, C channels at a time
template <class T, int D, int C, bool ADJ, bool VEC, bool X8, int MT>
__device__ __forceinline__ void add_chunks(const Place& p, const LanePart<T, C>& l, const Term& term, int n,
                                           int64_t base, int rows, T* lds, typename Mfma<T>::Acc (&acc)[MT][D]) {
  constexpr int KS = C / 4, P = pitch_of<T>(D, C), TA = 16 * MT * (64 / C);
  const int K = term.src.K, own = rows - 16 * MT * l.wa;
  if constexpr (sizeof(T) == 4 && ADJ && D == 1 && VEC) {  // the next channels are on their way while some are multiplied
    Mover<T, C * D, TA, P, VEC, X8> mover;
    T w[KS], next[KS];
    mover.issue(p, term.src, base, rows, 0, min(C, K), D);
    load_weights<T, KS, ADJ>(term, n, l.g4, 0, min(C, K), next);
    for (int k0 = 0; k0 < K; k0 += C) {
      const int count = min(C, K - k0), after = min(C, K - k0 - C);
#pragma unroll
      for (int s = 0; s < KS; ++s) w[s] = next[s];
      __syncthreads();
      mover.land(p, lds, rows, count * D);
      if (count < C) clear_channels<T, D, C, P>(p, lds, TA, count);
      __syncthreads();
      if (after > 0) {
        mover.issue(p, term.src, base, rows, k0 + C, after, D);
        load_weights<T, KS, ADJ>(term, n, l.g4, k0 + C, after, next);
      }
      multiply<T, D, KS, MT, P>(lds + 16 * MT * l.wa * P, l.i16, l.g4, own, w, acc);
    }
    return;
  }
  for (int k0 = 0; k0 < K; k0 += C) {
    const int count = min(C, K - k0);
    T w[KS];
    load_weights<T, KS, ADJ>(term, n, l.g4, k0, count, w);
    __syncthreads();
    stage<T, C * D, TA, P, VEC, X8>(p, term.src, lds, base, rows, k0, count, D);
    if (count < C) clear_channels<T, D, C, P>(p, lds, TA, count);
    __syncthreads();
    multiply<T, D, KS, MT, P>(lds + 16 * MT * l.wa * P, l.i16, l.g4, own, w, acc);
  }
}

// A map with more channels, or with a second term.
template <class T, int D, int C, int MODE, bool VEC, bool X8>
__device__ __forceinline__ void chunked_job(const DenseArgs& a, const DenseJob& j, int n0, int index, T* lds) {
  constexpr int MT = tiles_of<T>(D), TA = atoms_of<T>(D, C);
  constexpr bool kGates = has_gates(MODE), kExtra = MODE == kLinear || has_grad(MODE);
  using Acc = typename Mfma<T>::Acc;
  const Place p;
  const LanePart<T, C> l(p, n0, j.N, j.bias >= 0 ? static_cast<const T*>(a.bias) + j.bias : nullptr);
  const int64_t n_tiles = (a.n_rows + TA - 1) / TA;
  const bool with_extra = has_grad(MODE) || (MODE == kLinear && a.extra != nullptr);
  for (int64_t t = index; t < n_tiles; t += j.blocks) {
    const int64_t base = t * TA;
    const int rows = static_cast<int>(min<int64_t>(TA, a.n_rows - base)), own = rows - 16 * MT * l.wa;
    Acc z[kGates ? MT : 1][1], slope[MODE == kGatedGrad ? MT : 1], u[MT][D];
    if constexpr (kGates) {
      clear_sums<T, MT, 1>(z);
      add_chunks<T, 1, C, false, VEC, X8, MT>(p, l, j.gate, j.gate0 + l.n, base, rows, lds, z);
      activate_gates<T, MT, MODE == kGatedGrad>(j.act, l.bias, z, slope);
    }
    clear_sums<T, MT, D>(u);
    add_chunks<T, D, C, MODE == kTransposed, VEC, X8, MT>(p, l, j.main, l.n, base, rows, lds, u);
    if constexpr (MODE == kTransposed && D == 1)
      if (j.gate.src.K > 0) add_chunks<T, 1, C, true, VEC, X8, MT>(p, l, j.gate, l.n, base, rows, lds, u);
    T extra[kExtra ? MT : 1][4 * D];
    if constexpr (kExtra)
      if (with_extra) load_extra<T, D, C, MODE, MT>(a, j, l, base, own, extra);
    finish<T, D, C, MODE, MT>(a, j, l, base, own, with_extra, u, z, slope, extra);
  }
}

template <class T, int D, int C, int MODE, bool X8>
__device__ __forceinline__ void run_job(const DenseArgs& a, const DenseJob& j, int n0, int index, T* lds) {
  const bool vec = j.main.src.packed && (j.gate.src.K == 0 || j.gate.src.packed);
  if constexpr (sizeof(T) == 4) {  // fp64 has no registers for the tile ahead
    if (j.main.src.K <= C && j.gate.src.K <= C && !(MODE == kTransposed && j.gate.src.K > 0)) {
      if (vec)
        whole_job<T, D, C, MODE, true, X8>(a, j, n0, index, lds);
      else
        whole_job<T, D, C, MODE, false, X8>(a, j, n0, index, lds);
      return;
    }
  }
  if (vec)
    chunked_job<T, D, C, MODE, true, X8>(a, j, n0, index, lds);
  else
    chunked_job<T, D, C, MODE, false, X8>(a, j, n0, index, lds);
}

template <class T, int C, int MODE, bool X8>
__global__ __launch_bounds__(64 * kWaves, sizeof(T) == 4 && MODE != kGatedGrad ? 3 : 2) void k_dense(DenseArgs a) {
  extern __shared__ char dynamic[];
  int ji = 0;
  while (ji + 1 < a.n_jobs && static_cast<int>(blockIdx.x) >= a.job[ji + 1].first) ++ji;
  const DenseJob j = a.job[ji];
  // blocks with the same tiles and other channels run on one XCD (blocks go round them), so rows are fetched once there
  const int b = blockIdx.x - j.first, eight = b / (8 * j.shares), in = b - eight * 8 * j.shares;
  const int n0 = (in >> 3) * C, index = eight * 8 + (in & 7);
  if (index >= j.blocks) return;
  T* const lds = reinterpret_cast<T*>(dynamic);
  if constexpr (MODE == kLinearGrad) {
    run_job<T, 1, C, MODE, X8>(a, j, n0, index, lds);
  } else {
    switch (j.d) {
      case 1: run_job<T, 1, C, MODE, X8>(a, j, n0, index, lds); break;
      case 3: run_job<T, 3, C, MODE, X8>(a, j, n0, index, lds); break;
      case 5: run_job<T, 5, C, MODE, X8>(a, j, n0, index, lds); break;
      case 7: run_job<T, 7, C, MODE, X8>(a, j, n0, index, lds); break;
      case 9: run_job<T, 9, C, MODE, X8>(a, j, n0, index, lds); break;
      default: break;
    }
  }
}

// -------------------------------------------------------------------- host
// Blocks for each of n jobs of tiles[i] tiles that take cost[i] each, `most` in
// all (but one for each job), so that the last to end ends early: the shortest
// time in which whole numbers of tiles fit, within 2 %, and what is left over
// where most is to do, so that all jobs last as long (their segments lie at
// different places of the rows, and a job alone keeps some memory channels idle).
// Blocks go round the 8 XCDs, and a job's are a multiple of 8, so one XCD has the
// same rows of all jobs.  (28000 rows' gated gradients in one pass, 512 blocks:
// 167 us; without what is left over 183, and not in multiples of 8 193.)
inline void share_out(int n, const int64_t* tiles, const int64_t* cost, const int32_t* shares, int64_t most,
                      int32_t* blocks) {
  auto in_eights = [](int64_t b) { return (b + 7) / 8 * 8; };
  double time = 0;
  for (int i = 0; i < n; ++i) time += double(tiles[i]) * double(cost[i]) * shares[i];
  time /= double(most);
  int64_t used = 0;
  for (;; time *= 1.02) {
    used = 0;
    bool fewest = true;
    for (int i = 0; i < n; ++i) {
      const int64_t each = std::max<int64_t>(1, static_cast<int64_t>(time / double(cost[i])));
      blocks[i] = static_cast<int32_t>(std::min(in_eights((tiles[i] + each - 1) / each), tiles[i]));
      used += in_eights(blocks[i]) * shares[i];
      fewest = fewest && blocks[i] <= 8;
    }
    if (used <= most || fewest) break;
  }
  for (;;) {
    int best = -1;
    for (int i = 0; i < n; ++i)
      if (blocks[i] + 8 <= tiles[i] && used + 8 * shares[i] <= most &&
          (best < 0 || double(tiles[i]) * double(cost[i]) / blocks[i] >
                           double(tiles[best]) * double(cost[best]) / blocks[best]))
        best = i;
    if (best < 0) return;
    blocks[best] += 8;
    used += 8 * shares[best];
  }
}

// Blocks of a launch, two for each that a CU holds at a time (28000 rows of 64 channels l <= 3, linear and its
// transposed products: 512 blocks 109 and 87 us, 768: 95 and 77, 1024: 95 and 76, 1536: 88 and 74).
constexpr int64_t kDenseBlocks = 1536;

// Blocks of the jobs, LDS and launch; the jobs' sizes and terms are set.
template <class T, int C, int MODE, bool X8>
hipError_t launch_jobs(DenseArgs& a, hipStream_t s) {
  size_t lds = 0;
  int64_t tiles[kMaxMaps], cost[kMaxMaps];
  int32_t shares[kMaxMaps], of[kMaxMaps];
  for (int i = 0; i < a.n_jobs; ++i) {
    DenseJob& j = a.job[i];
    const int atoms = atoms_of<T>(j.d, C);
    shares[i] = j.shares = (j.N + C - 1) / C;
    tiles[i] = (a.n_rows + atoms - 1) / atoms;
    cost[i] = atoms * ((j.main.src.K + C - 1) / C * j.d + (j.gate.src.K + C - 1) / C);
    lds = std::max(lds, sizeof(T) * atoms * (pitch_of<T>(j.d, C) + (j.gate.src.K > 0 ? pitch_of<T>(1, C) : 0)));
  }
  share_out(a.n_jobs, tiles, cost, shares, kDenseBlocks, of);
  int32_t blocks = 0;
  for (int i = 0; i < a.n_jobs; ++i) {
    DenseJob& j = a.job[i];
    j.first = blocks;
    j.blocks = of[i];
    blocks += (j.blocks + 7) / 8 * 8 * j.shares;
  }
  auto* const f = k_dense<T, C, MODE, X8>;
  if (lds > 64 * 1024) {  // above the default limit of dynamic LDS
    const hipError_t he = hipFuncSetAttribute(reinterpret_cast<const void*>(f),
                                              hipFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(lds));
    if (he != hipSuccess) return he;
  }
  hipLaunchKernelGGL(f, dim3(blocks), dim3(64 * kWaves), lds, s, a);
  return hipGetLastError();
}

// ------------------------------------------------ gradients in one pass (fp32)
struct BackJob {
  Term main, gate;      // x and the maps; gated: the rows of 0e and the gates' weights
  RowSource g;          // grad_out
  int32_t d, K, N, K0;  // channels of x, of the result, of 0e
  int32_t x_off;        // first column in a row of grad_x
  int32_t bias, gate0, act;
  int32_t even;         // the even scalars' map
  int32_t first, blocks;
  int64_t at;           // first value of the job's parts: K x N, gated: K0 x N, N column sums
};

struct BackArgs {
  int64_t n_rows;
  int32_t ld_x, ld_g, n_gates, n_scalars;
  int32_t n_jobs;
  int32_t params;       // parameters' gradients are wanted
  const void* bias;
  float* grad_x;        // or NULL
  float* dz;            // gated: [n_rows][n_gates]
  float* du;            // gated: the even scalars' [n_rows][n_scalars]
  float* part;
  BackJob job[kMaxMaps];
};

// Blocks of that pass, 512: two to a CU.  Several linear maps get 768, whose last take the place of those that end
// first: a gain where the maps' tiles last unequally long, a loss where they are alike (the shares know the products, not
// the waits).  With the sums' join (us), linear, 768 and 512 blocks: 28000 rows of 64 channels l <= 3 118 and 143, of 48
// 109 and 133, of 64 l <= 2 88 and 93, of 32 l <= 3 81 and 78, of 64 l <= 1 51 and 43, 80000 rows of these 309 and 384,
// 283 and 352, 193 and 228, 215 and 196, 129 and 112; 4096 of the first 36 and 33.  214648 rows of one map of 64 scalars
// 97 and 82, of 32 55 and 57.  Gated, 28000 rows of 64 channels l <= 3 204 and 174, of 32 145 and 135 with the forward.
constexpr int back_blocks(bool gated, int n_jobs) { return gated || n_jobs == 1 ? 512 : 768; }

template <bool GATED, bool X8>
hipError_t run_back(BackArgs& a, int C, hipStream_t s);

// Blocks of the jobs for n_rows, and where their parts start; returns the parts' values.
int64_t cut_back(BackArgs& a, int C, bool gated);

// All jobs of a pass; node_dense_rows.hip holds one of each for a type and mode.
template <class T, int MODE, bool X8>
hipError_t run_dense(DenseArgs& a, hipStream_t s);

}  // namespace dense
}  // namespace tpconv
