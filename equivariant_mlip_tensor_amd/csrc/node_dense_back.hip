// node_dense_back.hip -- the gradients of gated and linear maps in one pass over
// the rows, for fp32 maps of up to 64 channels and l <= 3 (wider ones, and rows
// that cannot be taken 16 bytes at a time: node_dense.hip).
//
// A block keeps one map and goes over tiles of atoms.  With x and grad_out's rows
// G of a tile it forms, gated, the products and gates again, and from them
//   du = a(z) G,   dz = a'(z) sum_m G u        (linear: du = G, 0e a'(z) G),
// puts both into LDS beside x, and from there
//   grad_x = M du,   dM += x^T du,   dWg += x_0e^T dz,   db += dz,
// the sums over atoms staying in registers until the block's last tile.  So x
// and grad_out are read once, grad_x is written once, and du never leaves the CU;
// only the gates' rows dz (and du of 0e) do, for the even scalars' grad_x, which
// sums over all maps.  Blocks' sums go to the workspace and are added in order.
//
// Bound by the matrix units and, in turn with them, the wait for a tile's rows:
// two blocks a CU hold 4 tiles of LDS.  28000 fp32 rows of 64 channels l <= 3:
// gated 167 us (373 MB, 2.2 TB/s; 12.7 GFLOP, 76 TFLOP/s, the matrix units busy
// for 48 % of the time), linear 112 us (344 MB, 3.1 TB/s, 66 TFLOP/s), and 5-7 us
// for the sums' join.  As three kernels, du in memory between them: 645 and 228.
#include "node_dense.hpp"

namespace tpconv {
namespace dense {

namespace {

// TA atoms of LDS rows: acc[i][k] += sum over atoms and components of
// x[atom][u] g[atom][v], u = tu + 16 i + .., v = tv + 16 k + ...  A matrix
// instruction takes atoms four apart: their rows start 16 banks apart, and 16
// channels at one component fall between (2l+1 is odd).
template <int D, int TA, int PX, int PG, int F>
__device__ __forceinline__ void outer(const float* x, const float* g, int i16, int g4, int tu, int tv, int rows,
                                      Mfma<float>::Acc (&acc)[F][F]) {
  const float* const xp = x + 4 * g4 * PX + (tu + i16) * D;
  const float* const gp = g + 4 * g4 * PG + (tv + i16) * D;
#pragma unroll
  for (int t = 0; t < TA; t += 16) {
    if (t >= rows) break;
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int m = 0; m < D; ++m) {
        float xv[F], gv[F];
#pragma unroll
        for (int i = 0; i < F; ++i) {
          xv[i] = xp[(t + s) * PX + 16 * i * D + m];
          gv[i] = gp[(t + s) * PG + 16 * i * D + m];
        }
#pragma unroll
        for (int i = 0; i < F; ++i)
#pragma unroll
          for (int k = 0; k < F; ++k) acc[i][k] = Mfma<float>::step(xv[i], gv[k], acc[i][k]);
      }
  }
}

template <int F>
__device__ __forceinline__ void write_outer(float* to, const Mfma<float>::Acc (&acc)[F][F], int i16, int g4, int tu,
                                            int tv, int U, int V) {
#pragma unroll
  for (int i = 0; i < F; ++i)
#pragma unroll
    for (int k = 0; k < F; ++k)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int u = tu + 16 * i + Mfma<float>::row(g4, q), v = tv + 16 * k + i16;
        if (u < U && v < V) to[u * V + v] = acc[i][k][q];
      }
}

template <int CTRL>
__device__ __forceinline__ float moved(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, true));
}
// over the 16 lanes of a row of lanes
__device__ __forceinline__ float sum16(float v) {
  v += moved<0xB1>(v);
  v += moved<0x4E>(v);
  v += moved<0x141>(v);
  return v + moved<0x140>(v);
}

template <int D, int C, bool GATED, bool X8>
__device__ __forceinline__ void back_job(const BackArgs& a, const BackJob& j, int index, float* lds) {
  using Acc = Mfma<float>::Acc;
  constexpr int KS = C / 4, MT = tiles_of<float>(D), TA = atoms_of<float>(D, C), P = pitch_of<float>(D, C),
                P0 = pitch_of<float>(1, C), H = C / 2, F = H / 16;
  const Place p;
  const LanePart<float, C> v(p, 0, j.N, j.bias >= 0 ? static_cast<const float*>(a.bias) + j.bias : nullptr);
  const LanePart<float, C> u(p, 0, j.K, nullptr);  // the channels of x
  const int i16 = v.i16, g4 = v.g4, tu = (p.wave >> 1) * H, tv = (p.wave & 1) * H, first = 16 * MT * v.wa;
  const bool same = GATED && D == 1 && j.main.src.off == j.gate.src.off;  // the gates' rows are the map's
  const bool sloped = !GATED && D == 1 && j.even && j.act != TPCONV_ACT_IDENTITY;
  const bool again = GATED || sloped;                                      // products are formed again
  const bool sums = GATED || (D == 1 && j.even);                           // column sums: the bias's gradient
  const bool to_x = a.grad_x != nullptr && !(GATED && D == 1 && j.even);
  float* const xs = lds;
  float* const gs = xs + TA * P;
  float* const x0s = gs + TA * P;
  float* const dzs = x0s + (same ? 0 : TA * P0);
  Mover<float, C * D, TA, P, true, X8> mx;
  Mover<float, C, TA, P0, true, X8> m0;
  Mover<float, C * D, TA, P, true, false> mg;
  int64_t base = int64_t(index) * TA;
  int rows = static_cast<int>(min<int64_t>(TA, a.n_rows - base));
  auto issue = [&]() __attribute__((always_inline)) {
    mx.issue(p, j.main.src, base, rows, 0, j.K, D);
    if (GATED && !same) m0.issue(p, j.gate.src, base, rows, 0, j.K0, 1);
    if (!GATED && !again) mg.issue(p, j.g, base, rows, 0, j.N, D);
  };
  issue();
  float w[KS], wt[KS], wg[GATED ? KS : 1];
  if (again) load_weights<float, KS, false>(j.main, v.n, g4, 0, j.K, w);
  // the transposed ones with grad_x alone: without it a linear map may have none to read (weights NULL)
#pragma unroll
  for (int s = 0; s < KS; ++s) wt[s] = 0;
  if (to_x) load_weights<float, KS, true>(j.main, u.n, g4, 0, j.N, wt);
  if constexpr (GATED) load_weights<float, KS, false>(j.gate, j.gate0 + v.n, g4, 0, j.K0, wg);
  // channels that are not there stay zero
  if (j.K < C) clear_channels<float, D, C, P>(p, xs, TA, j.K);
  if (j.N < C) clear_channels<float, D, C, P>(p, gs, TA, j.N);
  if (GATED && !same && j.K0 < C) clear_channels<float, 1, C, P0>(p, x0s, TA, j.K0);
  if (GATED && j.N < C) clear_channels<float, 1, C, P0>(p, dzs, TA, j.N);
  Acc dm[F][F], dw[GATED ? F : 1][GATED ? F : 1];
#pragma unroll
  for (int i = 0; i < F; ++i)
#pragma unroll
    for (int k = 0; k < F; ++k) {
      dm[i][k] = Acc{0, 0, 0, 0};
      if constexpr (GATED) dw[i][k] = Acc{0, 0, 0, 0};
    }
  float column[4] = {0, 0, 0, 0};
  for (int64_t t = int64_t(index) * TA; t < a.n_rows; t += int64_t(j.blocks) * TA) {
    const int64_t here = base;
    const int held = rows, own = held - first;
    __syncthreads();  // the last tile is multiplied
    mx.land(p, xs, held, j.K * D);
    if (GATED && !same) m0.land(p, x0s, held, j.K0);
    if (!GATED && !again) mg.land(p, gs, held, j.N * D);
    if (held < TA) {  // atoms that are not there count for nothing in the sums
      for (int q = p.tid; q < (TA - held) * P; q += 64 * kWaves) {
        xs[held * P + q] = 0;
        if (!again) gs[held * P + q] = 0;
      }
      if (GATED && !same)
        for (int q = p.tid; q < (TA - held) * P0; q += 64 * kWaves) x0s[held * P0 + q] = 0;
    }
    __syncthreads();
    float g[MT][4 * D];
    if (again) {
#pragma unroll
      for (int i = 0; i < MT; ++i) {
#pragma unroll
        for (int e = 0; e < 4 * D; ++e) g[i][e] = 0;
        if (16 * i + i16 < own && v.there > 0)
          load_run<float, D>(g[i],
                             static_cast<const float*>(j.g.rows) + (here + first + 16 * i + i16) * a.ld_g + j.g.off +
                                 v.c0 * D,
                             true, 4);
      }
    }
    if (t + int64_t(j.blocks) * TA < a.n_rows) {
      base = t + int64_t(j.blocks) * TA;
      rows = static_cast<int>(min<int64_t>(TA, a.n_rows - base));
      issue();
    }
    if (again) {
      Acc z[MT][1], slope[MT], pr[MT][D];
      if constexpr (GATED) {
        clear_sums<float, MT, 1>(z);
        if (D == 1 && same)
          multiply<float, 1, KS, MT, P>(xs + first * P, i16, g4, own, wg, z);
        else
          multiply<float, 1, KS, MT, P0>(x0s + first * P0, i16, g4, own, wg, z);
        activate_gates<float, MT, true>(j.act, v.bias, z, slope);
      }
      clear_sums<float, MT, D>(pr);
      multiply<float, D, KS, MT, P>(xs + first * P, i16, g4, own, w, pr);
      if constexpr (!GATED && D == 1)
        for_activation(j.act, [&](auto kind) __attribute__((always_inline)) {
#pragma unroll
          for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) pr[i][0][q] = slope_of<decltype(kind)::value>(pr[i][0][q] + v.bias[q]);
        });
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const bool in = 16 * i + i16 < own;
        const int64_t row = here + first + 16 * i + i16;
        float dz[4] = {0, 0, 0, 0};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
#pragma unroll
          for (int m = 0; m < D; ++m) {
            const float r = pr[i][m][q];
            float& e = g[i][q * D + m];
            if constexpr (GATED) {
              dz[q] = fma(e, r, dz[q]);
              e = in ? e * z[i][0][q] : 0.0f;
            } else {
              e = in ? e * r : 0.0f;
            }
          }
          if constexpr (GATED) dz[q] = in ? dz[q] * slope[i][q] : 0.0f;
          if (sums) column[q] += GATED ? dz[q] : g[i][q];
        }
        if (v.there > 0) {
          store_run<float, D>(g[i], gs + (first + 16 * i + i16) * P + v.c0 * D, true, 4);
          if constexpr (GATED) {
            store_run<float, 1>(dz, dzs + (first + 16 * i + i16) * P0 + v.c0, true, 4);
            if (in && a.grad_x != nullptr) {
              store_run<float, 1>(dz, a.dz + row * a.n_gates + j.gate0 + v.c0, true, 4);
              if (D == 1 && j.even) store_run<float, D>(g[i], a.du + row * a.n_scalars + v.c0, true, 4);
            }
          }
        }
      }
      __syncthreads();
    } else if (sums) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
        if (16 * i + i16 < own && v.there > 0)
#pragma unroll
          for (int q = 0; q < 4; ++q) column[q] += gs[(first + 16 * i + i16) * P + v.c0 + q];
    }
    if (to_x) {
      Acc acc[MT][D];
      clear_sums<float, MT, D>(acc);
      multiply<float, D, KS, MT, P>(gs + first * P, i16, g4, own, wt, acc);
#pragma unroll
      for (int i = 0; i < MT; ++i)
        if (16 * i + i16 < own && u.there > 0) {
          float out[4 * D];
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int m = 0; m < D; ++m) out[q * D + m] = acc[i][m][q];
          store_run<float, D>(out, a.grad_x + (here + first + 16 * i + i16) * a.ld_x + j.x_off + u.c0 * D, true, 4);
        }
    }
    if (a.params) {
      outer<D, TA, P, P, F>(xs, gs, i16, g4, tu, tv, held, dm);
      if constexpr (GATED) {
        if (D == 1 && same)
          outer<1, TA, P, P0, F>(xs, dzs, i16, g4, tu, tv, held, dw);
        else
          outer<1, TA, P0, P0, F>(x0s, dzs, i16, g4, tu, tv, held, dw);
      }
    }
  }
  if (!a.params) return;
  const int64_t numel = int64_t(j.K) * j.N, gated = GATED ? int64_t(j.K0) * j.N : 0;
  float* const to = a.part + j.at + index * (numel + gated + (sums ? j.N : 0));
  write_outer<F>(to, dm, i16, g4, tu, tv, j.K, j.N);
  if constexpr (GATED) write_outer<F>(to + numel, dw, i16, g4, tu, tv, j.K0, j.N);
  if (sums) {  // over the lanes' atoms, then the wavefronts with the same channels, in order
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 4; ++q) column[q] = sum16(column[q]);
    if (i16 == 0)
#pragma unroll
      for (int q = 0; q < 4; ++q) lds[v.wa * C + v.c0 + q] = column[q];
    __syncthreads();
    if (p.tid < j.N) {
      float s = lds[p.tid];
#pragma unroll
      for (int q = 1; q < 64 / C; ++q) s += lds[q * C + p.tid];
      to[numel + gated + p.tid] = s;
    }
  }
}

template <int C, bool GATED, bool X8>
__global__ __launch_bounds__(64 * kWaves, 2) void k_back(BackArgs a) {
  extern __shared__ char dynamic[];
  int ji = 0;
  while (ji + 1 < a.n_jobs && static_cast<int>(blockIdx.x) >= a.job[ji + 1].first) ++ji;
  const BackJob j = a.job[ji];
  const int index = static_cast<int>(blockIdx.x) - j.first;
  if (index >= j.blocks) return;
  float* const lds = reinterpret_cast<float*>(dynamic);
  switch (j.d) {
    case 1: back_job<1, C, GATED, X8>(a, j, index, lds); break;
    case 3: back_job<3, C, GATED, X8>(a, j, index, lds); break;
    case 5: back_job<5, C, GATED, X8>(a, j, index, lds); break;
    case 7: back_job<7, C, GATED, X8>(a, j, index, lds); break;
    default: break;
  }
}

template <int C, bool GATED, bool X8>
hipError_t launch_back(BackArgs& a, hipStream_t s) {
  size_t lds = 0;
  for (int i = 0; i < a.n_jobs; ++i) {
    const BackJob& j = a.job[i];
    const bool same = j.main.src.off == j.gate.src.off && j.d == 1;
    lds = std::max(lds, sizeof(float) * atoms_of<float>(j.d, C) *
                            (2 * pitch_of<float>(j.d, C) + (GATED ? (same ? 1 : 2) * pitch_of<float>(1, C) : 0)));
  }
  const BackJob& last = a.job[a.n_jobs - 1];
  auto* const f = k_back<C, GATED, X8>;
  if (lds > 64 * 1024) {  // above the default limit of dynamic LDS
    const hipError_t he = hipFuncSetAttribute(reinterpret_cast<const void*>(f),
                                              hipFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(lds));
    if (he != hipSuccess) return he;
  }
  hipLaunchKernelGGL(f, dim3(last.first + last.blocks), dim3(64 * kWaves), lds, s, a);
  return hipGetLastError();
}

}  // namespace

template <bool GATED, bool X8>
hipError_t run_back(BackArgs& a, int C, hipStream_t s) {
  return C == 32 ? launch_back<32, GATED, X8>(a, s) : launch_back<64, GATED, X8>(a, s);
}

template hipError_t run_back<TPCONV_GATED, false>(BackArgs&, int, hipStream_t);
template hipError_t run_back<TPCONV_GATED, true>(BackArgs&, int, hipStream_t);

}  // namespace dense
}  // namespace tpconv
