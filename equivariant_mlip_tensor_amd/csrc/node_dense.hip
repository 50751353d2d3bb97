// node_dense.hip -- the linear and gated maps' parameters' gradients, and the
// passes that make up their calls (the products themselves: node_dense.hpp).
#include "node_dense.hpp"

namespace tpconv {
namespace dense {
namespace {

// --------------------------------------------------------- parameters' gradients
// dM[u][v] = sum over atoms and components of x[i][u][m] g[i][v][m]: a matrix
// product whose inner dimension is the (atom, component) pairs.  A block takes
// one S x S tile of a map's matrix and a run of atoms, a few of them at a time
// in LDS as they lie in memory (the pitch makes the next atom's channels go on
// where the 16 of one end, so 4 atoms times 16 channels fall into as many banks);
// its 4 wavefronts share the tile.  Runs' matrices go to the workspace and are
// added in order; one run writes the gradient itself.  The first row of tiles
// also sums its columns of g, for the bias.
// Only plans that the one pass over the rows does not take come here.  Bound by
// latency at their sizes: 2048 fp64 rows of 16 channels l <= 4, with gates, 10 us
// (x and du: 13 MB); 28000 fp32 rows of 64 channels l <= 3 by this way took 97 us
// (229 MB, 2.4 TB/s).
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
  ParamJob job[kMaxMaps + 1];
};

template <class T>
constexpr int tile_side() {
  return sizeof(T) == 4 ? 64 : 32;
}
// atoms of a stage, a multiple of 4
constexpr int stage_atoms(int d) { return d == 1 ? 32 : (d == 3 ? 16 : 8); }

template <class T, int D, bool VEC, bool X8>
__device__ __forceinline__ void param_tile(const ParamArgs& a, const ParamJob& j, int uv, int run, T* lds) {
  constexpr int S = tile_side<T>(), SA = stage_atoms(D), P = S * D + 16, H = S / 2, F = H / 16;
  using Acc = typename Mfma<T>::Acc;
  const Place p;
  const int tid = p.tid, w = p.wave, i16 = p.lane & 15, g4 = p.lane >> 4;
  const int u0 = uv / j.nv * S, v0 = uv % j.nv * S;
  const int nu = min(S, j.x.K - u0), nv = min(S, j.g.K - v0);
  const int64_t from = run * j.run, upto = min(from + j.run, a.n_rows);
  T* const xs = lds;
  T* const gs = lds + SA * P;
  Mover<T, S * D, SA, P, VEC, X8> mx;
  Mover<T, S * D, SA, P, VEC, false> mg;
  auto issue = [&](int64_t base) {
    const int rows = static_cast<int>(min<int64_t>(SA, upto - base));
    mx.issue(p, j.x, base, rows, u0, nu, D);
    mg.issue(p, j.g, base, rows, v0, nv, D);
  };
  if (from < upto) issue(from);
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
    mx.land(p, xs, rows, nu * D);
    mg.land(p, gs, rows, nv * D);
    for (int q = tid; q < (SA - rows) * P; q += 256) xs[rows * P + q] = gs[rows * P + q] = T(0);
    __syncthreads();
    if (base + SA < upto) issue(base + SA);
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

template <class T, bool X8>
__global__ __launch_bounds__(64 * kWaves, 2) void k_param(ParamArgs a) {
  extern __shared__ char dynamic[];
  const int block = static_cast<int>(blockIdx.x);
  int ji = 0;
  while (ji + 1 < a.n_jobs && block >= a.job[ji + 1].first) ++ji;
  const ParamJob j = a.job[ji];
  const int r = block - j.first, uv = r % (j.nu * j.nv), run = r / (j.nu * j.nv);
  T* const lds = reinterpret_cast<T*>(dynamic);
  const bool vec = j.x.packed && j.g.packed;
#define TPCONV_PARAM(D)                                \
  case D:                                              \
    if (vec)                                           \
      param_tile<T, D, true, X8>(a, j, uv, run, lds);  \
    else                                               \
      param_tile<T, D, false, X8>(a, j, uv, run, lds); \
    break;
  switch (j.d) {
    TPCONV_PARAM(1)
    TPCONV_PARAM(3)
    TPCONV_PARAM(5)
    TPCONV_PARAM(7)
    TPCONV_PARAM(9)
    default: break;
  }
#undef TPCONV_PARAM
}

// The runs' matrices and column sums, added in order in 64 bits: 64 values a
// block, its 16 wavefronts every 16th run.
struct JoinJob {
  int64_t at, per;          // first value; values of a run
  int32_t rows, cols, sums; // a matrix, and column sums after it, of those values
  int32_t ld;               // of the matrix in the gradient
  int32_t runs, first;
  void *matrix, *columns;
};
struct JoinArgs {
  int32_t n_jobs;
  JoinJob job[2 * kMaxMaps];
};

template <class T>
__global__ __launch_bounds__(1024) void k_param_join(JoinArgs a, const T* __restrict__ part) {
  __shared__ double sums[16][64];
  int ji = 0;
  while (ji + 1 < a.n_jobs && static_cast<int>(blockIdx.x) >= a.job[ji + 1].first) ++ji;
  const JoinJob j = a.job[ji];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int q = (static_cast<int>(blockIdx.x) - j.first) * 64 + lane, numel = j.rows * j.cols, held = numel + j.sums;
  double v = 0;
  if (q < held) {
#pragma unroll 4
    for (int r = w; r < j.runs; r += 16) v += double(part[j.at + r * j.per + q]);
  }
  sums[w][lane] = v;
  __syncthreads();
  if (w > 0 || q >= held) return;
  v = 0;
#pragma unroll
  for (int r = 0; r < 16; ++r) v += sums[r][lane];
  if (q < numel) {
    if (j.matrix != nullptr) static_cast<T*>(j.matrix)[q / j.cols * j.ld + q % j.cols] = static_cast<T>(v);
  } else if (j.columns != nullptr) {
    static_cast<T*>(j.columns)[q - numel] = static_cast<T>(v);
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

// Whether rows' channels can be taken four at a time, 16 bytes apart or a multiple of it.
template <class T>
bool in_fours(const void* p, int64_t ld, int64_t off, int64_t channels) {
  constexpr int per = 16 / sizeof(T);
  return aligned16(p) && ld % per == 0 && off % per == 0 && channels % 4 == 0;
}

// x's segment s_in as a source
template <class T>
RowSource source_of(const Dense& p, const DenseInput& x, int32_t off, int32_t mul, int d, int seg) {
  RowSource r{};
  r.ld = static_cast<int32_t>(p.dim_in);
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
  r.ld = static_cast<int32_t>(ld);
  r.off = off;
  r.K = mul;
  r.packed = pieces16<T>(rows, ld, off, int64_t(mul) * d);
  return r;
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
  a.ld_out = static_cast<int32_t>(p.dim_out);
  a.n_gates = static_cast<int32_t>(p.n_gates);
  a.out = out;
  a.extra = residual;
  forward_jobs<T>(p, DenseInput{x, nullptr, nullptr}, weights, gate_weights, bias, a, false);
  for (int i = 0; i < a.n_jobs; ++i) {
    DenseJob& j = a.job[i];
    j.packed_out = in_fours<T>(out, p.dim_out, j.out_off, j.N) && aligned16(residual);
  }
  return p.gated ? run_dense<T, kGated, false>(a, s) : run_dense<T, kLinear, false>(a, s);
}

}  // namespace

int64_t cut_back(BackArgs& a, int C, bool gated) {
  int64_t parts = 0, tiles[kMaxMaps], cost[kMaxMaps];
  int32_t shares[kMaxMaps], of[kMaxMaps];
  for (int i = 0; i < a.n_jobs; ++i) {
    const BackJob& j = a.job[i];
    const int atoms = atoms_of<float>(j.d, C);
    tiles[i] = (a.n_rows + atoms - 1) / atoms;
    // products a tile: the map's, its transposed one (but gated 0e's) and its gradient's, the gates' and their gradient's;
    // linear: what the tile's way through LDS takes beside them (with the sums' join, with and without it, 28000 rows of
    // 64 channels l <= 3: 118 and 124 us, of 48 109 and 115, of 64 l <= 2 88 and 84, l <= 1 51 and 46, 80000 of the last
    // two 193 and 224, 129 and 128)
    const bool sloped = !gated && j.even && j.act != TPCONV_ACT_IDENTITY;
    cost[i] = atoms * (gated ? 3 * j.d + 2 - (j.even ? 1 : 0) : 2 * j.d + (sloped ? 1 : 0)) + (gated ? 0 : 128);
    shares[i] = 1;
  }
  share_out(a.n_jobs, tiles, cost, shares, back_blocks(gated, a.n_jobs), of);
  int32_t blocks = 0;
  for (int i = 0; i < a.n_jobs; ++i) {
    BackJob& j = a.job[i];
    j.first = blocks;
    j.blocks = of[i];
    blocks += (j.blocks + 7) / 8 * 8;
    j.at = parts;
    parts += j.blocks * (int64_t(j.K) * j.N + int64_t(j.K0) * j.N + (gated || (j.d == 1 && j.even) ? j.N : 0));
  }
  return parts;
}

namespace {

// How the atoms of the parameters' jobs are cut into runs: about kParamBlocks
// blocks of equal work, a run a whole number of stages.
constexpr int kParamBlocks = 1024;  // 4 for each CU

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
  size_t gates, parts, total;  // du of the rows, or the even scalars' gradient, stands at 0
};

// Whether the gradients' one pass over the rows takes the plan (its LDS and registers hold 64 channels of l <= 3 in
// fp32), and with how many channels; 0: it does not.
int back_channels(const Dense& p) {
  int most = p.gated ? p.scalar_mul : 1;
  if (p.f64) return 0;
  for (const DenseMap& m : p.maps) {
    if (m.d > 7 || m.mul_in % 4 != 0 || m.mul_out % 4 != 0) return 0;
    most = std::max({most, m.mul_in, m.mul_out});
  }
  return most <= 32 ? 32 : (most <= 64 ? 64 : 0);
}

// The jobs' sizes for the one pass.
void back_jobs(const Dense& p, BackArgs& a) {
  a.n_jobs = 0;
  for (const DenseMap& m : p.maps) {
    BackJob& j = a.job[a.n_jobs++];
    j.d = m.d;
    j.K = m.mul_in;
    j.N = m.mul_out;
    j.K0 = p.gated ? p.scalar_mul : 0;
    j.x_off = m.in_off;
    j.gate0 = m.gate;
    j.act = m.act;
    j.even = m.even;
  }
}

template <class T>
DenseSpace dense_space(const Dense& p, int64_t n_rows) {
  DenseSpace w{};
  const ParamShape h = param_shape<T>(p, n_rows);
  size_t at = 0;
  if (p.gated) {
    at = align_up(sizeof(T) * static_cast<size_t>(n_rows) * p.dim_out);
    w.gates = at;
    at += align_up(sizeof(T) * static_cast<size_t>(n_rows) * p.n_gates);
  } else if (p.sloped()) {
    at = align_up(sizeof(T) * static_cast<size_t>(n_rows) * p.scalar_out_mul);
  }
  w.parts = at;
  size_t parts = h.single ? 0 : align_up(sizeof(T) * static_cast<size_t>(h.total));
  if (const int C = back_channels(p)) {
    BackArgs a{};
    a.n_rows = n_rows;
    back_jobs(p, a);
    parts = std::max(parts, align_up(sizeof(T) * static_cast<size_t>(cut_back(a, C, p.gated))));
  }
  w.total = at + parts;
  return w;
}

template <class T>
hipError_t clear_bare(const Dense& p, int64_t n_rows, void* grad_x, hipStream_t s) {
  for (const ColumnRun& r : p.bare_in) {
    const int64_t b = (n_rows * r.len + 255) / 256;
    hipLaunchKernelGGL(k_clear_columns<T>, dim3(static_cast<unsigned>(b > 65536 ? 65536 : b)), dim3(256), 0, s, n_rows,
                       p.dim_in, r.off, r.len, static_cast<T*>(grad_x));
    const hipError_t he = hipGetLastError();
    if (he != hipSuccess) return he;
  }
  return hipSuccess;
}

// A job of the transposed products: grad_x of channels N from rows `src`.
template <class T>
void transposed_job(DenseJob& j, const RowSource& src, const void* weights, int32_t ldw, int d, int N, int32_t off,
                    void* grad_x, int64_t ld) {
  j.main.src = src;
  j.main.weights = weights;
  j.main.ldw = ldw;
  j.main.packed = pieces16<T>(weights, ldw, 0, 0);
  j.d = d;
  j.N = N;
  j.out_off = off;
  j.bias = -1;
  j.packed_out = in_fours<T>(grad_x, ld, off, N);
}

// Gated: the even scalars' gradient, from their own map's rows (`du`, or none) and the gates'.
template <class T>
void even_job(const Dense& p, DenseJob& j, const RowSource* du, const DenseMap* m, const T* dz, const void* weights,
              const void* gate_weights, void* grad_x) {
  const RowSource gates = source_rows<T>(dz, p.n_gates, 0, static_cast<int32_t>(p.n_gates), 1);
  const int32_t ldg = static_cast<int32_t>(p.n_gates);
  if (du == nullptr) {
    transposed_job<T>(j, gates, gate_weights, ldg, 1, p.scalar_mul, p.scalar_off, grad_x, p.dim_in);
    return;
  }
  transposed_job<T>(j, *du, static_cast<const T*>(weights) + m->woff, m->mul_out, 1, p.scalar_mul, p.scalar_off, grad_x,
                    p.dim_in);
  j.gate.src = gates;
  j.gate.weights = gate_weights;
  j.gate.ldw = ldg;
  j.gate.packed = pieces16<T>(gate_weights, ldg, 0, 0);
}

// The gradients in one pass over the rows (node_dense_back.hip), where the plan and the rows' places allow it.
hipError_t back_in_one(const Dense& p, int64_t n_rows, const DenseInput& x, const void* weights,
                       const void* gate_weights, const void* bias, const void* grad_out, void* grad_x,
                       void* grad_weights, void* grad_gate_weights, void* grad_bias, char* mem,
                       const DenseSpace& space, hipStream_t s, bool& done) {
  using T = float;
  const int C = back_channels(p);
  const bool params = grad_weights != nullptr || grad_gate_weights != nullptr || grad_bias != nullptr;
  // rows alone of a linear map without activation have nothing to share
  if (C == 0 || n_rows == 0 || (!params && !p.gated && !p.sloped())) return hipSuccess;
  const bool x8 = x.codes != nullptr;
  BackArgs a{};
  a.n_rows = n_rows;
  back_jobs(p, a);
  cut_back(a, C, p.gated);
  bool fits = in_fours<T>(grad_out, p.dim_out, 0, 0) && (grad_x == nullptr || in_fours<T>(grad_x, p.dim_in, 0, 0));
  for (int i = 0; i < a.n_jobs; ++i) {
    const DenseMap& m = p.maps[i];
    BackJob& j = a.job[i];
    j.main.src = source_of<T>(p, x, m.in_off, m.mul_in, m.d, m.seg_in);
    j.main.weights = static_cast<const T*>(weights) + m.woff;
    j.main.ldw = m.mul_out;
    j.main.packed = pieces16<T>(j.main.weights, m.mul_out, 0, 0);
    j.g = source_rows<T>(grad_out, p.dim_out, m.out_off, m.mul_out, m.d);
    j.bias = -1;
    fits = fits && j.main.src.packed && j.g.packed && m.in_off % 4 == 0;
    if (p.gated) {
      j.gate.src = source_of<T>(p, x, p.scalar_off, p.scalar_mul, 1, p.scalar_seg);
      j.gate.weights = gate_weights;
      j.gate.ldw = static_cast<int32_t>(p.n_gates);
      fits = fits && j.gate.src.packed && m.gate % 4 == 0;
      if (bias != nullptr) j.bias = m.gate;
    } else if (m.even && bias != nullptr) {
      j.bias = 0;
    }
  }
  if (!fits) return hipSuccess;
  done = true;
  a.ld_x = static_cast<int32_t>(p.dim_in);
  a.ld_g = static_cast<int32_t>(p.dim_out);
  a.n_gates = static_cast<int32_t>(p.n_gates);
  a.n_scalars = p.scalar_out_mul;
  a.params = params;
  a.bias = bias;
  a.grad_x = static_cast<T*>(grad_x);
  a.du = reinterpret_cast<T*>(mem);
  a.dz = reinterpret_cast<T*>(mem + space.gates);
  a.part = reinterpret_cast<T*>(mem + space.parts);
  hipError_t he = p.gated ? (x8 ? run_back<true, true>(a, C, s) : run_back<true, false>(a, C, s))
                          : (x8 ? run_back<false, true>(a, C, s) : run_back<false, false>(a, C, s));
  if (he != hipSuccess) return he;
  if (grad_x != nullptr) {
    if (p.gated) {
      const DenseMap* even = nullptr;
      for (const DenseMap& m : p.maps)
        if (m.even) even = &m;
      RowSource du{};
      if (even != nullptr) du = source_rows<T>(a.du, p.scalar_out_mul, 0, even->mul_out, 1);
      DenseArgs t{};
      t.n_rows = n_rows;
      t.out = grad_x;
      t.ld_out = static_cast<int32_t>(p.dim_in);
      t.n_jobs = 1;
      even_job<T>(p, t.job[0], even != nullptr ? &du : nullptr, even, a.dz, weights, gate_weights, grad_x);
      he = run_dense<T, kTransposed, false>(t, s);
      if (he != hipSuccess) return he;
    }
    he = clear_bare<T>(p, n_rows, grad_x, s);
    if (he != hipSuccess) return he;
  }
  if (!params) return hipSuccess;
  JoinArgs join{};
  int joins = 0;
  auto add = [&](const BackJob& j, int64_t at, int rows, int sums, int ld, T* matrix, T* columns) {
    if (matrix == nullptr && columns == nullptr) return;
    const int64_t per = int64_t(j.K + j.K0) * j.N + (p.gated || (j.d == 1 && j.even) ? j.N : 0);
    join.job[join.n_jobs++] = JoinJob{j.at + at, per, rows, j.N, sums, ld, j.blocks, joins, matrix, columns};
    joins += (rows * j.N + sums + 63) / 64;
  };
  for (int i = 0; i < a.n_jobs; ++i) {
    const BackJob& j = a.job[i];
    T* const gw = grad_weights != nullptr ? static_cast<T*>(grad_weights) + p.maps[i].woff : nullptr;
    const int64_t numel = int64_t(j.K) * j.N;
    if (p.gated) {
      add(j, 0, j.K, 0, j.N, gw, nullptr);
      add(j, numel, j.K0, j.N, static_cast<int>(p.n_gates),
          grad_gate_weights != nullptr ? static_cast<T*>(grad_gate_weights) + j.gate0 : nullptr,
          grad_bias != nullptr ? static_cast<T*>(grad_bias) + j.gate0 : nullptr);
    } else {
      add(j, 0, j.K, j.d == 1 && j.even ? j.N : 0, j.N, gw, j.even ? static_cast<T*>(grad_bias) : nullptr);
    }
  }
  if (joins == 0) return hipSuccess;
  hipLaunchKernelGGL(k_param_join<T>, dim3(static_cast<unsigned>(joins)), dim3(1024), 0, s, join,
                     static_cast<const T*>(a.part));
  return hipGetLastError();
}

template <class T>
hipError_t dense_backward(const Dense& p, int64_t n_rows, const DenseInput& x, const void* weights,
                          const void* gate_weights, const void* bias, const void* grad_out, void* grad_x,
                          void* grad_weights, void* grad_gate_weights, void* grad_bias, void* ws, hipStream_t s) {
  const DenseSpace space = dense_space<T>(p, n_rows);
  char* const mem = static_cast<char*>(ws);
  if constexpr (sizeof(T) == 4) {
    bool done = false;
    const hipError_t he = back_in_one(p, n_rows, x, weights, gate_weights, bias, grad_out, grad_x, grad_weights,
                                      grad_gate_weights, grad_bias, mem, space, s, done);
    if (he != hipSuccess || done) return he;
  }
  // grad_out through the activations: rows (gated), their gates, or the even scalars alone (linear)
  T* const dz = reinterpret_cast<T*>(p.gated ? mem + space.gates : mem);
  const T* du = static_cast<const T*>(grad_out);
  if (p.gated || p.sloped()) {
    DenseArgs a{};
    a.n_rows = n_rows;
    a.ld_g = static_cast<int32_t>(p.dim_out);
    a.n_gates = static_cast<int32_t>(p.n_gates);
    a.extra = grad_out;
    forward_jobs<T>(p, x, weights, gate_weights, bias, a, !p.gated);
    if (p.gated) {
      du = reinterpret_cast<T*>(mem);
      a.out = mem;
      a.ld_out = static_cast<int32_t>(p.dim_out);
      a.dz = dz;
    } else {
      a.out = dz;
      a.ld_out = p.scalar_out_mul;
      a.job[0].out_off = 0;
    }
    for (int i = 0; i < a.n_jobs; ++i) {
      DenseJob& j = a.job[i];
      j.packed_g = in_fours<T>(grad_out, p.dim_out, j.g_off, j.N);
      j.packed_out = in_fours<T>(a.out, a.ld_out, j.out_off, j.N);
      j.packed_dz = p.gated && in_fours<T>(a.dz, a.n_gates, j.gate0, j.N);
    }
    const bool x8 = x.codes != nullptr;
    auto go = [&](auto codes) {
      return p.gated ? run_dense<T, kGatedGrad, decltype(codes)::value>(a, s)
                     : run_dense<T, kLinearGrad, decltype(codes)::value>(a, s);
    };
    hipError_t he;
    if constexpr (sizeof(T) == 4)
      he = x8 ? go(std::true_type{}) : go(std::false_type{});
    else
      he = go(std::false_type{});
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
    a.ld_out = static_cast<int32_t>(p.dim_in);
    for (const DenseMap& m : p.maps) {
      const RowSource src = grad_rows(m);
      if (p.gated && m.even)
        even_job<T>(p, a.job[a.n_jobs++], &src, &m, dz, weights, gate_weights, grad_x);
      else
        transposed_job<T>(a.job[a.n_jobs++], src, static_cast<const T*>(weights) + m.woff, m.mul_out, m.d, m.mul_in,
                          m.in_off, grad_x, p.dim_in);
    }
    if (p.gated && !p.even_out)  // the even scalars reach the gates alone
      even_job<T>(p, a.job[a.n_jobs++], nullptr, nullptr, dz, weights, gate_weights, grad_x);
    hipError_t he = run_dense<T, kTransposed, false>(a, s);
    if (he == hipSuccess) he = clear_bare<T>(p, n_rows, grad_x, s);
    if (he != hipSuccess) return he;
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
    q = JoinJob{h.at[i], h.per[i], h.U[i], h.V[i], h.sums[i] ? h.V[i] : 0, h.V[i], h.runs[i], joins, matrix, sums};
    joins += static_cast<int>((h.per[i] + 63) / 64);
    lds = std::max(lds, sizeof(T) * 2 * stage_atoms(j.d) * (tile_side<T>() * j.d + 16));
  }
  join.n_jobs = a.n_jobs;
  if (a.n_jobs == 0) return hipSuccess;
  auto* f = k_param<T, false>;
  if constexpr (sizeof(T) == 4)
    if (x.codes != nullptr) f = k_param<T, true>;
  hipLaunchKernelGGL(f, dim3(static_cast<unsigned>(blocks)), dim3(64 * kWaves), lds, s, a);
  hipError_t he = hipGetLastError();
  if (he != hipSuccess || h.single) return he;
  hipLaunchKernelGGL(k_param_join<T>, dim3(static_cast<unsigned>(joins)), dim3(1024), 0, s, join,
                     static_cast<const T*>(a.part));
  return hipGetLastError();
}

}  // namespace
}  // namespace dense

using namespace dense;

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
