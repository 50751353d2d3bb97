// node_experts.hip -- the experts' equivariant maps on irreps rows and their
// gradients:
//   out[i][v][m]    = sum_a g_ia sum_u M_e[u][v] x[i][u][m],  e = e(i, a)
//   grad_x[i][u][m] = sum_a g_ia sum_v M_e[u][v] G[i][v][m]
//   grad_g[i][a]    = sum_{u,m} x[i][u][m] (M_e G_i)[u][m]
//   grad_M_e[u][v]  = sum_{(i,a): e(i,a) = e} g_ia sum_m x[i][u][m] G[i][v][m]
// for each pair of equal (l, parity) segments.  A row has 2l+1 components that
// all see the same matrix, so a map is a matrix product whose rows are the
// (atom, component) pairs of an expert's atoms; it runs on the matrix cores
// (v_mfma_f32_16x16x4f32, v_mfma_f64_16x16x4f64: the library's data types).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "node_internal.hpp"

namespace tpconv {
namespace {

// ------------------------------------------------------------ matrix cores
// D[i][j] += sum_k A[i][k] B[k][j], 16 x 16 x 4: lane holds A[lane % 16]
// [lane / 16], B[lane / 16][lane % 16] and the four D[row(lane / 16, r)][lane % 16].
template <class T>
struct Mfma;
template <>
struct Mfma<float> {
  typedef float Acc __attribute__((ext_vector_type(4)));
  static __device__ __forceinline__ Acc step(float a, float b, Acc c) {
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ int row(int g, int r) { return 4 * g + r; }
};
template <>
struct Mfma<double> {
  typedef double Acc __attribute__((ext_vector_type(4)));
  static __device__ __forceinline__ Acc step(double a, double b, Acc c) {
    return __builtin_amdgcn_mfma_f64_16x16x4f64(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ int row(int g, int r) { return 4 * r + g; }
};

template <class T>
struct alignas(16) Pack {  // one 16-byte load
  T v[16 / sizeof(T)];
};

int blocks_for(int64_t n, int block) {
  const int64_t g = (n + block - 1) / block;
  return static_cast<int>(g < 1 ? 1 : (g > 65536 ? 65536 : g));
}

size_t align_up(size_t v) { return (v + 255) / 256 * 256; }

// ------------------------------------------------------------------ layout
// Rows are taken in groups of kGroup (or n / 64 when that is more, so that
// there are at most 64 groups); each group is sorted by itself, which needs
// no exchange between blocks: one launch whatever the size.
//   order    the group's rows by the pair (smallest, next) of their experts, so
//            that a tile of consecutive rows meets few experts
//   entries  the group's entries (row * top_k + place) by expert, entries of an
//            expert in ascending order (the sums over them are taken in it)
//   first    [group][X + 1] where each expert's entries start in `entries`,
//            relative to the group's first
//   piece    [group][X + 1] the same in pieces of at most kPiece entries
constexpr int64_t kGroup = 2048;
constexpr int kMaxBins = 4096;
constexpr int kPiece = 256;

struct LayoutShape {
  int64_t group, n_groups;
  int64_t max_pieces;  // pieces of a group, at most
  size_t order, entries, first, pieces, total;
};

LayoutShape layout_shape(int64_t n, int X, int k) {
  LayoutShape L{};
  L.group = std::max<int64_t>(kGroup, (n + 63) / 64);
  L.n_groups = std::max<int64_t>(1, (n + L.group - 1) / L.group);
  const int64_t most = std::min(L.group, std::max<int64_t>(n, 1)) * k;
  L.max_pieces = most / kPiece + X;
  size_t o = 0;
  auto take = [&](int64_t ints) {
    const size_t at = o;
    o = align_up(o + sizeof(int32_t) * static_cast<size_t>(ints));
    return at;
  };
  L.order = take(n);
  L.entries = take(n * k);
  L.first = take(L.n_groups * (X + 1));
  L.pieces = take(L.n_groups * (X + 1));
  L.total = std::max<size_t>(o, 256);
  return L;
}

// Exclusive sum over the block's values (one per thread) plus the total.
__device__ __forceinline__ int block_exclusive(int v, int* wave_sums, int& total) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, nw = blockDim.x >> 6;
  int s = v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int t = __shfl_up(s, o, 64);
    if (lane >= o) s += t;
  }
  __syncthreads();
  if (lane == 63) wave_sums[w] = s;
  __syncthreads();
  int before = 0;
  total = 0;
  for (int q = 0; q < nw; ++q) {
    const int t = wave_sums[q];
    before += q < w ? t : 0;
    total += t;
  }
  return before + s - v;
}

// In-place exclusive sums of n counters in LDS; returns their total.
__device__ int scan_counters(int* c, int n, int* wave_sums) {
  int carry = 0;
  const int per = (n + blockDim.x - 1) / blockDim.x;
  const int at = threadIdx.x * per, end = min(n, at + per);
  int mine = 0;
  for (int q = at; q < end; ++q) mine += c[q];
  int total;
  carry = block_exclusive(mine, wave_sums, total);
  for (int q = at; q < end; ++q) {
    const int t = c[q];
    c[q] = carry;
    carry += t;
  }
  __syncthreads();
  return total;
}

// One block per group.  Bins of the row order: (smallest expert) * H + (next
// * H / X), H = min(X, 4096 / X); rows without experts last.  Rows of one bin
// come in no fixed order (an integer atomic hands out the places): a row's
// results do not depend on its neighbours.  Entries are ranked by counting in
// order, so theirs is fixed.  Latency bound: 28000 rows are 14 blocks.
__global__ __launch_bounds__(1024) void k_layout(int64_t n, int X, int k, int H, int64_t group,
                                                 const int32_t* __restrict__ experts, int32_t* __restrict__ order,
                                                 int32_t* __restrict__ entries, int32_t* __restrict__ first,
                                                 int32_t* __restrict__ pieces) {
  __shared__ int bins[kMaxBins + 1];
  __shared__ int wave_sums[16];
  const int64_t r0 = blockIdx.x * group;
  const int rows = static_cast<int>(min(group, n - r0));
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, nw = blockDim.x >> 6;
  const int32_t* ex = experts + r0 * k;

  auto bin_of = [&](int r) {
    int lo = X, hi = X;
    for (int a = 0; a < k; ++a) {
      const int e = ex[int64_t(r) * k + a];
      if (e < 0 || e >= X) continue;
      if (e < lo) {
        hi = lo;
        lo = e;
      } else if (e > lo && e < hi) {
        hi = e;
      }
    }
    if (lo == X) return X * H;
    if (hi == X) hi = lo;
    return lo * H + hi * H / X;
  };
  for (int q = tid; q <= X * H; q += blockDim.x) bins[q] = 0;
  __syncthreads();
  for (int r = tid; r < rows; r += blockDim.x) atomicAdd(&bins[bin_of(r)], 1);
  __syncthreads();
  scan_counters(bins, X * H + 1, wave_sums);
  for (int r = tid; r < rows; r += blockDim.x)
    order[r0 + atomicAdd(&bins[bin_of(r)], 1)] = static_cast<int32_t>(r0 + r);
  __syncthreads();

  // entries by expert: each wavefront counts, then places, its own run of them;
  // counters [expert][wavefront], scanned in that order
  const int total = rows * k;
  const int run = ((total + nw - 1) / nw + 63) / 64 * 64;
  const int q0 = w * run, q1 = min(total, q0 + run);
  for (int q = tid; q < X * nw; q += blockDim.x) bins[q] = 0;
  __syncthreads();
  for (int q = q0 + lane; q < q1; q += 64) {
    const int e = ex[q];
    if (e >= 0 && e < X) atomicAdd(&bins[e * nw + w], 1);
  }
  __syncthreads();
  const int placed = scan_counters(bins, X * nw, wave_sums);
  int32_t* const fst = first + blockIdx.x * int64_t(X + 1);
  int32_t* const pcs = pieces + blockIdx.x * int64_t(X + 1);
  int mine = 0;  // X <= 256 <= blockDim
  if (tid < X) {
    const int at = bins[tid * nw], end = tid + 1 < X ? bins[(tid + 1) * nw] : placed;
    fst[tid] = at;
    mine = static_cast<int>((end - at + kPiece - 1) / kPiece);
  }
  int n_pieces;
  const int before = block_exclusive(mine, wave_sums, n_pieces);
  if (tid < X) pcs[tid] = before;
  if (tid == 0) {
    fst[X] = placed;
    pcs[X] = n_pieces;
  }
  __syncthreads();
  for (int q = q0; q < q1; q += 64) {
    const int e = q + lane < q1 ? ex[q + lane] : -1;
    const bool live = e >= 0 && e < X;
    uint64_t peers = __ballot(live);  // lanes of this pass with the same expert
#pragma unroll
    for (int b = 0; b < 8; ++b) {
      const uint64_t on = __ballot(live && ((e >> b) & 1));
      peers &= ((e >> b) & 1) ? on : ~on;
    }
    if (live) {
      const int rank = __popcll(peers & ((uint64_t(1) << lane) - 1));
      int base = 0;
      if (rank == 0) base = atomicAdd(&bins[e * nw + w], __popcll(peers));
      base = __shfl(base, __ffsll(static_cast<unsigned long long>(peers)) - 1, 64);
      entries[r0 * k + base + rank] = static_cast<int32_t>(r0 * k + q + lane);
    }
  }
}

// entries of each expert, summed over the groups
__global__ void k_load(int X, int64_t n_groups, const int32_t* __restrict__ first, int32_t* __restrict__ load) {
  const int e = threadIdx.x;
  if (e >= X) return;
  int c = 0;
  for (int64_t g = 0; g < n_groups; ++g) c += first[g * (X + 1) + e + 1] - first[g * (X + 1) + e];
  load[e] = c;
}

// ----------------------------------------------------- rows: out and grad_x
// A block takes a tile of rows (in the layout's order) and one map: the tile's
// segment goes to LDS once, the tile's experts are listed with their member
// rows, and for each expert the members' (row, component) pairs are packed
// into 16-row matrix tiles, so a tile that meets many experts still fills the
// matrix cores.  The products, times the gates, are added into the tile's
// output in LDS, which is written once: x is read once and out written once
// whatever top_k, and each row's sum runs over its experts in ascending order.
// A wavefront owns 16 output channels at a time, so no two wavefronts add into
// the same place.  ADJ runs the transposed maps on grad_out; GG also dots the
// ungated products with x for the gates' gradient (a partial sum per map).
struct RowMap {
  int32_t src_off, dst_off;  // first columns in a row of src / dst
  int32_t K, N;              // channels summed over / produced
  int32_t V;                 // row length of the map's weights
  int32_t d, woff;
  int32_t tile;              // rows of a tile, at most 32
  int32_t ld_src, ld_dst;    // LDS elements between a tile's rows
  int32_t matrix_rows;       // of a tile, at most
  int32_t first;             // first block of this map
  int32_t vec;               // bit 0 / 1: 16-byte aligned rows of src / dst; bit 2: of the weights along K
  uint32_t inv_src, inv_dst; // ceil(2^32 / pieces of a src / dst segment), 0 for one piece
};

struct RowArgs {
  int64_t n_rows, ld_src, ld_dst, weight_numel;
  int32_t X, k, n_maps, waves;
  RowMap map[kMaxMaps];
};

// LDS of a block (byte offsets), for the map that needs most.
struct RowLds {
  uint32_t src, acc, dot, rowsum, mask, start, list, rtab, rgate, rowid, graw, ents, total;
};

// Matrix rows of a tile, each expert's rounded up to 16.
int matrix_rows(int tile, int X, int k, int d) { return tile * k * d + 15 * std::min(X, tile * k); }

RowLds row_lds(const RowMap& m, int X, int k, int waves, bool gg, size_t size) {
  RowLds L{};
  uint32_t o = 0;
  auto take = [&](size_t n, size_t each) {
    const uint32_t at = o;
    o = static_cast<uint32_t>((o + n * each + 15) / 16 * 16);
    return at;
  };
  const size_t t = m.tile, r = matrix_rows(m.tile, X, k, m.d);
  L.src = take(t * m.ld_src, size);
  L.acc = take((t + 1) * m.ld_dst, size);  // the last row takes what the matrix rows past an expert's last one give
  L.dot = take(gg ? (t + 1) * m.ld_dst : 0, size);
  L.rowsum = take(gg ? (t * k * m.d + 1) * waves : 0, size);
  L.mask = take(X, 4);
  L.start = take(X, 4);
  L.list = take(4 * (t * k + 1), 4);
  L.rtab = take(r, 4);
  L.rgate = take(r, size);
  L.rowid = take(t, 8);
  L.graw = take(t * k, size);
  L.ents = take(t * k, 4);
  L.total = o;
  return L;
}

// Sum over the 16 lanes of a row of lanes, in all of them.
template <int CTRL>
__device__ __forceinline__ float rotate16(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, false));
}
template <int CTRL>
__device__ __forceinline__ double rotate16(double v) {
  return __hiloint2double(__builtin_amdgcn_update_dpp(0, __double2hiint(v), CTRL, 0xF, 0xF, false),
                          __builtin_amdgcn_update_dpp(0, __double2loint(v), CTRL, 0xF, 0xF, false));
}
template <class T>
__device__ __forceinline__ T sum16(T v) {  // rotations by 8, 4, 2, 1
  v += rotate16<0x128>(v);
  v += rotate16<0x124>(v);
  v += rotate16<0x122>(v);
  return v + rotate16<0x121>(v);
}

// Visits the `pieces` pieces of each of `rows` rows, kBatch of them a thread at
// a time: every load of a batch is issued before the first is waited for (one
// after the other, a tile of 16 rows took 8 trips to memory).
constexpr int kBatch = 8;

template <class V, class Load, class Store>
__device__ __forceinline__ void move_rows(int rows, int pieces, uint32_t inv, Load load, Store store) {
  const int total = rows * pieces;
  for (int i0 = threadIdx.x; i0 < total; i0 += kBatch * blockDim.x) {
    V v[kBatch];
    int s[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int i = i0 + j * blockDim.x;
      s[j] = inv != 0 ? static_cast<int>(__umulhi(static_cast<uint32_t>(i), inv)) : i;
      if (i < total) v[j] = load(s[j], i - s[j] * pieces);
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int i = i0 + j * blockDim.x;
      if (i < total) store(s[j], i - s[j] * pieces, v[j]);
    }
  }
}

template <class T, int KS, bool ADJ, bool GG>
__global__ __launch_bounds__(256) void k_rows(RowArgs a, RowLds L0, const T* __restrict__ src,
                                              const T* __restrict__ weights, const int32_t* __restrict__ experts,
                                              const T* __restrict__ gates, const int32_t* __restrict__ order,
                                              T* __restrict__ dst, const T* __restrict__ other,
                                              T* __restrict__ gate_part) {
  extern __shared__ char lds[];
  int mi = 0;
  while (mi + 1 < a.n_maps && static_cast<int>(blockIdx.x) >= a.map[mi + 1].first) ++mi;
  const RowMap m = a.map[mi];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, k = a.k, d = m.d;
  const int64_t base = int64_t(static_cast<int>(blockIdx.x) - m.first) * m.tile;
  const int rows = static_cast<int>(min<int64_t>(m.tile, a.n_rows - base));
  T* const xs = reinterpret_cast<T*>(lds + L0.src);
  T* const acc = reinterpret_cast<T*>(lds + L0.acc);
  T* const dot = reinterpret_cast<T*>(lds + L0.dot);
  T* const rowsum = reinterpret_cast<T*>(lds + L0.rowsum);
  uint32_t* const mask = reinterpret_cast<uint32_t*>(lds + L0.mask);  // members of each expert, a bit per row
  uint32_t* const start = reinterpret_cast<uint32_t*>(lds + L0.start);  // their first place << 16 | matrix row
  int* const list = reinterpret_cast<int*>(lds + L0.list);  // the tile's experts: expert, first matrix row, rows, place
  uint32_t* const rtab = reinterpret_cast<uint32_t*>(lds + L0.rtab);  // matrix row -> LDS places in dst << 16 | src
  T* const rgate = reinterpret_cast<T*>(lds + L0.rgate);
  int64_t* const rowid = reinterpret_cast<int64_t*>(lds + L0.rowid);
  T* const graw = reinterpret_cast<T*>(lds + L0.graw);
  int* const ents = reinterpret_cast<int*>(lds + L0.ents);

  // a thread's entry of the tile (tile * k <= blockDim), read once
  const int n_entries = rows * k, my_s = tid / k;
  int64_t my_at = 0;
  int my_e = -1;
  T my_g = 0;
  if (tid < n_entries) {
    const int64_t row = order != nullptr ? order[base + my_s] : base + my_s;
    my_at = row * k + (tid - my_s * k);
    const int e = experts[my_at];
    my_e = e >= 0 && e < a.X ? e : -1;
    if (my_e >= 0) my_g = gates[my_at];
    if (tid == my_s * k) rowid[my_s] = row;
    ents[tid] = my_e;
    graw[tid] = my_g;
  }
  for (int q = tid; q < a.X; q += blockDim.x) mask[q] = 0;
  const int spare = m.tile * m.ld_dst;
  for (int q = tid; q < m.matrix_rows; q += blockDim.x) {
    rtab[q] = uint32_t(spare) << 16;
    rgate[q] = T(0);
  }
  __syncthreads();
  if (my_e >= 0) atomicOr(&mask[my_e], 1u << my_s);

  // the tile's rows
  constexpr int kPer = 16 / sizeof(T);
  const int len = m.K * d, olen = m.N * d;
  auto stage = [&](const T* from, int64_t ld, int n, uint32_t inv, bool vec, T* to, int to_ld) {
    if (vec)
      move_rows<Pack<T>>(rows, n / kPer, inv,
                         [&](int s, int c) { return *reinterpret_cast<const Pack<T>*>(from + rowid[s] * ld + c * kPer); },
                         [&](int s, int c, const Pack<T>& p) {
#pragma unroll
                           for (int q = 0; q < kPer; ++q) to[s * to_ld + c * kPer + q] = p.v[q];
                         });
    else
      move_rows<T>(rows, n, inv, [&](int s, int c) { return from[rowid[s] * ld + c]; },
                   [&](int s, int c, T v) { to[s * to_ld + c] = v; });
  };
  stage(src + m.src_off, a.ld_src, len, m.inv_src, m.vec & 1, xs, m.ld_src);
  if (GG) stage(other + m.dst_off, a.ld_dst, olen, m.inv_dst, m.vec & 2, dot, m.ld_dst);
  // channels up to the next multiple of 4 KS are summed over too: zero
  const int padded = (m.K + 4 * KS - 1) / (4 * KS) * 4 * KS * d;
  for (int s = w; s < rows && padded > len; s += a.waves)
    for (int c = len + lane; c < padded; c += 64) xs[s * m.ld_src + c] = T(0);
  for (int q = tid; q < rows * m.ld_dst; q += blockDim.x) acc[q] = T(0);
  const int sums = m.tile * k * d + 1;  // a wavefront's sums of the gates' gradient, and a spare place
  if (GG)
    for (int q = tid; q < a.waves * sums; q += blockDim.x) rowsum[q] = T(0);
  __syncthreads();
  // experts present, ascending: places (members before) and matrix rows before, summed as one word
  if (w == 0) {
    int n_here = 0;
    uint32_t before = 0;
    for (int e0 = 0; e0 < a.X; e0 += 64) {
      const uint32_t c = __popc(e0 + lane < a.X ? mask[e0 + lane] : 0);
      const uint32_t mine = c << 16 | ((c * d + 15) & ~15u);
      uint32_t s = mine;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const uint32_t t = __shfl_up(s, o, 64);
        if (lane >= o) s += t;
      }
      const uint32_t at = before + s - mine;
      const uint64_t here = __ballot(c > 0);
      if (c > 0) {
        int* const to = list + 4 * (n_here + __popcll(here & ((uint64_t(1) << lane) - 1)));
        to[0] = e0 + lane;
        to[1] = at & 0xFFFF;
        to[2] = c * d;
        to[3] = at >> 16;
      }
      if (e0 + lane < a.X) start[e0 + lane] = at;
      before += __shfl(s, 63, 64);
      n_here += __popcll(here);
    }
    if (lane == 0) list[4 * n_here] = -1;
  }
  __syncthreads();
  // members' gates (an expert that stands twice in a row: their sum) and matrix rows
  int my_place = 0;
  if (my_e >= 0) {
    bool leads = true;
    T g = 0;
    for (int b = 0; b < k; ++b) {
      const int q = my_s * k + b;
      if (ents[q] == my_e) {
        leads = leads && q >= tid;
        g += graw[q];
      }
    }
    const uint32_t at = start[my_e], nth = __popc(mask[my_e] & ((1u << my_s) - 1));
    my_place = (at >> 16) + nth;
    if (leads) {
      const int r = (at & 0xFFFF) + nth * d;
      for (int c = 0; c < d; ++c) {
        rtab[r + c] = uint32_t(my_s * m.ld_dst + c) << 16 | uint32_t(my_s * m.ld_src + c);
        rgate[r + c] = g;
      }
    }
  }
  __syncthreads();

  // each wavefront: 16 output channels, all experts of the tile, the next
  // expert's weights on their way while one's are in use
  const int i16 = lane & 15, g4 = lane >> 4;
  T* const my_sums = GG ? rowsum + w * sums : nullptr;
  for (int n0 = w * 16; n0 < m.N; n0 += a.waves * 16) {
    const int col = min(n0 + i16, m.N - 1);  // a lane past the last channel fills a column that is not written
    const int to = (n0 + i16) * d;
    for (int k0 = 0; k0 < m.K; k0 += 4 * KS) {
      const int kk = k0 + g4 * KS;  // lane's channels of the sum: kk .. kk + KS - 1
      const bool full = k0 + 4 * KS <= m.K;
      auto load_weights = [&](int e, T* b) {  // zero past the last channel of the sum
        const T* wp = weights + e * a.weight_numel + m.woff;
        if (ADJ) {
          const T* row = wp + col * m.V;
          if (KS >= kPer && full && (m.vec & 4)) {
#pragma unroll
            for (int s = 0; s < KS; s += kPer) {
              const Pack<T> p = *reinterpret_cast<const Pack<T>*>(row + kk + s);
#pragma unroll
              for (int q = 0; q < kPer; ++q) b[s + q] = p.v[q];
            }
          } else {
#pragma unroll
            for (int s = 0; s < KS; ++s) b[s] = row[min(kk + s, m.K - 1)];
          }
        } else if (full) {
#pragma unroll
          for (int s = 0; s < KS; ++s) b[s] = wp[(kk + s) * m.V + col];
        } else {
#pragma unroll
          for (int s = 0; s < KS; ++s) b[s] = wp[min(kk + s, m.K - 1) * m.V + col];
        }
      };
      T b[KS], next[KS];
      int e = __builtin_amdgcn_readfirstlane(list[0]);
      if (e >= 0) load_weights(e, next);
      for (int j = 0; e >= 0; ++j) {
#pragma unroll
        for (int s = 0; s < KS; ++s) b[s] = full || kk + s < m.K ? next[s] : T(0);
        e = __builtin_amdgcn_readfirstlane(list[4 * j + 4]);
        if (e >= 0) load_weights(e, next);
        const int r0 = __builtin_amdgcn_readfirstlane(list[4 * j + 1]);
        const int n_rows = __builtin_amdgcn_readfirstlane(list[4 * j + 2]);
        const int place = __builtin_amdgcn_readfirstlane(list[4 * j + 3]) * d;
        for (int r = 0; r < n_rows; r += 16) {
          const T* ap = xs + (rtab[r0 + r + i16] & 0xFFFF) + kk * d;
          T av[KS];
#pragma unroll
          for (int s = 0; s < KS; ++s) av[s] = ap[s * d];
          int at[4];
          T gate[4], sofar[4], other_row[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int rr = r0 + r + Mfma<T>::row(g4, q);
            at[q] = static_cast<int>(rtab[rr] >> 16) + to;
            gate[q] = rgate[rr];
          }
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            sofar[q] = acc[at[q]];
            if (GG) other_row[q] = dot[at[q]];
          }
          typename Mfma<T>::Acc prod = {0, 0, 0, 0};
#pragma unroll
          for (int s = 0; s < KS; ++s) prod = Mfma<T>::step(av[s], b[s], prod);
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[at[q]] = sofar[q] + gate[q] * prod[q];
          if (GG) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int rr = r + Mfma<T>::row(g4, q);
              const T v = sum16(n0 + i16 < m.N ? prod[q] * other_row[q] : T(0));
              if (i16 == 0) my_sums[rr < n_rows ? place + rr : sums - 1] += v;
            }
          }
        }
      }
    }
  }
  __syncthreads();
  if (dst != nullptr) {
    T* const to = dst + m.dst_off;
    if (m.vec & 2)
      move_rows<Pack<T>>(rows, olen / kPer, m.inv_dst,
                         [&](int s, int c) {
                           Pack<T> p;
#pragma unroll
                           for (int q = 0; q < kPer; ++q) p.v[q] = acc[s * m.ld_dst + c * kPer + q];
                           return p;
                         },
                         [&](int s, int c, const Pack<T>& p) {
                           *reinterpret_cast<Pack<T>*>(to + rowid[s] * a.ld_dst + c * kPer) = p;
                         });
    else
      move_rows<T>(rows, olen, m.inv_dst, [&](int s, int c) { return acc[s * m.ld_dst + c]; },
                   [&](int s, int c, T v) { to[rowid[s] * a.ld_dst + c] = v; });
  }
  if (GG && tid < n_entries) {
    T v = 0;
    if (my_e >= 0)
      for (int ww = 0; ww < a.waves; ++ww)
        for (int c = 0; c < d; ++c) v += rowsum[ww * sums + my_place * d + c];
    gate_part[mi * (a.n_rows * k) + my_at] = v;
  }
}

template <class T>
__global__ void k_zero_columns(int64_t n_rows, int64_t dim, int32_t off, int32_t len, T* __restrict__ out) {
  const int64_t total = n_rows * len, step = int64_t(gridDim.x) * blockDim.x;
  for (int64_t q = blockIdx.x * int64_t(blockDim.x) + threadIdx.x; q < total; q += step)
    out[(q / len) * dim + off + q % len] = T(0);
}

// ------------------------------------------------------- weights' gradient
// grad_M_e = sum over e's entries and components of x (gate G)^T: a matrix
// product whose inner dimension is the (entry, component) pairs of an expert.
// A block takes one piece (at most kPiece entries of one expert and group), one
// map and one S x S tile of it.  Stages of a few entries are gathered into LDS
// with the components split out ([component row][channel]), while the next
// stage's loads are in flight in registers; 4 wavefronts share the tile (S =
// 16: they share the rows, and are added in order at the end).  Each piece's
// matrix goes to the workspace; k_join adds an expert's pieces in order.
struct WgradMap {
  int32_t in_off, out_off, U, V, d, woff;
  int32_t nu, nv;     // S x S tiles of the matrix
  int32_t per_stage;  // entries of a stage, a multiple of 4
  int32_t inv_d;      // ceil(65536 / d): c / d = c * inv_d >> 16 for c below 64 d
  int32_t first;      // first block of this map
};

struct WgradArgs {
  int64_t dim_in, dim_out, weight_numel;
  int64_t max_pieces, group;
  int64_t slots;  // pieces of all groups, at most
  int32_t X, k, n_maps;
  int32_t direct;  // every expert has one piece at most: straight into grad_weights, zeros for those without
  WgradMap map[kMaxMaps];
};

constexpr int kStage = 2304;  // channels times rows of a stage, at most

template <int S>
constexpr int stage_pitch() {  // rows (4 at a time) start 16 banks apart
  return S == 16 ? 16 : S + 16;
}

template <class T, int S, bool VEC>
__global__ __launch_bounds__(256) void k_wgrad(WgradArgs a, const T* __restrict__ x, const T* __restrict__ gates,
                                               const T* __restrict__ grad, const int32_t* __restrict__ entries,
                                               const int32_t* __restrict__ first, const int32_t* __restrict__ pieces,
                                               T* __restrict__ out) {
  constexpr int P = stage_pitch<S>(), kPer = VEC ? 16 / sizeof(T) : 1;
  constexpr int kLoads = (kStage / kPer + 255) / 256;  // a thread's loads of a stage and operand
  constexpr int kTiles = S == 64 ? 2 : 1;
  constexpr int kRows = kStage / S;
  __shared__ T xs[kRows * P], gs[kRows * P];
  __shared__ int64_t at_row[kPiece];
  __shared__ T at_gate[kPiece];
  __shared__ int found[2];
  int mi = 0;
  while (mi + 1 < a.n_maps && static_cast<int>(blockIdx.x) >= a.map[mi + 1].first) ++mi;
  const WgradMap m = a.map[mi];
  const int64_t r = int64_t(blockIdx.x) - m.first;
  const int64_t slot = r % a.slots;
  const int uv = static_cast<int>(r / a.slots), u0 = uv / m.nv * S, v0 = uv % m.nv * S;
  const int64_t grp = slot / a.max_pieces;
  const int p = static_cast<int>(slot - grp * a.max_pieces);
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, d = m.d;
  const int32_t* const pcs = pieces + grp * (a.X + 1);
  const int32_t* const fst = first + grp * (a.X + 1);
  // the piece's expert and entries
  int e, from, count;
  if (a.direct) {
    e = p;
    from = fst[e];
    count = fst[e + 1] - from;
  } else {
    if (p >= pcs[a.X]) return;
    if (tid < a.X && pcs[tid] <= p && p < pcs[tid + 1]) {
      found[0] = tid;
      found[1] = p - pcs[tid];
    }
    __syncthreads();
    e = found[0];
    from = fst[e] + found[1] * kPiece;
    count = min(kPiece, fst[e + 1] - from);
  }
  if (tid < count) {
    const int64_t q = entries[grp * a.group * a.k + from + tid];
    at_row[tid] = q / a.k;
    at_gate[tid] = gates[q];
  }
  __syncthreads();

  // a thread's part of a stage: entry `es`, LDS place of its first element
  const int ulen = min(S, m.U - u0) * d, vlen = min(S, m.V - v0) * d;
  auto split = [&](int q, int len, int& es, int& c) {
    const int idx = (tid + q * 256) * kPer;
    es = idx / len;
    c = idx - es * len;
  };
  int xe[kLoads], xc[kLoads], ge[kLoads], gc[kLoads];
#pragma unroll
  for (int q = 0; q < kLoads; ++q) {
    split(q, ulen, xe[q], xc[q]);
    split(q, vlen, ge[q], gc[q]);
  }
  T px[kLoads][kPer], pg[kLoads][kPer];
  const T* const xb = x + m.in_off + u0 * d;
  const T* const gb = grad + m.out_off + v0 * d;
  auto load = [&](int s0) {  // entries s0 .. of the piece; zeros past its end
#pragma unroll
    for (int q = 0; q < kLoads; ++q) {
      const int ex = s0 + xe[q], eg = s0 + ge[q];
      const bool inx = xe[q] < m.per_stage && ex < count, ing = ge[q] < m.per_stage && eg < count;
      const T g = ing ? at_gate[eg] : T(0);
      if (VEC) {
        const Pack<T> a0 = inx ? *reinterpret_cast<const Pack<T>*>(xb + at_row[ex] * a.dim_in + xc[q]) : Pack<T>{};
        const Pack<T> b0 = ing ? *reinterpret_cast<const Pack<T>*>(gb + at_row[eg] * a.dim_out + gc[q]) : Pack<T>{};
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          px[q][j] = a0.v[j];
          pg[q][j] = b0.v[j] * g;
        }
      } else {
        px[q][0] = inx ? xb[at_row[ex] * a.dim_in + xc[q]] : T(0);
        pg[q][0] = ing ? gb[at_row[eg] * a.dim_out + gc[q]] * g : T(0);
      }
    }
  };
  auto store = [&](T* to, int es, int c, const T* v) {
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int u = (c + j) * m.inv_d >> 16, comp = c + j - u * d;
      to[(es * d + comp) * P + u] = v[j];
    }
  };

  const int i16 = lane & 15, g4 = lane >> 4;
  const int tu = S == 64 ? (w >> 1) * 32 : (S == 32 ? (w >> 1) * 16 : 0);
  const int tv = S == 64 ? (w & 1) * 32 : (S == 32 ? (w & 1) * 16 : 0);
  typename Mfma<T>::Acc acc[kTiles][kTiles];
#pragma unroll
  for (int i = 0; i < kTiles; ++i)
#pragma unroll
    for (int j = 0; j < kTiles; ++j) acc[i][j] = typename Mfma<T>::Acc{0, 0, 0, 0};
  const int steps = m.per_stage * d / 4;
  load(0);
  for (int s0 = 0; s0 < count; s0 += m.per_stage) {
#pragma unroll
    for (int q = 0; q < kLoads; ++q) {
      if (xe[q] < m.per_stage) store(xs, xe[q], xc[q], px[q]);
      if (ge[q] < m.per_stage) store(gs, ge[q], gc[q], pg[q]);
    }
    __syncthreads();
    if (s0 + m.per_stage < count) load(s0 + m.per_stage);
    for (int st = S == 16 ? w : 0; st < steps; st += S == 16 ? 4 : 1) {
      const T* xr = xs + (4 * st + g4) * P + tu + i16;
      const T* gr = gs + (4 * st + g4) * P + tv + i16;
#pragma unroll
      for (int i = 0; i < kTiles; ++i)
#pragma unroll
        for (int j = 0; j < kTiles; ++j) acc[i][j] = Mfma<T>::step(xr[16 * i], gr[16 * j], acc[i][j]);
    }
    __syncthreads();
  }
  T* const to = out + (a.direct ? e : slot) * a.weight_numel + m.woff;
  if (S == 16) {  // the wavefronts' shares of the rows, added in order
#pragma unroll
    for (int q = 0; q < 4; ++q) xs[w * 256 + Mfma<T>::row(g4, q) * 16 + i16] = acc[0][0][q];
    __syncthreads();
    const int u = u0 + tid / 16, v = v0 + tid % 16;
    if (u < m.U && v < m.V) to[u * m.V + v] = ((xs[tid] + xs[256 + tid]) + xs[512 + tid]) + xs[768 + tid];
    return;
  }
#pragma unroll
  for (int i = 0; i < kTiles; ++i)
#pragma unroll
    for (int j = 0; j < kTiles; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int u = u0 + tu + 16 * i + Mfma<T>::row(g4, q), v = v0 + tv + 16 * j + i16;
        if (u < m.U && v < m.V) to[u * m.V + v] = acc[i][j][q];
      }
}

// Adds what the kernels above left in parts, in order: an expert's pieces
// (blocks [0, X nw): nw blocks of 256 weights each) and the maps' shares of the
// gates' gradient (the blocks after them).
template <class T>
__global__ __launch_bounds__(256) void k_join(int X, int nw, int64_t numel, int n_groups, int64_t max_pieces,
                                              const int32_t* __restrict__ pieces, const T* __restrict__ part,
                                              T* __restrict__ out, int64_t n_gates, int n_maps,
                                              const T* __restrict__ gate_part, T* __restrict__ gate_out) {
  __shared__ int lo[64], upto[64], list[256];
  const int b = blockIdx.x, tid = threadIdx.x;
  if (b >= X * nw) {
    const int64_t q = int64_t(b - X * nw) * 256 + tid;
    if (q >= n_gates) return;
    T s = 0;
    for (int p = 0; p < n_maps; ++p) s += gate_part[p * n_gates + q];
    gate_out[q] = s;
    return;
  }
  const int e = b / nw;
  const int64_t c = int64_t(b - e * nw) * 256 + tid;
  // pieces of the expert in the groups (64 at most) up to and including each
  if (tid < 64) {
    const int64_t at = int64_t(tid) * (X + 1) + e;
    const int p0 = tid < n_groups ? pieces[at] : 0;
    int n = tid < n_groups ? pieces[at + 1] - p0 : 0;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int t = __shfl_up(n, o, 64);
      if (tid >= o) n += t;
    }
    lo[tid] = p0;
    upto[tid] = n;
  }
  __syncthreads();
  const int total = upto[63];
  T s = 0;
  for (int q0 = 0; q0 < total; q0 += 256) {
    const int q = q0 + tid;
    if (q < total) {
      int g = 0;  // first group whose count exceeds q
#pragma unroll
      for (int step = 32; step > 0; step >>= 1)
        if (upto[g + step - 1] <= q) g += step;
      list[tid] = static_cast<int>(g * max_pieces + lo[g] + q - (g > 0 ? upto[g - 1] : 0));
    }
    __syncthreads();
    const int here = min(256, total - q0);
    if (c < numel) {
#pragma unroll 8
      for (int j = 0; j < here; ++j) s += part[list[j] * numel + c];
    }
    __syncthreads();
  }
  if (c < numel) out[e * numel + c] = s;
}

// -------------------------------------------------------------------- host
bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

template <class T, int KS, bool ADJ, bool GG>
hipError_t rows_ks(const RowArgs& a, const RowLds& L, int64_t blocks, const T* src, const T* weights,
                   const int32_t* experts, const T* gates, const int32_t* order, T* dst, const T* other, T* part,
                   hipStream_t s) {
  auto* const f = k_rows<T, KS, ADJ, GG>;
  if (L.total > 64 * 1024) {  // above the default limit of dynamic LDS
    const hipError_t he = hipFuncSetAttribute(reinterpret_cast<const void*>(f),
                                              hipFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(L.total));
    if (he != hipSuccess) return he;
  }
  hipLaunchKernelGGL(f, dim3(static_cast<unsigned>(blocks)), dim3(64 * a.waves), L.total, s, a, L, src, weights, experts, gates, order, dst,
                     other, part);
  return hipGetLastError();
}

template <class T, bool ADJ, bool GG>
hipError_t rows(const Experts& p, int64_t n, const T* src, const T* weights, const int32_t* experts, const T* gates,
                const int32_t* order, T* dst, const T* other, T* part, hipStream_t s) {
  RowArgs a{};
  a.n_rows = n;
  a.ld_src = ADJ ? p.dim_out : p.dim_in;
  a.ld_dst = ADJ ? p.dim_in : p.dim_out;
  a.weight_numel = p.weight_numel;
  a.X = p.n_experts;
  a.k = p.top_k;
  a.n_maps = static_cast<int32_t>(p.maps.size());
  const int per = 16 / static_cast<int>(sizeof(T));
  int maxK = 0, maxN = 0;
  for (int q = 0; q < a.n_maps; ++q) {
    const ExpertMap& e = p.maps[q];
    RowMap& m = a.map[q];
    m.src_off = ADJ ? e.out_off : e.in_off;
    m.dst_off = ADJ ? e.in_off : e.out_off;
    m.K = ADJ ? e.mul_out : e.mul_in;
    m.N = ADJ ? e.mul_in : e.mul_out;
    m.V = e.mul_out;
    m.d = e.d;
    m.woff = e.woff;
    const bool vs = aligned16(src) && a.ld_src % per == 0 && m.src_off % per == 0 && (m.K * m.d) % per == 0;
    const bool vd = (dst == nullptr || aligned16(dst)) && (!GG || aligned16(other)) && a.ld_dst % per == 0 &&
                    m.dst_off % per == 0 && (m.N * m.d) % per == 0;
    const bool vw = aligned16(weights) && a.weight_numel % per == 0 && m.woff % per == 0 && m.V % per == 0;
    m.vec = (vs ? 1 : 0) | (vd ? 2 : 0) | (vw ? 4 : 0);
    maxK = std::max(maxK, m.K);
    maxN = std::max(maxN, m.N);
  }
  const int KS = maxK <= 16 ? 4 : (maxK <= 32 ? 8 : 16);
  a.waves = std::min(4, (maxN + 15) / 16);
  // Tile: as many rows (32 at most: a bit each) as leave LDS for 8 wavefronts
  // on a CU, 20 KiB for each of the block's; a thread for each entry, one row
  // at least.  With few rows
  // the tiles are made smaller, to have two blocks for each of the 256 CUs.
  std::sort(a.map, a.map + a.n_maps, [](const RowMap& x, const RowMap& y) {
    return int64_t(x.K) * x.N * x.d > int64_t(y.K) * y.N * y.d;  // long maps first
  });
  uint32_t region[sizeof(RowLds) / 4] = {};
  const int64_t spread = std::max<int64_t>(1, n * a.n_maps / 512);
  int64_t blocks = 0;
  for (int q = 0; q < a.n_maps; ++q) {
    RowMap& m = a.map[q];
    // rows in LDS start d (rounded up to 4) banks apart, modulo the 64 banks
    auto pitch = [&](int channels) {
      const int want = (m.d + 3) / 4 * 4, full = channels * m.d;
      return full + ((want - full) % 64 + 64) % 64;
    };
    m.ld_src = pitch((m.K + 4 * KS - 1) / (4 * KS) * 4 * KS);
    m.ld_dst = pitch((m.N + 15) / 16 * 16);
    auto inverse = [](int pieces) { return pieces > 1 ? uint32_t((0xFFFFFFFFull + pieces) / pieces) : 0u; };
    m.inv_src = inverse(m.K * m.d / (m.vec & 1 ? per : 1));
    m.inv_dst = inverse(m.N * m.d / (m.vec & 2 ? per : 1));
    RowLds one{};
    for (m.tile = std::min(32, 64 * a.waves / a.k); m.tile > 1; --m.tile) {
      one = row_lds(m, a.X, a.k, a.waves, GG, sizeof(T));
      if (m.tile <= spread && one.total <= 20480u * a.waves) break;
    }
    one = row_lds(m, a.X, a.k, a.waves, GG, sizeof(T));
    m.matrix_rows = matrix_rows(m.tile, a.X, a.k, m.d);
    m.first = static_cast<int32_t>(blocks);
    blocks += (n + m.tile - 1) / m.tile;
    if (blocks > INT32_MAX) return hipErrorInvalidValue;
    // one launch for all maps: each region as large as the map that needs most
    for (size_t f = 0; f < sizeof(RowLds) / 4; ++f) {
      const uint32_t* const from = reinterpret_cast<const uint32_t*>(&one) + f;
      region[f] = std::max(region[f], f > 0 ? from[0] - from[-1] : 0u);
    }
  }
  RowLds L{};  // the regions' sizes, to offsets
  for (size_t f = 1; f < sizeof(RowLds) / 4; ++f) {
    uint32_t* const at = reinterpret_cast<uint32_t*>(&L) + f;
    at[0] = at[-1] + region[f];
  }
  if (L.total > 160 * 1024) return hipErrorInvalidValue;
  for (const ColumnRun& r : ADJ ? p.bare_in : p.bare_out)
    if (dst != nullptr)
      hipLaunchKernelGGL(k_zero_columns<T>, dim3(blocks_for(n * r.len, 256)), dim3(256), 0, s, n, a.ld_dst, r.off,
                         r.len, dst);
  switch (KS) {
    case 4: return rows_ks<T, 4, ADJ, GG>(a, L, blocks, src, weights, experts, gates, order, dst, other, part, s);
    case 8: return rows_ks<T, 8, ADJ, GG>(a, L, blocks, src, weights, experts, gates, order, dst, other, part, s);
    default: return rows_ks<T, 16, ADJ, GG>(a, L, blocks, src, weights, experts, gates, order, dst, other, part, s);
  }
}

const int32_t* order_in(const Experts& p, int64_t n, const void* layout) {
  if (layout == nullptr) return nullptr;
  const LayoutShape L = layout_shape(n, p.n_experts, p.top_k);
  return reinterpret_cast<const int32_t*>(static_cast<const char*>(layout) + L.order);
}

// Workspace of the backward: the maps' shares of the gates' gradient, then the
// pieces' matrices.
struct BackwardSpace {
  size_t gates, parts, total;
};

BackwardSpace backward_space(const Experts& p, int64_t n) {
  const size_t size = p.f64 ? 8 : 4;
  const LayoutShape L = layout_shape(n, p.n_experts, p.top_k);
  BackwardSpace w{};
  w.parts = align_up(p.maps.size() * n * p.top_k * size);
  w.total = std::max<size_t>(256, w.parts + align_up(L.n_groups * L.max_pieces * p.weight_numel * size));
  return w;
}

template <class T, int S, bool VEC>
hipError_t wgrad_launch(const WgradArgs& a, int64_t blocks, const T* x, const T* gates, const T* grad,
                        const int32_t* entries, const int32_t* first, const int32_t* pieces, T* out, hipStream_t s) {
  hipLaunchKernelGGL((k_wgrad<T, S, VEC>), dim3(static_cast<unsigned>(blocks)), dim3(256), 0, s, a, x, gates, grad,
                     entries, first, pieces, out);
  return hipGetLastError();
}

template <class T>
hipError_t backward(const Experts& p, int64_t n, const T* x, const T* weights, const int32_t* experts, const T* gates,
                    const void* layout, const T* grad, T* gx, T* gw, T* gg, void* ws, hipStream_t s) {
  const int32_t* order = order_in(p, n, layout);
  const int64_t n_gates = gg != nullptr ? n * p.top_k : 0;
  const int n_maps = static_cast<int>(p.maps.size()), X = p.n_experts;
  const BackwardSpace space = backward_space(p, n);
  T* const gate_part = static_cast<T*>(ws);
  hipError_t he = hipSuccess;
  if (n_gates > 0)
    he = rows<T, true, true>(p, n, grad, weights, experts, gates, order, gx, x, gate_part, s);
  else if (n > 0 && gx != nullptr)
    he = rows<T, true, false>(p, n, grad, weights, experts, gates, order, gx, nullptr, nullptr, s);
  if (he != hipSuccess) return he;
  const int64_t gate_blocks = (n_gates + 255) / 256;
  if (gw == nullptr) {
    if (gate_blocks > 0)
      hipLaunchKernelGGL(k_join<T>, dim3(static_cast<unsigned>(gate_blocks)), dim3(256), 0, s, 0, 0, p.weight_numel, 0,
                         int64_t(0), nullptr, nullptr, nullptr, n_gates, n_maps, gate_part, gg);
    return hipGetLastError();
  }
  const LayoutShape L = layout_shape(n, X, p.top_k);
  const char* const at = static_cast<const char*>(layout);
  auto ints = [&](size_t off) { return n > 0 ? reinterpret_cast<const int32_t*>(at + off) : nullptr; };
  WgradArgs a{};
  a.dim_in = p.dim_in;
  a.dim_out = p.dim_out;
  a.weight_numel = p.weight_numel;
  a.max_pieces = L.max_pieces;
  a.group = L.group;
  a.X = X;
  a.k = p.top_k;
  a.n_maps = n_maps;
  // with at most a piece's entries in all, an expert's one piece is its sum
  a.direct = n * p.top_k <= kPiece;
  a.slots = a.direct ? X : L.n_groups * L.max_pieces;
  const int per = 16 / static_cast<int>(sizeof(T));
  bool vec = aligned16(x) && aligned16(grad) && p.dim_in % per == 0 && p.dim_out % per == 0;
  int widest = 0;
  for (const ExpertMap& e : p.maps) {
    widest = std::max({widest, e.mul_in, e.mul_out});
    vec = vec && e.in_off % per == 0 && e.out_off % per == 0 && (e.mul_in * e.d) % per == 0 &&
          (e.mul_out * e.d) % per == 0;
  }
  const int S = widest <= 16 ? 16 : (widest <= 32 ? 32 : 64);
  int64_t blocks = 0;
  for (int q = 0; q < n_maps; ++q) {
    const ExpertMap& e = p.maps[q];
    a.map[q] = WgradMap{e.in_off, e.out_off, e.mul_in, e.mul_out, e.d, e.woff, (e.mul_in + S - 1) / S,
                        (e.mul_out + S - 1) / S, kStage / S / e.d / 4 * 4, (65536 + e.d - 1) / e.d, 0};
  }
  std::sort(a.map, a.map + n_maps, [](const WgradMap& l, const WgradMap& r) {
    return l.d > r.d;  // long maps first
  });
  for (int q = 0; q < n_maps; ++q) {
    a.map[q].first = static_cast<int32_t>(blocks);
    blocks += a.slots * a.map[q].nu * a.map[q].nv;
  }
  if (blocks > INT32_MAX) return hipErrorInvalidValue;
  T* const parts = reinterpret_cast<T*>(static_cast<char*>(ws) + space.parts);
  T* const to = a.direct ? gw : parts;
  const int32_t *entries = ints(L.entries), *first = ints(L.first), *pcs = ints(L.pieces);
  if (n > 0) {
    if (S == 16)
      he = vec ? wgrad_launch<T, 16, true>(a, blocks, x, gates, grad, entries, first, pcs, to, s)
               : wgrad_launch<T, 16, false>(a, blocks, x, gates, grad, entries, first, pcs, to, s);
    else if (S == 32)
      he = vec ? wgrad_launch<T, 32, true>(a, blocks, x, gates, grad, entries, first, pcs, to, s)
               : wgrad_launch<T, 32, false>(a, blocks, x, gates, grad, entries, first, pcs, to, s);
    else
      he = vec ? wgrad_launch<T, 64, true>(a, blocks, x, gates, grad, entries, first, pcs, to, s)
               : wgrad_launch<T, 64, false>(a, blocks, x, gates, grad, entries, first, pcs, to, s);
    if (he != hipSuccess) return he;
  }
  const int nw = a.direct && n > 0 ? 0 : static_cast<int>((p.weight_numel + 255) / 256);  // n = 0: zeros
  if (nw > 0 || gate_blocks > 0)
    hipLaunchKernelGGL(k_join<T>, dim3(static_cast<unsigned>(int64_t(X) * nw + gate_blocks)), dim3(256), 0, s, X, nw,
                       p.weight_numel, n > 0 ? static_cast<int>(L.n_groups) : 0, L.max_pieces, pcs, parts, gw, n_gates,
                       n_maps, gate_part, gg);
  return hipGetLastError();
}

}  // namespace

size_t experts_layout_bytes(const Experts& p, int64_t n) { return layout_shape(n, p.n_experts, p.top_k).total; }

size_t experts_workspace(const Experts& p, int64_t n) { return backward_space(p, n).total; }

hipError_t launch_experts_layout(const Experts& p, int64_t n, const int32_t* experts, void* layout, int32_t* load,
                                 hipStream_t s) {
  const int X = p.n_experts;
  const LayoutShape L = layout_shape(n, X, p.top_k);
  char* const at = static_cast<char*>(layout);
  auto ints = [&](size_t off) { return reinterpret_cast<int32_t*>(at + off); };
  const int H = std::min(X, kMaxBins / X);
  const int threads = std::min(L.group, n) > 1024 ? 1024 : 256;
  hipLaunchKernelGGL(k_layout, dim3(static_cast<unsigned>(L.n_groups)), dim3(threads), 0, s, n, X, p.top_k, H,
                     L.group, experts, ints(L.order), ints(L.entries), ints(L.first), ints(L.pieces));
  if (load != nullptr) hipLaunchKernelGGL(k_load, dim3(1), dim3(256), 0, s, X, L.n_groups, ints(L.first), load);
  return hipGetLastError();
}

hipError_t launch_experts_forward(const Experts& p, int64_t n, const void* x, const void* weights,
                                  const int32_t* experts, const void* gates, const void* layout, void* out,
                                  hipStream_t s) {
  const int32_t* order = order_in(p, n, layout);
  if (p.f64)
    return rows<double, false, false>(p, n, static_cast<const double*>(x), static_cast<const double*>(weights),
                                      experts, static_cast<const double*>(gates), order, static_cast<double*>(out),
                                      nullptr, nullptr, s);
  return rows<float, false, false>(p, n, static_cast<const float*>(x), static_cast<const float*>(weights), experts,
                                   static_cast<const float*>(gates), order, static_cast<float*>(out), nullptr,
                                   nullptr, s);
}

hipError_t launch_experts_backward(const Experts& p, int64_t n, const void* x, const void* weights,
                                   const int32_t* experts, const void* gates, const void* layout, const void* grad_out,
                                   void* grad_x, void* grad_weights, void* grad_gates, void* ws, hipStream_t s) {
  if (p.f64)
    return backward(p, n, static_cast<const double*>(x), static_cast<const double*>(weights), experts,
                    static_cast<const double*>(gates), layout, static_cast<const double*>(grad_out),
                    static_cast<double*>(grad_x), static_cast<double*>(grad_weights),
                    static_cast<double*>(grad_gates), ws, s);
  return backward(p, n, static_cast<const float*>(x), static_cast<const float*>(weights), experts,
                  static_cast<const float*>(gates), layout, static_cast<const float*>(grad_out),
                  static_cast<float*>(grad_x), static_cast<float*>(grad_weights), static_cast<float*>(grad_gates), ws,
                  s);
}

}  // namespace tpconv
