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

#include "node_device.hpp"
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

int blocks_for(int64_t n, int block) {
  const int64_t g = (n + block - 1) / block;
  return static_cast<int>(g < 1 ? 1 : (g > 65536 ? 65536 : g));
}

// ------------------------------------------------------------------ layout
// Rows are taken in groups of kGroup, fewer where top_k makes more than twice
// as many entries of them, more where n / 64 or 64 entries an expert are more
// (at most 64 groups, and a group's experts have entries enough for their
// pieces); each group is sorted by itself, which needs no exchange between
// blocks: one launch whatever the size.
//   order    the group's rows by the pair (smallest, next) of their experts, so
//            that a tile of consecutive rows meets few experts
//   listed   the rows' experts in that order (a tile's are then one run, known
//            without its row numbers)
//   entries  the group's entries (row * top_k + place) by expert, entries of an
//            expert in ascending order (the sums over them are taken in it)
//   first    [group][X + 1] where each expert's entries start in `entries`,
//            relative to the group's first
//   pieces   [group][X + 1] the same in pieces of at most `piece` entries
constexpr int64_t kGroup = 2048;
constexpr int kMaxBins = 4096;
constexpr int kPiece = 128, kLeastPiece = 32;

struct LayoutShape {
  int64_t group, n_groups;
  int32_t piece;       // entries of a piece, at most
  int64_t max_pieces;  // pieces of a group, at most
  size_t order, listed, entries, first, pieces, total;
};

LayoutShape layout_shape(const Experts& p, int64_t n) {
  const int X = p.n_experts, k = p.top_k;
  LayoutShape L{};
  // pieces of all maps for 4 blocks a CU (2048 fp64 rows of 16 channels l <= 4, 2 of 8 experts: 12 us in pieces of
  // 32, 22 us of 128); longer ones (fewer sums to add) where there are entries enough
  L.piece = kLeastPiece;
  while (L.piece < kPiece && n * k * int64_t(p.maps.size()) > int64_t(1024) * L.piece) L.piece *= 2;
  // An expert has a piece of its own in every group, so with many experts the groups have to be longer: 28000 rows, 2
  // of 256 experts, 64 channels l <= 3: 104 MB of pieces, gradients in 499 us, layout in 24; in groups of 2048 rows 268
  // MB, 588 and 11 us
  L.group = std::max<int64_t>({std::min<int64_t>(kGroup, 2 * kGroup / k), (n + 63) / 64, 64 * X / k});
  L.n_groups = std::max<int64_t>(1, (n + L.group - 1) / L.group);
  const int64_t most = std::min(L.group, std::max<int64_t>(n, 1)) * k;
  L.max_pieces = most / L.piece + X;
  size_t o = 0;
  auto take = [&](int64_t ints) {
    const size_t at = o;
    o = align_up(o + sizeof(int32_t) * static_cast<size_t>(ints));
    return at;
  };
  L.order = take(n);
  L.listed = take(n * k);
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

// Two blocks per group.  Bins of the row order: (smallest expert) * H + (next
// * H / X), H = min(X, 4096 / X); rows without experts last.  Rows of one bin
// come in no fixed order (an integer atomic hands out the places): a row's
// results do not depend on its neighbours.  Entries are ranked by counting in
// order, so theirs is fixed.  Latency bound, so the group's experts are read
// once, into LDS, where they fit, and the two sorts run in blocks of their own:
// 10.5 us at 28000 rows of 2 entries over 16 experts, 24 us over 256, 9.4 us at
// 4096 rows of 4 over 32, 3.8 us for one row.
constexpr int kStaged = 16384;

__global__ __launch_bounds__(1024) void k_layout(int64_t n, int X, int k, int H, int64_t group, int piece,
                                                 const int32_t* __restrict__ experts, int32_t* __restrict__ order,
                                                 int32_t* __restrict__ listed, int32_t* __restrict__ entries,
                                                 int32_t* __restrict__ first, int32_t* __restrict__ pieces) {
  __shared__ int bins[kMaxBins + 1];
  __shared__ int wave_sums[16];
  __shared__ uint16_t staged[kStaged];
  const int64_t grp = blockIdx.x >> 1, r0 = grp * group;
  const int rows = static_cast<int>(min(group, n - r0));
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, nw = blockDim.x >> 6;
  const int32_t* ex = experts + r0 * k;
  const int total = rows * k;
  const bool in_lds = total <= kStaged;
  auto clean = [&](int e) { return e >= 0 && e < X ? e : X; };  // X: none
  if (in_lds)
    for (int q0 = tid; q0 < total; q0 += 8 * blockDim.x) {
      int e[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) e[j] = ex[min(q0 + j * int(blockDim.x), total - 1)];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (q0 + j * int(blockDim.x) < total) staged[q0 + j * blockDim.x] = static_cast<uint16_t>(clean(e[j]));
    }
  auto expert = [&](int q) { return in_lds ? int(staged[q]) : clean(ex[q]); };

  if ((blockIdx.x & 1) == 0) {
    auto bin_of = [&](int r) {
      int lo = X, hi = X;
      for (int a = 0; a < k; ++a) {
        const int e = expert(r * k + a);
        hi = e < lo ? lo : (e > lo && e < hi ? e : hi);
        lo = min(lo, e);
      }
      if (lo == X) return X * H;
      return lo * H + (hi == X ? lo : hi) * H / X;
    };
    auto put = [&](int r, int at) {
      order[r0 + at] = static_cast<int32_t>(r0 + r);
      for (int a = 0; a < k; ++a) listed[(r0 + at) * k + a] = expert(r * k + a);
    };
    for (int q = tid; q <= X * H; q += blockDim.x) bins[q] = 0;
    __syncthreads();
    constexpr int kKept = 2;  // rows of a thread whose bins are kept (all of them in a group of 2048)
    int kept[kKept];
#pragma unroll
    for (int j = 0; j < kKept; ++j) {
      const int r = tid + j * blockDim.x;
      kept[j] = r < rows ? bin_of(r) : 0;
      if (r < rows) atomicAdd(&bins[kept[j]], 1);
    }
    for (int r = tid + kKept * blockDim.x; r < rows; r += blockDim.x) atomicAdd(&bins[bin_of(r)], 1);
    __syncthreads();
    scan_counters(bins, X * H + 1, wave_sums);
#pragma unroll
    for (int j = 0; j < kKept; ++j) {
      const int r = tid + j * blockDim.x;
      if (r < rows) put(r, atomicAdd(&bins[kept[j]], 1));
    }
    for (int r = tid + kKept * blockDim.x; r < rows; r += blockDim.x) put(r, atomicAdd(&bins[bin_of(r)], 1));
    return;
  }

  // entries by expert: each wavefront counts, then places, its own run of them;
  // counters [expert][wavefront], scanned in that order
  const int run = ((total + nw - 1) / nw + 63) / 64 * 64;
  const int q0 = w * run, q1 = min(total, q0 + run);
  for (int q = tid; q < X * nw; q += blockDim.x) bins[q] = 0;
  __syncthreads();
  for (int q = q0 + lane; q < q1; q += 64) {
    const int e = expert(q);
    if (e < X) atomicAdd(&bins[e * nw + w], 1);
  }
  __syncthreads();
  const int placed = scan_counters(bins, X * nw, wave_sums);
  int32_t* const fst = first + grp * (X + 1);
  int32_t* const pcs = pieces + grp * (X + 1);
  int mine = 0;  // X <= 256 <= blockDim
  if (tid < X) {
    const int at = bins[tid * nw], end = tid + 1 < X ? bins[(tid + 1) * nw] : placed;
    fst[tid] = at;
    mine = static_cast<int>((end - at + piece - 1) / piece);
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
    const int e = q + lane < q1 ? expert(q + lane) : X;
    const bool live = e < X;
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
    wave_sync();  // the next pass's entries take the places after these
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
// A block takes a tile of up to 16 rows (in the layout's order), one map and up
// to 64 of its output channels, and lists the tile's experts with their member
// rows.  The tile's (row, component) pairs are its matrix rows, 16 at a time:
// 2l+1 chunks.
// The segment goes to LDS with the channels apart ([channel][matrix row], so
// that every read of the loop is one address register and a constant), the
// chunks' sums stay in registers, and for each expert of the tile the chunks
// that hold one of its rows are multiplied and added times the rows' gates (0
// where a row is not the expert's; 4 multiplications for a chunk, where gates
// on the rows would take 16, which compete with the fp32 matrix instructions
// for the vector units).  So x is read once, out is written once
// whatever top_k, and a row's sum runs over its experts in ascending order.
// The next expert's weights are on their way while one's are in use.  A
// wavefront owns 16 output channels.  ADJ runs the transposed maps on
// grad_out; GG also dots the products with x for the gates' gradient.
// 28000 fp32 rows of 64 channels l <= 3, 2 of 16 experts: 145 us, and 213 us
// transposed with the gates' gradient; 229 MB and 344 MB are 46 and 69 us at the
// rate of a copy and 7.3 GFLOP are 48 us at that of a library product.  No unit
// is full: the matrix units are busy in 35 % of the cycles (24 % transposed; 1.12
// times the needed products, since chunks that hold some of an expert's rows are
// multiplied whole) and the vector units in 32 % (35 %); a wavefront waits in 40 %
// (50 %) of its cycles for memory, LDS or a barrier, with four (three) wavefronts
// a SIMD to take its place.  (Transposed with the gates' gradient, two wavefronts
// and no spilled registers: 245 us.)  Where few tiles leave two wavefronts a SIMD,
// the trips to memory and the matrix instructions of one wavefront's experts in
// turn decide: 4096 rows of 32 channels, 4 of 32 experts, 35 us (2.2 times the
// needed products, matrix units 17 %); 2048 fp64 rows of 16 channels l <= 4, 2 of
// 8, 17 us and 24 us (matrix units 3 %).
// (32 output channels a wavefront: 213 us for the first; sums in LDS with the
// members packed into full chunks: 171 us; all maps of a tile in one block: 199.)
constexpr int kTile = 16;

struct RowMap {
  int32_t src_off, dst_off;  // first columns in a row of src / dst
  int32_t K, N;              // channels summed over / produced
  int32_t V;                 // row length of the map's weights
  int32_t d, woff;
  int32_t packed;            // bit 0: 16-byte pieces of src, bit 1: of dst, bit 2: of the weights along K
};

// LDS of a block (byte offsets)
struct RowLds {
  uint32_t tile, gates, mask, start, list, rows, graw, grow, esum, wsum, rsum, ents, total;
};

struct RowArgs {
  int32_t first[kMaxMaps];  // first share (a map's block of output channels) of each map, INT32_MAX past the last map
  int64_t n_rows, ld_src, ld_dst, weight_numel;
  int32_t X, k, n_maps, waves;
  int32_t tile;       // rows of a tile, at most kTile
  int32_t n_tiles;
  int32_t block0;     // this launch's first block
  RowLds lds;
  RowMap map[kMaxMaps];
};

// Matrix rows of a tile are D runs of 16; a channel's row of them is padded to
// 4 more than a multiple of 16, which puts the four channels that a matrix
// instruction reads 16 banks apart.
constexpr int pitch_of(int d) { return 16 * d + 4; }

// Four values of each of the 16 lanes of a row of lanes, each summed over the
// lanes: lane q of every four holds the q-th sum.  The first two steps halve
// the values while they add (11 additions and selections for 16).
template <int CTRL>
__device__ __forceinline__ float moved(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, true));
}
template <int CTRL>
__device__ __forceinline__ double moved(double v) {
  return __hiloint2double(__builtin_amdgcn_update_dpp(0, __double2hiint(v), CTRL, 0xF, 0xF, true),
                          __builtin_amdgcn_update_dpp(0, __double2loint(v), CTRL, 0xF, 0xF, true));
}
template <class T>
__device__ __forceinline__ T sums16(const T (&v)[4], int lane) {
  const bool odd = lane & 1, high = lane & 2;
  const T a = (odd ? v[1] : v[0]) + moved<0xB1>(odd ? v[0] : v[1]);  // with the lane next to it
  const T b = (odd ? v[3] : v[2]) + moved<0xB1>(odd ? v[2] : v[3]);
  T s = (high ? b : a) + moved<0x4E>(high ? a : b);  // with the pair next to it
  s += moved<0x124>(s);                              // and the other fours: rotations by 4 and 8
  return s + moved<0x128>(s);
}

// A value the compiler takes for new: what is computed from it stays where it
// is used (kept from one phase to the next, places in LDS took 60 registers).
__device__ __forceinline__ int fresh(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// The tile's rows of a segment of n channels (CH at most), global <-> LDS:
// element c of row s is [c / D][s D + c % D] there.  A wavefront takes whole
// rows, several at a time where they are short, kBatch pieces in flight.
constexpr int kBatch = 8;

template <class T, int D, int CH, int PER>
struct TileMover {
  static constexpr int kPieces = CH * D / PER;
  static constexpr int lanes() {
    int l = 1;
    while (l < 64 && l < kPieces) l *= 2;
    return l;
  }
  static constexpr int kLanes = lanes(), kRows = 64 / kLanes, kSteps = (kPieces + 63) / 64;
  static constexpr int P = pitch_of(D);

  // c / D as a 24-bit product (c < 64 D): 32-bit ones, which a division compiles to, run at a quarter of the rate
  static __device__ __forceinline__ int place(int s, int c) {
    return __mul24(__umul24(c, (65536 + D - 1) / D) >> 16, P - D) + __mul24(s, D) + c;
  }

  // (row, first element) of a lane's q-th piece; false where there is none
  static __device__ __forceinline__ bool piece(int tid, int q, int rows, int pieces, int waves, int& s, int& c) {
    const int lane = tid & 63;
    s = (q / kSteps * waves + (tid >> 6)) * kRows + lane / kLanes;
    c = q % kSteps * 64 + lane % kLanes;
    const bool in = s < rows && c < pieces;
    s = min(s, rows - 1);
    c = min(c, pieces - 1) * PER;
    return in;
  }
  static __device__ __forceinline__ int trips(int rows, int waves) {
    return (rows + waves * kRows - 1) / (waves * kRows) * kSteps;
  }

  T v[kBatch][PER];

  // a batch of pieces, from the q0-th on; start(s): where row s of the tile starts
  template <class Start>
  __device__ __forceinline__ void issue(int q0, const T* from, Start start, int rows, int n, int waves) {
    const int tid = fresh(threadIdx.x);
    int64_t row[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      int s, c;
      piece(tid, q0 + j, rows, n * D / PER, waves, s, c);
      row[j] = start(s) + c;
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const T* at = from + row[j];
      if constexpr (PER > 1) {
        const Pack<T> p = *reinterpret_cast<const Pack<T>*>(at);
#pragma unroll
        for (int e = 0; e < PER; ++e) v[j][e] = p.v[e];
      } else {
        v[j][0] = *at;
      }
    }
  }
  // puts the first batch, issued before, into LDS, and fetches what it left
  template <class Start>
  __device__ __forceinline__ void finish(T* lds, const T* from, Start start, int rows, int n, int waves) {
    for (int q0 = 0;;) {
      const int tid = fresh(threadIdx.x);
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        int s, c;
        if (piece(tid, q0 + j, rows, n * D / PER, waves, s, c))
#pragma unroll
          for (int e = 0; e < PER; ++e) lds[place(s, c + e)] = v[j][e];
      }
      q0 += kBatch;
      if (q0 >= trips(rows, waves)) break;
      issue(q0, from, start, rows, n, waves);
    }
  }

  template <class Start>
  static __device__ __forceinline__ void store(const T* lds, T* to, Start start, int rows, int n, int waves) {
    const int tid = fresh(threadIdx.x);
    for (int q = 0; q < trips(rows, waves); ++q) {
      int s, c;
      if (!piece(tid, q, rows, n * D / PER, waves, s, c)) continue;
      T* const at = to + start(s) + c;
      if constexpr (PER > 1) {
        Pack<T> p;
#pragma unroll
        for (int e = 0; e < PER; ++e) p.v[e] = lds[place(s, c + e)];
        *reinterpret_cast<Pack<T>*>(at) = p;
      } else {
        *at = lds[place(s, c)];
      }
    }
  }
};

// One block's work on a map of components D, the rows' starts being in LDS.
// KS: channels summed over in a pass / 4; VS, VD: 16-byte pieces of src / dst;
// experts: in the rows' order here.
template <class T, int D, int KS, bool ADJ, bool GG, bool VS, bool VD>
__device__ __forceinline__ void map_rows(const RowArgs& a, const RowMap& m, int share, int n_base, int64_t base,
                                         int rows, char* lds, const T* __restrict__ src, const T* __restrict__ weights,
                                         const int32_t* __restrict__ experts, const T* __restrict__ gates,
                                         const int32_t* __restrict__ order, T* __restrict__ dst,
                                         const T* __restrict__ other, T* __restrict__ gate_part) {
  constexpr int kPer = 16 / sizeof(T), CH = 4 * KS, P = pitch_of(D);
  using Acc = typename Mfma<T>::Acc;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, k = a.k;
  const int i16 = lane & 15, g4 = lane >> 4;
  T* const xs = reinterpret_cast<T*>(lds + a.lds.tile);
  T* const gtab = reinterpret_cast<T*>(lds + a.lds.gates);  // gate of each expert of the tile and row
  uint32_t* const mask = reinterpret_cast<uint32_t*>(lds + a.lds.mask);  // members of each expert, a bit per row
  int* const start = reinterpret_cast<int*>(lds + a.lds.start);          // each expert's place in the list
  int* const list = reinterpret_cast<int*>(lds + a.lds.list);  // the tile's: expert, members' bits, members before
  int* const rowid = reinterpret_cast<int*>(lds + a.lds.rows);
  T* const graw = reinterpret_cast<T*>(lds + a.lds.graw);
  int* const ents = reinterpret_cast<int*>(lds + a.lds.ents);
  T* const grow = reinterpret_cast<T*>(lds + a.lds.grow) + w * 16 * 9;  // a wavefront's: gates of an expert's rows
  T* const esum = reinterpret_cast<T*>(lds + a.lds.esum);  // GG: entries' sums; each wavefront's; a wavefront's rows
  T* const wsum = reinterpret_cast<T*>(lds + a.lds.wsum);
  T* const rsum = reinterpret_cast<T*>(lds + a.lds.rsum) + w * 16 * 9;

  // The tile's entries, then its rows, are on their way while its experts are
  // listed: one trip to memory for the row numbers, one for all that they name.
  const int n_here = min(16 * a.waves, m.N - n_base);
  const int n_entries = rows * k;
  auto row_of = [&](int s) -> int64_t { return order != nullptr ? order[base + s] : base + s; };
  auto src_row = [&](int s) { return rowid[s] * a.ld_src; };
  auto dst_row = [&](int s) { return rowid[s] * a.ld_dst; };
  const int q0 = min(tid, n_entries - 1), s0 = q0 / k;
  const int e0 = experts[base * k + q0];
  const int64_t row0 = row_of(s0);
  const T g0 = gates[row0 * k + (q0 - s0 * k)];
  TileMover<T, D, CH, VS ? kPer : 1> mover;
  TileMover<T, D, 64, VD ? kPer : 1> mover_dst;
  const T* const src_from = src + m.src_off;
  const T* const other_from = GG ? other + m.dst_off + n_base * D : nullptr;
  auto first = [&](auto row) {
    if (GG) mover_dst.issue(0, other_from, [&](int s) { return row(s) * a.ld_dst; }, rows, n_here, a.waves);
    mover.issue(0, src_from, [&](int s) { return row(s) * a.ld_src; }, rows, min(CH, m.K), a.waves);
  };
  if (order != nullptr)
    first([&](int s) -> int64_t { return order[base + s]; });
  else
    first([&](int s) -> int64_t { return base + s; });

  for (int q = tid; q < a.X; q += blockDim.x) mask[q] = 0;
  for (int q = tid; q < n_entries * kTile; q += blockDim.x) gtab[q] = T(0);
  __syncthreads();
  auto note = [&](int q, int s, int64_t row, int e, T g) {
    const bool live = e >= 0 && e < a.X;
    ents[q] = live ? e : -1;
    graw[q] = live ? g : T(0);
    if (GG) esum[q] = T(0);
    if (live) atomicOr(&mask[e], 1u << s);
    if (q == s * k) rowid[s] = static_cast<int>(row);
  };
  if (tid < n_entries) note(q0, s0, row0, e0, g0);
  for (int q = tid + blockDim.x; q < n_entries; q += blockDim.x) {
    const int s = q / k;
    const int64_t row = row_of(s);
    note(q, s, row, experts[base * k + q], gates[row * k + (q - s * k)]);
  }
  __syncthreads();
  if (w == 0) {  // experts present, ascending, and the members before each
    int n_experts = 0, places = 0;
    for (int e0 = 0; e0 < a.X; e0 += 64) {
      const uint32_t mk = e0 + lane < a.X ? mask[e0 + lane] : 0;
      const int c = __popc(mk);
      int s = c;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int t = __shfl_up(s, o, 64);
        if (lane >= o) s += t;
      }
      const uint64_t here = __ballot(c > 0);
      if (c > 0) {
        const int j = n_experts + __popcll(here & ((uint64_t(1) << lane) - 1));
        list[4 * j] = e0 + lane;
        list[4 * j + 1] = static_cast<int>(mk);
        list[4 * j + 2] = places + s - c;
        start[e0 + lane] = j;
      }
      places += __shfl(s, 63, 64);
      n_experts += __popcll(here);
    }
    if (lane == 0) list[4 * n_experts] = -1;
  }
  __syncthreads();
  for (int q = tid; q < n_entries; q += blockDim.x) {
    const int e = ents[q], s = q / k;
    if (e < 0) continue;
    T g = 0;  // of an expert that stands twice in a row: the sum
    bool leads = true;
    for (int b = s * k; b < s * k + k; ++b)
      if (ents[b] == e) {
        leads = leads && b >= q;
        g += graw[b];
      }
    if (leads) gtab[start[e] * kTile + s] = g;
  }

  const int col = min(n_base + 16 * w + i16, m.N - 1);  // past the last channel: a column that is not written
  const bool whole = n_base + 16 * w + 16 <= m.N;       // the wavefront has a channel in every column
  T mine[GG ? D : 1][4];                                // GG: this lane's x
  if (GG) {
    mover_dst.finish(xs, other_from, dst_row, rows, n_here, a.waves);
    __syncthreads();
    const bool col_in = n_base + 16 * w + i16 < m.N;
#pragma unroll
    for (int c = 0; c < (GG ? D : 1); ++c)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        mine[c][q] = col_in ? xs[(16 * w + i16) * P + 16 * c + Mfma<T>::row(g4, q)] : T(0);
    __syncthreads();
  }
  Acc acc[D];
#pragma unroll
  for (int c = 0; c < D; ++c) acc[c] = Acc{0, 0, 0, 0};
  for (int k0 = 0; k0 < m.K; k0 += CH) {
    const int k_here = min(CH, m.K - k0);
    // lane's channels of the sum: 16 a + 4 g4 + b for its 4 a + b-th value; its place in the matrix is a part
    // of its own (bytes) after a part common to the wavefront
    const uint32_t mine_at = sizeof(T) * (ADJ ? col * m.V + 4 * g4 : 4 * g4 * m.V + col);
    const bool full = k_here == CH;
    auto load_weights = [&](int e, T (&b)[KS]) {
      const T* const we = weights + m.woff + e * a.weight_numel + (ADJ ? int64_t(k0) : int64_t(k0) * m.V);
      if (ADJ && full && (m.packed & 4)) {
#pragma unroll
        for (int s = 0; s < KS; s += kPer) {
          const Pack<T> p = *reinterpret_cast<const Pack<T>*>(reinterpret_cast<const char*>(we + s / 4 * 16 + s % 4) +
                                                              mine_at);
#pragma unroll
          for (int q = 0; q < kPer; ++q) b[s + q] = p.v[q];
        }
      } else if (full) {
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          const int u = s / 4 * 16 + s % 4;
          b[s] = *reinterpret_cast<const T*>(reinterpret_cast<const char*>(we + (ADJ ? u : u * m.V)) + mine_at);
        }
      } else {
        int last = k_here - 1;
        asm volatile("" : "+v"(last));  // keeps the places below out of the registers around the loop
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          const int u = min(s / 4 * 16 + 4 * g4 + s % 4, last);
          b[s] = we[ADJ ? col * m.V + u : u * m.V + col];
        }
      }
    };
    T b[KS], next[KS];
    int e = __builtin_amdgcn_readfirstlane(list[0]);
    if (e >= 0) load_weights(e, next);
    if (k0 > 0) mover.issue(0, src_from + k0 * D, src_row, rows, k_here, a.waves);
    mover.finish(xs, src_from + k0 * D, src_row, rows, k_here, a.waves);
    for (int q = tid; q < (CH - k_here) * P; q += blockDim.x) xs[k_here * P + q] = T(0);
    __syncthreads();
    const T* const ap = xs + 4 * g4 * P + i16;
    for (int j = 0; e >= 0; ++j) {
      const int members = __builtin_amdgcn_readfirstlane(list[4 * j + 1]);
#pragma unroll
      for (int s = 0; s < KS; ++s) b[s] = full || s / 4 * 16 + 4 * g4 + s % 4 < k_here ? next[s] : T(0);
      e = __builtin_amdgcn_readfirstlane(list[4 * j + 4]);
      if (e >= 0) load_weights(e, next);
      wave_sync();  // the last expert's gates and sums are read
#pragma unroll
      for (int r = 0; r < 16 * D; r += 64)
        if (r + lane < 16 * D) grow[r + lane] = gtab[j * kTile + (r + lane) / D];
      wave_sync();
#pragma unroll
      for (int c = 0; c < D; ++c) {
        constexpr auto bits = [](int chunk) {  // rows of the tile in the chunk
          int v = 0;
          for (int s = 16 * chunk / D; s <= (16 * chunk + 15) / D; ++s) v |= 1 << s;
          return v;
        };
        if ((members & bits(c)) == 0) continue;
        T av[KS];
#pragma unroll
        for (int s = 0; s < KS; ++s) av[s] = ap[(s / 4 * 16 + s % 4) * P + 16 * c];
        Acc prod = {0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < KS; ++s) prod = Mfma<T>::step(av[s], b[s], prod);
#pragma unroll
        for (int q = 0; q < 4; ++q) {  // a row that is not the expert's takes nothing, infinities and NaN included
          const T g = grow[16 * c + Mfma<T>::row(g4, q)];
          acc[c][q] = fma(g, g != T(0) ? prod[q] : T(0), acc[c][q]);
        }
        if (GG) {
          T v[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) v[q] = prod[q] * mine[GG ? c : 0][q];
          if (!whole)  // an infinite product in the place of a channel that is not there is no NaN in the sum
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] = n_base + 16 * w + i16 < m.N ? v[q] : T(0);
          const T s = sums16(v, i16);
          if (i16 < 4) rsum[16 * c + Mfma<T>::row(g4, i16)] = s;
        }
      }
      if (GG) wave_sync();
      if (GG && lane < kTile && ((members >> lane) & 1)) {  // the expert's rows, each over its components
        T v = 0;
#pragma unroll
        for (int c = 0; c < D; ++c) v += rsum[lane * D + c];
        wsum[w * kTile * k + list[4 * j + 2] + __popc(members & ((1 << lane) - 1))] = v;
      }
    }
    __syncthreads();
    if (GG)
      for (int q = tid; q < n_entries; q += blockDim.x) {
        if (ents[q] < 0) continue;
        const int s = q / k, j = start[ents[q]];
        const int place = list[4 * j + 2] + __popc(list[4 * j + 1] & ((1 << s) - 1));
        T v = esum[q];
        for (int ww = 0; ww < a.waves; ++ww) v += wsum[ww * kTile * k + place];
        esum[q] = v;
      }
  }
  if (dst != nullptr) {
#pragma unroll
    for (int c = 0; c < D; ++c)
#pragma unroll
      for (int q = 0; q < 4; ++q) xs[(16 * w + i16) * P + 16 * c + Mfma<T>::row(g4, q)] = acc[c][q];
    __syncthreads();
    mover_dst.store(xs, dst + m.dst_off + n_base * D, dst_row, rows, n_here, a.waves);
  }
  if (GG)
    for (int q = tid; q < n_entries; q += blockDim.x)
      gate_part[share * (a.n_rows * k) + int64_t(rowid[q / k]) * k + q % k] = esum[q];
}

template <class T, int KS, bool ADJ, bool GG>
__global__ __launch_bounds__(256, sizeof(T) == 8 ? 2 : (ADJ ? 3 : 4)) void k_rows(
    RowArgs a, const T* __restrict__ src, const T* __restrict__ weights, const int32_t* __restrict__ experts,
    const T* __restrict__ gates, const int32_t* __restrict__ order, T* __restrict__ dst, const T* __restrict__ other,
    T* __restrict__ gate_part) {
  extern __shared__ char lds[];
  const int block = a.block0 + static_cast<int>(blockIdx.x), share = block / a.n_tiles;
  int mi = 0;
#pragma unroll
  for (int q = 1; q < kMaxMaps; ++q) mi += share >= a.first[q];
  const RowMap& m = a.map[mi];
  const int64_t base = int64_t(block - share * a.n_tiles) * a.tile;
  const int rows = static_cast<int>(min<int64_t>(a.tile, a.n_rows - base));
  const int n_base = (share - a.first[mi]) * 16 * a.waves;
#define TPCONV_MAP_ROWS(D)                                                                                         \
  case D:                                                                                                          \
    if ((m.packed & 3) == 3)                                                                                       \
      map_rows<T, D, KS, ADJ, GG, true, true>(a, m, share, n_base, base, rows, lds, src, weights, experts, gates,  \
                                              order, dst, other, gate_part);                                       \
    else                                                                                                           \
      map_rows<T, D, KS, ADJ, GG, false, false>(a, m, share, n_base, base, rows, lds, src, weights, experts,        \
                                                gates, order, dst, other, gate_part);                              \
    break;
  switch (m.d) {
    TPCONV_MAP_ROWS(1)
    TPCONV_MAP_ROWS(3)
    TPCONV_MAP_ROWS(5)
    TPCONV_MAP_ROWS(7)
    TPCONV_MAP_ROWS(9)
    default: break;
  }
#undef TPCONV_MAP_ROWS
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
// A block takes one piece (at most 128 entries of one expert and group), one
// map and one S x S tile of it.  Stages of a few entries are gathered into LDS
// with the components split out ([component row][channel]), while the next
// stage's loads are in flight in registers; 4 wavefronts share the tile (S =
// 16: they share the rows, and are added in order at the end).  Each piece's
// matrix goes to the workspace; k_join adds an expert's pieces in order.
// Bound by the gathers and the products in turn: each entry's rows of x and G
// once, 459 MB in 137 us (3.3 TB/s; matrix units busy in 33 % of the cycles,
// wavefronts waiting in 39 % of theirs) at 28000 fp32 rows of 64 channels l <= 3
// with 2 of 16 experts; 11.5 us for 2048 fp64 rows of 16 channels l <= 4, 2 of 8.
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
  int32_t X, k, n_maps, piece;
  int32_t block0;  // this launch's first block
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
  const int block = a.block0 + static_cast<int>(blockIdx.x);
  while (mi + 1 < a.n_maps && block >= a.map[mi + 1].first) ++mi;
  const WgradMap m = a.map[mi];
  const int64_t r = block - m.first;
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
    from = fst[e] + found[1] * a.piece;
    count = min(a.piece, fst[e + 1] - from);
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
// (blocks [0, X nw): nw blocks of 256 weights each) and the shares of the
// gates' gradient (the blocks after them).  Bound by latency and the read of the
// pieces: 13-16 us for 16 experts' 16384 weights and 56000 gates, 6 us for 8
// experts' 1280 weights and 4096 gates in fp64.
template <class T>
__global__ __launch_bounds__(256) void k_join(int X, int nw, int64_t numel, int n_groups, int64_t max_pieces,
                                              const int32_t* __restrict__ pieces, const T* __restrict__ part,
                                              T* __restrict__ out, int64_t n_gates, int n_parts,
                                              const T* __restrict__ gate_part, T* __restrict__ gate_out) {
  __shared__ int lo[64], upto[64], list[256];
  const int b = blockIdx.x, tid = threadIdx.x;
  if (b >= X * nw) {
    const int64_t q = int64_t(b - X * nw) * 256 + tid;
    if (q >= n_gates) return;
    T s = 0;
    for (int p = 0; p < n_parts; ++p) s += gate_part[p * n_gates + q];
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
template <class T, int KS, bool ADJ, bool GG>
hipError_t rows_ks(RowArgs a, int64_t blocks, const T* src, const T* weights, const int32_t* experts,
                   const T* gates, const int32_t* order, T* dst, const T* other, T* part, hipStream_t s) {
  auto* const f = k_rows<T, KS, ADJ, GG>;
  if (a.lds.total > 64 * 1024) {  // above the default limit of dynamic LDS
    const hipError_t he =
        hipFuncSetAttribute(reinterpret_cast<const void*>(f), hipFuncAttributeMaxDynamicSharedMemorySize,
                            static_cast<int>(a.lds.total));
    if (he != hipSuccess) return he;
  }
  in_launches(blocks, 64 * a.waves, [&](int64_t block0, unsigned n) {
    a.block0 = static_cast<int32_t>(block0);
    hipLaunchKernelGGL(f, dim3(n), dim3(64 * a.waves), a.lds.total, s, a, src, weights, experts, gates, order, dst,
                       other, part);
  });
  return hipGetLastError();
}

// The rows' order and their experts in it; both NULL without a layout.
struct RowOrder {
  const int32_t *order = nullptr, *listed = nullptr;
};

RowOrder order_in(const Experts& p, int64_t n, const void* layout) {
  if (layout == nullptr) return {};
  const LayoutShape L = layout_shape(p, n);
  const char* const at = static_cast<const char*>(layout);
  return {reinterpret_cast<const int32_t*>(at + L.order), reinterpret_cast<const int32_t*>(at + L.listed)};
}

// n_parts: into how many partial sums the gates' gradient went, one for each
// block of output channels of each map.
template <class T, bool ADJ, bool GG>
hipError_t rows(const Experts& p, int64_t n, const T* src, const T* weights, const int32_t* experts, const T* gates,
                const RowOrder& layout, T* dst, const T* other, T* part, T* gate_grad, int& n_parts, hipStream_t s) {
  RowArgs a{};
  a.n_rows = n;
  a.ld_src = ADJ ? p.dim_out : p.dim_in;
  a.ld_dst = ADJ ? p.dim_in : p.dim_out;
  a.weight_numel = p.weight_numel;
  a.X = p.n_experts;
  a.k = p.top_k;
  a.n_maps = static_cast<int32_t>(p.maps.size());
  const int per = 16 / static_cast<int>(sizeof(T));
  int maxK = 0, maxN = 0, maxD = 0;
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
    const bool ps = aligned16(src) && a.ld_src % per == 0 && m.src_off % per == 0 && (m.K * m.d) % per == 0;
    const bool pd = (dst == nullptr || aligned16(dst)) && (!GG || aligned16(other)) && a.ld_dst % per == 0 &&
                    m.dst_off % per == 0 && (m.N * m.d) % per == 0;
    const bool pw = aligned16(weights) && a.weight_numel % per == 0 && m.woff % per == 0 && m.V % per == 0;
    // 28000 rows of 64 channels: 148 us by 16 bytes, 163 by single elements
    m.packed = (ps ? 1 : 0) | (pd ? 2 : 0) | (pw ? 4 : 0);
    maxK = std::max(maxK, m.K);
    maxN = std::max(maxN, m.N);
    maxD = std::max(maxD, m.d);
  }
  std::sort(a.map, a.map + a.n_maps, [](const RowMap& x, const RowMap& y) {
    return int64_t(x.K) * x.N * x.d > int64_t(y.K) * y.N * y.d;  // long maps first
  });
  // the fewest steps that hold a map's channels, 64 channels at a time above (zeros are multiplied like others: 4096
  // rows of 32 channels take 36 us in 8 steps, 58 in 16; 2048 fp64 rows of 16 take 17 us in 4, 52 in 16)
  const int KS = maxK <= 16 ? 4 : (maxK <= 32 ? 8 : 16);
  a.waves = std::min(4, (maxN + 15) / 16);
  // With few rows the tiles are made smaller, to have two wavefronts for each
  // of the 1024 SIMDs: 2048 fp64 rows of 16 channels take 17 us and, transposed
  // with the gates' gradient, 24 us, in tiles of 16 rows 28 us and 46 us.
  n_parts = 0;
  std::fill(a.first, a.first + kMaxMaps, INT32_MAX);
  for (int q = 0; q < a.n_maps; ++q) {
    a.first[q] = n_parts;
    n_parts += (a.map[q].N + 16 * a.waves - 1) / (16 * a.waves);
  }
  a.tile = static_cast<int32_t>(std::min<int64_t>(kTile, std::max<int64_t>(1, n * n_parts * a.waves / 2048)));
  const int64_t tiles = (n + a.tile - 1) / a.tile;
  if (tiles * n_parts > INT32_MAX) return hipErrorInvalidValue;
  a.n_tiles = static_cast<int32_t>(tiles);
  uint32_t o = 0;
  auto take = [&](size_t count, size_t each) {
    const uint32_t at = o;
    o = static_cast<uint32_t>((o + count * each + 15) / 16 * 16);
    return at;
  };
  const size_t entries = size_t(a.tile) * a.k, size = sizeof(T);
  a.lds.tile = take(std::max(4 * KS, 16 * a.waves) * pitch_of(maxD), size);
  a.lds.gates = take(entries * kTile, size);
  a.lds.mask = take(a.X, 4);
  a.lds.start = take(a.X, 4);
  a.lds.list = take(4 * (entries + 1), 4);
  a.lds.rows = take(kTile, 4);
  a.lds.graw = take(entries, size);
  a.lds.grow = take(16 * 9 * a.waves, size);
  a.lds.esum = take(GG ? entries : 0, size);
  a.lds.wsum = take(GG ? size_t(kTile) * a.k * a.waves : 0, size);
  a.lds.rsum = take(GG ? 16 * 9 * a.waves : 0, size);
  a.lds.ents = take(entries, 4);
  a.lds.total = o;
  if (a.lds.total > 160 * 1024) return hipErrorInvalidValue;
  const int64_t blocks = tiles * n_parts;
  T* const gg = n_parts == 1 ? gate_grad : part;
  for (const ColumnRun& r : ADJ ? p.bare_in : p.bare_out)
    if (dst != nullptr)
      hipLaunchKernelGGL(k_zero_columns<T>, dim3(blocks_for(n * r.len, 256)), dim3(256), 0, s, n, a.ld_dst, r.off,
                         r.len, dst);
  const int32_t* const order = layout.order;
  if (layout.listed != nullptr) experts = layout.listed;
  if (KS == 4) return rows_ks<T, 4, ADJ, GG>(a, blocks, src, weights, experts, gates, order, dst, other, gg, s);
  if (KS == 8) return rows_ks<T, 8, ADJ, GG>(a, blocks, src, weights, experts, gates, order, dst, other, gg, s);
  return rows_ks<T, 16, ADJ, GG>(a, blocks, src, weights, experts, gates, order, dst, other, gg, s);
}

// Workspace of the backward: the maps' shares of the gates' gradient, then the
// pieces' matrices.
struct BackwardSpace {
  size_t gates, parts, total;
};

BackwardSpace backward_space(const Experts& p, int64_t n) {
  const size_t size = p.f64 ? 8 : 4;
  const LayoutShape L = layout_shape(p, n);
  BackwardSpace w{};
  size_t shares = 0;  // as rows() counts them, with the fewest wavefronts a map's channels can get
  for (const ExpertMap& m : p.maps) shares += (m.mul_in + 15) / 16;
  w.parts = align_up(shares * n * p.top_k * size);
  w.total = std::max<size_t>(256, w.parts + align_up(L.n_groups * L.max_pieces * p.weight_numel * size));
  return w;
}

template <class T, int S, bool VEC>
hipError_t wgrad_launch(WgradArgs a, int64_t blocks, const T* x, const T* gates, const T* grad,
                        const int32_t* entries, const int32_t* first, const int32_t* pieces, T* out, hipStream_t s) {
  in_launches(blocks, 256, [&](int64_t block0, unsigned n) {
    a.block0 = static_cast<int32_t>(block0);
    hipLaunchKernelGGL((k_wgrad<T, S, VEC>), dim3(n), dim3(256), 0, s, a, x, gates, grad, entries, first, pieces, out);
  });
  return hipGetLastError();
}

template <class T>
hipError_t backward(const Experts& p, int64_t n, const T* x, const T* weights, const int32_t* experts, const T* gates,
                    const void* layout, const T* grad, T* gx, T* gw, T* gg, void* ws, hipStream_t s) {
  const RowOrder order = order_in(p, n, layout);
  int64_t n_gates = gg != nullptr ? n * p.top_k : 0;
  const int n_maps = static_cast<int>(p.maps.size()), X = p.n_experts;
  int n_parts = 1;
  const BackwardSpace space = backward_space(p, n);
  T* const gate_part = static_cast<T*>(ws);
  hipError_t he = hipSuccess;
  if (n_gates > 0)
    he = rows<T, true, true>(p, n, grad, weights, experts, gates, order, gx, x, gate_part, gg, n_parts, s);
  else if (n > 0 && gx != nullptr)
    he = rows<T, true, false>(p, n, grad, weights, experts, gates, order, gx, nullptr, nullptr, nullptr,
                             n_parts, s);
  if (he != hipSuccess) return he;
  if (n_parts == 1) n_gates = 0;  // they are whole
  const int64_t gate_blocks = (n_gates + 255) / 256;
  if (gw == nullptr) {
    if (gate_blocks > 0)
      hipLaunchKernelGGL(k_join<T>, dim3(static_cast<unsigned>(gate_blocks)), dim3(256), 0, s, 0, 0, p.weight_numel, 0,
                         int64_t(0), nullptr, nullptr, nullptr, n_gates, n_parts, gate_part, gg);
    return hipGetLastError();
  }
  const LayoutShape L = layout_shape(p, n);
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
  a.piece = L.piece;
  a.direct = n * p.top_k <= L.piece;
  a.slots = a.direct ? X : L.n_groups * L.max_pieces;
  const int per = 16 / static_cast<int>(sizeof(T));
  bool vec = aligned16(x) && aligned16(grad) && p.dim_in % per == 0 && p.dim_out % per == 0;
  int widest = 0;
  for (const ExpertMap& e : p.maps) {
    widest = std::max({widest, e.mul_in, e.mul_out});
    vec = vec && e.in_off % per == 0 && e.out_off % per == 0 && (e.mul_in * e.d) % per == 0 &&
          (e.mul_out * e.d) % per == 0;
  }
  // the smallest tile that holds the widest segment, several of 64 above: 2048 fp64 rows of 16 channels take 12 us in
  // tiles of 16, 30 us in tiles of 64; `vec`: 28000 rows of 64 channels take 141 us by 16 bytes, 277 by single elements
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
                       n_parts, gate_part, gg);
  return hipGetLastError();
}

}  // namespace

size_t experts_layout_bytes(const Experts& p, int64_t n) { return layout_shape(p, n).total; }

size_t experts_workspace(const Experts& p, int64_t n) { return backward_space(p, n).total; }

hipError_t launch_experts_layout(const Experts& p, int64_t n, const int32_t* experts, void* layout, int32_t* load,
                                 hipStream_t s) {
  const int X = p.n_experts;
  const LayoutShape L = layout_shape(p, n);
  char* const at = static_cast<char*>(layout);
  auto ints = [&](size_t off) { return reinterpret_cast<int32_t*>(at + off); };
  const int H = std::min(X, kMaxBins / X);
  const int threads = std::min(L.group, n) * p.top_k > 1024 ? 1024 : 256;
  hipLaunchKernelGGL(k_layout, dim3(static_cast<unsigned>(2 * L.n_groups)), dim3(threads), 0, s, n, X, p.top_k,
                     H, L.group, L.piece, experts, ints(L.order), ints(L.listed), ints(L.entries), ints(L.first),
                     ints(L.pieces));
  if (load != nullptr) hipLaunchKernelGGL(k_load, dim3(1), dim3(256), 0, s, X, L.n_groups, ints(L.first), load);
  return hipGetLastError();
}

hipError_t launch_experts_forward(const Experts& p, int64_t n, const void* x, const void* weights,
                                  const int32_t* experts, const void* gates, const void* layout, void* out,
                                  hipStream_t s) {
  const RowOrder order = order_in(p, n, layout);
  int n_parts;
  if (p.f64)
    return rows<double, false, false>(p, n, static_cast<const double*>(x), static_cast<const double*>(weights),
                                      experts, static_cast<const double*>(gates), order, static_cast<double*>(out),
                                      nullptr, nullptr, nullptr, n_parts, s);
  return rows<float, false, false>(p, n, static_cast<const float*>(x), static_cast<const float*>(weights), experts,
                                   static_cast<const float*>(gates), order, static_cast<float*>(out), nullptr,
                                   nullptr, nullptr, n_parts, s);
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
