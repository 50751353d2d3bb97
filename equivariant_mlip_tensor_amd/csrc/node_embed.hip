// node_embed.hip -- species embedding: out = scale * table[type], and the
// table's gradient.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "node_device.hpp"
#include "node_internal.hpp"

namespace tpconv {
namespace {

// -------------------------------------------------------------------- forward
// A copy: the table stays in cache, out is streamed.  Lanes share a row in
// groups of a power of two, so no lane divides by the row's length.  Bound by
// the writes: 250001 fp32 rows of 128 take 34 us (3.8 TB/s), 28000 rows of 64
// into rows of 1024 take 4.5 us, 16 fp64 rows 1.6 us (the launch).
template <class T, bool VEC>
__global__ __launch_bounds__(256) void k_embed(EmbedArgs a, int lg, const T* __restrict__ table,
                                               T* __restrict__ out) {
  constexpr int kPer = VEC ? 16 / sizeof(T) : 1;
  const T scale = static_cast<T>(a.scale);
  const int64_t pieces = a.dim / kPer, step = int64_t(gridDim.x) * 256 >> lg;
  const int lane = threadIdx.x & ((1 << lg) - 1);
  for (int64_t i = (int64_t(blockIdx.x) * 256 + threadIdx.x) >> lg; i < a.n_rows; i += step) {
    const int64_t t = a.types[i];
    const bool in = t >= 0 && t < a.n_types;
    for (int64_t c = lane; c < pieces; c += 1 << lg) {
      T* const to = out + i * a.stride + c * kPer;
      const T* const from = table + (in ? t : 0) * a.dim + c * kPer;
      if constexpr (VEC) {
        Pack<T> p = {};
        if (in) p = *reinterpret_cast<const Pack<T>*>(from);
#pragma unroll
        for (int q = 0; q < kPer; ++q) p.v[q] = in ? scale * p.v[q] : T(0);
        *reinterpret_cast<Pack<T>*>(to) = p;
      } else {
        *to = in ? scale * *from : T(0);
      }
    }
  }
}

// ------------------------------------------------------------------- backward
// Each block sorts its rows by type (rows of a type stay in order) and sums its
// runs of equal types.
// The sorted rows are cut into equal slices, one for each group of lanes that
// holds a row; a group sums its slice run by run.  A run that lies in one
// slice is written by its group; the parts of one that crosses slices go
// through LDS and are added in order.  So no group waits for another however
// unequal the runs are.  A block's sums are rows of `part`, its types a sorted
// list in `runs`; the second kernel adds each type's sums over the blocks, in
// order.  (A walk over all atoms by each type's own threads reads the types as
// often as there are types: 41 ms at 250001 rows.)  250001 fp32 rows of 128, 97
// types: 38 us, 3.4 TB/s: each block's sort, then its reads, in turn, so that
// wavefronts wait in 71 % of their cycles (blocks of half the length: 37 us and
// 3.4 more for the join); 28000 rows of 64, 5 types: 9.2 us (latency); 16 fp64
// rows in one block: 5.7 us.  Narrow rows have many groups and so short slices:
// with rows of one piece 512 groups share a block, and a run over many slices is
// joined by one of them, part after part: 250001 rows of one column take 44 us
// with 2 types, 28 with 5, 15 with 97.
constexpr int kRows = 1024;  // rows of a block, at most
constexpr int kThreads = 512;
constexpr int kCounters = 4096;  // of the sort by counting: 16 KiB of LDS, four blocks still share a CU's

struct EmbedSpace {
  int64_t rows, blocks;  // rows of a block
  size_t runs, part, total;
};

EmbedSpace embed_space(int64_t n, int64_t n_types, int64_t dim, size_t size) {
  EmbedSpace s{};
  // Blocks for the 256 CUs first, then long blocks: the longer, the fewer sums are left to add.  28000 rows:
  // sums and join 14.6 us, with 64 rows a block 17.7; 250001 rows: 45, with 512 rows a block 48.
  s.rows = 64;
  while (s.rows < kRows && s.rows * 256 < n) s.rows *= 2;
  s.blocks = (n + s.rows - 1) / s.rows;
  const int64_t most = std::min<int64_t>(s.rows, n_types);  // runs of a block
  size_t o = align_up(sizeof(int32_t) * s.blocks * (most + 1));
  s.part = o;
  s.total = std::max<size_t>(256, o + align_up(size * s.blocks * most * dim));
  return s;
}

// The block's rows by type, rows of a type in their order: put(place, type,
// row).  Each wavefront counts the types of its own run of rows, lanes of a type
// found by a ballot for each of its bits, in counters [type][wavefront]; their
// running sums are the places.
template <class Put>
__device__ __forceinline__ void sort_by_counting(const EmbedArgs& a, int64_t r0, int rows, int waves, int* count,
                                                 int* sums, Put put) {
  constexpr int kRounds = kRows / kThreads;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int none = static_cast<int>(a.n_types), n = (none + 1) * waves, bits = 32 - __clz(none);
  const int rounds = (rows + kThreads - 1) / kThreads;
  for (int q = tid; q < n; q += kThreads) count[q] = 0;
  int type[kRounds], place[kRounds];
#pragma unroll
  for (int j = 0; j < kRounds; ++j) {
    const int q = (w * rounds + j) * 64 + lane;
    const int t = a.types[r0 + min(q, rows - 1)];
    type[j] = j < rounds && q < rows ? (t >= 0 && t < none ? t : none) : -1;
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kRounds; ++j) {
    uint64_t peers = __ballot(type[j] >= 0);
    for (int b = 0; b < bits; ++b) {
      const uint64_t on = __ballot((type[j] >> b) & 1);
      peers &= (type[j] >> b) & 1 ? on : ~on;
    }
    const int rank = __popcll(peers & ((uint64_t(1) << lane) - 1));
    int base = 0;
    if (type[j] >= 0 && rank == 0) base = atomicAdd(&count[type[j] * waves + w], __popcll(peers));
    place[j] = __shfl(base, type[j] >= 0 ? __ffsll(static_cast<unsigned long long>(peers)) - 1 : 0, 64) + rank;
    wave_sync();  // the next round's rows take the places after these
  }
  __syncthreads();
  const int per = (n + kThreads - 1) / kThreads, q0 = min(n, tid * per), q1 = min(n, q0 + per);
  int mine = 0;
  for (int q = q0; q < q1; ++q) mine += count[q];
  int before = mine;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int t = __shfl_up(before, o, 64);
    if (lane >= o) before += t;
  }
  if (lane == 63) sums[w] = before;
  __syncthreads();
  before -= mine;
  for (int q = 0; q < w; ++q) before += sums[q];
  for (int q = q0; q < q1; ++q) {
    const int c = count[q];
    count[q] = before;
    before += c;
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kRounds; ++j)
    if (type[j] >= 0) put(count[type[j] * waves + w] + place[j], type[j], (w * rounds + j) * 64 + lane);
  __syncthreads();
}

// A group's columns: kCols pieces a lane at a time, 16 bytes or one element.
template <class T, bool VEC>
__global__ __launch_bounds__(kThreads) void k_embed_runs(EmbedArgs a, int lg, int block_rows, int most,
                                                         const T* __restrict__ grad,
                                                         int32_t* __restrict__ runs, T* __restrict__ part,
                                                         T* __restrict__ table) {
  constexpr int kPer = VEC ? 16 / sizeof(T) : 1;
  __shared__ uint64_t key[kRows];
  __shared__ int run_of[kRows];  // sorted row -> its run
  __shared__ int sums[kThreads / 64];
  __shared__ int count[kCounters];
  extern __shared__ char lds[];
  T* const head = reinterpret_cast<T*>(lds);  // a group's part of the run its slice starts in
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int64_t r0 = int64_t(blockIdx.x) * block_rows;
  const int rows = static_cast<int>(min<int64_t>(block_rows, a.n_rows - r0));
  // types outside the table come after all others
  auto key_of = [&](int64_t t, int q) {
    return (t >= 0 && t < a.n_types ? uint64_t(t) : uint64_t(1) << 40) << 10 | uint64_t(q);
  };
  // by counting where the counters fit (1024 rows: up to 511 types), else by a bitonic sort of the keys, which
  // takes any types: 250001 rows of 128 and 97 types in 38 us, by the other 48; 28000 rows of 64 in 9.2 and 12.4
  const int waves = (min(rows, kThreads) + 63) / 64;  // wavefronts with rows
  if ((a.n_types + 1) * waves <= kCounters) {
    sort_by_counting(a, r0, rows, waves, count, sums, [&](int at, int t, int q) { key[at] = key_of(t, q); });
  } else {
    int size = 2;
    while (size < rows) size *= 2;
    for (int q = tid; q < size; q += kThreads) key[q] = key_of(q < rows ? a.types[r0 + q] : -1, q);
    __syncthreads();
    for (int k = 2; k <= size; k *= 2)
      for (int j = k / 2; j > 0; j /= 2) {
        for (int q = tid; q < size / 2; q += kThreads) {
          const int lo = 2 * q - (q & (j - 1)), hi = lo + j;
          const uint64_t x = key[lo], y = key[hi];
          if ((x > y) == ((lo & k) == 0)) {
            key[lo] = y;
            key[hi] = x;
          }
        }
        __syncthreads();
      }
  }
  // number the runs: kEach sorted rows a thread
  constexpr int kEach = kRows / kThreads;
  int starts[kEach], mine = 0;
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    const int q = tid * kEach + j;
    const bool live = q < rows && (key[q] >> 50) == 0;
    starts[j] = live && (q == 0 || (key[q] >> 10) != (key[q - 1] >> 10));
    mine += starts[j];
  }
  int before = mine;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int t = __shfl_up(before, o, 64);
    if (lane >= o) before += t;
  }
  if (lane == 63) sums[w] = before;
  __syncthreads();
  int n_runs = 0;
  before -= mine;
  for (int q = 0; q < kThreads / 64; ++q) {
    if (q < w) before += sums[q];
    n_runs += sums[q];
  }
  // the only block's sums are the table itself: a run's row there is its type
  const bool whole = table != nullptr;
  int32_t* const my_runs = runs + blockIdx.x * int64_t(most + 1);
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    const int q = tid * kEach + j;
    before += starts[j];
    if (q < rows) run_of[q] = (key[q] >> 50) != 0 ? -1 : (whole ? static_cast<int>(key[q] >> 10) : before - 1);
    if (starts[j] && !whole) my_runs[before - 1] = static_cast<int32_t>(key[q] >> 10);
  }
  if (tid == 0 && !whole) my_runs[most] = n_runs;
  if (whole)
    for (int64_t q = tid; q < a.n_types * a.dim; q += kThreads) table[q] = T(0);
  __syncthreads();

  const int groups = kThreads >> lg, g = tid >> lg, sub = tid & ((1 << lg) - 1);
  const int slice = (rows + groups - 1) / groups, q0 = min(rows, g * slice), q1 = min(rows, q0 + slice);
  const T scale = static_cast<T>(a.scale);
  T* const my_part = whole ? table : part + blockIdx.x * int64_t(most) * a.dim;
  const int64_t pieces = a.dim / kPer;
  for (int64_t c0 = 0; c0 < pieces; c0 += 1 << lg) {
    const bool in = c0 + sub < pieces;
    const int64_t col = (in ? c0 + sub : 0) * kPer;
    T* const my_head = head + tid * kPer;
    Pack<T> s = {};
    int run = q0 < q1 ? run_of[q0] : -1;
    // a run that this slice starts in the middle of, or ends in
    const bool inherits = q0 > 0 && q0 < q1 && run >= 0 && run_of[q0 - 1] == run;
    bool first = inherits;
    Pack<T> mine_first = {};
    auto flush = [&]() {  // the run's sum within the slice
      if (first)
        mine_first = s;
      else if (in && run >= 0) {
#pragma unroll
        for (int e = 0; e < kPer; ++e) my_part[int64_t(run) * a.dim + col + e] = scale * s.v[e];
      }
      first = false;
    };
    constexpr int kAhead = 8;  // rows loaded before they are added
    for (int q = q0; q < q1; q += kAhead) {
      Pack<T> v[kAhead];
      int r[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int at = min(q + j, q1 - 1);
        r[j] = run_of[at];
        const T* from = grad + (r0 + int(key[at] & 1023)) * a.stride + col;
        if constexpr (VEC)
          v[j] = *reinterpret_cast<const Pack<T>*>(from);
        else
          v[j].v[0] = *from;
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        if (q + j >= q1) continue;
        if (r[j] != run) {
          flush();
          run = r[j];
          s = Pack<T>{};
        }
#pragma unroll
        for (int e = 0; e < kPer; ++e) s.v[e] += v[j].v[e];
      }
    }
    if (q0 < q1) flush();
    // parts of runs that began in an earlier slice: added to it by the group that began them, in order
#pragma unroll
    for (int e = 0; e < kPer; ++e) my_head[e] = mine_first.v[e];
    __syncthreads();
    if (q0 < q1 && in) {
      const int last = run_of[q1 - 1];
      const bool began_here = last >= 0 && !(inherits && run_of[q0] == last);
      if (began_here && q1 < rows && run_of[q1] == last) {
        Pack<T> t = s;  // this slice's own part of its last run
        for (int h = g + 1; h < groups; ++h) {
          const int at = h * slice;
          if (at >= rows || run_of[at] != last) break;
#pragma unroll
          for (int e = 0; e < kPer; ++e) t.v[e] += head[((h << lg) + sub) * kPer + e];
        }
#pragma unroll
        for (int e = 0; e < kPer; ++e) my_part[int64_t(last) * a.dim + col + e] = scale * t.v[e];
      }
    }
    __syncthreads();
  }
}

// One block per type and 64 columns: the blocks that have the type, found by
// a search of their sorted lists (a thread for each), are listed in order; the
// wavefronts each add a run of the list, 8 sums on their way at a time, and
// their results are added in order.  Bound by the latency of search, list and
// sums in turn: 7.3 us for 97 types of 245 blocks, 5.3 us for 5 types of 219.
constexpr int kList = 1024;

template <class T>
__global__ __launch_bounds__(1024) void k_embed_join(int64_t block0, int64_t dim, int64_t chunks, int64_t blocks,
                                                     int most, const int32_t* __restrict__ runs,
                                                     const T* __restrict__ part, T* __restrict__ out) {
  __shared__ int64_t list[kList];
  __shared__ int counts[16];
  __shared__ T sums[16][64];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, nw = blockDim.x >> 6;
  const int64_t block = block0 + blockIdx.x, t = block / chunks, c = (block - t * chunks) * 64 + lane;
  const int64_t col = min(c, dim - 1);
  T total = 0;
  for (int64_t b0 = 0; b0 < blocks; b0 += blockDim.x) {
    const int64_t b = b0 + tid;
    int at = -1;
    if (b < blocks) {
      const int32_t* const r = runs + b * (most + 1);
      const int n = r[most];
      int lo = 0, hi = n;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (r[mid] < t)
          lo = mid + 1;
        else
          hi = mid;
      }
      if (lo < n && r[lo] == t) at = lo;
    }
    const uint64_t have = __ballot(at >= 0);
    if (lane == 0) counts[w] = __popcll(have);
    __syncthreads();
    int before = 0, n = 0;
    for (int q = 0; q < nw; ++q) {
      if (q < w) before += counts[q];
      n += counts[q];
    }
    if (at >= 0) list[before + __popcll(have & ((uint64_t(1) << lane) - 1))] = b * most + at;
    __syncthreads();
    const int each = (n + nw - 1) / nw, q1 = min(n, (w + 1) * each);
    T s = 0;
    for (int q = w * each; q < q1; q += 8) {
      T v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = part[list[min(q + j, q1 - 1)] * dim + col];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (q + j < q1) s += v[j];
    }
    sums[w][lane] = s;
    __syncthreads();
    if (w == 0)
      for (int q = 0; q < nw; ++q) total += sums[q][lane];
  }
  if (w == 0 && c < dim) out[t * dim + c] = total;
}

// lanes (a power of two, 2^lg) that share a row of `pieces` pieces
int lanes_for(int64_t pieces, int most) {
  int lg = 0;
  while (lg < most && (int64_t(1) << lg) < pieces) ++lg;
  return lg;
}

template <class T>
hipError_t forward(const EmbedArgs& a, const T* table, T* out, hipStream_t s) {
  constexpr int kPer = 16 / sizeof(T);
  // 16 bytes a lane where all rows allow it: 250001 rows of 128 in 33 us, one element a lane 48
  const bool vec = aligned16(table) && aligned16(out) && a.dim % kPer == 0 && a.stride % kPer == 0;
  const int lg = lanes_for(vec ? a.dim / kPer : a.dim, 6);
  const int64_t blocks = std::min<int64_t>(((a.n_rows << lg) + 255) / 256, 16384);
  if (vec)
    hipLaunchKernelGGL((k_embed<T, true>), dim3(static_cast<unsigned>(blocks)), dim3(256), 0, s, a, lg, table, out);
  else
    hipLaunchKernelGGL((k_embed<T, false>), dim3(static_cast<unsigned>(blocks)), dim3(256), 0, s, a, lg, table, out);
  return hipGetLastError();
}

template <class T>
hipError_t backward(const EmbedArgs& a, const T* grad, T* grad_table, void* ws, hipStream_t s) {
  constexpr int kPer = 16 / sizeof(T);
  const EmbedSpace space = embed_space(a.n_rows, a.n_types, a.dim, sizeof(T));
  if (space.blocks > INT32_MAX) return hipErrorInvalidValue;
  char* const at = static_cast<char*>(ws);
  int32_t* const runs = reinterpret_cast<int32_t*>(at + space.runs);
  T* const part = reinterpret_cast<T*>(at + space.part);
  const int block_rows = static_cast<int>(space.rows);
  const int most = static_cast<int>(std::min<int64_t>(block_rows, a.n_types));
  // one block and a small table: no sums left to add (16 fp64 rows: 5.8 us, by way of the workspace 6.0 + 3.2)
  T* const table = space.blocks == 1 && a.n_types * a.dim <= 16384 ? grad_table : nullptr;
  if (a.n_rows > 0) {
    // 16 bytes a lane where all rows allow it, for the same reason as above
    const bool vec = aligned16(grad) && a.dim % kPer == 0 && a.stride % kPer == 0;
    const int lg = lanes_for(vec ? a.dim / kPer : a.dim, 9);
    const dim3 grid(static_cast<unsigned>(space.blocks));
    if (vec)
      hipLaunchKernelGGL((k_embed_runs<T, true>), grid, dim3(kThreads), kThreads * 16, s, a, lg, block_rows, most,
                         grad, runs, part, table);
    else
      hipLaunchKernelGGL((k_embed_runs<T, false>), grid, dim3(kThreads), kThreads * sizeof(T), s, a, lg,
                         block_rows, most, grad, runs, part, table);
  }
  if (table != nullptr) return hipGetLastError();
  const int64_t chunks = (a.dim + 63) / 64;
  if (a.n_types * chunks > INT32_MAX) return hipErrorInvalidValue;
  // a wavefront for each 16 blocks to add, 16 at most
  const int threads = 64 * static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(16, (space.blocks + 15) / 16)));
  in_launches(a.n_types * chunks, threads, [&](int64_t first, unsigned blocks) {
    hipLaunchKernelGGL(k_embed_join<T>, dim3(blocks), dim3(threads), 0, s, first, a.dim, chunks, space.blocks, most, runs,
                       part, grad_table);
  });
  return hipGetLastError();
}

}  // namespace

size_t embed_workspace(bool f64, int64_t n_rows, int64_t n_types, int64_t dim) {
  return embed_space(n_rows, n_types, dim, f64 ? 8 : 4).total;
}

hipError_t launch_embed_forward(bool f64, const EmbedArgs& a, const void* table, void* out, hipStream_t s) {
  return f64 ? forward(a, static_cast<const double*>(table), static_cast<double*>(out), s)
             : forward(a, static_cast<const float*>(table), static_cast<float*>(out), s);
}

hipError_t launch_embed_backward(bool f64, const EmbedArgs& a, const void* grad, void* grad_table, void* ws,
                                 hipStream_t s) {
  return f64 ? backward(a, static_cast<const double*>(grad), static_cast<double*>(grad_table), ws, s)
             : backward(a, static_cast<const float*>(grad), static_cast<float*>(grad_table), ws, s);
}

}  // namespace tpconv
