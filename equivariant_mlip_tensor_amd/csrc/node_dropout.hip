// node_dropout.hip -- dropout on irreps rows from a counter-based generator.
#include <hip/hip_runtime.h>

#include "node_internal.hpp"

namespace tpconv {
namespace {

// Philox4x32-10 (Salmon et al., "Parallel random numbers: as easy as 1, 2, 3",
// 2011): ten rounds of two 32x32->64 bit products, the key stepped by Weyl
// constants.  Word w of the block with counter (block, offset).
struct Words {
  uint32_t w[4];
};

__device__ __forceinline__ Words philox(uint64_t block, uint64_t offset, uint64_t seed) {
  uint32_t c0 = uint32_t(block), c1 = uint32_t(block >> 32), c2 = uint32_t(offset), c3 = uint32_t(offset >> 32);
  uint32_t k0 = uint32_t(seed), k1 = uint32_t(seed >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = uint64_t(c0) * 0xD2511F53u, b = uint64_t(c2) * 0xCD9E8D57u;
    c0 = uint32_t(b >> 32) ^ c1 ^ k0;
    c1 = uint32_t(b);
    c2 = uint32_t(a >> 32) ^ c3 ^ k1;
    c3 = uint32_t(a);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return Words{{c0, c1, c2, c3}};
}

// One thread per element, its draw computed for it alone: for rows whose
// column table does not fit LDS (above 16384 columns; the generator then runs
// four times a block of draws, or 2l+1 times that).
template <class T>
__global__ void k_dropout_wide(DropArgs a, const T* x, const T* residual, T* out) {
  const T scale = static_cast<T>(a.scale);
  const int64_t total = a.n_rows * a.dim, step = int64_t(gridDim.x) * blockDim.x;
  for (int64_t q = blockIdx.x * int64_t(blockDim.x) + threadIdx.x; q < total; q += step) {
    const int64_t i = q / a.dim;
    const int32_t col = static_cast<int32_t>(q - i * a.dim);
    int s = 0;
    while (col >= a.seg[s].end) ++s;
    const int64_t ch = i * a.channels + a.seg[s].channel + (col - a.seg[s].off) / a.seg[s].d;
    const Words w = philox(uint64_t(ch) >> 2, a.offset, a.seed);
    const T base = residual != nullptr ? residual[q] : T(0);
    out[q] = w.w[ch & 3] >= a.threshold ? base + scale * x[q] : base;
  }
}

// Memory bound: a block takes tiles of rows, draws the tile's channels (four
// to a generator call) into LDS, a byte each, and streams the tile's pieces of
// 16 bytes past them; a table in LDS says which channel a column belongs to.
// The next kAhead pieces are loaded while the draws are made.  28000 fp32 rows
// of 1024 columns: 67 us with a residual (344 MB, 5.1 TB/s), 40 us without (229
// MB, 5.7 TB/s), at the rate of a copy; 1024 rows of 288: 4 us (latency).
constexpr int kThreads = 256, kAhead = 4;
constexpr int kTableColumns = 16384, kTileBytes = 16384;

template <class T, bool VEC, bool RES>
__global__ __launch_bounds__(kThreads) void k_dropout(DropArgs a, int tile, uint32_t inv, const T* x,
                                                      const T* residual, T* out) {
  constexpr int kPer = VEC ? 16 / sizeof(T) : 1;
  struct alignas(kPer * sizeof(T)) Piece {
    T v[kPer];
  };
  extern __shared__ uint16_t channel_of[];  // [dim], then a byte for each channel of the tile
  const int dim = static_cast<int>(a.dim), channels = static_cast<int>(a.channels);
  uint8_t* const keep = reinterpret_cast<uint8_t*>(channel_of + (dim + 7) / 8 * 8);
  const int tid = threadIdx.x;
  for (int s = 0; s < a.n_segs; ++s)
    for (int c = a.seg[s].off + tid; c < a.seg[s].end; c += kThreads)
      channel_of[c] = static_cast<uint16_t>(a.seg[s].channel + (c - a.seg[s].off) / a.seg[s].d);
  const T scale = static_cast<T>(a.scale);
  const int pieces = dim / kPer;
  for (int64_t i0 = int64_t(blockIdx.x) * tile; i0 < a.n_rows; i0 += int64_t(gridDim.x) * tile) {
    const int rows = static_cast<int>(min<int64_t>(tile, a.n_rows - i0)), total = rows * pieces;
    const Piece* const xp = reinterpret_cast<const Piece*>(x + i0 * dim);
    const Piece* const rp = reinterpret_cast<const Piece*>(residual + (RES ? i0 * dim : 0));
    Piece* const op = reinterpret_cast<Piece*>(out + i0 * dim);
    Piece vx[kAhead], vr[kAhead];
    auto load = [&](int q0) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int q = min(q0 + j * kThreads, total - 1);
        vx[j] = xp[q];
        if (RES) vr[j] = rp[q];
      }
    };
    load(tid);
    __syncthreads();  // the last tile's draws are no longer read
    const int64_t c0 = i0 * channels;
    const int n = rows * channels, lead = static_cast<int>(c0 & 3);  // channels of the first call that are not ours
    for (int g = tid; g * 4 < n + lead; g += kThreads) {
      const Words w = philox((uint64_t(c0) >> 2) + g, a.offset, a.seed);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = g * 4 + j - lead;
        if (c >= 0 && c < n) keep[c] = w.w[j] >= a.threshold;
      }
    }
    __syncthreads();
    for (int q0 = tid; q0 < total; q0 += kAhead * kThreads) {
      if (q0 != tid) load(q0);
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int q = q0 + j * kThreads;
        if (q >= total) continue;
        const int row = inv != 0 ? static_cast<int>(__umulhi(static_cast<uint32_t>(q), inv)) : q;
        const uint16_t* const ch = channel_of + (q - row * pieces) * kPer;
        const uint8_t* const kept = keep + row * channels;
        Piece p;
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
          const T base = RES ? vr[j].v[e] : T(0);
          p.v[e] = kept[ch[e]] ? base + scale * vx[j].v[e] : base;
        }
        op[q] = p;
      }
    }
  }
}

template <class T>
hipError_t dropout(const DropArgs& a, const T* x, const T* residual, T* out, hipStream_t s) {
  constexpr int kPer = 16 / sizeof(T);
  if (a.dim > kTableColumns) {
    const int64_t g = (a.n_rows * a.dim + 255) / 256;
    hipLaunchKernelGGL(k_dropout_wide<T>, dim3(static_cast<unsigned>(g > 65536 ? 65536 : g)), dim3(256), 0, s, a, x,
                       residual, out);
    return hipGetLastError();
  }
  // 28000 rows of 1024 columns: 67 us by 16 bytes, 79 by single elements
  const bool vec = a.dim % kPer == 0 && aligned16(x) && aligned16(residual) && aligned16(out);
  const int pieces = static_cast<int>(a.dim) / (vec ? kPer : 1);
  // a tile: as many rows as make 16 KiB of x, one at least; fewer where that leaves CUs without a tile (1024 rows of
  // 288: 4.2 us, with whole tiles 4.5)
  int64_t tile = kTileBytes / (a.dim * int64_t(sizeof(T)));
  tile = tile < 1 ? 1 : tile;
  while (tile > 1 && (a.n_rows + tile - 1) / tile < 512) tile = (tile + 1) / 2;
  int64_t blocks = (a.n_rows + tile - 1) / tile;
  blocks = blocks < 2048 ? blocks : 2048;  // 8 blocks for each CU, the table built once for all of a block's tiles
  const uint32_t inv = pieces > 1 ? uint32_t((0xFFFFFFFFull + pieces) / pieces) : 0u;
  const size_t lds = (a.dim + 7) / 8 * 16 + tile * a.channels;
  const dim3 grid(static_cast<unsigned>(blocks));
#define TPCONV_DROP(V, R)                                                                                         \
  hipLaunchKernelGGL((k_dropout<T, V, R>), grid, dim3(kThreads), lds, s, a, static_cast<int>(tile), inv, x, residual, \
                     out)
  if (vec && residual != nullptr)
    TPCONV_DROP(true, true);
  else if (vec)
    TPCONV_DROP(true, false);
  else if (residual != nullptr)
    TPCONV_DROP(false, true);
  else
    TPCONV_DROP(false, false);
#undef TPCONV_DROP
  return hipGetLastError();
}

}  // namespace

hipError_t launch_dropout(bool f64, const DropArgs& a, const void* x, const void* residual, void* out,
                          hipStream_t s) {
  return f64 ? dropout(a, static_cast<const double*>(x), static_cast<const double*>(residual),
                       static_cast<double*>(out), s)
             : dropout(a, static_cast<const float*>(x), static_cast<const float*>(residual), static_cast<float*>(out),
                       s);
}

}  // namespace tpconv
