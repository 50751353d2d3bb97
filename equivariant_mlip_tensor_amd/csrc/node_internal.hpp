// node_internal.hpp -- what the node operators' host side (node_api.cpp) and
// kernels (node_*.hip) share.
#pragma once

#include <cstdint>
#include <vector>

#include "tpconv_internal.hpp"
#include "tpconv_node.h"

namespace tpconv {

constexpr int kMaxMaps = 2 * (kMaxL + 1);  // one per (l, parity)
constexpr int kMaxDropSegs = 32;

inline bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

inline size_t align_up(size_t v) { return (v + 255) / 256 * 256; }

// A grid of 2^32 threads or more is taken without an error and not run as asked,
// so blocks go out in launches of fewer: launch(first block, blocks).
template <class F>
void in_launches(int64_t blocks, int threads, F&& launch) {
  const int64_t most = ((int64_t(1) << 32) - 1) / threads;
  for (int64_t b = 0; b < blocks; b += most) launch(b, static_cast<unsigned>(blocks - b < most ? blocks - b : most));
}

// ------------------------------------------------------------- embedding
struct EmbedArgs {
  int64_t n_rows, n_types, dim, stride;
  const int32_t* types;
  double scale;
};
size_t embed_workspace(bool f64, int64_t n_rows, int64_t n_types, int64_t dim);
hipError_t launch_embed_forward(bool f64, const EmbedArgs& a, const void* table, void* out, hipStream_t s);
hipError_t launch_embed_backward(bool f64, const EmbedArgs& a, const void* grad, void* grad_table, void* ws,
                                 hipStream_t s);

// --------------------------------------------------------------- routing
struct RouteArgs {
  int64_t n_rows;
  int32_t X, k, groups, top_groups;
  bool sigmoid, renorm;
  double scale;
};
hipError_t launch_route_forward(bool f64, const RouteArgs& a, const void* logits, const void* bias, int32_t* experts,
                                void* gates, hipStream_t s);
hipError_t launch_route_backward(bool f64, const RouteArgs& a, const void* logits, const int32_t* experts,
                                 const void* grad_gates, void* grad_logits, hipStream_t s);

// --------------------------------------------------------------- experts
// One pair of equal (l, parity) segments.
struct ExpertMap {
  int32_t in_off, out_off;  // first column of the segment in a row of x / out
  int32_t mul_in, mul_out;
  int32_t d;                // 2 l + 1
  int32_t woff;             // first weight within an expert
};

// Columns of a row that no map writes: a run to be filled with zeros.
struct ColumnRun {
  int32_t off, len;
};

struct Experts {
  std::vector<ExpertMap> maps;
  std::vector<int64_t> listing;  // seg_in, seg_out, l, woff per map
  std::vector<ColumnRun> bare_out, bare_in;
  int32_t n_experts = 0, top_k = 0;
  int64_t dim_in = 0, dim_out = 0, weight_numel = 0;
  bool f64 = false;
};

size_t experts_layout_bytes(const Experts& p, int64_t n_rows);
size_t experts_workspace(const Experts& p, int64_t n_rows);
hipError_t launch_experts_layout(const Experts& p, int64_t n_rows, const int32_t* experts, void* layout,
                                 int32_t* load, hipStream_t s);
hipError_t launch_experts_forward(const Experts& p, int64_t n_rows, const void* x, const void* weights,
                                  const int32_t* experts, const void* gates, const void* layout, void* out,
                                  hipStream_t s);
hipError_t launch_experts_backward(const Experts& p, int64_t n_rows, const void* x, const void* weights,
                                   const int32_t* experts, const void* gates, const void* layout, const void* grad_out,
                                   void* grad_x, void* grad_weights, void* grad_gates, void* ws, hipStream_t s);

// --------------------------------------------------------------- dropout
struct DropSeg {
  int32_t off, end;  // columns [off, end)
  int32_t d;         // 2 l + 1
  int32_t channel;   // first channel
};
struct DropArgs {
  int64_t n_rows, dim, channels;
  uint64_t seed, offset;
  uint32_t threshold;
  double scale;
  int32_t n_segs;
  DropSeg seg[kMaxDropSegs];
};
hipError_t launch_dropout(bool f64, const DropArgs& a, const void* x, const void* residual, void* out, hipStream_t s);

// ------------------------------------------------------------ norm, 8 bits
constexpr int kMaxNormSegs = 32;

struct NormSeg {
  int32_t off, end;  // columns [off, end)
  int32_t d;         // 2 l + 1
  int32_t channel;   // first channel
};
struct NormArgs {
  int64_t n_rows;
  int32_t dim, n_segs, channels;
  int32_t lanes;     // of a row (the kernels' own)
  bool row_scope;
  double eps;
  NormSeg seg[kMaxNormSegs];
};
size_t norm_workspace(bool f64, const NormArgs& a, int64_t n_rows);
hipError_t launch_norm_forward(bool f64, const NormArgs& a, const void* x, const void* residual, const void* gamma,
                               void* sum, void* out, uint8_t* codes, float* scales, hipStream_t s);
hipError_t launch_norm_backward(bool f64, const NormArgs& a, const void* h, const void* gamma, const void* grad_out,
                                const void* grad_sum, void* grad_x, void* grad_gamma, void* ws, hipStream_t s);
hipError_t launch_pack8(const NormArgs& a, const float* x, uint8_t* codes, float* scales, hipStream_t s);
hipError_t launch_unpack8(NormArgs a, const uint8_t* codes, const float* scales, float* x, hipStream_t s);

// -------------------------------------------------------- gated and linear
// One pair of equal (l, parity) segments.
struct DenseMap {
  int32_t in_off, out_off, mul_in, mul_out;
  int32_t d;       // 2 l + 1
  int32_t woff;    // first weight
  int32_t seg_in;  // segment of irreps_in
  int32_t gate;    // first channel of the output segment
  int32_t act;
  bool even;       // 0e
};

struct Dense {
  std::vector<DenseMap> maps;
  std::vector<int64_t> listing;  // seg_in, seg_out, l, woff per map
  std::vector<ColumnRun> bare_in;
  int64_t dim_in = 0, dim_out = 0, weight_numel = 0, n_gates = 0;
  int32_t n_segs_in = 0;
  int32_t scalar_off = 0, scalar_mul = 0, scalar_seg = 0;  // gated: irreps_in's 0e
  int32_t scalar_out_mul = 0;                              // linear: mul of irreps_out's 0e
  int32_t act = TPCONV_ACT_IDENTITY;                       // linear
  bool gated = false, f64 = false;
  bool even_out = false;                                   // irreps_out has 0e
  // linear: grad_out's even scalars pass an activation
  bool sloped() const { return !gated && even_out && act != TPCONV_ACT_IDENTITY; }
};

// Rows, or 8-bit codes and scales of them.
struct DenseInput {
  const void* rows;
  const uint8_t* codes;
  const float* scales;
};

size_t dense_workspace(const Dense& p, int64_t n_rows);
hipError_t launch_dense_forward(const Dense& p, int64_t n_rows, const void* x, const void* weights,
                                const void* gate_weights, const void* bias, const void* residual, void* out,
                                hipStream_t s);
hipError_t launch_dense_backward(const Dense& p, int64_t n_rows, const DenseInput& x, const void* weights,
                                 const void* gate_weights, const void* bias, const void* grad_out, void* grad_x,
                                 void* grad_weights, void* grad_gate_weights, void* grad_bias, void* ws,
                                 hipStream_t s);

}  // namespace tpconv
