// node_block_api.cpp -- C entry points of the feed-forward block's operators
// (norm, rows in 8 bits, gated and linear maps): argument checks, plans, and
// dispatch to the kernels of node_norm.hip and node_dense.hip.
#include <cmath>
#include <string>

#include "node_check.hpp"
#include "node_internal.hpp"

namespace tpconv {
namespace {

struct Norm {
  NormArgs args;
  bool f64;
};

const Norm* norm_of(tpconv_norm_t h) { return reinterpret_cast<const Norm*>(h); }
const Dense* dense_of(tpconv_dense_t h) { return reinterpret_cast<const Dense*>(h); }

tpconv_status check_rows(int64_t n_rows) {
  if (n_rows < 0 || n_rows >= kMaxRows) return bad("row count must be in [0, 2^31)");
  return TPCONV_OK;
}

// The row's segments as the norm's and the 8-bit kernels take them.
tpconv_status rows_of(const char* irreps, NormArgs& a) {
  if (irreps == nullptr) return bad("NULL irreps string");
  std::vector<Segment> segs;
  std::string why;
  if (!parse_irreps(irreps, segs, why)) return fail(TPCONV_E_IRREPS, "irreps: " + why);
  if (segs.size() > kMaxNormSegs) return fail(TPCONV_E_UNSUPPORTED, "norm: more than 32 segments");
  a = NormArgs{};
  int64_t col = 0, ch = 0;
  for (const Segment& s : segs) {
    if (s.l > kMaxL) return fail(TPCONV_E_UNSUPPORTED, "l = " + std::to_string(s.l) + " exceeds TPCONV_MAX_L");
    const int64_t end = col + int64_t(s.mul) * (2 * s.l + 1);
    if (end > TPCONV_MAX_NORM_DIM) return fail(TPCONV_E_UNSUPPORTED, "norm: a row has more than 8192 columns");
    a.seg[a.n_segs++] = NormSeg{int32_t(col), int32_t(end), 2 * s.l + 1, int32_t(ch)};
    col = end;
    ch += s.mul;
  }
  a.dim = static_cast<int32_t>(col);
  a.channels = static_cast<int32_t>(ch);
  return TPCONV_OK;
}

// The rows of a call on 8 bits.
tpconv_status rows8(const char* irreps, int64_t n_rows, int64_t dim, const void* p, const void* q, const void* r,
                    NormArgs& a) {
  tpconv_status st = rows_of(irreps, a);
  if (st != TPCONV_OK) return st;
  st = check_rows(n_rows);
  if (st != TPCONV_OK) return st;
  if (dim != a.dim) return bad("rows of this irreps string have " + std::to_string(a.dim) + " columns");
  if (n_rows > 0 && (p == nullptr || q == nullptr || r == nullptr)) return bad("NULL x, codes or scales");
  a.n_rows = n_rows;
  return TPCONV_OK;
}

tpconv_status dense_plan(bool gated, const char* irreps_in, const char* irreps_out, int scalar_act, int gate_act,
                         tpconv_dtype dtype, tpconv_dense_t* out) {
  if (out == nullptr) return bad("NULL output handle");
  *out = nullptr;
  if (irreps_in == nullptr || irreps_out == nullptr) return bad("NULL irreps string");
  if (!known(dtype)) return bad("unknown dtype");
  for (int act : {scalar_act, gate_act})
    if (act < TPCONV_ACT_IDENTITY || act > TPCONV_ACT_GELU) return bad("unknown activation");
  std::vector<Segment> in, ou;
  std::string why;
  if (!parse_irreps(irreps_in, in, why)) return fail(TPCONV_E_IRREPS, "irreps_in: " + why);
  if (!parse_irreps(irreps_out, ou, why)) return fail(TPCONV_E_IRREPS, "irreps_out: " + why);
  for (const auto* v : {&in, &ou}) {
    bool seen[kMaxL + 1][2] = {};
    for (const Segment& s : *v) {
      if (s.l > kMaxL) return fail(TPCONV_E_UNSUPPORTED, "l = " + std::to_string(s.l) + " exceeds TPCONV_MAX_L");
      if (s.mul > TPCONV_MAX_DENSE_MUL) return fail(TPCONV_E_UNSUPPORTED, "multiplicity above 1024");
      bool& was = seen[s.l][s.p > 0];
      if (was) return fail(TPCONV_E_UNSUPPORTED, "an (l, parity) appears twice in one irreps string");
      was = true;
    }
  }
  auto even = [](const Segment& s) { return s.l == 0 && s.p > 0; };
  Dense p;
  p.gated = gated;
  p.f64 = dtype == TPCONV_F64;
  p.act = scalar_act;
  p.n_segs_in = static_cast<int32_t>(in.size());
  std::vector<int32_t> out_at, channel_at;
  int32_t channels = 0;
  for (const Segment& s : ou) {
    out_at.push_back(static_cast<int32_t>(p.dim_out));
    channel_at.push_back(channels);
    p.dim_out += int64_t(s.mul) * (2 * s.l + 1);
    channels += s.mul;
    if (even(s)) {
      p.even_out = true;
      p.scalar_out_mul = s.mul;
    }
  }
  if (gated) p.n_gates = channels;
  std::vector<bool> paired(ou.size(), false);
  for (size_t i = 0; i < in.size(); ++i) {
    const int d = 2 * in[i].l + 1;
    const int32_t off = static_cast<int32_t>(p.dim_in);
    p.dim_in += int64_t(in[i].mul) * d;
    if (gated && even(in[i])) {
      p.scalar_off = off;
      p.scalar_mul = in[i].mul;
      p.scalar_seg = static_cast<int32_t>(i);
    }
    bool any = gated && even(in[i]);
    for (size_t k = 0; k < ou.size(); ++k) {
      if (ou[k].l != in[i].l || ou[k].p != in[i].p) continue;
      const bool e = even(in[i]);
      const int32_t act = gated ? (e ? scalar_act : gate_act) : (e ? scalar_act : TPCONV_ACT_IDENTITY);
      p.maps.push_back(DenseMap{off, out_at[k], in[i].mul, ou[k].mul, d, int32_t(p.weight_numel), int32_t(i),
                                channel_at[k], act, e});
      p.listing.insert(p.listing.end(), {int64_t(i), int64_t(k), int64_t(in[i].l), p.weight_numel});
      p.weight_numel += int64_t(in[i].mul) * ou[k].mul;
      any = paired[k] = true;
    }
    if (!any) p.bare_in.push_back(ColumnRun{off, in[i].mul * d});
  }
  for (size_t k = 0; k < ou.size(); ++k)
    if (!paired[k]) return fail(TPCONV_E_NO_PATHS, "a segment of irreps_out has no partner in irreps_in");
  if (gated && p.scalar_mul == 0) return fail(TPCONV_E_NO_PATHS, "gated: irreps_in has no even scalars (0e)");
  *out = reinterpret_cast<tpconv_dense_t>(new Dense(std::move(p)));
  return TPCONV_OK;
}

tpconv_status check_dense(tpconv_dense_t h, bool gated, int64_t n_rows) {
  if (h == nullptr) return bad("NULL plan");
  if (dense_of(h)->gated != gated) return bad(gated ? "not a gated plan" : "not a linear plan");
  return check_rows(n_rows);
}

// x, or its codes and scales.
tpconv_status check_input(const Dense& p, const void* x, const uint8_t* codes, const float* scales) {
  if (codes == nullptr && scales == nullptr) return x != nullptr ? TPCONV_OK : bad("NULL x");
  if (codes == nullptr || scales == nullptr) return bad("codes and scales go together");
  if (x != nullptr) return bad("x and codes: one of them");
  if (p.f64) return bad("rows in 8 bits need an F32 plan");
  return TPCONV_OK;
}

}  // namespace
}  // namespace tpconv

using namespace tpconv;

// --------------------------------------------------------------------- norm
extern "C" tpconv_status tpconv_norm_plan(const char* irreps, int scope, double eps, tpconv_dtype dtype,
                                          tpconv_norm_t* out) {
  return guarded([&]() -> tpconv_status {
    if (out == nullptr) return bad("NULL output handle");
    *out = nullptr;
    if (!known(dtype)) return bad("unknown dtype");
    if (scope != TPCONV_NORM_SEGMENT && scope != TPCONV_NORM_ROW) return bad("norm: unknown scope");
    if (!(std::isfinite(eps) && eps >= 0x1p-126)) return bad("norm: eps must be finite and at least 2^-126");
    Norm p{};
    const tpconv_status st = rows_of(irreps, p.args);
    if (st != TPCONV_OK) return st;
    p.args.row_scope = scope == TPCONV_NORM_ROW;
    p.args.eps = eps;
    p.f64 = dtype == TPCONV_F64;
    *out = reinterpret_cast<tpconv_norm_t>(new Norm(p));
    return TPCONV_OK;
  });
}

extern "C" tpconv_status tpconv_norm_query(tpconv_norm_t h, tpconv_norm_info* info) {
  return guarded([&]() -> tpconv_status {
    if (h == nullptr || info == nullptr) return bad("NULL norm plan or info");
    const Norm& p = *norm_of(h);
    *info = tpconv_norm_info{p.args.dim,
                             p.args.channels,
                             p.args.n_segs,
                             p.args.row_scope ? TPCONV_NORM_ROW : TPCONV_NORM_SEGMENT,
                             p.f64 ? TPCONV_F64 : TPCONV_F32,
                             0,
                             p.args.eps};
    return TPCONV_OK;
  });
}

extern "C" void tpconv_norm_destroy(tpconv_norm_t h) { delete reinterpret_cast<Norm*>(h); }

extern "C" tpconv_status tpconv_norm_forward(tpconv_norm_t h, int64_t n_rows, const void* x, const void* residual,
                                             const void* gamma, void* sum, void* out, uint8_t* codes, float* scales,
                                             hipStream_t stream) {
  return guarded([&]() -> tpconv_status {
    if (h == nullptr) return bad("NULL norm plan");
    const tpconv_status st = check_rows(n_rows);
    if (st != TPCONV_OK) return st;
    const Norm& p = *norm_of(h);
    if (n_rows == 0) return TPCONV_OK;
    if ((codes == nullptr) != (scales == nullptr)) return bad("codes and scales go together");
    if (codes != nullptr && p.f64) return bad("rows in 8 bits need an F32 plan");
    if (x == nullptr) return bad("NULL x");
    if (sum == nullptr && out == nullptr && codes == nullptr) return bad("norm: no output asked for");
    NormArgs a = p.args;
    a.n_rows = n_rows;
    return launched(launch_norm_forward(p.f64, a, x, residual, gamma, sum, out, codes, scales, stream),
                    "norm forward");
  });
}

extern "C" size_t tpconv_norm_workspace_bytes(tpconv_norm_t h, int64_t n_rows) {
  if (h == nullptr || n_rows < 0 || n_rows >= kMaxRows) return 0;
  return norm_workspace(norm_of(h)->f64, norm_of(h)->args, n_rows);
}

extern "C" tpconv_status tpconv_norm_backward(tpconv_norm_t h, int64_t n_rows, const void* rows, const void* gamma,
                                              const void* grad_out, const void* grad_sum, void* grad_x,
                                              void* grad_gamma, void* workspace, size_t workspace_bytes,
                                              hipStream_t stream) {
  return guarded([&]() -> tpconv_status {
    if (h == nullptr) return bad("NULL norm plan");
    tpconv_status st = check_rows(n_rows);
    if (st != TPCONV_OK) return st;
    if (grad_x == nullptr && grad_gamma == nullptr) return TPCONV_OK;
    if (n_rows > 0 && (rows == nullptr || grad_out == nullptr)) return bad("NULL h or grad_out");
    if (grad_gamma != nullptr) {
      st = check_workspace(workspace, workspace_bytes, tpconv_norm_workspace_bytes(h, n_rows), "norm workspace");
      if (st != TPCONV_OK) return st;
    }
    if (n_rows == 0 && grad_gamma == nullptr) return TPCONV_OK;
    const Norm& p = *norm_of(h);
    NormArgs a = p.args;
    a.n_rows = n_rows;
    return launched(launch_norm_backward(p.f64, a, rows, gamma, grad_out, grad_sum, grad_x, grad_gamma, workspace,
                                         stream),
                    "norm backward");
  });
}

// -------------------------------------------------------------------- 8 bits
extern "C" tpconv_status tpconv_pack8(const char* irreps, int64_t n_rows, int64_t dim, const float* x, uint8_t* codes,
                                      float* scales, hipStream_t stream) {
  return guarded([&]() -> tpconv_status {
    NormArgs a;
    const tpconv_status st = rows8(irreps, n_rows, dim, x, codes, scales, a);
    if (st != TPCONV_OK || n_rows == 0) return st;
    return launched(launch_pack8(a, x, codes, scales, stream), "pack8");
  });
}

extern "C" tpconv_status tpconv_unpack8(const char* irreps, int64_t n_rows, int64_t dim, const uint8_t* codes,
                                        const float* scales, float* x, hipStream_t stream) {
  return guarded([&]() -> tpconv_status {
    NormArgs a;
    const tpconv_status st = rows8(irreps, n_rows, dim, x, codes, scales, a);
    if (st != TPCONV_OK || n_rows == 0) return st;
    return launched(launch_unpack8(a, codes, scales, x, stream), "unpack8");
  });
}

// ----------------------------------------------------------- gated and linear
extern "C" tpconv_status tpconv_gated_plan(const char* irreps_in, const char* irreps_out, int scalar_act, int gate_act,
                                           tpconv_dtype dtype, tpconv_dense_t* out) {
  return guarded([&] { return dense_plan(true, irreps_in, irreps_out, scalar_act, gate_act, dtype, out); });
}

extern "C" tpconv_status tpconv_linear_plan(const char* irreps_in, const char* irreps_out, int act, tpconv_dtype dtype,
                                            tpconv_dense_t* out) {
  return guarded([&] { return dense_plan(false, irreps_in, irreps_out, act, act, dtype, out); });
}

extern "C" tpconv_status tpconv_dense_query(tpconv_dense_t h, tpconv_dense_info* info) {
  return guarded([&]() -> tpconv_status {
    if (h == nullptr || info == nullptr) return bad("NULL plan or info");
    const Dense& p = *dense_of(h);
    *info = tpconv_dense_info{p.dim_in,
                              p.dim_out,
                              p.weight_numel,
                              int64_t(p.maps.size()),
                              p.n_gates,
                              p.scalar_mul,
                              p.gated ? p.n_gates : int64_t(p.scalar_out_mul),
                              p.n_segs_in,
                              p.f64 ? TPCONV_F64 : TPCONV_F32};
    return TPCONV_OK;
  });
}

extern "C" tpconv_status tpconv_dense_maps(tpconv_dense_t h, int64_t* maps) {
  return guarded([&]() -> tpconv_status {
    if (h == nullptr || maps == nullptr) return bad("NULL plan or buffer");
    const Dense& p = *dense_of(h);
    for (size_t i = 0; i < p.listing.size(); ++i) maps[i] = p.listing[i];
    return TPCONV_OK;
  });
}

extern "C" void tpconv_dense_destroy(tpconv_dense_t h) { delete reinterpret_cast<Dense*>(h); }

extern "C" tpconv_status tpconv_gated_forward(tpconv_dense_t h, int64_t n_rows, const void* x, const void* weights,
                                              const void* gate_weights, const void* gate_bias, void* out,
                                              hipStream_t stream) {
  return guarded([&]() -> tpconv_status {
    const tpconv_status st = check_dense(h, true, n_rows);
    if (st != TPCONV_OK || n_rows == 0) return st;
    if (x == nullptr || weights == nullptr || gate_weights == nullptr || out == nullptr)
      return bad("NULL x, weights, gate_weights or out");
    return launched(launch_dense_forward(*dense_of(h), n_rows, x, weights, gate_weights, gate_bias, nullptr, out,
                                         stream),
                    "gated forward");
  });
}

extern "C" tpconv_status tpconv_linear_forward(tpconv_dense_t h, int64_t n_rows, const void* x, const void* weights,
                                               const void* bias, const void* residual, void* out,
                                               hipStream_t stream) {
  return guarded([&]() -> tpconv_status {
    const tpconv_status st = check_dense(h, false, n_rows);
    if (st != TPCONV_OK || n_rows == 0) return st;
    if (x == nullptr || weights == nullptr || out == nullptr) return bad("NULL x, weights or out");
    return launched(launch_dense_forward(*dense_of(h), n_rows, x, weights, nullptr, bias, residual, out, stream),
                    "linear forward");
  });
}

extern "C" size_t tpconv_dense_workspace_bytes(tpconv_dense_t h, int64_t n_rows) {
  if (h == nullptr || n_rows < 0 || n_rows >= kMaxRows) return 0;
  return dense_workspace(*dense_of(h), n_rows);
}

extern "C" tpconv_status tpconv_gated_backward(tpconv_dense_t h, int64_t n_rows, const void* x, const uint8_t* codes,
                                               const float* scales, const void* weights, const void* gate_weights,
                                               const void* gate_bias, const void* grad_out, void* grad_x,
                                               void* grad_weights, void* grad_gate_weights, void* grad_gate_bias,
                                               void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return guarded([&]() -> tpconv_status {
    tpconv_status st = check_dense(h, true, n_rows);
    if (st != TPCONV_OK) return st;
    if (grad_x == nullptr && grad_weights == nullptr && grad_gate_weights == nullptr && grad_gate_bias == nullptr)
      return TPCONV_OK;
    const Dense& p = *dense_of(h);
    if (n_rows > 0) {
      st = check_input(p, x, codes, scales);
      if (st != TPCONV_OK) return st;
      if (weights == nullptr || gate_weights == nullptr || grad_out == nullptr)
        return bad("NULL weights, gate_weights or grad_out");
    }
    st = check_workspace(workspace, workspace_bytes, dense_workspace(p, n_rows), "gated workspace");
    if (st != TPCONV_OK) return st;
    return launched(launch_dense_backward(p, n_rows, DenseInput{x, codes, scales}, weights, gate_weights, gate_bias,
                                          grad_out, grad_x, grad_weights, grad_gate_weights, grad_gate_bias,
                                          workspace, stream),
                    "gated backward");
  });
}

extern "C" tpconv_status tpconv_linear_backward(tpconv_dense_t h, int64_t n_rows, const void* x, const uint8_t* codes,
                                                const float* scales, const void* weights, const void* bias,
                                                const void* grad_out, void* grad_x, void* grad_weights,
                                                void* grad_bias, void* workspace, size_t workspace_bytes,
                                                hipStream_t stream) {
  return guarded([&]() -> tpconv_status {
    tpconv_status st = check_dense(h, false, n_rows);
    if (st != TPCONV_OK) return st;
    if (grad_x == nullptr && grad_weights == nullptr && grad_bias == nullptr) return TPCONV_OK;
    const Dense& p = *dense_of(h);
    const bool params = grad_weights != nullptr || grad_bias != nullptr;
    if (n_rows > 0) {
      if (params || p.sloped() || x != nullptr || codes != nullptr || scales != nullptr) {
        st = check_input(p, x, codes, scales);
        if (st != TPCONV_OK) return st;
      }
      if (grad_out == nullptr) return bad("NULL grad_out");
      if (weights == nullptr && (grad_x != nullptr || p.sloped())) return bad("NULL weights");
    }
    if (params || p.sloped()) {
      st = check_workspace(workspace, workspace_bytes, dense_workspace(p, n_rows), "linear workspace");
      if (st != TPCONV_OK) return st;
    }
    return launched(launch_dense_backward(p, n_rows, DenseInput{x, codes, scales}, weights, nullptr, bias, grad_out,
                                          grad_x, grad_weights, nullptr, grad_bias, workspace, stream),
                    "linear backward");
  });
}
