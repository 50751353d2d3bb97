// node_api.cpp -- the node operators' C entry points: argument checks, the
// experts' plan, and dispatch to the kernels of node_*.hip.
#include <cmath>
#include <string>

#include "node_check.hpp"
#include "node_internal.hpp"

namespace tpconv {
namespace {

tpconv_status check_embedding(tpconv_dtype dt, int64_t n_rows, int64_t n_types, int64_t dim, int64_t stride) {
  if (!known(dt)) return bad("unknown dtype");
  if (n_rows < 0 || n_types < 0) return bad("negative row or type count");
  if (n_rows >= kMaxRows || n_types >= kMaxRows) return bad("row and type counts must be below 2^31");
  if (dim < 1 || dim >= kMaxRows) return bad("dim must be at least 1 and below 2^31");
  if (stride < dim) return bad("row stride below dim");
  return TPCONV_OK;
}

tpconv_status check_route(tpconv_dtype dt, int64_t n_rows, const tpconv_route_config* c, RouteArgs& a) {
  if (c == nullptr) return bad("NULL routing config");
  if (!known(dt)) return bad("unknown dtype");
  if (n_rows < 0 || n_rows >= kMaxRows) return bad("row count must be in [0, 2^31)");
  if (c->n_experts < 1 || c->top_k < 1 || c->n_groups < 1 || c->top_groups < 1)
    return bad("routing: n_experts, top_k, n_groups and top_groups must be positive");
  if (c->n_experts > TPCONV_MAX_EXPERTS || c->top_k > TPCONV_MAX_TOP_K || c->n_groups > 64)
    return fail(TPCONV_E_UNSUPPORTED, "routing: at most 256 experts, top_k 8, 64 groups");
  if (c->n_experts % c->n_groups != 0) return bad("routing: n_groups must divide n_experts");
  if (c->top_groups > c->n_groups) return bad("routing: top_groups exceeds n_groups");
  if (c->top_k > c->top_groups * (c->n_experts / c->n_groups))
    return bad("routing: top_k exceeds the experts in top_groups groups");
  if (c->score != TPCONV_ROUTE_SOFTMAX && c->score != TPCONV_ROUTE_SIGMOID) return bad("routing: unknown score");
  if (c->renormalise != 0 && c->renormalise != 1) return bad("routing: renormalise must be 0 or 1");
  if (!std::isfinite(c->scale)) return bad("routing: scale must be finite");
  a = RouteArgs{n_rows,          c->n_experts, c->top_k, c->n_groups, c->top_groups, c->score == TPCONV_ROUTE_SIGMOID,
                c->renormalise != 0, c->scale};
  return TPCONV_OK;
}

const Experts* experts_of(tpconv_experts_t h) { return reinterpret_cast<const Experts*>(h); }

// Whether rows times top_k is in [0, 2^31), without the product.
bool few_enough(const Experts& p, int64_t n_rows) { return n_rows >= 0 && n_rows <= (kMaxRows - 1) / p.top_k; }

tpconv_status check_experts(tpconv_experts_t h, int64_t n_rows) {
  if (h == nullptr) return bad("NULL experts plan");
  if (!few_enough(*experts_of(h), n_rows)) return bad("rows times top_k must be in [0, 2^31)");
  return TPCONV_OK;
}

tpconv_status dropout(const char* irreps, tpconv_dtype dt, int64_t n_rows, int64_t dim, double p, uint64_t seed,
                      uint64_t offset, const void* x, const void* residual, void* out, hipStream_t stream) {
  if (irreps == nullptr) return bad("NULL irreps string");
  if (!known(dt)) return bad("unknown dtype");
  if (n_rows < 0 || n_rows >= kMaxRows) return bad("row count must be in [0, 2^31)");
  if (!(p >= 0.0 && p < 1.0)) return bad("dropout: p must be in [0, 1)");
  std::vector<Segment> segs;
  std::string why;
  if (!parse_irreps(irreps, segs, why)) return fail(TPCONV_E_IRREPS, "irreps: " + why);
  if (segs.size() > kMaxDropSegs) return fail(TPCONV_E_UNSUPPORTED, "dropout: more than 32 segments");
  DropArgs a{};
  int64_t col = 0, ch = 0;
  for (const Segment& s : segs) {
    if (s.l > kMaxL) return fail(TPCONV_E_UNSUPPORTED, "l = " + std::to_string(s.l) + " exceeds TPCONV_MAX_L");
    const int64_t end = col + int64_t(s.mul) * (2 * s.l + 1);
    if (end >= (int64_t(1) << 24)) return fail(TPCONV_E_UNSUPPORTED, "dropout: a row has 2^24 or more columns");
    a.seg[a.n_segs++] = DropSeg{int32_t(col), int32_t(end), 2 * s.l + 1, int32_t(ch)};
    col = end;
    ch += s.mul;
  }
  if (dim != col) return bad("dropout: rows of this irreps string have " + std::to_string(col) + " columns");
  if (n_rows == 0) return TPCONV_OK;
  if (x == nullptr || out == nullptr) return bad("NULL input or output");
  a.n_rows = n_rows;
  a.dim = col;
  a.channels = ch;
  a.seed = seed;
  a.offset = offset;
  a.threshold = static_cast<uint32_t>(std::floor(p * 4294967296.0));
  a.scale = 1.0 / (1.0 - p);
  return launched(launch_dropout(dt == TPCONV_F64, a, x, residual, out, stream), "dropout");
}

}  // namespace
}  // namespace tpconv

using namespace tpconv;

// ---------------------------------------------------------------- embedding
extern "C" tpconv_status tpconv_embedding_forward(tpconv_dtype dtype, int64_t n_rows, int64_t n_types, int64_t dim,
                                                  const int32_t* types, const void* table, double scale, void* out,
                                                  int64_t out_stride, hipStream_t stream) {
  return guarded([&]() -> tpconv_status {
    const tpconv_status st = check_embedding(dtype, n_rows, n_types, dim, out_stride);
    if (st != TPCONV_OK || n_rows == 0) return st;
    if (types == nullptr || out == nullptr || (n_types > 0 && table == nullptr))
      return bad("NULL types, table or out");
    const EmbedArgs a{n_rows, n_types, dim, out_stride, types, scale};
    return launched(launch_embed_forward(dtype == TPCONV_F64, a, table, out, stream), "embedding forward");
  });
}

extern "C" size_t tpconv_embedding_workspace_bytes(tpconv_dtype dtype, int64_t n_rows, int64_t n_types, int64_t dim) {
  if (!known(dtype) || n_rows < 0 || n_types < 0 || dim < 1 || n_rows >= kMaxRows || n_types >= kMaxRows ||
      dim >= kMaxRows)
    return 0;
  return embed_workspace(dtype == TPCONV_F64, n_rows, n_types, dim);
}

extern "C" tpconv_status tpconv_embedding_backward(tpconv_dtype dtype, int64_t n_rows, int64_t n_types, int64_t dim,
                                                   const int32_t* types, const void* grad_out, int64_t grad_stride,
                                                   double scale, void* grad_table, void* workspace,
                                                   size_t workspace_bytes, hipStream_t stream) {
  return guarded([&]() -> tpconv_status {
    tpconv_status st = check_embedding(dtype, n_rows, n_types, dim, grad_stride);
    if (st != TPCONV_OK || n_types == 0) return st;
    if (grad_table == nullptr || (n_rows > 0 && (types == nullptr || grad_out == nullptr)))
      return bad("NULL types, grad_out or grad_table");
    st = check_workspace(workspace, workspace_bytes, tpconv_embedding_workspace_bytes(dtype, n_rows, n_types, dim),
                         "embedding workspace");
    if (st != TPCONV_OK) return st;
    const EmbedArgs a{n_rows, n_types, dim, grad_stride, types, scale};
    return launched(launch_embed_backward(dtype == TPCONV_F64, a, grad_out, grad_table, workspace, stream),
                    "embedding backward");
  });
}

// ------------------------------------------------------------------ routing
extern "C" tpconv_status tpconv_route_forward(tpconv_dtype dtype, int64_t n_rows, const tpconv_route_config* config,
                                              const void* logits, const void* bias, int32_t* experts, void* gates,
                                              hipStream_t stream) {
  return guarded([&]() -> tpconv_status {
    RouteArgs a{};
    const tpconv_status st = check_route(dtype, n_rows, config, a);
    if (st != TPCONV_OK || n_rows == 0) return st;
    if (logits == nullptr || experts == nullptr || gates == nullptr) return bad("NULL logits, experts or gates");
    return launched(launch_route_forward(dtype == TPCONV_F64, a, logits, bias, experts, gates, stream),
                    "routing forward");
  });
}

extern "C" tpconv_status tpconv_route_backward(tpconv_dtype dtype, int64_t n_rows, const tpconv_route_config* config,
                                               const void* logits, const int32_t* experts, const void* grad_gates,
                                               void* grad_logits, hipStream_t stream) {
  return guarded([&]() -> tpconv_status {
    RouteArgs a{};
    const tpconv_status st = check_route(dtype, n_rows, config, a);
    if (st != TPCONV_OK || n_rows == 0) return st;
    if (logits == nullptr || experts == nullptr || grad_gates == nullptr || grad_logits == nullptr)
      return bad("NULL logits, experts, grad_gates or grad_logits");
    return launched(launch_route_backward(dtype == TPCONV_F64, a, logits, experts, grad_gates, grad_logits, stream),
                    "routing backward");
  });
}

// ------------------------------------------------------------------ experts
extern "C" tpconv_status tpconv_experts_plan(const char* irreps_in, const char* irreps_out, int n_experts, int top_k,
                                             tpconv_dtype dtype, tpconv_experts_t* out) {
  return guarded([&]() -> tpconv_status {
    if (out == nullptr) return bad("NULL output handle");
    *out = nullptr;
    if (irreps_in == nullptr || irreps_out == nullptr) return bad("NULL irreps string");
    if (!known(dtype)) return bad("unknown dtype");
    if (n_experts < 1 || top_k < 1) return bad("experts: n_experts and top_k must be positive");
    if (n_experts > TPCONV_MAX_EXPERTS || top_k > TPCONV_MAX_TOP_K)
      return fail(TPCONV_E_UNSUPPORTED, "experts: at most 256 experts and top_k 8");
    std::vector<Segment> in, ou;
    std::string why;
    if (!parse_irreps(irreps_in, in, why)) return fail(TPCONV_E_IRREPS, "irreps_in: " + why);
    if (!parse_irreps(irreps_out, ou, why)) return fail(TPCONV_E_IRREPS, "irreps_out: " + why);
    for (const auto* v : {&in, &ou}) {
      bool seen[kMaxL + 1][2] = {};
      for (const Segment& s : *v) {
        if (s.l > kMaxL) return fail(TPCONV_E_UNSUPPORTED, "l = " + std::to_string(s.l) + " exceeds TPCONV_MAX_L");
        if (s.mul > TPCONV_MAX_EXPERT_MUL)
          return fail(TPCONV_E_UNSUPPORTED, "experts: multiplicity above 256");
        bool& was = seen[s.l][s.p > 0];
        if (was) return fail(TPCONV_E_UNSUPPORTED, "experts: an (l, parity) appears twice in one irreps string");
        was = true;
      }
    }
    Experts p;
    p.n_experts = n_experts;
    p.top_k = top_k;
    p.f64 = dtype == TPCONV_F64;
    auto starts = [](const std::vector<Segment>& v, int64_t& total) {
      std::vector<int32_t> at;
      total = 0;
      for (const Segment& s : v) {
        at.push_back(static_cast<int32_t>(total));
        total += int64_t(s.mul) * (2 * s.l + 1);
      }
      return at;
    };
    const std::vector<int32_t> in_at = starts(in, p.dim_in), out_at = starts(ou, p.dim_out);
    std::vector<bool> paired(ou.size(), false);
    for (size_t i = 0; i < in.size(); ++i) {
      const int d = 2 * in[i].l + 1;
      bool any = false;
      for (size_t j = 0; j < ou.size(); ++j) {
        if (ou[j].l != in[i].l || ou[j].p != in[i].p) continue;
        p.maps.push_back(ExpertMap{in_at[i], out_at[j], in[i].mul, ou[j].mul, d, int32_t(p.weight_numel)});
        p.listing.insert(p.listing.end(), {int64_t(i), int64_t(j), int64_t(in[i].l), p.weight_numel});
        p.weight_numel += int64_t(in[i].mul) * ou[j].mul;
        any = paired[j] = true;
      }
      if (!any) p.bare_in.push_back(ColumnRun{in_at[i], in[i].mul * d});
    }
    for (size_t j = 0; j < ou.size(); ++j)
      if (!paired[j]) p.bare_out.push_back(ColumnRun{out_at[j], ou[j].mul * (2 * ou[j].l + 1)});
    if (p.maps.empty()) return fail(TPCONV_E_NO_PATHS, "experts: no segment of irreps_in has a partner in irreps_out");
    *out = reinterpret_cast<tpconv_experts_t>(new Experts(std::move(p)));
    return TPCONV_OK;
  });
}

extern "C" tpconv_status tpconv_experts_query(tpconv_experts_t h, tpconv_experts_info* info) {
  return guarded([&]() -> tpconv_status {
    if (h == nullptr || info == nullptr) return bad("NULL experts plan or info");
    const Experts& p = *experts_of(h);
    *info = tpconv_experts_info{p.dim_in,    p.dim_out, p.weight_numel, int64_t(p.maps.size()),
                                p.n_experts, p.top_k,   p.f64 ? TPCONV_F64 : TPCONV_F32, 0};
    return TPCONV_OK;
  });
}

extern "C" tpconv_status tpconv_experts_maps(tpconv_experts_t h, int64_t* maps) {
  return guarded([&]() -> tpconv_status {
    if (h == nullptr || maps == nullptr) return bad("NULL experts plan or buffer");
    const Experts& p = *experts_of(h);
    for (size_t i = 0; i < p.listing.size(); ++i) maps[i] = p.listing[i];
    return TPCONV_OK;
  });
}

extern "C" void tpconv_experts_destroy(tpconv_experts_t h) { delete reinterpret_cast<Experts*>(h); }

extern "C" size_t tpconv_experts_layout_bytes(tpconv_experts_t h, int64_t n_rows) {
  if (h == nullptr || !few_enough(*experts_of(h), n_rows)) return 0;
  return experts_layout_bytes(*experts_of(h), n_rows);
}

extern "C" tpconv_status tpconv_experts_layout(tpconv_experts_t h, int64_t n_rows, const int32_t* experts,
                                               void* layout, size_t layout_bytes, int32_t* load, hipStream_t stream) {
  return guarded([&]() -> tpconv_status {
    tpconv_status st = check_experts(h, n_rows);
    if (st != TPCONV_OK) return st;
    if (n_rows > 0 && experts == nullptr) return bad("NULL experts");
    st = check_workspace(layout, layout_bytes, tpconv_experts_layout_bytes(h, n_rows), "experts layout");
    if (st != TPCONV_OK) return st;
    return launched(launch_experts_layout(*experts_of(h), n_rows, experts, layout, load, stream), "experts layout");
  });
}

extern "C" tpconv_status tpconv_experts_forward(tpconv_experts_t h, int64_t n_rows, const void* x,
                                                const void* weights, const int32_t* experts, const void* gates,
                                                const void* layout, void* out, hipStream_t stream) {
  return guarded([&]() -> tpconv_status {
    const tpconv_status st = check_experts(h, n_rows);
    if (st != TPCONV_OK || n_rows == 0) return st;
    if (x == nullptr || weights == nullptr || experts == nullptr || gates == nullptr || out == nullptr)
      return bad("NULL x, weights, experts, gates or out");
    if (layout != nullptr && reinterpret_cast<uintptr_t>(layout) % 256 != 0)
      return bad("experts layout must be 256-byte aligned");
    return launched(launch_experts_forward(*experts_of(h), n_rows, x, weights, experts, gates, layout, out, stream),
                    "experts forward");
  });
}

extern "C" size_t tpconv_experts_workspace_bytes(tpconv_experts_t h, int64_t n_rows) {
  if (h == nullptr || !few_enough(*experts_of(h), n_rows)) return 0;
  return experts_workspace(*experts_of(h), n_rows);
}

extern "C" tpconv_status tpconv_experts_backward(tpconv_experts_t h, int64_t n_rows, const void* x,
                                                 const void* weights, const int32_t* experts, const void* gates,
                                                 const void* layout, const void* grad_out, void* grad_x,
                                                 void* grad_weights, void* grad_gates, void* workspace,
                                                 size_t workspace_bytes, hipStream_t stream) {
  return guarded([&]() -> tpconv_status {
    tpconv_status st = check_experts(h, n_rows);
    if (st != TPCONV_OK) return st;
    if (grad_x == nullptr && grad_weights == nullptr && grad_gates == nullptr) return TPCONV_OK;
    if (n_rows > 0 && (experts == nullptr || gates == nullptr || grad_out == nullptr))
      return bad("NULL experts, gates or grad_out");
    if (n_rows > 0 && weights == nullptr && (grad_x != nullptr || grad_gates != nullptr)) return bad("NULL weights");
    if (n_rows > 0 && x == nullptr && (grad_weights != nullptr || grad_gates != nullptr)) return bad("NULL x");
    if (n_rows > 0 && grad_weights != nullptr && layout == nullptr)
      return bad("grad_weights needs the experts layout");
    if (layout != nullptr && reinterpret_cast<uintptr_t>(layout) % 256 != 0)
      return bad("experts layout must be 256-byte aligned");
    if (grad_weights != nullptr || grad_gates != nullptr) {
      st = check_workspace(workspace, workspace_bytes, tpconv_experts_workspace_bytes(h, n_rows),
                           "experts workspace");
      if (st != TPCONV_OK) return st;
    }
    return launched(launch_experts_backward(*experts_of(h), n_rows, x, weights, experts, gates, layout, grad_out,
                                            grad_x, grad_weights, grad_gates, workspace, stream),
                    "experts backward");
  });
}

// ------------------------------------------------------------------ dropout
extern "C" tpconv_status tpconv_dropout_forward(const char* irreps, tpconv_dtype dtype, int64_t n_rows, int64_t dim,
                                                double p, uint64_t seed, uint64_t offset, const void* x,
                                                const void* residual, void* out, hipStream_t stream) {
  return guarded([&] { return dropout(irreps, dtype, n_rows, dim, p, seed, offset, x, residual, out, stream); });
}

extern "C" tpconv_status tpconv_dropout_backward(const char* irreps, tpconv_dtype dtype, int64_t n_rows, int64_t dim,
                                                 double p, uint64_t seed, uint64_t offset, const void* grad_out,
                                                 void* grad_x, hipStream_t stream) {
  return guarded([&] { return dropout(irreps, dtype, n_rows, dim, p, seed, offset, grad_out, nullptr, grad_x, stream); });
}
