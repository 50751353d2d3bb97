/*
 * tpconv_node.h -- C ABI of libtpconv.so's node operators: what a
 * mixture-of-experts potential runs on its atoms around the convolution of
 * tpconv.h.
 *
 *   embedding   species -> the first node features, and the table's gradient
 *   routing     each atom's router logits -> top_k experts and their gates
 *   experts     equivariant linear maps on irreps rows, one set per expert,
 *               summed over an atom's experts with its gates
 *   dropout     on irreps rows, equivariant, from a counter-based generator
 *
 * The pages behind this library name mixture-of-experts potentials (MatRIS-
 * MoE and the Janus system; UMA in the TrimSO(2) abstract) and print no
 * formula for them: each formula below is the plain reading.
 *
 * Conventions are those of tpconv.h: device pointers, row-major contiguous
 * tensors (but for the row strides that the embedding takes), irreps rows
 * stored segment after segment as [mul][2l+1], caller-owned buffers, status
 * codes with tpconv_last_error(), work queued on `stream` without
 * synchronising it, no floating-point atomics (repeated calls give bitwise
 * identical outputs).  Data types: TPCONV_F32 and TPCONV_F64, the library's
 * own; sums and softmax statistics are held in the data type (32 bits or
 * more).  Outputs may overlap neither inputs nor each other, but where a call
 * says so.  Row counts are below 2^31; offsets are 64-bit.  Nothing here
 * allocates or clears memory through the runtime, so every call can be
 * captured into a HIP graph.
 */
#ifndef TPCONV_NODE_H
#define TPCONV_NODE_H

#include "tpconv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* -------------------------------------------------------------- embedding --
 * tpconv_embedding_forward: out[i][0..dim) = scale * table[types[i]], with
 * rows out_stride elements apart (out_stride >= dim), so the result can be
 * written straight into the scalar columns of wider feature rows; other
 * columns are not touched.  A type outside [0, n_types) -- the -1 of a
 * padding atom -- gets a row of zeros.
 *   types [n_rows] int32, table [n_types][dim], out [n_rows] rows.
 * Errors: TPCONV_E_INVALID_ARG (negative size, dim < 1, out_stride < dim, bad
 * dtype, NULL pointer to a non-empty tensor, n_rows or n_types >= 2^31),
 * TPCONV_E_HIP. */
tpconv_status tpconv_embedding_forward(tpconv_dtype dtype, int64_t n_rows, int64_t n_types, int64_t dim,
                                       const int32_t* types, const void* table, double scale, void* out,
                                       int64_t out_stride, hipStream_t stream);

/* Workspace bytes of tpconv_embedding_backward (0 for bad sizes). */
size_t tpconv_embedding_workspace_bytes(tpconv_dtype dtype, int64_t n_rows, int64_t n_types, int64_t dim);

/* tpconv_embedding_backward: grad_table[t] = scale * sum of grad_out[i] over
 * the rows of type t (overwritten; zero for a type no row has).  Rows are
 * sorted by type block by block, each block sums its runs of equal types and
 * the blocks' sums are added in order: no atomics, whatever the number of
 * types or how unequal their counts.  grad_out rows are grad_stride elements
 * apart.  workspace: caller-owned device memory, 256-byte aligned, at least
 * tpconv_embedding_workspace_bytes; it holds nothing between calls.  Errors:
 * as the forward, TPCONV_E_WORKSPACE (too small or misaligned). */
tpconv_status tpconv_embedding_backward(tpconv_dtype dtype, int64_t n_rows, int64_t n_types, int64_t dim,
                                        const int32_t* types, const void* grad_out, int64_t grad_stride,
                                        double scale, void* grad_table, void* workspace, size_t workspace_bytes,
                                        hipStream_t stream);

/* ---------------------------------------------------------------- routing --
 * For each row: scores s = softmax(logits) or sigmoid(logits); selection keys
 * s + bias; experts with logit -inf or bias -inf are masked and never chosen
 * (a bias leaves scores and gates as they are, -inf too).  With
 * n_groups > 1 the experts form n_groups equal runs: a group's key is the sum
 * of its two largest unmasked keys (of the one it has, if it has one), and
 * only the top_groups groups with the largest keys stay.  The top_k largest
 * keys are chosen, in descending order.  Experts whose keys are equal in the
 * data type (scores that round to 0 or 1) go by their logits, the larger first;
 * what ties in these too, and groups that tie, go to the lowest index.  A row with fewer than top_k experts left (all masked:
 * a padding atom) gets index -1 and gate 0 in its last places.
 * Gates: scale * s of the chosen, or, with renormalise, scale * s / (sum of s
 * over the chosen), formed from the logits so that scores which all underflow
 * still give gates that sum to scale.  The bias moves the selection only.
 * A NaN logit (with softmax also +inf) orders below every number but before
 * the masked ones and makes the gates it enters NaN; NaN keys go by their
 * index.  In a group's key, NaN and a key below half the type's lowest value
 * count as that half, so a group is dropped for its rank alone. */
#define TPCONV_MAX_EXPERTS 256
#define TPCONV_MAX_TOP_K 8

typedef enum { TPCONV_ROUTE_SOFTMAX = 0, TPCONV_ROUTE_SIGMOID = 1 } tpconv_route_score;

typedef struct {
  int32_t n_experts;   /* 1 .. TPCONV_MAX_EXPERTS */
  int32_t top_k;       /* 1 .. min(TPCONV_MAX_TOP_K, top_groups * (n_experts / n_groups)) */
  int32_t n_groups;    /* divides n_experts, at most 64; 1 = no groups */
  int32_t top_groups;  /* 1 .. n_groups */
  int32_t score;       /* tpconv_route_score */
  int32_t renormalise; /* 0 or 1 */
  double scale;
} tpconv_route_config;

/* tpconv_route_forward: logits [n_rows][n_experts], bias [n_experts] or NULL
 * -> experts [n_rows][top_k] int32, gates [n_rows][top_k].  Errors:
 * TPCONV_E_INVALID_ARG (NULL config or pointer to a non-empty tensor, sizes
 * or enum out of the ranges above), TPCONV_E_UNSUPPORTED (n_experts, top_k or
 * n_groups above the limits), TPCONV_E_HIP. */
tpconv_status tpconv_route_forward(tpconv_dtype dtype, int64_t n_rows, const tpconv_route_config* config,
                                   const void* logits, const void* bias, int32_t* experts, void* gates,
                                   hipStream_t stream);

/* tpconv_route_backward: grad_logits [n_rows][n_experts] (overwritten) of
 * <grad_gates, gates> for the forward's `experts` (the selection is a
 * constant).  With w the gates, g their gradient, c = scale:
 *   renormalised: d_a = w_a (g_a - sum_b g_b w_b / c), times (1 - s_a) for sigmoid;
 *   softmax: c s_j ([j chosen] g_j - sum_a g_a s_a) for every j;
 *   sigmoid: c g_a s_a (1 - s_a).
 * Renormalised, w is formed from the chosen logits and no others are read: NaN
 * in these or in grad_gates makes the entries of the chosen NaN, NaN elsewhere
 * in the row does not (the forward's gates show it).  Not renormalised, a NaN
 * score makes NaN of the entries whose formula has it.  Masked experts get 0.
 * Entries with index -1 are skipped whatever grad_gates holds there.  An
 * index outside [0, n_experts) is taken as -1; an expert that stands twice in
 * a row gets both gradients.  Errors as the forward. */
tpconv_status tpconv_route_backward(tpconv_dtype dtype, int64_t n_rows, const tpconv_route_config* config,
                                    const void* logits, const int32_t* experts, const void* grad_gates,
                                    void* grad_logits, hipStream_t stream);

/* ---------------------------------------------------------------- experts --
 * out[i][s'][v][m] = sum_a gates[i][a] sum_s sum_u M_e[p][u][v] x[i][s][u][m],
 * e = experts[i][a], p the map from segment s of irreps_in to segment s' of
 * irreps_out, for every pair of equal (l, parity): equivariant for any gates.
 * weights [n_experts][weight_numel]; map p at its offset, [mul_in][mul_out],
 * maps in the order of irreps_in's segments.  An output segment without a
 * partner is zero, and so is a row without experts.  experts entries outside
 * [0, n_experts) are skipped (their gate is not read into any sum and their
 * gate gradient is 0); an expert that stands twice counts twice.  Infinities
 * and NaN in an expert's weights reach the rows that have it with a gate other
 * than 0, and no others. */
#define TPCONV_MAX_EXPERT_MUL 256

typedef struct tpconv_experts_s* tpconv_experts_t;

typedef struct {
  int64_t dim_in, dim_out; /* row widths of x and out */
  int64_t weight_numel;    /* weights of one expert */
  int64_t n_maps;
  int32_t n_experts, top_k;
  int32_t dtype; /* tpconv_dtype */
  int32_t reserved;
} tpconv_experts_info;

/* tpconv_experts_plan: host only.  Irreps strings as for tpconv_plan, but
 * multiplicities may differ between segments and between the two strings:
 * each is 1 .. TPCONV_MAX_EXPERT_MUL, each (l, parity) at most once per
 * string, l <= TPCONV_MAX_L.  Errors: TPCONV_E_INVALID_ARG, TPCONV_E_IRREPS,
 * TPCONV_E_UNSUPPORTED, TPCONV_E_NO_PATHS (no pair of equal segments). */
tpconv_status tpconv_experts_plan(const char* irreps_in, const char* irreps_out, int n_experts, int top_k,
                                  tpconv_dtype dtype, tpconv_experts_t* out);
tpconv_status tpconv_experts_query(tpconv_experts_t plan, tpconv_experts_info* info);
/* Map list, host buffer of n_maps*4 int64: segment of irreps_in, segment of
 * irreps_out, l, weight offset. */
tpconv_status tpconv_experts_maps(tpconv_experts_t plan, int64_t* maps);
void tpconv_experts_destroy(tpconv_experts_t plan);

/* tpconv_experts_layout: from experts [n_rows][top_k], the order in which the
 * kernels below walk the rows (rows with the same experts together) and, for
 * the weights' gradient, the entries by expert; one per routing, into
 * caller-owned device memory of at least tpconv_experts_layout_bytes, 256-byte
 * aligned, which must outlive its uses.  load (device int32 [n_experts], may
 * be NULL) gets the entries of each expert, what a balance bias is updated
 * from.  Errors: TPCONV_E_INVALID_ARG, TPCONV_E_WORKSPACE, TPCONV_E_HIP. */
size_t tpconv_experts_layout_bytes(tpconv_experts_t plan, int64_t n_rows);
tpconv_status tpconv_experts_layout(tpconv_experts_t plan, int64_t n_rows, const int32_t* experts, void* layout,
                                    size_t layout_bytes, int32_t* load, hipStream_t stream);

/* tpconv_experts_forward: x [n_rows][dim_in], weights [n_experts]
 * [weight_numel], experts, gates [n_rows][top_k] -> out [n_rows][dim_out]
 * (overwritten).  layout: of these `experts`, or NULL, which takes the rows as
 * they come (the same result bit by bit; for a handful of rows it saves a
 * call).  Errors: TPCONV_E_INVALID_ARG, TPCONV_E_HIP. */
tpconv_status tpconv_experts_forward(tpconv_experts_t plan, int64_t n_rows, const void* x, const void* weights,
                                     const int32_t* experts, const void* gates, const void* layout, void* out,
                                     hipStream_t stream);

/* Workspace bytes of tpconv_experts_backward.  Most of them hold parts of
 * grad_weights, matrices of weight_numel each: at most n_rows top_k / 32 +
 * n_experts of them above 131072 entries (n_rows top_k times n_maps), n_rows
 * top_k / 8 + n_experts below.  32768 rows, 8 of 256 experts, 64 channels l <= 3
 * in fp32: 0.4 GB; 256 channels: 6.5 GB. */
size_t tpconv_experts_workspace_bytes(tpconv_experts_t plan, int64_t n_rows);

/* tpconv_experts_backward: gradients of <grad_out, out>:
 *   grad_x [n_rows][dim_in], grad_weights [n_experts][weight_numel] (zero for
 *   an expert no row has), grad_gates [n_rows][top_k].
 * Each is overwritten; NULL skips one.  layout is needed for grad_weights and
 * may be NULL without it.  workspace: caller-owned, 256-byte aligned, at least
 * tpconv_experts_workspace_bytes, holds nothing between calls; needed for
 * grad_weights and grad_gates.  Errors: TPCONV_E_INVALID_ARG,
 * TPCONV_E_WORKSPACE, TPCONV_E_HIP. */
tpconv_status tpconv_experts_backward(tpconv_experts_t plan, int64_t n_rows, const void* x, const void* weights,
                                      const int32_t* experts, const void* gates, const void* layout,
                                      const void* grad_out, void* grad_x, void* grad_weights, void* grad_gates,
                                      void* workspace, size_t workspace_bytes, hipStream_t stream);

/* ---------------------------------------------------------------- dropout --
 * tpconv_dropout_forward: out = residual + keep * x / (1 - p) on irreps rows
 * (residual NULL: without it), one draw for the 2l+1 components of a channel,
 * so the result stays equivariant.  The mask is never stored: with the row's
 * channels counted over all segments (C of them), channel c of row i has
 * number q = i C + c and takes word q mod 4 of Philox4x32-10 (Salmon et al.,
 * "Parallel random numbers: as easy as 1, 2, 3", 2011) with key `seed` and
 * counter (q / 4, offset), both 64-bit little end first; it is kept where
 * the word is at least floor(p 2^32).  A dropped channel is exactly the
 * residual (zero without one) whatever x holds.  0 <= p < 1.  x, residual and
 * out [n_rows][dim]; out may be x or residual itself, but no other overlap;
 * dim is the width of a row of `irreps`.
 * irreps as for tpconv_experts_plan, but mul may be any and an (l, parity)
 * may repeat.  Errors: TPCONV_E_INVALID_ARG (NULL, p, dim not the width of
 * `irreps`), TPCONV_E_IRREPS, TPCONV_E_UNSUPPORTED (l > TPCONV_MAX_L, over 32 segments, a row of 2^24 or
 * more columns), TPCONV_E_HIP.
 *
 * tpconv_dropout_backward: grad_x = keep * grad_out / (1 - p) with the
 * forward's seed and offset (the residual's gradient is grad_out itself). */
tpconv_status tpconv_dropout_forward(const char* irreps, tpconv_dtype dtype, int64_t n_rows, int64_t dim, double p,
                                     uint64_t seed, uint64_t offset, const void* x, const void* residual, void* out,
                                     hipStream_t stream);
tpconv_status tpconv_dropout_backward(const char* irreps, tpconv_dtype dtype, int64_t n_rows, int64_t dim, double p,
                                      uint64_t seed, uint64_t offset, const void* grad_out, void* grad_x,
                                      hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* TPCONV_NODE_H */
