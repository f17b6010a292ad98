/*
 * moe_routed.h -- C ABI of the routed mixture-of-experts layer for AMD
 * Instinct MI355X (gfx950): routing plan, activation gather, grouped expert
 * FFN (gate/up projection + SwiGLU, weighted down projection) and a
 * fixed-order combine.
 *
 * Sources of the operations (web pages, cited by title and section):
 *  [P1] "Round 4 Track C: Prefill MoE Plan (mm_clear + mm_hist + mm_scan +
 *       mm_place) & Epilogue / Gather Audit" -- s.1 findings 1-4, s.2
 *       Table 2.1, s.3 Bitwise & Numerical Parity.
 *  [P3] "Batched resident MoE experts on Apple Silicon: a flat parallel expert
 *       pass" -- s.1 Contribution (job list of (token, expert, weight);
 *       gate/up -> gated activation -> weighted down projection), s.3
 *       Results (fixed per-token top-k summation order).
 *  [P4] "Add --moe-mode sweep-prefill: streamed expert supply for CPU
 *       mul_mat_id" -- Mechanism (experts in ascending id order over
 *       contiguous slices).
 *
 * Common conventions
 *  - Entry i = t*K + k: token t's k-th routed expert (token-major), k in the
 *    router's order.
 *  - Element types (enum moe_dtype): activations x, gathered rows xs, expert
 *    weights and the SwiGLU output h share one type D. Accumulation is fp32.
 *    Router weights w, the per-row weight sw, expert outputs y and the layer
 *    output are fp32.
 *  - Weight layouts, row-major: w_gate and w_up [E][d][f] (input index, then
 *    output index), w_down [E][f][d].
 *  - Pointers: every array argument is a DEVICE pointer (hipMalloc'd or
 *    equivalent), owned by the caller. The library allocates and frees no
 *    device memory and keeps no state between calls. Arrays must not alias,
 *    except that a scratch/workspace buffer may be reused by later calls on
 *    the same stream. Structs passed by pointer (sizes, timers) live on the
 *    host.
 *  - Streams: every call enqueues its kernels on `stream` (a hipStream_t; NULL
 *    is the default stream) and returns without waiting. Data-dependent
 *    scalars (row counts) stay on the device in `meta` and are read there by
 *    later calls.
 *  - Outputs need no clearing: every element a call defines is written on
 *    every call.
 *  - Errors: each call returns MOE_OK or an error code; nothing prints, throws
 *    or aborts. MOE_EINVAL: a NULL or misaligned pointer (data arrays need
 *    16-byte alignment, index arrays 4-byte), a size out of range, an
 *    undersized scratch or workspace. MOE_EUNSUPPORTED: a valid request this
 *    build does not implement (E > MOE_MAX_EXPERTS). MOE_EHIP: the HIP
 *    runtime refused a launch (e.g. no device). Argument checks happen before
 *    any HIP call.
 *  - Ids: -1 marks a skipped entry ([P1] s.3: experts skipped by tail
 *    skipping); it gets no row and pos = -1. Any other id outside [0, E) is
 *    counted in meta[MOE_META_NBAD] and treated the same way.
 *  - Inconsistent plan arrays passed to the later calls (made up rather than
 *    produced by moe_plan) give unspecified values but never an access
 *    outside the stated array sizes: row and token indices are clamped to
 *    their bounds on the device.
 */
#ifndef MOE_ROUTED_H
#define MOE_ROUTED_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef void *moe_stream_t; /* hipStream_t */

enum moe_dtype { MOE_F32 = 0, MOE_F16 = 1, MOE_BF16 = 2 };

enum moe_status {
    MOE_OK = 0,
    MOE_EINVAL = 1,
    MOE_EUNSUPPORTED = 2,
    MOE_EHIP = 3,
    MOE_ENOSPACE = 4 /* larger than the fixed buffer of moe_forward_packed_noalloc */
};

/* Fields of the device array meta[MOE_META_N] written by moe_plan. */
enum moe_meta_field {
    MOE_META_NENT = 0,    /* T*K entries */
    MOE_META_NBLK = 1,    /* plan blocks of MOE_PLAN_BLOCK entries */
    MOE_META_NR = 2,      /* rows of the expert-sorted list, pads included */
    MOE_META_NT = 3,      /* tiles of tm rows: nr / tm */
    MOE_META_NACTIVE = 4, /* experts with at least one entry */
    MOE_META_MAXCNT = 5,  /* largest entry count of one expert */
    MOE_META_NSKIP = 6,   /* entries with id -1 */
    MOE_META_NBAD = 7,    /* entries with another id outside [0, E) */
    MOE_META_TM = 8,
    MOE_META_E = 9,
    MOE_META_K = 10,
    MOE_META_N = 11
};

#define MOE_MAX_EXPERTS 1024 /* one plan counter per expert in LDS ([P1] s.1 finding 1: 1024 counters) */
#define MOE_PLAN_BLOCK 1024  /* entries per plan block (the page's block size) */

#define MOE_ROUTE_MAX_K 64     /* picks per token of moe_route_topk (one wave lane each) */

/*
 * moe_route_topk -- the router step before the plan ([P1] s.1 finding 5 and
 * s.3 name route_topk, which writes the routed ids). Per token: a softmax over
 * the E logits, the K largest probabilities kept and renormalised to sum to
 * one -- equivalently the K largest logits, weight k = exp(l_k - m) / sum over
 * the K picks of exp(l_j - m), m the largest logit. Picks are in descending
 * order; equal logits go to the lower expert id; NaN logits are never picked
 * and if fewer than K logits are not NaN the remaining picks are id -1 with
 * weight 0. fp32 arithmetic, exponentials summed in pick order.
 * In:  logits [T][E] fp32. Out: ids [T*K] int32, w [T*K] fp32 (the inputs of
 * moe_plan / moe_forward).
 * Errors: MOE_EINVAL for T, E or K < 1, K > E, NULL/misaligned pointers;
 * MOE_EUNSUPPORTED for E > MOE_MAX_EXPERTS or K > MOE_ROUTE_MAX_K; MOE_EHIP
 * on a failed launch.
 */
int moe_route_topk(const float *logits, int T, int E, int K, int32_t *ids, float *w,
                   moe_stream_t stream);

/* Host-side sizes of a plan. */
typedef struct {
    int64_t nent;         /* T*K */
    int64_t nblk;         /* ceil(nent / MOE_PLAN_BLOCK) */
    int64_t max_rows;     /* upper bound of nr: rows to allocate for stok, sw, xs, h, y */
    int64_t max_tiles;    /* max_rows / tm */
    size_t scratch_bytes; /* device scratch moe_plan needs */
} moe_plan_sizes_t;

/*
 * moe_plan_sizes -- host only, no HIP call.
 * max_rows = ceil((T*K + min(E, T*K)*(tm-1)) / tm) * tm: every valid entry has
 * a row and each active expert adds at most tm-1 pad rows.
 * Returns MOE_EINVAL if T, K, E or tm < 1, T*K >= 2^31 or max_rows >= 2^31;
 * MOE_EUNSUPPORTED if E > MOE_MAX_EXPERTS.
 */
int moe_plan_sizes(int T, int K, int E, int tm, moe_plan_sizes_t *out);

/*
 * moe_plan -- the routing plan ([P1] s.1 findings 1 and 2; s.3 lists the
 * outputs): a per-block expert histogram, a prefix scan of the per-expert
 * counts padded up to a multiple of tm (pad rows marked -1 in the same pass),
 * and a placement of every entry into an expert-sorted row list. Experts are
 * laid out in ascending id order ([P4] Mechanism). Inside one expert the rows
 * follow entry order (stable by token, then k), so the plan is unique.
 *
 * In:  ids [T*K] int32, w [T*K] fp32 (router weight of each entry).
 * Out: cnt [E]            entries per expert
 *      eoff [E+1]         first row of each expert; eoff[E] = nr
 *      tiles [max_tiles]  expert of each tm-row tile, tiles [0, nt) written
 *      stok [max_rows]    token of each row; -1 on pad rows; rows [0, nr) written
 *      sw [max_rows]      router weight of each row (bit copy of w); +0.0 on pad rows
 *      pos [T*K]          row of each entry; -1 for skipped/bad entries
 *      boff [nblk*E]      entries of expert e in the blocks before block b, at [b*E + e]
 *      meta [MOE_META_N]  see enum moe_meta_field
 * scratch: device buffer of at least moe_plan_sizes().scratch_bytes.
 * Errors: as moe_plan_sizes, plus MOE_EINVAL for NULL/misaligned pointers or
 * a small scratch; MOE_EHIP on a failed launch.
 */
int moe_plan(const int32_t *ids, const float *w, int T, int K, int E, int tm, int32_t *cnt,
             int32_t *eoff, int32_t *tiles, int32_t *stok, float *sw, int32_t *pos, int32_t *boff,
             int32_t *meta, void *scratch, size_t scratch_bytes, moe_stream_t stream);

/*
 * moe_gather -- [P1] s.1 finding 4: copy each routed token's row of the
 * half-precision activation into expert-contiguous rows, bit for bit.
 * xs[r][:] = x[stok[r]][:] for r < min(meta[MOE_META_NR], max_rows); pad rows
 * (stok[r] < 0) become all-zero bits. Rows >= nr are not touched.
 * In:  x [T][d] of dtype, stok [max_rows], meta [MOE_META_N] (device, from moe_plan).
 * Out: xs [max_rows][d] of dtype.
 * Errors: MOE_EINVAL for d < 8 or d % 8 != 0, T < 1, max_rows < 1, bad dtype,
 * NULL/misaligned pointers; MOE_EHIP on a failed launch.
 */
int moe_gather(const void *x, int dtype, int T, int d, const int32_t *stok, const int32_t *meta,
               int64_t max_rows, void *xs, moe_stream_t stream);

/*
 * moe_ffn_scratch_bytes -- host only: scratch moe_expert_ffn needs for a plan
 * of at most max_rows rows over E experts with tile tm, hidden size d,
 * intermediate size f and element type dtype (the work list, plus fp32
 * partial sums when a projection is split along its reduction, see
 * moe_ffn_splits).
 * Errors: MOE_EINVAL for NULL bytes, E/tm/max_rows < 1, d or f not positive
 * multiples of 8, bad dtype; MOE_EUNSUPPORTED for E > MOE_MAX_EXPERTS.
 */
int moe_ffn_scratch_bytes(int E, int d, int f, int tm, int64_t max_rows, int dtype,
                          size_t *bytes);

/*
 * moe_ffn_splits -- host only: into how many reduction ranges moe_expert_ffn
 * (and moe_forward) split the gate/up projection (over d) and the down
 * projection (over f) for these sizes. A projection is split when the bound on
 * its work items is too small to occupy the GPU (decode-sized batches); the
 * partial sums are then added in a fixed order, so results stay deterministic
 * run to run but differ in rounding from the unsplit order. Same argument
 * checks as moe_ffn_scratch_bytes.
 */
int moe_ffn_splits(int E, int d, int f, int tm, int64_t max_rows, int dtype, int *split_gateup,
                   int *split_down);

/*
 * moe_ffn_big_cells -- host only: which projections of the packed entry
 * points (moe_expert_ffn_packed, moe_forward_packed) with fp16 or bf16 run
 * each expert's runs of 4 work items (256 rows) on 512-thread workgroups of
 * 256 rows x 256 weight columns whose operands are staged in LDS (a separate
 * launch before the other work items): *on bit 0 = the gate/up projection,
 * bit 1 = the down projection. Used when the plan bound averages at least 64
 * rows per expert, for a projection that is not split. The results are the
 * same bits either way. Same argument checks as moe_ffn_scratch_bytes.
 */
int moe_ffn_big_cells(int E, int d, int f, int tm, int64_t max_rows, int dtype, int *on);

/*
 * moe_expert_ffn -- the grouped expert FFN over the expert-sorted rows
 * ([P3] s.1: gate/up projection, gated activation, weighted down projection
 * per job; [P1] s.1 finding 5 names the SwiGLU and down-projection epilogue
 * kernels). For every row r in expert e's range [eoff[e], eoff[e+1]):
 *   g = xs[r] . w_gate[e],  u = xs[r] . w_up[e]            (fp32 accumulation)
 *   h[r][j] = D( silu(g[j]) * u[j] ),  silu(z) = z / (1 + exp(-z))
 *   y[r][c] = sw[r] * sum_j h[r][j] * w_down[e][j][c]      (fp32)
 * h is stored in D (the operand type of the down projection, like the page's
 * half SwiGLU output) for every row of every expert range; y is stored only
 * on rows with stok[r] >= 0 (pad rows are never read by moe_combine).
 * In:  xs [max_rows][d], w_gate/w_up [E][d][f], w_down [E][f][d] (dtype),
 *      eoff [E+1], stok [max_rows], sw [max_rows], meta [MOE_META_N].
 * Out: h [max_rows][f] (dtype), y [max_rows][d] fp32.
 * scratch: at least moe_ffn_scratch_bytes().
 * Errors: MOE_EINVAL for d or f not positive multiples of 8 or above 2^22,
 * one expert matrix of 2 GiB or more, bad dtype, NULL/misaligned pointers,
 * small scratch, tm < 1, more workgroups than a launch of 2^32 threads holds
 * (items of 64 rows, by max_rows, E and tm, times groups of 256 columns of h or
 * 512 of y: 2^24 of them; packed 16-bit weights with 64 rows an expert or more,
 * 193 rows times 128 columns of h or 256 of y: 2^23); MOE_EUNSUPPORTED for E > MOE_MAX_EXPERTS; MOE_EHIP
 * on a failed launch.
 */
int moe_expert_ffn(const void *xs, const void *w_gate, const void *w_up, const void *w_down,
                   int dtype, int E, int d, int f, int tm, const int32_t *eoff, const int32_t *stok,
                   const float *sw, const int32_t *meta, int64_t max_rows, void *h, float *y,
                   void *scratch, size_t scratch_bytes, moe_stream_t stream);

/* Which matrices a packed weight buffer holds. */
enum moe_wkind {
    MOE_W_GATE_UP = 0, /* W_gate or W_up: [E][d][f] */
    MOE_W_DOWN = 1     /* W_down: [E][f][d] */
};

/*
 * moe_packed_weight_bytes -- host only: size of one packed matrix set (see
 * moe_pack_weights) for E experts, hidden size d, intermediate size f, dtype.
 * Errors: MOE_EINVAL for NULL bytes, E < 1, d or f not positive multiples of
 * 8, bad dtype or kind; MOE_EUNSUPPORTED for E > MOE_MAX_EXPERTS.
 */
int moe_packed_weight_bytes(int E, int d, int f, int dtype, int kind, size_t *bytes);

/*
 * moe_pack_weights -- rearrange one set of expert matrices, once (at model
 * load), into the tile layout the grouped FFN streams: for each expert,
 * column group of 4 slices, K-step and slice, one contiguous 4 KB tile per
 * 64-column stream (gate/up: one stream of 64 columns per slice; down: two)
 * holding, for each of the 64 MFMA lanes, the 4 B-operand words of that step
 * in the order the lane consumes them (16-bit types: 8 consecutive K of one
 * column; fp32: 4 consecutive columns of one K-row). Bits are copied, nothing
 * is converted; positions past d or f hold zeros. The grouped GEMMs then read
 * each workgroup's K range of a column group as one contiguous run, with
 * 16-byte loads and no transposes: a reorganisation of [P3]'s resident expert
 * weights for the MI355X memory system, not a change of the arithmetic
 * (moe_forward_packed returns the same bits as moe_forward).
 * In:  w = W_gate or W_up [E][d][f] (kind MOE_W_GATE_UP) or W_down [E][f][d]
 *      (MOE_W_DOWN) of dtype, 16-byte aligned.
 * Out: packed [moe_packed_weight_bytes], 16-byte aligned; owned by the caller.
 * Errors: as moe_packed_weight_bytes, plus MOE_EINVAL for misaligned pointers,
 * packed_bytes too small, or one matrix of 2 GiB or more; MOE_EHIP on a failed
 * launch.
 */
int moe_pack_weights(const void *w, int dtype, int E, int d, int f, int kind, void *packed,
                     size_t packed_bytes, moe_stream_t stream);

/*
 * moe_expert_ffn_packed -- moe_expert_ffn with packed expert weights
 * (pw_gate, pw_up: moe_pack_weights(..., MOE_W_GATE_UP); pw_down:
 * MOE_W_DOWN). Same arguments, results (bit for bit) and errors otherwise.
 */
int moe_expert_ffn_packed(const void *xs, const void *pw_gate, const void *pw_up,
                          const void *pw_down, int dtype, int E, int d, int f, int tm,
                          const int32_t *eoff, const int32_t *stok, const float *sw,
                          const int32_t *meta, int64_t max_rows, void *h, float *y, void *scratch,
                          size_t scratch_bytes, moe_stream_t stream);

/*
 * moe_combine -- sum each token's expert outputs in the fixed top-k order
 * ([P3] s.3: the same per-token top-k summation order gives bit-identical
 * results): out[t][c] = +0.0f, then += y[pos[t*K+k]][c] for k = 0..K-1 in fp32,
 * skipping pos < 0 (and pos >= max_rows). One correct fp32 result exists for
 * this order, and this call produces it.
 * In:  y [max_rows][d] fp32, pos [T*K]. Out: out [T][d] fp32.
 * Errors: MOE_EINVAL for d % 8 != 0, T/K < 1, NULL/misaligned pointers;
 * MOE_EHIP on a failed launch.
 */
int moe_combine(const float *y, int64_t max_rows, const int32_t *pos, int T, int K, int d,
                float *out, moe_stream_t stream);

/*
 * moe_forward_workspace -- host only: bytes of the workspace moe_forward
 * carves its intermediates from (plan arrays, xs, h, y, scratch).
 */
int moe_forward_workspace(int T, int K, int E, int d, int f, int tm, int dtype, size_t *bytes);

/*
 * moe_forward -- one routed MoE layer: the results of moe_plan, moe_gather,
 * moe_expert_ffn and moe_combine in sequence on one stream, intermediates in
 * `workspace`. Fewer launches than calling them one by one: for T*K <= 32768
 * the plan is one kernel that also writes the FFN's work list; for T*K <= 64
 * with tm dividing 64 (and x below 2 GiB) that plan runs inside the gate/up
 * kernel, whose workgroups find their work items from the ids themselves (the
 * workspace's plan arrays get the same values); and when x is smaller than 2
 * GiB the gate/up kernel reads its rows from x through stok (the gather is
 * fused; the workspace's xs rows are then left unwritten).
 * For fp16 and bf16 layers the expert outputs y are kept in a compact format,
 * half the bytes of fp32 rows: each row is cut into blocks of 128 columns, a
 * block holds binary16 values s and one exponent e (int8) and stands for
 * s * 2^-e exactly; e puts the block's largest magnitude in [2^14, 2^15) (e =
 * 15 - k for a maximum m * 2^k, m in [1/2, 1), clamped to [-112, 100]; 0 for
 * an all-zero or infinite block) and s = y * 2^e rounded to binary16 (nearest
 * even), a relative error of at most 2^-12 per value near the block maximum.
 * The combine decodes each value exactly and sums in the same fixed order, so
 * the result is deterministic; it differs in rounding from the four calls
 * (whose y is fp32) but not from the same call again. In the workspace
 * (moe_forward_layout) the y region then holds the binary16 rows [max_rows][d]
 * followed by their exponents, block-major: [ceil(d/128)][max_rows]. fp32
 * layers keep fp32 y and equal the four calls bit for bit.
 * In:  x [T][d] (dtype), ids [T*K], w [T*K], expert weights as above.
 * Out: out [T][d] fp32.
 * Errors: the union of the four calls' errors.
 */
int moe_forward(const void *x, const int32_t *ids, const float *w, const void *w_gate,
                const void *w_up, const void *w_down, int dtype, int T, int K, int E, int d, int f,
                int tm, void *workspace, size_t ws_bytes, float *out, moe_stream_t stream);

/*
 * moe_forward_packed -- moe_forward with packed expert weights (see
 * moe_pack_weights); same workspace, results (bit for bit) and errors.
 */
int moe_forward_packed(const void *x, const int32_t *ids, const float *w, const void *pw_gate,
                       const void *pw_up, const void *pw_down, int dtype, int T, int K, int E,
                       int d, int f, int tm, void *workspace, size_t ws_bytes, float *out,
                       moe_stream_t stream);

/*
 * Expert weights in microscaled 4-bit floating point: 4.25 bits a weight with its
 * share of a scale, 17/64 of the 16-bit weights' bytes.
 *
 * Format: 32 weights that follow one another along the reduction (the input
 * index; the last block of a column may be shorter) share a scale 2^(s - 127), s a
 * byte, 255 meaning NaN; each weight is a 4-bit e2m1 code (sign, 2 exponent bits,
 * 1 fraction bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6) and stands for code * 2^(s - 127).
 * The packed layout is moe_pack_weights' for 16-bit types (expert, column group,
 * K-step, slice, stream), a tile of 32 x 64 weights being 1024 bytes of codes and
 * 64 of scales: byte 16 l + 4 c + i / 2 (low half for even i) holds the code of
 * K-value 8 (l / 16) + i, column 4 (l % 16) + c; byte 1024 + j the scale of column
 * j. Positions past d or f hold zeros.
 *
 * moe_mx4_weight_bytes -- host only: size of one packed matrix set. Errors: as
 * moe_packed_weight_bytes; MOE_EINVAL also for matrices of more than 2^30 weights.
 *
 * moe_mx4_quantize -- from w [E][d][f] (MOE_W_GATE_UP) or [E][f][d] (MOE_W_DOWN)
 * of dtype. With M a block's largest magnitude, s - 127 is the least e with M <=
 * 6 * 2^e, within [-110, 120] (-110 for M = 0), and codes are nearest, ties to the
 * even code: no value is clamped but magnitudes above 6 * 2^120. The relative error
 * is at most 1/5 for magnitudes of at least 2^e, the absolute one at most 2^(e-2)
 * below that. A block with a value that is not finite has s = 255. Weights that are
 * values of this format already, by scales from 2^-110 to 2^120 (whatever rule chose
 * them), are kept exactly.
 *
 * moe_mx4_dequantize -- the values that packed weights stand for, row-major, in
 * dtype (rounded to nearest even where the type does not hold them).
 *
 * moe_forward_mx4 -- moe_forward_packed with such weights (pw_gate, pw_up:
 * MOE_W_GATE_UP; pw_down: MOE_W_DOWN) and 16-bit activations: a weight is its
 * value in dtype, products are summed in fp32 and h is kept in dtype: the layer on
 * the dequantised weights, though sums may be cut along the reduction elsewhere than
 * moe_forward_packed cuts them. With MOE_BF16 the expert outputs are kept in the
 * compact format of moe_forward, with MOE_F16 in fp32 (that format's rounding is as
 * large as fp16's own).
 * In:  x, ids, w as moe_forward; dtype MOE_F16 or MOE_BF16.
 * Out: out [T][d] of out_dtype (dtype or MOE_F32; one rounding of the fp32 sum).
 * workspace: moe_forward_workspace() bytes.
 * Errors: those of moe_forward; MOE_EUNSUPPORTED for MOE_F32; MOE_EINVAL also for
 * another out_dtype and for an out that is another argument.
 */
int moe_mx4_weight_bytes(int E, int d, int f, int kind, size_t *bytes);
int moe_mx4_quantize(const void *w, int dtype, int E, int d, int f, int kind, void *packed,
                     size_t packed_bytes, moe_stream_t stream);
int moe_mx4_dequantize(const void *packed, size_t packed_bytes, int E, int d, int f, int kind,
                       void *w, int dtype, moe_stream_t stream);
int moe_forward_mx4(const void *x, const int32_t *ids, const float *w, const void *pw_gate,
                    const void *pw_up, const void *pw_down, int dtype, int T, int K, int E, int d,
                    int f, int tm, void *workspace, size_t ws_bytes, void *out, int out_dtype,
                    moe_stream_t stream);

/*
 * Expert weights in host memory, for layers whose experts do not all fit in
 * device memory ("#372 Prompt path: an MMQ group's experts gathered in one
 * launch, after one wait, released by one event", description: the routed
 * experts are streamed into a ring of device slots, ring entries the routing
 * does not use are skipped; "Add --moe-mode sweep-prefill: streamed expert
 * supply for CPU mul_mat_id", Mechanism: the used experts in ascending order).
 * The weights stay in host memory that is pinned and mapped for the device
 * (hipHostMalloc; torch pin_memory): w_gate_host, w_up_host [E][d][f] and
 * w_down_host [E][f][d], or the packed arrays of moe_pack_weights (packed = 1).
 * A device cache holds `slots` experts (each slot one expert's three
 * matrices) and the state of a ring over the slots.
 *
 * moe_host_cache_bytes -- host only: the cache's device bytes for `slots`
 * slots (0: the fewest that serve a call of T tokens, min(E, T*K)).
 * Errors: MOE_EINVAL / MOE_EUNSUPPORTED as moe_forward_workspace; MOE_EINVAL
 * also for packed other than 0 or 1 and for slots (other than 0) below
 * min(E, T*K) or above E.
 *
 * moe_host_cache_init -- mark every slot of a cache empty (one launch on
 * `stream`). Needed before a cache's first use, and again after the host
 * weights it has copied change. Errors: MOE_EINVAL for a small or unaligned
 * cache or bad sizes (1 <= slots <= E).
 *
 * moe_forward_host_weights -- moe_forward (packed = 0) or moe_forward_packed
 * (packed = 1) with the weights in host memory. After the plan, one launch
 * keeps the slot of every routed expert the cache already holds, gives every
 * other routed expert (ascending) the next slot of the ring that holds no
 * expert this call routes to (evicting the expert it held), and renumbers the
 * work list to slots; a second launch copies the newly placed experts'
 * matrices from host memory, the GPU reading it over the host link. The
 * grouped FFN then reads the cache. The call enqueues on the stream like
 * moe_forward and never waits for the GPU. Calls that share a cache must be
 * ordered (one stream).
 * In:  the host weights as above; slots as at moe_host_cache_init (>=
 *      min(E, T*K)); the rest as moe_forward.
 * cache: device, 256-byte aligned, >= moe_host_cache_bytes for `slots`, made
 *      by moe_host_cache_init with the same sizes; updated by the call.
 * Out: out [T][d] fp32, the same bits as moe_forward / moe_forward_packed on
 *      device copies of the same weights, whatever the cache held.
 * Errors: those of moe_forward; MOE_EINVAL also for a small or unaligned
 *      cache, slots below min(E, T*K), and weight pointers that are not
 *      pinned, device-mapped host memory (pageable memory is refused before
 *      any launch).
 */
int moe_host_cache_bytes(int T, int K, int E, int d, int f, int dtype, int packed, int slots,
                         size_t *bytes);
int moe_host_cache_init(void *cache, size_t cache_bytes, int E, int d, int f, int dtype,
                        int packed, int slots, moe_stream_t stream);
int moe_forward_host_weights(const void *x, const int32_t *ids, const float *w,
                             const void *w_gate_host, const void *w_up_host,
                             const void *w_down_host, int packed, int dtype, int T, int K, int E,
                             int d, int f, int tm, int slots, void *cache, size_t cache_bytes,
                             void *workspace, size_t ws_bytes, float *out, moe_stream_t stream);

/* Byte offsets of moe_forward's intermediates inside the workspace (host only),
 * so that a caller can inspect them after a call. */
typedef struct {
    size_t cnt, eoff, tiles, stok, sw, pos, boff, meta, plan_scratch, xs, h, y, ffn_scratch, total;
} moe_forward_layout_t;
int moe_forward_layout(int T, int K, int E, int d, int f, int tm, int dtype,
                       moe_forward_layout_t *out);

/* ---- per-kernel timing (HIP events recorded around each kernel) ---- */

enum moe_stage {
    MOE_STAGE_HIST = 0,
    MOE_STAGE_SCAN,
    MOE_STAGE_PLACE,
    MOE_STAGE_GATHER,
    MOE_STAGE_WORKLIST,
    MOE_STAGE_GATEUP,
    MOE_STAGE_DOWN,
    MOE_STAGE_COMBINE,
    MOE_STAGE_N
};

typedef struct moe_timer moe_timer_t;

/* Create a timer that can hold `capacity` recorded calls (host object; its
 * HIP events are created on the current device). Only the stages whose bit
 * (1 << stage) is set in stage_mask are timed, so that a caller timing one
 * kernel adds no event records around the others. */
int moe_timer_create(moe_timer_t **out, int capacity, unsigned stage_mask);
int moe_timer_destroy(moe_timer_t *timer);
/* Wait for the recorded events, add each stage's elapsed milliseconds into
 * total_ms[MOE_STAGE_N] and its launch count into launches[MOE_STAGE_N], then
 * forget the recorded calls. */
int moe_timer_read(moe_timer_t *timer, double *total_ms, int64_t *launches);

/* moe_forward with an event pair recorded around every kernel into `timer`
 * (NULL: identical to moe_forward). MOE_EINVAL when the timer is full. */
int moe_forward_timed(const void *x, const int32_t *ids, const float *w, const void *w_gate,
                      const void *w_up, const void *w_down, int dtype, int T, int K, int E, int d,
                      int f, int tm, void *workspace, size_t ws_bytes, float *out,
                      moe_stream_t stream, moe_timer_t *timer);

/* moe_forward_packed with an event pair recorded around every kernel into
 * `timer` (NULL: identical to moe_forward_packed). */
int moe_forward_packed_timed(const void *x, const int32_t *ids, const float *w,
                             const void *pw_gate, const void *pw_up, const void *pw_down,
                             int dtype, int T, int K, int E, int d, int f, int tm,
                             void *workspace, size_t ws_bytes, float *out, moe_stream_t stream,
                             moe_timer_t *timer);

/*
 * moe_forward_packed_noalloc -- for callers that cannot allocate device memory
 * (code under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc): moe_forward_packed with its workspace taken from a fixed buffer
 * inside this library instead of a caller argument. The caller still passes
 * the inputs and `out`, as for moe_forward_packed; results are the same bits.
 *  - The buffer is MOE_NOALLOC_WORKSPACE_BYTES of device memory per GPU,
 *    reserved when the library's code is loaded on that GPU and held until the
 *    process ends. It covers decode-sized batches (e.g. 4 tokens, hidden 2816,
 *    128 experts, top-8, intermediate 704 needs 22.7 MiB).
 *  - A request whose moe_forward_workspace() exceeds the buffer returns
 *    MOE_ENOSPACE before any HIP call.
 *  - The first call on each device looks up that device's buffer address
 *    (hipGetSymbolAddress); make that first call outside graph capture. Later
 *    calls allocate nothing, clear nothing with memset and never wait on the
 *    host, so they can be captured.
 *  - `stream` must belong to the current device (MOE_EINVAL otherwise); NULL
 *    is the current device's default stream.
 *  - All calls on one GPU share that GPU's buffer, which keeps the last call's
 *    contents (nothing in it needs to start at zero): calls that can overlap on
 *    one GPU (different streams or threads without ordering between them) race
 *    on it and must be serialised by the caller.
 * Errors: those of moe_forward_packed, plus MOE_ENOSPACE, and
 * MOE_EUNSUPPORTED for a device ordinal of 64 or more.
 */
#define MOE_NOALLOC_WORKSPACE_BYTES (64u * 1024u * 1024u)
int moe_forward_packed_noalloc(const void *x, const int32_t *ids, const float *w,
                               const void *pw_gate, const void *pw_up, const void *pw_down,
                               int dtype, int T, int K, int E, int d, int f, int tm, float *out,
                               moe_stream_t stream);

/*
 * ---- Dense operators beside the routed layer ----
 *
 * The router's own product and the dense (shared) expert that every token
 * takes, with the gradients that train them: a matrix product with bias,
 * activation and residual; the router's balance losses with the gradient of
 * its logits; an activation whose inputs are kept for the backward pass in 8
 * bits. Conventions as above (device pointers, the caller's stream and
 * workspace, no host wait, argument checks before any HIP call); in addition
 *  - matrices are row-major with a row stride in elements (ld >= row length,
 *    at most 2^20); every size and stride from 1 on is served, rows that are not
 *    whole 16-byte chunks at the price of a copy in the workspace. The first
 *    element of a matrix, bias or bias gradient lies at a 16-byte boundary
 *    (MOE_EINVAL otherwise: a slice that starts elsewhere is to be copied);
 *  - products are accumulated and epilogues computed in fp32 and rounded once
 *    to the result's type;
 *  - a workspace is needed only where its size is not 0 (then 256-byte
 *    aligned); it starts with any contents, and calls that may overlap need
 *    one each;
 *  - an output, or a workspace that is needed, overlaps no other argument, but
 *    where a call names one that an output may be: then it is that array itself,
 *    from its first element and with its stride. An output whose address is
 *    another argument's is refused otherwise (MOE_EINVAL), but where a call says
 *    that it does not look; ranges that overlap from different addresses, and a
 *    workspace that is an input, are the caller's to avoid;
 *  - results do not depend on timing: the same call gives the same bits.
 */

/* Activations: relu max(z, 0); silu z / (1 + exp(-z)); gelu z Phi(z), Phi the
 * normal distribution function (erf form). NaN gives NaN. */
enum moe_act { MOE_ACT_NONE = 0, MOE_ACT_RELU = 1, MOE_ACT_SILU = 2, MOE_ACT_GELU = 3 };

/*
 * moe_linear -- out = act(x W + bias) + residual: router logits (fp32 out,
 * the input of moe_route_topk), or a projection of a dense expert, whose last
 * product adds the routed layer's output (residual = moe_forward's out, fp32).
 * In:  x [T][d] stride ldx, w [d][n] stride ldw (input index, then output
 *      index, as the expert weights), bias [n] or NULL: all of dtype;
 *      residual [T][n] stride ldr of residual_dtype (dtype or MOE_F32) or
 *      NULL. It may be out itself (same type and stride).
 * Out: out [T][n] stride ldo of out_dtype (dtype or MOE_F32). Only columns
 *      [0, n) of its rows are written.
 * workspace: moe_linear_workspace() bytes (padded copies of operands whose
 *      stride or row length is not a multiple of 16 bytes; fp32 partial sums
 *      when few tiles are cut along d).
 * moe_linear_shape -- host only: the tile (64, 128 or 256 rows and columns of a
 *      workgroup) and the ranges of K that a product of M x N outputs over K is
 *      computed in: the forward product is T x n over d, dx is T x d over n, dw
 *      d x n over T. Errors: MOE_EINVAL for a size < 1, a bad dtype, NULL.
 * Errors: MOE_EINVAL for T, d or n < 1, a stride below the row length or above
 *      2^20, a bad dtype or act, NULL or misaligned pointers, an out that is
 *      another argument, a small workspace, a product of more than 2^23 tiles
 *      (moe_linear_shape); MOE_EHIP on a failed launch.
 */
int moe_linear_shape(int M, int N, int K, int dtype, int *tile, int *split);
int moe_linear_workspace(int T, int d, int n, int64_t ldx, int64_t ldw, int dtype, size_t *bytes);
int moe_linear(const void *x, int64_t ldx, const void *w, int64_t ldw, const void *bias,
               const void *residual, int64_t ldr, int residual_dtype, int dtype, int act, int T,
               int d, int n, void *workspace, size_t ws_bytes, void *out, int64_t ldo,
               int out_dtype, moe_stream_t stream);

/*
 * moe_linear_backward -- the gradients of z = x W + bias from dz [T][n] (of
 * dtype, stride lddz):
 *   dx = dz W^T [T][d] (dtype),  dw = x^T dz [d][n],  db = sum over t of dz [n]
 * (dw and db of grad_dtype: dtype or MOE_F32). A NULL dx, dw or db is not
 * computed, and an operand that only it reads (w for dx, x for dw) may be
 * NULL; one at least is asked for. With an activation behind z, dz is what
 * moe_act_backward gives; the residual's gradient is the output's own.
 * grads (workspace size): the MOE_GRAD_ bits of what is asked for.
 * Errors: as moe_linear.
 */
enum moe_grad { MOE_GRAD_X = 1, MOE_GRAD_W = 2, MOE_GRAD_BIAS = 4 };
int moe_linear_backward_workspace(int T, int d, int n, int64_t ldx, int64_t ldw, int64_t lddz,
                                  int dtype, int grads, size_t *bytes);
int moe_linear_backward(const void *x, int64_t ldx, const void *w, int64_t ldw, const void *dz,
                        int64_t lddz, int dtype, int T, int d, int n, void *workspace,
                        size_t ws_bytes, void *dx, int64_t lddx, void *dw, int64_t lddw, void *db,
                        int grad_dtype, moe_stream_t stream);

/*
 * moe_balance_loss -- the router's auxiliary losses over a batch of T tokens.
 * p_t = softmax of token t's logits; a token is valid if one of its ids is in
 * [0, E) (padding has ids -1); n_t valid tokens, c_e entries routed to expert
 * e, n_a their sum:
 *   prob[e] = (1 / n_t) sum over valid t of p_te
 *   loss[0] = E sum_e (c_e / n_a) prob[e]               (balance)
 *   loss[1] = (1 / n_t) sum over valid t of (log sum_e exp(logits_te))^2   (z)
 * NaN and -inf logits are absent experts (p = 0); a row of only such logits
 * adds nothing to prob and the z loss. +inf gives NaN. With no valid token
 * both losses and prob are 0.
 * In:  logits [T][E] fp32, ids [T*K] (moe_route_topk's).
 * Out: cnt [E+2] int32: c_e, then n_t at cnt[E] and n_a at cnt[E+1];
 *      prob [E] fp32; loss [2] fp32.
 * Errors: as moe_route_topk; MOE_EINVAL also for a small workspace, and for an
 *      output that is another argument or the workspace (not looked at where
 *      logits and ids are one address).
 */
int moe_balance_workspace(int T, int E, int K, size_t *bytes);
int moe_balance_loss(const float *logits, const int32_t *ids, int T, int E, int K, void *workspace,
                     size_t ws_bytes, int32_t *cnt, float *prob, float *loss, moe_stream_t stream);

/*
 * moe_route_backward -- the gradient of the router logits, of both the losses
 * above and the renormalised weights of moe_route_topk, in one pass:
 *   dlogits_te = p_te (dloss[0] (E / n_t) (c_e / n_a - sum_j c_j / n_a p_tj)
 *                      + dloss[1] (2 / n_t) lse_t)              for valid t
 *                + sum over t's entries k with id e: w_k (dw_k - sum_j w_j dw_j)
 * (the sum over j: t's entries with a valid id; 0 elsewhere).
 * In:  logits, ids, as above; w [T*K] fp32 (moe_route_topk's weights) and dw
 *      [T*K] fp32 their gradient, or dw NULL (w is then not read): no second
 *      term; cnt [E+2] from moe_balance_loss; dloss [2] fp32, the gradient of
 *      the training loss by loss[0] and loss[1], on the device, or NULL: no
 *      first term. Not both NULL. Values of w and dw at invalid ids are not used.
 * Out: dlogits [T][E] of dtype (MOE_F32, or the type of the router's product,
 *      whose moe_linear_backward takes it as dz). Every element is written.
 * Errors: as moe_route_topk; MOE_EINVAL also for a dlogits that is one of the
 *      arrays that are read.
 */
int moe_route_backward(const float *logits, const int32_t *ids, const float *w, const float *dw,
                       const int32_t *cnt, const float *dloss, int T, int E, int K, void *dlogits,
                       int dtype, moe_stream_t stream);

/*
 * moe_act_forward -- h = act(g) * u (gated: SwiGLU with MOE_ACT_SILU), or h =
 * act(g) with u NULL; and, unless g8 is NULL, the checkpoint its backward
 * starts from: 8 bits an element instead of g and u themselves.
 * Checkpoint of a matrix z [T][f]: rows are cut into blocks of
 * MOE_ACT8_BLOCK columns (the last may be shorter); a block has one scale byte
 * s and each element one e4m3 code (4 exponent bits, bias 7, 3 fraction bits,
 * largest 448, 0x7f NaN) and stands for code * 2^(s - 127) exactly. With M the
 * block's largest finite magnitude, s - 127 is the least e with M <= 448 * 2^e,
 * within [-110, 120] (-110 for M = 0); the code is z * 2^-e rounded once
 * (nearest, ties to even). Elements that are not finite have code 0x7f. The
 * relative error is at most 2^-4 for magnitudes of at least 2^(e-6), and below
 * that the absolute error is at most 2^(e-10).
 * In:  g, u [T][f] of dtype, strides ldg, ldu. act: not MOE_ACT_NONE.
 * Out: h [T][f] of dtype, stride ldh (may be g or u itself); g8 [T][f] codes and gs [T][ceil(f / 32)]
 *      scales, contiguous (g8 16-byte aligned); u8 and us likewise, given
 *      exactly when g8 and u are.
 * Errors: MOE_EINVAL for T or f < 1, a bad stride, dtype or act, NULL or
 *      misaligned pointers, a checkpoint given in part, codes or scales that are
 *      another argument; MOE_EHIP on a failed launch.
 *
 * moe_act_backward -- from that checkpoint (g, u: the values it stands for; in a
 * block of the largest scale, 2^120, they are read times 1 - 2^-24, so that 2^128,
 * which magnitudes of 248 * 2^120 and more are rounded to, is fp32's largest
 * value) and dh [T][f] of dtype:
 *   dg = dh * u * act'(g),  du = dh * act(g),  h = act(g) * u
 * (u8, us and du NULL: dg = dh * act'(g), h = act(g)). relu'(0) = 0.
 * h may be NULL; it is the operand x of the following product's dw. One of dg,
 * du and h may be dh itself. Errors: as above; MOE_EINVAL also for an output
 * that is one of the codes or scales (not looked at where it is dh itself).
 */
#define MOE_ACT8_BLOCK 32
int moe_act_forward(const void *g, int64_t ldg, const void *u, int64_t ldu, int dtype, int act,
                    int T, int f, void *h, int64_t ldh, uint8_t *g8, uint8_t *gs, uint8_t *u8,
                    uint8_t *us, moe_stream_t stream);
int moe_act_backward(const uint8_t *g8, const uint8_t *gs, const uint8_t *u8, const uint8_t *us,
                     const void *dh, int64_t lddh, int dtype, int act, int T, int f, void *dg,
                     int64_t lddg, void *du, int64_t lddu, void *h, int64_t ldh,
                     moe_stream_t stream);

/*
 * ---- Operators around the routed layer's block ----
 *
 * The router's other forms and the norms that a block stands between. Conventions
 * as for the dense operators.
 *
 * moe_route_scored -- routing by scores. Per token, over the experts that are
 * there (NaN and -inf logits mark an absent expert):
 *   s_e = softmax of the logits, or 1 / (1 + exp(-l_e))
 *   c_e = s_e + bias_e                          (bias NULL: c_e = s_e)
 * An expert whose bias is NaN or -inf is never picked and adds to no group.
 * The experts form `groups` groups of E / groups neighbours; a group is worth the
 * sum of its group_top largest c (of fewer if fewer are there), and the `keep`
 * groups of the largest worth stay (groups = keep = 1: no groups). Of their
 * experts the K with the largest c are picked, in descending order, and
 *   w_k = scale s_k / (sum over the picks of s_j)    (renorm != 0)
 *   w_k = scale s_k                                  (renorm == 0)
 * Equal c, and groups of equal worth, go to the lower index. Choices are those of c
 * and worth in 64-bit arithmetic (without a bias experts go by their logits, of which
 * s is a rising function); weights are within a few roundings of fp32.
 * Where fewer than K experts are there, the remaining picks are id -1 with weight
 * 0. A softmax with +inf logits is shared evenly among them.
 * In:  logits [T][E] fp32, bias [E] fp32 or NULL. score: enum moe_score.
 * Out: ids [T*K] int32, w [T*K] fp32 (the inputs of moe_plan / moe_forward).
 * Errors: as moe_route_topk; MOE_EINVAL also for an unknown score, groups that do
 *      not divide E, keep outside [1, groups], group_top outside [1, E / groups],
 *      K above keep E / groups, a scale that is not finite, an output that is
 *      another argument; MOE_EUNSUPPORTED for more than MOE_SCORE_MAX_GROUPS groups
 *      or group_top above 2.
 *
 * moe_route_scored_backward -- the gradient of the logits from dw, that of w, for
 * the choice made (ids, as moe_route_scored gave them). With u_k = scale dw_k over
 * the entries with a valid id (others have no part; an id may come twice):
 *   renorm:  g_k = (s_k / S) (u_k - sum_j (s_j / S) u_j),  S = sum_j s_j
 *   else:    g_k = s_k u_k
 *   sigmoid:               dl_e = sum over k of e: g_k (1 - s_e)
 *   softmax, renorm:       dl_e = sum over k of e: g_k
 *   softmax, not renorm:   dl_e = (sum over k of e: g_k) - s_e sum_j g_j
 * (the softmax over the experts that are there; dl_e = 0 for those that are not).
 * In:  logits [T][E] fp32, ids [T*K], dw [T*K] fp32; add [T][E] of dtype or NULL:
 *      a gradient that is added (the balance loss's, say). It may be dlogits.
 * Out: dlogits [T][E] of dtype. Every element is written.
 * Errors: as moe_route_backward; MOE_EINVAL also for an unknown score and a scale
 *      that is not finite.
 */
enum moe_score { MOE_SCORE_SOFTMAX = 0, MOE_SCORE_SIGMOID = 1 };
#define MOE_SCORE_MAX_GROUPS 64
int moe_route_scored(const float *logits, const float *bias, int score, int T, int E, int K,
                     int groups, int keep, int group_top, int renorm, float scale, int32_t *ids,
                     float *w, moe_stream_t stream);
int moe_route_scored_backward(const float *logits, const int32_t *ids, const float *dw,
                              const void *add, int score, int T, int E, int K, int renorm,
                              float scale, void *dlogits, int dtype, moe_stream_t stream);

/*
 * moe_norm -- the norms after and before a block, with its gate, scale and
 * residual, in one pass (rms(v) = sqrt(mean of v^2 + eps), per row):
 *   n = y / rms(y) * w_post      (w_post NULL: n = y)
 *   z = r + alpha * gate * n     (gate NULL: 1; y NULL: z = r)
 *   h = z / rms(z) * w_pre       (w_pre NULL: no h)
 * In:  r [T][d] of r_dtype, the residual stream; y [T][d] of y_dtype (each dtype or
 *      MOE_F32) or NULL, the block's output (the routed layer's, say); w_post and
 *      w_pre [d] and the gate of dtype. gate_kind: enum moe_gate -- one value per
 *      token [T], per channel [d], or per element [T][d] (stride ldgate).
 *      y or w_pre is given; w_post and gate only with y.
 * Out: z [T][d] of r_dtype (given exactly when y is; it may be r itself); h [T][d]
 *      of dtype, the next block's input (given exactly when w_pre is; it may be y
 *      itself); stats [T][2] fp32 or NULL: 1 / rms(y) and 1 / rms(z), 0 where there
 *      is no such norm (what moe_norm_backward takes). h comes from z before its
 *      rounding.
 * Sums are in fp32; rows whose squares overflow it are summed scaled.
 * Errors: MOE_EINVAL for T or d < 1, a bad stride, dtype or gate kind, eps below
 *      2^-100 or not finite, alpha not finite, NULL or misaligned pointers, arguments that
 *      do not go together, an output that is another argument; MOE_EUNSUPPORTED for
 *      d > MOE_NORM_MAX_D; MOE_EHIP on a failed launch.
 *
 * moe_norm_backward -- from dz [T][d] of r_dtype (the gradient that reaches z from
 * behind, or NULL) and dh [T][d] of dtype (given exactly when w_pre is). With
 * zn = z * stats[1], yn = y * stats[0]:
 *   dr = dz + stats[1] (dh w_pre - zn mean(dh w_pre zn))       w_pre: the mean over d
 *   dw_pre = sum over t of dh zn
 *   dgate = alpha dr n, summed over the elements that share a gate's value
 *   q = alpha gate dr;  dw_post = sum over t of q yn
 *   dy = stats[0] (q w_post - yn mean(q w_post yn))            (w_post NULL: dy = q)
 * dr here is in fp32, before its rounding. z: the forward's (r without y).
 * Out: dr [T][d] of r_dtype (may be dz itself); dy [T][d] of y_dtype; dgate in the
 *      gate's shape, of dtype -- but per channel of grad_dtype; dw_post, dw_pre [d]
 *      of grad_dtype (dtype or MOE_F32). dy, dgate, dw_post and dw_pre may each be
 *      NULL: not computed.
 * workspace: moe_norm_backward_workspace() bytes (partial column sums).
 * Errors: as moe_norm.
 */
enum moe_gate {
    MOE_GATE_NONE = 0,
    MOE_GATE_TOKEN = 1,
    MOE_GATE_CHANNEL = 2,
    MOE_GATE_FULL = 3
};
#define MOE_NORM_MAX_D 32768
int moe_norm(const void *r, int64_t ldr, int r_dtype, const void *y, int64_t ldy, int y_dtype,
             const void *w_post, const void *gate, int64_t ldgate, int gate_kind,
             const void *w_pre, int dtype, int T, int d, float alpha, float eps, void *z,
             int64_t ldz, void *h, int64_t ldh, float *stats, moe_stream_t stream);
int moe_norm_backward_workspace(int T, int d, size_t *bytes);
int moe_norm_backward(const void *dz, int64_t lddz, const void *dh, int64_t lddh, const void *z,
                      int64_t ldz, int r_dtype, const void *y, int64_t ldy, int y_dtype,
                      const void *w_post, const void *gate, int64_t ldgate, int gate_kind,
                      const void *w_pre, const float *stats, int dtype, int T, int d, float alpha,
                      void *workspace, size_t ws_bytes, void *dr, int64_t lddr, void *dy,
                      int64_t lddy, void *dgate, int64_t lddgate, void *dw_post, void *dw_pre,
                      int grad_dtype, moe_stream_t stream);

/* Static description of a status code. */
const char *moe_status_str(int status);

#ifdef __cplusplus
}
#endif

#endif /* MOE_ROUTED_H */
