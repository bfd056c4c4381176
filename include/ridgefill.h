/*
 * ridgefill.h -- C ABI of the RidgeFill upper-layer KV fill, its one-pass calibration
 * and its closed-form ridge solve, for AMD Instinct MI355X (gfx950).
 *
 * Method source: the English RidgeFill review (jaehun.me, "paper-2611-09709v1", English
 * edition).  Each entry point names the section it implements.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - Pointers marked "device" point to GPU memory the caller allocated; pointers
 *    marked "host" point to CPU memory.  The library allocates no device memory,
 *    keeps no device state between calls and creates no streams (the streamed fill
 *    creates five HIP events per host thread and device on first use and reuses them;
 *    ridgefill_fill_noalloc works in a fixed array of RIDGEFILL_NOALLOC_SCRATCH_BYTES
 *    that is part of the library's device code, one per device, whose contents the
 *    next such call on that device overwrites).
 *    Every buffer it needs beyond inputs and outputs is a caller-owned workspace whose
 *    size a *_workspace_bytes / *_state_bytes query returns.
 *  - bf16 tensors are passed as uint16_t bit patterns (bfloat16, round-to-nearest-
 *    even where the library produces them).  All matrices are row-major.
 *  - `stream` is a hipStream_t (NULL = the null stream).  Device work is enqueued
 *    on it and the call returns without waiting, except where stated.  ridgefill_fill
 *    with resident maps (plain or folded) and the cache calls (ridgefill_rope to
 *    ridgefill_evict_rows, ridgefill_norm_rope to ridgefill_cache_attention) enqueue kernels only (the status word is cleared by a kernel,
 *    not a memset), so they can be captured into a HIP graph and replayed; workspaces,
 *    index lists and pools must then stay at their addresses.
 *  - Errors found on the host (null pointers, shapes, sizes, workspace too small,
 *    invalid parameters) return a non-zero rf_status before anything is enqueued;
 *    ridgefill_last_error() then gives a description.  A failed launch returns
 *    RF_E_HIP.  Errors that only the device can see (an index out of range, a
 *    non-increasing index list, a non-positive pivot) set bits in the status word
 *    at the start of the workspace; ridgefill_read_status() returns them.  Rows whose
 *    index is invalid are skipped: the library never writes outside the rows it was
 *    given and never aborts.
 *  - Calls that share a workspace or state buffer must not run concurrently.
 */
#ifndef RIDGEFILL_H
#define RIDGEFILL_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum rf_status {
  RF_OK = 0,
  RF_E_INVALID = 1,      /* null pointer or invalid scalar parameter            */
  RF_E_SHAPE = 2,        /* unsupported or inconsistent sizes                   */
  RF_E_WORKSPACE = 3,    /* workspace / state buffer too small or mismatched    */
  RF_E_HIP = 4,          /* a HIP runtime call or kernel launch failed          */
  RF_E_NOT_SPD = 5,      /* device: X^T X + alpha I was not positive definite   */
  RF_E_ROWS = 6,         /* device: an index was out of range or not increasing */
  RF_E_UNSUPPORTED = 7   /* the requested variant is not built                  */
} rf_status;

/* Model shape shared by all layers of one fill call. */
typedef struct rf_shape {
  int32_t d;            /* hidden size of the upper layers (the map's output width);
                           multiple of 256                                             */
  int32_t n_kv_heads;   /* KV heads; n_kv_heads * head_dim must be a multiple of 128 */
  int32_t head_dim;     /* 64 or 128                                                 */
  float rms_eps;        /* RMSNorm epsilon (inside the square root), >= 0; also the
                           epsilon of the per-head key norm when one is given        */
  double rope_theta;    /* RoPE base, > 1                                            */
  int32_t d_in;         /* width of x_S, the map's input (section "Ridge map ...", map
                           size paragraph: a map's input width may differ from its
                           output width).  0 means d.  Multiple of 64.                */
  int32_t reserved;     /* must be 0                                                  */
} rf_shape;

/* One upper layer l >= S.  Every pointer is a device pointer owned by the caller.   */
typedef struct rf_layer {
  const uint16_t* A;       /* bf16 [d][d_in]: x_hat = A x_S + b (A[out][in]); NULL when
                              the map is given in int8 (A_q)                            */
  const float* b;          /* fp32 [d]                                                 */
  const uint16_t* norm_w;  /* bf16 [d]: the layer's RMSNorm weight                     */
  const uint16_t* W_K;     /* bf16 [n_kv_heads*head_dim][d]: key projection, no bias   */
  const uint16_t* W_V;     /* bf16 [n_kv_heads*head_dim][d]: value projection, no bias */
  uint16_t* k_pages;       /* bf16 [num_pages][page_size][n_kv_heads][head_dim]        */
  uint16_t* v_pages;       /* bf16 [num_pages][page_size][n_kv_heads][head_dim]        */
  /* Optional parts (NULL = absent). */
  const uint16_t* k_norm_w; /* bf16 [head_dim]: per-head key RMSNorm (Qwen-style layers;
                               section "Hybrid layers and two corrections": the Qwen
                               models apply a norm to the keys), applied to each key head after W_K and
                               before RoPE                                               */
  const float* v_scale;     /* fp32 [n_kv_heads]: value-rescale factors (same section,
                               value rescale); head h of every filled value is
                               multiplied by v_scale[h].  ridgefill_value_scale computes
                               them.                                                    */
  const int8_t* A_q;        /* int8 [d][d_in] with A_scale: the map is A_q[o][i] *
                               A_scale[o] (section "Ridge map ...", map size paragraph:
                               int8 maps).  Exactly one of A and A_q is set.             */
  const float* A_scale;     /* fp32 [d]: per-output-row scale of A_q                    */
  const void* folded;       /* buffer of ridgefill_fold_bytes(shape) bytes made by
                               ridgefill_fold_maps, 256-byte aligned: the layer's folded
                               form (device memory; host memory, ideally page-locked, for
                               ridgefill_fill_streamed).  When set, the fill reads it
                               instead of A, A_q, A_scale, b, norm_w, W_K and W_V (which
                               may then be NULL).                                          */
} rf_layer;

/* Paged KV layout of one prompt, shared by every layer's k_pages / v_pages. */
typedef struct rf_paged_kv {
  const int32_t* block_table;   /* device int32 [n_logical]: logical page -> physical */
  int64_t n_logical;            /* entries in block_table (>= ceil(N / page_size))    */
  int32_t page_size;            /* rows per page, >= 1                                */
  int32_t num_pages;            /* physical pages in each k_pages / v_pages pool      */
} rf_paged_kv;

/* ------------------------------------------------------------------------------
 * Row partition.  Section "Method: ..." -> "Two numbers set the skip range": the last
 * T rows are the tail; the N - T rows before them are the prefix, whose rows are each
 * computed exactly or filled from the maps.  Host-only, integer, no GPU.
 *
 *   exact_mask  host uint8 [N - T]: nonzero marks an exact row (may be NULL = none)
 *   filled_idx  host int32 [N - T] out: the filled rows in ascending order
 *   n_filled    host out: their count (N - T - number of exact rows)
 * Returns RF_E_SHAPE unless 0 <= T <= N and N - T fits in int32.
 * ------------------------------------------------------------------------------ */
rf_status ridgefill_partition(int64_t N, int64_t T, const uint8_t* exact_mask,
                              int32_t* filled_idx, int64_t* n_filled);

/* ------------------------------------------------------------------------------
 * Exact-row selection from scores, on the device.  Section "Which rows to compute
 * exactly", attention selection: the prefix rows that receive the most attention are
 * computed exactly (10% of them in the reference study's "+rows" arm).  Given one score
 * per prefix row, the k rows with the largest score, ties broken toward the lower row
 * index, are the exact rows; the other P - k rows, in ascending order, are written to
 * filled_idx, ready for ridgefill_fill with n_filled = P - k.
 *
 *   scores      device fp32 [P]; -0.0 and +0.0 tie; a NaN score ranks lowest and sets
 *               RF_E_INVALID in the device status (ridgefill_read_status(ws))
 *   k           0 <= k <= P
 *   exact_mask  device uint8 [P] out (1 = exact), or NULL
 *   filled_idx  device int32 [P - k] out
 *   ws          device workspace >= ridgefill_select_workspace_bytes(P); its first 256
 *               bytes hold the status
 * Integer and order decisions only: the result is exact and deterministic.
 * ------------------------------------------------------------------------------ */
size_t ridgefill_select_workspace_bytes(int64_t P);
rf_status ridgefill_select_rows(const float* scores, int64_t P, int64_t k, uint8_t* exact_mask,
                                int32_t* filled_idx, void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------------
 * Fill.  Section "Ridge map: predict the input, and the original projection runs
 * unchanged" (prediction equation; the paragraph on feeding the predicted input to the
 * layer's norm and K/V projections; Fig. 2):
 * for every filled row t and every given upper layer l,
 *     x_hat = A_l x_S[t] + b_l          (A_l = A_q,l * A_scale,l for an int8 map)
 *     h     = x_hat / sqrt(mean(x_hat^2) + eps) * norm_w_l
 *     k     = W_K,l h,  then per head k / sqrt(mean(k^2) + eps) * k_norm_w_l if given
 *     k     = RoPE_t(k)   (pairs (j, j + head_dim/2), angle t * theta^(-2j/head_dim))
 *     v     = W_V,l h,  times v_scale_l[head] if given
 * and k, v are written to row t of layer l's paged cache (page block_table[t /
 * page_size], slot t % page_size).  Nothing else in the caches is touched; with
 * n_filled = 0 or n_layers = 0 only the status word is cleared (if ws is given).  Layers
 * are independent, so a caller may also split them over several calls.
 *
 *   x_S         device bf16 [N][x_stride]: split-layer states of all prompt rows
 *               (x_stride >= d_in); the prefix rows must span at most 4 GiB
 *               ((N - T) x x_stride x 2 bytes), and x_stride is a multiple of 8
 *   filled_idx  device int32 [n_filled]: filled rows, strictly increasing, each
 *               < N - T (the tail never receives a filled entry).  Violations set
 *               RF_E_ROWS in the device status; out-of-range rows are skipped.
 *   layers      host array [n_layers] of device-pointer descriptors
 *   ws          device workspace of ws_bytes >= ridgefill_fill_workspace_bytes(shape,
 *               n_filled, 1); a larger workspace (up to the value for n_layers) lets
 *               more layers share one launch.  Its first 256 bytes hold the status.
 * Computation: bf16 inputs, fp32 accumulation, x_hat and the RMS in fp32, one bf16
 * rounding of x_hat * norm_w, one bf16 rounding of the stored k and v.  An int8 map's
 * codes are read by the map GEMM as they are and turned into bf16 numbers between LDS and
 * the matrix cores (exactly: |q| <= 127), and its row scale is applied to the fp32
 * product, so it adds no rounding of its own.  All
 * layers of one call must agree on which optional parts they use (int8 or bf16 map,
 * key norm); v_scale may be set per layer.
 * ------------------------------------------------------------------------------ */
size_t ridgefill_fill_workspace_bytes(const rf_shape* shape, int64_t n_filled,
                                      int32_t n_layers);
rf_status ridgefill_fill(const rf_shape* shape, const uint16_t* x_S, int64_t N, int64_t T,
                         int64_t x_stride, const int32_t* filled_idx, int64_t n_filled,
                         const rf_layer* layers, int32_t n_layers, const rf_paged_kv* kv,
                         void* ws, size_t ws_bytes, void* stream);

/* Map variants for the workspace query: RF_MAPS_INT8 when the layers carry A_q/A_scale
 * (the same workspace as for bf16 maps), RF_MAPS_STREAMED for
 * ridgefill_fill_streamed (two landing slots per layer), RF_MAPS_FOLDED when the layers
 * carry folded forms (no predicted-input buffer: a few MB per layer).  Returns 0 on
 * invalid input.
 * ridgefill_fill_workspace_bytes(...) is ridgefill_fill_workspace_bytes_ex(..., 0). */
#define RF_MAPS_INT8 1
#define RF_MAPS_STREAMED 2
#define RF_MAPS_FOLDED 4
size_t ridgefill_fill_workspace_bytes_ex(const rf_shape* shape, int64_t n_filled,
                                         int32_t n_layers, int32_t map_flags);

/* ------------------------------------------------------------------------------
 * Fill with host-resident maps.  Section "Ridge map ...", map size paragraph: maps can
 * stay in GPU memory or be streamed from host memory layer by layer.  Same
 * computation and arguments as ridgefill_fill, except that every layer's A (or A_q), or
 * for folded layers its whole folded buffer, is a HOST pointer, ideally page-locked
 * (hipHostMalloc) so that the copies run asynchronously.  Layers are processed in groups
 * sized by the workspace (ridgefill_fill_workspace_bytes_ex with RF_MAPS_STREAMED, plus
 * RF_MAPS_INT8 for int8 maps or RF_MAPS_FOLDED for folded layers); group g's maps (or
 * folded buffers) are copied on `copy_stream` into landing slot g % 2 while group g - 1
 * computes on `stream`.  Of a folded buffer only what the fill reads is copied: P, c, r1,
 * g, kappa, and R1 from each 256-row block's diagonal block rightwards (the zeros below the
 * diagonal blocks, about half of R, are not).  copy_stream must be a different stream; both must stay
 * valid until the work completes.  The first copy of a call waits for the work already
 * enqueued on `stream`, so back-to-back calls on one workspace are ordered.  The results
 * are bit-identical to ridgefill_fill's.
 * ------------------------------------------------------------------------------ */
rf_status ridgefill_fill_streamed(const rf_shape* shape, const uint16_t* x_S, int64_t N, int64_t T,
                                  int64_t x_stride, const int32_t* filled_idx, int64_t n_filled,
                                  const rf_layer* layers, int32_t n_layers, const rf_paged_kv* kv,
                                  void* ws, size_t ws_bytes, void* stream, void* copy_stream);

/* ------------------------------------------------------------------------------
 * For callers that cannot allocate device memory (code under HIP graph capture, serving
 * loops that must not call hipMalloc): the same computation and arguments as
 * ridgefill_fill with resident maps (plain bf16, int8 or folded layers), without a
 * workspace argument.  The library's own scratch array serves as the workspace:
 * RIDGEFILL_NOALLOC_SCRATCH_BYTES of device memory per device, part of the library's code
 * object (allocated when it is loaded on that device, held until the process ends).  The
 * call allocates nothing; layers are processed in groups as large as the scratch holds.
 *   status   device pointer to one uint32 (4-byte aligned) that receives the device status
 *            word of the call (cleared first); read it with ridgefill_read_status(status).
 * Returns RF_E_WORKSPACE, before anything is enqueued, when one layer's share of the
 * workspace (ridgefill_fill_workspace_bytes_ex(shape, n_filled, 1, flags)) exceeds the
 * scratch.  All calls on one device share its scratch, which keeps the last call's
 * contents: calls that overlap on one device (two streams, two threads) race and must be
 * ordered by the caller.  Nothing in the scratch needs to start at zero.
 * ------------------------------------------------------------------------------ */
#define RIDGEFILL_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)
rf_status ridgefill_fill_noalloc(const rf_shape* shape, const uint16_t* x_S, int64_t N, int64_t T,
                                 int64_t x_stride, const int32_t* filled_idx, int64_t n_filled,
                                 const rf_layer* layers, int32_t n_layers, const rf_paged_kv* kv,
                                 uint32_t* status, void* stream);

/* ------------------------------------------------------------------------------
 * Folded layers.  Section "Ridge map: predict the input, and the original projection runs
 * unchanged": after x_hat = A x_S + b the layer's RMSNorm weight w and its projections
 * W_K, W_V are linear, so they can be multiplied into the map once per layer; the only
 * non-linear quantity left is |x_hat|^2, which equals |R x_S + r|^2 + kappa with R the
 * upper-triangular factor of A^T A (R^T R = A^T A, positive diagonal),
 * r = R^-T A^T b and kappa = |b|^2 - |r|^2.  The fill of a folded layer then computes
 *     k, v = (P x_S + c) / sqrt((|R x_S + r|^2 + kappa) / d + eps)
 * with P = [W_K; W_V] diag(w) A and c = [W_K; W_V] (w * b), followed by the same key norm,
 * RoPE, value rescale and paged store as the plain fill.  Same result up to rounding;
 * R x_S needs half the multiply-adds of A x_S, and x_hat is never stored.
 *
 * A^T A is accumulated in fp32 from the exact bf16 products; its diagonal is lifted by a
 * relative 2^-16 before the fp64 Cholesky (so that the accumulation's rounding cannot make
 * the factorization meet a non-positive pivot for maps of large condition number), which
 * adds 2^-16 sum_i |A_i|^2 x_i^2 to |x_hat|^2 (about 1.5e-5 of it where the columns A_i x_i
 * do not cancel).  A zero column of A still gives a zero pivot.
 * R is stored with a unit diagonal: R = diag(g) R1 with g = diag(R) in fp32 and R1 in
 * bf16 whose diagonal entries are exactly 1, and r as r1 = r / g, so that
 * |R x_S + r|^2 = sum_f g_f^2 (R1_f x_S + r1_f)^2 and the diagonal term (through which
 * alone feature 0 reaches the sum) is not rounded to bf16.
 *
 * Folded buffer of one layer (offsets from its start, each 256-byte aligned):
 *     P bf16 [2 kv][d_in] (K rows, then V rows), R1 bf16 [d_in][d_in] (unit diagonal,
 *     zeros below it), c fp32 [2 kv], r1 fp32 [d_in], g fp32 [d_in], kappa fp32;
 *     kv = n_kv_heads * head_dim.
 * ridgefill_fold_bytes returns its size, 0 when the shape cannot be folded: A^T A must be
 * positive definite, so d_in <= d, and d_in must be a multiple of 256.
 *
 * ridgefill_fold_maps computes every given layer's folded buffer from its plain fields
 * (A bf16, or A_q int8 with A_scale; b, norm_w, W_K, W_V).  All layers of a call carry
 * bf16 maps or all carry int8 maps:
 *   folded     host array [n_layers] of device pointers, each >= ridgefill_fold_bytes
 *              bytes and 256-byte aligned
 *   ws         device workspace >= ridgefill_fold_workspace_bytes(shape) for bf16 maps,
 *              >= ridgefill_fold_workspace_bytes_maps(shape, 1, RF_MAPS_INT8) for int8
 *              maps (RF_E_WORKSPACE otherwise, before anything is enqueued); its first
 *              256 bytes hold the status: RF_E_NOT_SPD when some layer's A^T A had a
 *              non-positive pivot (A not of full column rank; that layer's buffer is
 *              then not usable).  A workspace of ridgefill_fold_workspace_bytes_ex(shape, G)
 *              bytes (ridgefill_fold_workspace_bytes_maps(shape, G, RF_MAPS_INT8) for int8
 *              maps) folds G layers side by side (their Cholesky factorizations share one
 *              sequence of launches); a smaller one folds as many as it holds, at least
 *              one (at most 64) at a time.  The results do not depend on G.
 * Arithmetic: P = bf16-split(W diag(w)) times A on the matrix cores (products exact,
 * fp32 accumulation, one bf16 rounding of P); A^T A with exact products and fp32
 * accumulation; Cholesky, r and kappa in fp64; R rounded to bf16 once; c in fp64
 * rounded to fp32.  An int8 map A = diag(A_scale) A_q folds through its codes, which
 * bf16 holds exactly: P = bf16-split(W diag(w A_scale)) times A_q, and
 * A^T A = A_q^T diag(A_scale^2) A_q with the scaled side split into two bf16 parts
 * (about 2^-17 of each entry), as above otherwise; the buffer is the same as from the
 * bf16 map A_q * A_scale up to those roundings.
 * Folded layers work with ridgefill_fill and, from host memory, ridgefill_fill_streamed;
 * all layers of a fill call must be folded or none.  ridgefill_value_scale takes folded
 * layers too (see there).
 * ------------------------------------------------------------------------------ */
size_t ridgefill_fold_bytes(const rf_shape* shape);
size_t ridgefill_fold_workspace_bytes(const rf_shape* shape);
/* Workspace that folds layers_at_once (>= 1) layers side by side; 0 for a shape that
 * cannot be folded or layers_at_once < 1. */
size_t ridgefill_fold_workspace_bytes_ex(const rf_shape* shape, int32_t layers_at_once);
/* The same for the map kind of the layers: map_flags 0 (bf16 maps, as the _ex query) or
 * RF_MAPS_INT8 (int8 maps, which take a second operand slot per layer); 0 for other flags. */
size_t ridgefill_fold_workspace_bytes_maps(const rf_shape* shape, int32_t layers_at_once,
                                           uint32_t map_flags);
rf_status ridgefill_fold_maps(const rf_shape* shape, const rf_layer* layers, int32_t n_layers,
                              void* const* folded, void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------------
 * int8 maps.  Section "Ridge map ...", map size paragraph: maps held in int8 (1.2 GiB
 * for 48 upper layers at hidden size 5120).  Symmetric, one scale per output row:
 *     A_scale[o] = max_i |A[o][i]| / 127,  A_q[o][i] = round-half-even(A[o][i] / A_scale[o])
 * clipped to [-127, 127]; a zero row gets scale 0 and zero codes.  All decisions in fp32
 * with correctly rounded division.  The fill then uses A_q * A_scale as the map.
 *   A        device fp32 [rows][cols] (e.g. one layer of ridgefill_solve's A_out)
 *   A_q      device int8 [rows][cols] out;  A_scale  device fp32 [rows] out
 * ------------------------------------------------------------------------------ */
rf_status ridgefill_quantize_map(const float* A, int64_t rows, int64_t cols, int8_t* A_q,
                                 float* A_scale, void* stream);

/* ------------------------------------------------------------------------------
 * Value-rescale factors.  Section "Hybrid layers and two corrections", value rescale:
 * for each upper layer, the values of the first c tail rows are computed from both the
 * true layer input and the mapped input; per KV head, the mean over those rows of
 * |exact value| / |predicted value| scales the filled values.  For layer l and head h:
 *     v_e(t) = W_V,l RMSNorm_l(x_l,exact[t]),  v_p(t) = W_V,l RMSNorm_l(A_l x_S[t] + b_l)
 *     v_scale_out[l][h] = (1/c) sum_t |v_e(t)_h| / |v_p(t)_h|
 * Pass v_scale_out + l * n_kv_heads as layer l's v_scale to ridgefill_fill.
 *
 *   x_S_tail     device bf16 [c][x_stride]: split-layer states of the first c tail rows
 *   x_l_tail     host array [n_layers] of device bf16 [c][d] (contiguous): each layer's
 *                exact input for the same rows
 *   layers       A or A_q/A_scale, b, norm_w, W_V of each layer (W_K is not read and
 *                may be null; K and the pages are not written); or, for
 *                folded layers (all or none), folded with norm_w and W_V: the predicted
 *                values then come from the folded form, v_p = (P_V x_S + c_V) / rms with
 *                |x_hat|^2 = |R x_S + r|^2 + kappa, and the exact ones from W_V and norm_w
 *   v_scale_out  device fp32 [n_layers][n_kv_heads]
 *   ws           >= ridgefill_value_scale_workspace_bytes(shape, c, 1, map_flags) with
 *                map_flags 0, RF_MAPS_INT8 or RF_MAPS_FOLDED (the last two exclusive); a
 *                larger one lets more layers share a launch (up to 64: the size query for
 *                n_layers covers min(n_layers, 64) layers)
 * Norms are taken in fp32 on the fp32 projections (before any bf16 rounding of v); the
 * inputs to W_V are rounded to bf16 once, as in the fill (for folded layers P_V is the
 * rounded operand).  The mean is added in row order in fp64.  A predicted norm of 0
 * gives an infinite factor.
 * ------------------------------------------------------------------------------ */
size_t ridgefill_value_scale_workspace_bytes(const rf_shape* shape, int64_t c, int32_t n_layers,
                                             int32_t map_flags);
rf_status ridgefill_value_scale(const rf_shape* shape, const uint16_t* x_S_tail, int64_t x_stride,
                                const uint16_t* const* x_l_tail, int64_t c, const rf_layer* layers,
                                int32_t n_layers, float* v_scale_out, void* ws, size_t ws_bytes,
                                void* stream);

/* ------------------------------------------------------------------------------
 * Calibration.  Same section, paragraph on alpha and the one-pass statistics: one pass
 * accumulates X^T X, Y_l^T X and the two means; a new lambda needs only a new solve.
 * The state belongs to one split (one x_S source) and is caller-owned device memory.
 * x_S is accumulated about a per-feature shift s (fp32 holding bf16 values), fixed by the
 * first call that adds rows: where that call has at least 64 rows, s_i is the bf16
 * rounding of the mean of feature i over them if that mean exceeds twice their standard
 * deviation, else 0; a first call of fewer rows fixes s = 0.  Each call accumulates
 * x'_S = bf16(x_S - s) (exact wherever x_S lies within [s/2, 2s]), so that a feature whose
 * mean dwarfs its spread keeps its centred moments in fp32 (raw moments would lose them
 * to cancellation).  Layout:
 *   [0, 256)   header: int64 row count n, int32 d, int32 n_layers, magic, int32 d,
 *              int32 shift fixed, int32 state marked bad, int32 (internal)
 *   then       fp64 sum_t x'_S         [d]
 *              fp64 sum_t x_l          [n_layers][d]
 *              fp32 sum_t x'_S x'_S^T  [d][d]   (lower triangle valid; i >= j)
 *              fp32 sum_t x_l x'_S^T   [n_layers][d][d]  (row = output feature of x_l)
 *              fp32 s                  [d]
 *              scratch: 16384 rows of bf16 [d] where each call stages x'_S (a call of
 *              more rows is processed in pieces of 16384)
 * Each region starts on a 256-byte boundary.  Saving the state is a device-to-host copy
 * of everything before the scratch area.
 *
 * ridgefill_calib_reset clears the state for (d, n_layers); later calls on the state
 * must pass the same d and n_layers.  A calibrate call whose sizes differ from the
 * header's changes nothing and marks the state bad; a later solve on it then reports
 * RF_E_WORKSPACE through ridgefill_read_status.
 * ridgefill_calibrate adds n_rows rows: x_S device bf16 [n_rows][d]; x_l host array
 * [n_layers] of device bf16 [n_rows][d] pointers.  Sums in fp32 per call and fp64
 * across calls for the means; moments accumulated in fp32.  d: multiple of 256;
 * n_layers: 1 .. 64.
 * ------------------------------------------------------------------------------ */
size_t ridgefill_calib_state_bytes(int32_t d, int32_t n_layers);
rf_status ridgefill_calib_reset(void* state, size_t state_bytes, int32_t d, int32_t n_layers,
                                void* stream);
rf_status ridgefill_calibrate(void* state, size_t state_bytes, int32_t d, int32_t n_layers,
                              const uint16_t* x_S, const uint16_t* const* x_l, int64_t n_rows,
                              void* stream);

/* The same for maps whose input width differs from their output width (section "Ridge
 * map ...", map-size paragraph): x_S rows are d_in wide, x_l rows d_out wide (both
 * multiples of 256).  The state then holds
 *   [0, 256)   header: int64 n, int32 d_out, int32 n_layers, magic, int32 d_in, ...
 *   then       fp64 sum_t x'_S [d_in], fp64 sum_t x_l [n_layers][d_out],
 *              fp32 sum_t x'_S x'_S^T [d_in][d_in] (lower triangle valid),
 *              fp32 sum_t x_l x'_S^T [n_layers][d_out][d_in], fp32 s [d_in],
 *              scratch bf16 [16384][d_in].
 * The plain calls are these with d_in = d_out = d. */
size_t ridgefill_calib_state_bytes_ex(int32_t d_in, int32_t d_out, int32_t n_layers);
rf_status ridgefill_calib_reset_ex(void* state, size_t state_bytes, int32_t d_in, int32_t d_out,
                                   int32_t n_layers, void* stream);
rf_status ridgefill_calibrate_ex(void* state, size_t state_bytes, int32_t d_in, int32_t d_out,
                                 int32_t n_layers, const uint16_t* x_S, const uint16_t* const* x_l,
                                 int64_t n_rows, void* stream);

/* ------------------------------------------------------------------------------
 * Solve.  Same section, closed-form equation and the scale-free penalty: with
 * mu = sums / n (mu_S of the shifted rows x'_S),  C = sum x'_S x'_S^T - n mu_S mu_S^T,
 * C_l = sum x_l x'_S^T - n mu_l mu_S^T,  alpha = lambda * tr(C) / d,
 *     A_l = C_l (C + alpha I)^-1,     b_l = mu_l - A_l (mu_S + s).
 * (C + alpha I) is factored by a device Cholesky in fp64 and inverted in fp64.  The
 * product C_l M (M = (C + alpha I)^-1) is a bf16 matrix-core GEMM on operands split into
 * bf16 parts, fp32 accumulation: two parts per operand (hi + mid, three products, about
 * 2^-17 relative per operand) while kappa_F = |C + alpha I|_F |M|_F <= 16 d, else three
 * parts (hi + mid + lo, six products, about 2^-25 per operand; the product then takes
 * twice as long).  The relative error of A grows about as 5e-6 kappa_F / d with two parts
 * and 1e-7 kappa_F / d with three.  b_l is accumulated in fp64.
 *
 *   A_out       device fp32 [n_layers][d][d] (may be NULL if A_bf16_out is given)
 *   b_out       device fp32 [n_layers][d]
 *   A_bf16_out  device bf16 [n_layers][d][d] or NULL: the map as the fill takes it
 *   ws          device workspace >= ridgefill_solve_workspace_bytes(d, n_layers);
 *               its first 256 bytes hold the status (RF_E_NOT_SPD on a bad pivot).
 * lambda must be >= 0 and finite.  Repeated solves reuse the state unchanged.
 * ------------------------------------------------------------------------------ */
size_t ridgefill_solve_workspace_bytes(int32_t d, int32_t n_layers);
rf_status ridgefill_solve(const void* state, size_t state_bytes, int32_t d, int32_t n_layers,
                          double lambda, float* A_out, float* b_out, uint16_t* A_bf16_out,
                          void* ws, size_t ws_bytes, void* stream);

/* The solve for a state made by the _ex calls: alpha = lambda tr(C) / d_in, the Cholesky
 * on the d_in x d_in side, A_out fp32 [n_layers][d_out][d_in], b_out fp32
 * [n_layers][d_out], A_bf16_out bf16 [n_layers][d_out][d_in]. */
size_t ridgefill_solve_workspace_bytes_ex(int32_t d_in, int32_t d_out, int32_t n_layers);
rf_status ridgefill_solve_ex(const void* state, size_t state_bytes, int32_t d_in, int32_t d_out,
                             int32_t n_layers, double lambda, float* A_out, float* b_out,
                             uint16_t* A_bf16_out, void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------------
 * The cache beyond the fill.  Exact rows, the tail and the generated tokens run the upper
 * layers themselves (section "Two numbers set the skip range"): their keys and values go
 * into the same paged cache, and their queries attend over it.  The calls below rotate and
 * append such rows, attend over the cache (up to 64 queries a sequence, its last rows; more
 * and others as sequences of their own), accumulate the attention weight that its rows
 * receive (the scores of section "Which rows to compute exactly"), and shorten it.  They
 * work on one layer's pools (the eviction on all of them) and on a batch of sequences.
 *
 * A batch of sequences in one pool.  Row t of sequence b lies in page
 * block_tables[b * table_stride + t / page_size], slot t % page_size.  Lengths are read on
 * the device, so a captured call replays with new ones; max_len is the host's bound on them
 * and sizes grids and workspaces.  A sequence whose length is not in [0, max_len] sets
 * RF_E_ROWS and is skipped (its outputs are left as they were); rows on a page outside
 * [0, num_pages) set RF_E_ROWS and are taken as not there.
 * ------------------------------------------------------------------------------ */
typedef struct rf_paged_batch {
  const int32_t* block_tables;  /* device int32 [batch][table_stride]                       */
  const int32_t* lengths;       /* device int32 [batch]: rows each sequence has in the cache
                                   (not read by ridgefill_append_rows, which takes NULL)    */
  int64_t table_stride;         /* >= ceil(max_len / page_size)                             */
  int32_t batch;                /* 1 .. 65535                                               */
  int32_t max_len;              /* 1 .. 2^30; batch * max_len <= 2^36                       */
  int32_t page_size, num_pages; /* >= 1; num_pages * page_size < 2^31                       */
  int32_t n_kv_heads;           /* 1 .. 256                                                 */
  int32_t head_dim;             /* 64 or 128; for ridgefill_append_rows a multiple of 16 up to 256 */
} rf_paged_batch;

/* ------------------------------------------------------------------------------
 * Rotary positions.  Pair j of a head (of rotary_dim / 2 pairs) turns by the angle
 * position * f_j, f_j = theta^(-2j / rotary_dim) where nothing is scaled:
 *     a' = m (a cos - b sin),   b' = m (b cos + a sin)
 * with (a, b) the features (j, j + rotary_dim/2) (RF_ROPE_HALF, as the fill rotates) or
 * (2j, 2j+1) (RF_ROPE_INTERLEAVED); features from rotary_dim on pass unchanged.  Scaling for
 * contexts s = factor times as long as the trained length L = orig_len:
 *   RF_ROPE_LINEAR  f_j / s
 *   RF_ROPE_NTK     theta * s^(r / (r - 2)) in place of theta, r = rotary_dim > 2
 *   RF_ROPE_BANDS   by turns n = L f_j / (2 pi) over the trained length: n < low: f_j / s;
 *                   n > high: f_j; between them (1 - t) f_j / s + t f_j,
 *                   t = (n - low) / (high - low)
 *   RF_ROPE_YARN    with d(n) = r ln(L / (2 pi n)) / (2 ln theta), p = max(floor d(high), 0),
 *                   q = min(ceil d(low), r - 1), t = clamp((j - p) / max(q - p, 0.001), 0, 1):
 *                   t f_j / s + (1 - t) f_j
 * m = mscale; 0 means 1, for RF_ROPE_YARN 0.1 ln s + 1.  Angles are formed in fp64, cos and
 * sin in fp32, and results rounded once to the output's type.
 * ------------------------------------------------------------------------------ */
#define RF_ROPE_HALF 0
#define RF_ROPE_INTERLEAVED 1
#define RF_ROPE_PLAIN 0
#define RF_ROPE_LINEAR 1
#define RF_ROPE_NTK 2
#define RF_ROPE_BANDS 3
#define RF_ROPE_YARN 4
typedef struct rf_rope {
  double theta;         /* base, > 1                                                     */
  int32_t rotary_dim;   /* 0: the whole head; else a multiple of 16, <= head_dim         */
  int32_t layout;       /* RF_ROPE_HALF or RF_ROPE_INTERLEAVED                           */
  int32_t scaling;      /* RF_ROPE_PLAIN .. RF_ROPE_YARN                                 */
  int32_t orig_len;     /* >= 1 for RF_ROPE_BANDS and RF_ROPE_YARN                       */
  double factor;        /* >= 1 where scaling is not RF_ROPE_PLAIN                       */
  double low, high;     /* 0 < low < high for RF_ROPE_BANDS and RF_ROPE_YARN             */
  double mscale;        /* >= 0                                                          */
} rf_rope;

/* Element types of ridgefill_rope. */
#define RF_TYPE_BF16 0
#define RF_TYPE_F32 1

/* Rotates x [n_rows][n_heads][head_dim] (rows x_stride elements apart) into out (the same,
 * out_stride apart; out = x with equal strides rotates in place, other overlaps are not
 * allowed).  transpose = 1 turns by the negative angle, times m: the transposed rotation,
 * which takes the gradient of out to the gradient of x.
 *   x, out      device, of x_type (RF_TYPE_BF16 or RF_TYPE_F32), 16-byte aligned; strides
 *               >= n_heads * head_dim and multiples of 8 (bf16) or 4 (fp32) elements
 *   positions   device int32 [n_rows]; any value, negative ones too
 * head_dim: a multiple of 16 up to 256; n_rows: 0 .. 2^23. */
rf_status ridgefill_rope(const rf_rope* rope, const void* x, int32_t x_type, int64_t n_rows,
                         int32_t n_heads, int32_t head_dim, int64_t x_stride,
                         const int32_t* positions, void* out, int64_t out_stride,
                         int32_t transpose, void* stream);

/* Appends n_rows rows to the paged cache of one layer: k is rotated (as it comes if rope is
 * NULL) and written with v to cache row rows[i] of sequence seq[i]; q, if given, is rotated
 * into q_out.  Everything in one pass over the rows.
 *   q           device bf16 [n_rows][n_q_heads][head_dim] or NULL (then n_q_heads = 0)
 *   q_out       device bf16, the same shape; q_out = q rotates in place (other overlaps of
 *               the rows with one another or with the pages are not allowed)
 *   k, v        device bf16 [n_rows][n_kv_heads][head_dim]; the strides (elements between
 *               rows) are multiples of 8, all pointers 16-byte aligned
 *   seq         device int32 [n_rows] or NULL (all rows belong to sequence 0); a negative
 *               entry marks a padding row: nothing of it is written
 *   rows        device int32 [n_rows]: cache rows in [0, kv->max_len)
 *   positions   device int32 [n_rows], the angles' positions, or NULL (the cache rows)
 *   status      device uint32 (4-byte aligned): receives the device status word of the
 *               call.  A sequence, row or page out of range sets RF_E_ROWS there and that
 *               row's k and v are not written (its q is rotated all the same).
 * The (seq, rows) pairs of one call must differ from one another.  n_rows: 0 .. 2^23. */
rf_status ridgefill_append_rows(const rf_rope* rope, const rf_paged_batch* kv, const uint16_t* q,
                                int32_t n_q_heads, int64_t q_stride, uint16_t* q_out,
                                int64_t q_out_stride, const uint16_t* k, int64_t k_stride,
                                const uint16_t* v, int64_t v_stride, int64_t n_rows,
                                const int32_t* seq, const int32_t* rows, const int32_t* positions,
                                uint16_t* k_pages, uint16_t* v_pages, uint32_t* status,
                                void* stream);

/* ------------------------------------------------------------------------------
 * Attention of the last rows of each sequence over its cache: a tree of drafted tokens, a
 * chain of them, or one token.  Queries q_start[b] .. q_start[b+1]-1 belong to sequence b
 * (n of them) and stand for the last n of its lengths[b] cached rows, which are in the cache
 * already; query i (0-based among them) sees the c = lengths[b] - n rows before, and of the
 * n rows those j whose bit is set in its word of tree_mask (without tree_mask: j <= i).
 *     s = scale q . k,   lse = ln sum exp s,   out = sum exp(s - lse) v
 * over the visible rows.  Query head h reads key head h / (n_q_heads / n_kv_heads).  A query
 * that sees no row, or only scores of -inf, gives out = 0 and lse = -inf; one that sees a score
 * of +inf or NaN gives NaN in both.  A row that a query does not see has no influence on it,
 * whatever the row holds (NaN included).  Sums of the values are fp32: magnitudes of v above
 * 2^88 may overflow.
 * Rows that are not the last of a sequence, or more than 64 of them, are sequences of their own
 * in the batch with a copy of the same block-table row, each ending with its own queries: the
 * last 150 rows of 300 as lengths 172, 236, 300 with 22, 64 and 64 queries.  Each such sequence
 * reads the cache once more.
 *   q           device bf16 [n_q][n_q_heads][head_dim], rows q_stride elements apart
 *               (multiple of 8), 16-byte aligned; n_q_heads a multiple of n_kv_heads
 *   q_start     device int32 [batch + 1], ascending; sequences may have no queries.  One
 *               with more than max_q queries, more queries than rows, or outside [0, n_q)
 *               sets RF_E_ROWS and is skipped.  Queries of no sequence are left as they were.
 *   max_q       1 .. 64: the host's bound on one sequence's queries;
 *               batch * n_q_heads * max_q <= 2^26
 *   tree_mask   device uint64 [n_q] or NULL
 *   out         device bf16 [n_q][n_q_heads][head_dim], rows out_stride elements apart
 *               (multiple of 8), 16-byte aligned, not overlapping q; or NULL (only lse; v_pages
 *               may then be NULL)
 *   lse         device fp32 [n_q][n_q_heads] or NULL (one of out, lse is needed)
 *   ws          >= ridgefill_tree_attention_workspace_bytes(kv, n_q_heads, max_q), 256-byte
 *               aligned; its first 256 bytes hold the status
 * Scores, maxima, sums and outputs are held in fp32; for the product with v exp(s - max) is two
 * bf16 operands of the matrix cores, which hold it to 2^-15; out is rounded once at the end
 * (a workgroup's sums of equal weights are exact up to 2^28 rows).  The same call on the
 * same inputs gives the same bits; a row's bits may differ between calls whose sequences have
 * other lengths, since long caches are split evenly over the batch.  Size query: 0 on invalid
 * input.
 * ------------------------------------------------------------------------------ */
size_t ridgefill_tree_attention_workspace_bytes(const rf_paged_batch* kv, int32_t n_q_heads,
                                                int32_t max_q);
rf_status ridgefill_tree_attention(const rf_paged_batch* kv, const uint16_t* k_pages,
                                   const uint16_t* v_pages, const uint16_t* q, int32_t n_q_heads,
                                   int64_t q_stride, const int32_t* q_start, int64_t n_q,
                                   int32_t max_q, const uint64_t* tree_mask, float scale,
                                   uint16_t* out, int64_t out_stride, float* lse, void* ws,
                                   size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------------
 * Accumulated attention weight.  For every row t of every sequence that has queries,
 *     acc_out[b][t] = decay * acc[b][t] + sum over queries i that see t, and heads h, of
 *                     exp(scale q_ih . k_t - lse_ih)
 * Queries, q_start, max_q, tree_mask and scale as in ridgefill_tree_attention, whose lse this
 * takes (entries of -inf give nothing).  With the last 64 tokens of a prompt as queries this
 * is the score of section "Which rows to compute exactly" that ridgefill_select_rows ranks.
 *   acc         device fp32 [batch][acc_stride] or NULL (nothing accumulated so far)
 *   acc_out     device fp32 [batch][acc_stride]; acc_out = acc accumulates in place.  Entries
 *               from lengths[b] on, and sequences without queries, are left as they were.
 *   acc_stride  >= max_len; batch * max_len <= 2^29
 *   ws          >= ridgefill_attention_weight_workspace_bytes(kv, n_q_heads, max_q)
 * Sums are held in fp32 and added in a fixed order: results do not vary between runs.
 * ------------------------------------------------------------------------------ */
size_t ridgefill_attention_weight_workspace_bytes(const rf_paged_batch* kv, int32_t n_q_heads,
                                                  int32_t max_q);
rf_status ridgefill_attention_weight(const rf_paged_batch* kv, const uint16_t* k_pages,
                                     const uint16_t* q, int32_t n_q_heads, int64_t q_stride,
                                     const int32_t* q_start, int64_t n_q, int32_t max_q,
                                     const uint64_t* tree_mask, float scale, const float* lse,
                                     float decay, const float* acc, float* acc_out,
                                     int64_t acc_stride, void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------------
 * Eviction.  Every sequence of more than n_keep rows is cut to n_keep, in every given
 * layer's pools.  The kept rows are, in this order, the protected ones (position < n_sink,
 * or among the n_recent highest positions: position > highest - n_recent) and the others by
 * falling weight; ties go to the lower cache row.  -0.0 ties with +0.0; a NaN weight ranks
 * lowest and sets RF_E_INVALID.  Kept rows below n_keep stay; the kept rows from n_keep on
 * move, in ascending order, into the rows below n_keep that were not kept, in ascending
 * order.  Keys carry their positions already, so attention does not depend on the order;
 * positions_out says which position each row holds.
 *   layers        host array [n_layers]; only k_pages and v_pages are used (16-byte aligned)
 *   acc           device fp32 [batch][stride]: weights (ridgefill_attention_weight)
 *   positions     device int32 [batch][stride]: position of each cached row
 *   acc_out, positions_out   device, the same shapes: those of the rows after the cut;
 *                 acc_out is 0 for the rows cut off (from the new length to the old one);
 *                 entries from the old length on are left as they were.  Each may be the input.
 *   lengths_out   device int32 [batch]: the new lengths; may be kv->lengths
 *   stride        >= max_len
 *   n_keep, n_sink, n_recent >= 0
 *   ws            >= ridgefill_evict_workspace_bytes(kv, n_keep), 256-byte aligned; its first
 *                 256 bytes hold the status.  A row that would move from or to a bad page is
 *                 lost: the place it would take keeps its own row, weight and position.
 * The cut off pages stay in the block table; their rows are free for new ones.  Sequences of
 * one call must not share pages that the cut writes.
 * ------------------------------------------------------------------------------ */
size_t ridgefill_evict_workspace_bytes(const rf_paged_batch* kv, int32_t n_keep);
rf_status ridgefill_evict_rows(const rf_paged_batch* kv, const rf_layer* layers, int32_t n_layers,
                               const float* acc, const int32_t* positions, int64_t stride,
                               int32_t n_keep, int32_t n_sink, int32_t n_recent, float* acc_out,
                               int32_t* positions_out, int32_t* lengths_out, void* ws,
                               size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------------
 * Norms of query and key heads with their rotation, in one pass (section "Hybrid layers and
 * two corrections": layers that norm their keys, as the fill does with k_norm_w).  For a head x
 * with weight w, r = (mean x^2 + eps)^(-1/2) over its head_dim features and R the rotation:
 *     y = R (w r x)
 * A tensor without a weight is only rotated.  Sums of squares are fp32 (magnitudes above 2^60
 * overflow them), results are rounded once.  With eps = 0 a head of zeros gives NaN, one whose
 * magnitudes are all below 2^-75 infinities, and r has fewer bits where they are all below 2^-58.
 * ------------------------------------------------------------------------------ */
typedef struct rf_head_norm {
  const void* q_w;              /* device [head_dim], of the tensors' type, 16-byte aligned;
                                   NULL: q is not normed                                     */
  const void* k_w;              /* the same for k                                            */
  float eps;                    /* >= 0                                                      */
  int32_t reserved;             /* must be 0                                                 */
} rf_head_norm;

/* q [n_rows][n_q_heads][head_dim] into q_out and k [n_rows][n_k_heads][head_dim] into k_out;
 * either may be NULL, with n_q_heads or n_k_heads 0.
 *   rope        NULL: no rotation (positions may then be NULL)
 *   norm        NULL: no norm
 *   q, k, q_out, k_out   device, all of `type` (RF_TYPE_BF16 or RF_TYPE_F32), 16-byte aligned;
 *               strides (elements between rows) >= heads * head_dim and multiples of 8 (bf16)
 *               or 4 (fp32); an output may be its input with equal strides, other overlaps are
 *               not allowed
 *   positions   device int32 [n_rows]
 * head_dim: a multiple of 16 up to 256; heads up to 4096 each; n_rows: 0 .. 2^23. */
rf_status ridgefill_norm_rope(const rf_rope* rope, const rf_head_norm* norm, int32_t type,
                              int64_t n_rows, int32_t head_dim, const int32_t* positions,
                              const void* q, int32_t n_q_heads, int64_t q_stride, void* q_out,
                              int64_t q_out_stride, const void* k, int32_t n_k_heads,
                              int64_t k_stride, void* k_out, int64_t k_out_stride, void* stream);

/* Its gradient: of the inputs q and k (as they went in) and the gradients gq and gk of the
 * outputs, q_grad and k_grad, and in fp32 [head_dim] those of the weights, qw_grad and kw_grad
 * (each may be NULL, not the same memory; not written for a tensor without a weight).  A weight that
 * q and k share has the sum of both as its gradient.  With g = R^T gy, xh = r x:
 *     q_grad = r (w g - xh mean(w g xh)),   qw_grad = sum over rows and heads of g xh
 * q and k may be NULL where they have no weight (their values are not needed), q_grad may be gq
 * and k_grad gk with equal strides.  The weights' sums are fp32, added in a fixed order.
 *   ws          >= ridgefill_norm_rope_grad_workspace_bytes(...), 256-byte aligned
 * Size query: 0 on invalid input. */
size_t ridgefill_norm_rope_grad_workspace_bytes(int64_t n_rows, int32_t n_q_heads,
                                                int32_t n_k_heads, int32_t head_dim);
rf_status ridgefill_norm_rope_grad(const rf_rope* rope, const rf_head_norm* norm, int32_t type,
                                   int64_t n_rows, int32_t head_dim, const int32_t* positions,
                                   const void* q, int32_t n_q_heads, int64_t q_stride,
                                   const void* gq, int64_t gq_stride, void* q_grad,
                                   int64_t q_grad_stride, float* qw_grad, const void* k,
                                   int32_t n_k_heads, int64_t k_stride, const void* gk,
                                   int64_t gk_stride, void* k_grad, int64_t k_grad_stride,
                                   float* kw_grad, void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------------
 * Caches in 16 or 8 bits.  RF_CACHE_BF16 is the cache of the calls above, which take no other: the
 * fill writes, and ridgefill_attention_weight and ridgefill_evict_rows read bf16 pools.  The others hold codes
 * of 8 bits (e4m3 floats, or whole numbers) in blocks of 32 features of a head that share a power
 * of two, much as in the OCP microscaling formats (there int8 codes count in steps of 2^-6 of the scale,
 * and e4m3 blocks above 1.75 2^k are cut off): for a block x, e is the smallest exponent with
 * max |x| <= M 2^e (M = 448 for e4m3, 127 for int8), kept to -110 .. 118; a code is x 2^-e rounded
 * to its type (ties to even, magnitudes above M to M) and stands for code * 2^e; the scale byte is
 * e + 127.  A block with an infinity or NaN is NaN altogether: scale byte 255, and codes 0 (int8) or
 * 0x7f (e4m3).  Every value that a cache can hold is exactly a bf16: reads give it as it is, and
 * attention over such a cache is attention over a bf16 cache of the same values (up to the order of
 * sums).  Other scale bytes than 17 .. 245 and such blocks are not allowed in a cache written
 * elsewhere; each pool of scales has to be readable to the end of its last word of 4 bytes.
 * ------------------------------------------------------------------------------ */
#define RF_CACHE_BF16 0
#define RF_CACHE_FP8 1
#define RF_CACHE_INT8 2
typedef struct rf_cache {       /* one layer's pools, device, 16-byte aligned                */
  int32_t type;
  int32_t reserved;             /* must be 0                                                 */
  void* k_pages;                /* bf16 or 8-bit codes [num_pages][page_size][n_kv_heads][head_dim] */
  void* v_pages;
  uint8_t* k_scales;            /* [num_pages][page_size][n_kv_heads][head_dim / 32]; NULL for bf16 */
  uint8_t* v_scales;
} rf_cache;

/* ridgefill_append_rows for a cache of any type and for layers with head norms: q and k are
 * normed where norm has a weight (bf16 [head_dim]), rotated, and k and v are rounded once to what
 * the cache holds.  Arguments as there; head_dim a multiple of 32 for 8 bits (16 for bf16).  With
 * norm NULL and a bf16 cache it does what that call does. */
rf_status ridgefill_append_cache(const rf_rope* rope, const rf_head_norm* norm,
                                 const rf_paged_batch* kv, const rf_cache* cache,
                                 const uint16_t* q, int32_t n_q_heads, int64_t q_stride,
                                 uint16_t* q_out, int64_t q_out_stride, const uint16_t* k,
                                 int64_t k_stride, const uint16_t* v, int64_t v_stride,
                                 int64_t n_rows, const int32_t* seq, const int32_t* rows,
                                 const int32_t* positions, uint32_t* status, void* stream);

/* Cached rows back: k_out[i] and v_out[i] receive cache row rows[i] of sequence seq[i].
 *   k_out, v_out   device [n_rows][n_kv_heads][head_dim] of `type` (RF_TYPE_BF16 or RF_TYPE_F32;
 *                  both exact), 16-byte aligned, strides as in ridgefill_norm_rope, no overlap; one
 *                  may be NULL
 *   seq, rows, status   as in ridgefill_append_rows, but the same row may come more than once;
 *                  rows that are out of range, on a bad page or padding are left as they were
 * kv->lengths is not read.  n_rows: 0 .. 2^23, n_rows * n_kv_heads * head_dim <= 2^34. */
rf_status ridgefill_read_rows(const rf_paged_batch* kv, const rf_cache* cache, int64_t n_rows,
                              const int32_t* seq, const int32_t* rows, int32_t type, void* k_out,
                              int64_t k_out_stride, void* v_out, int64_t v_out_stride,
                              uint32_t* status, void* stream);

/* ------------------------------------------------------------------------------
 * Attention over a cache of any type, also of sequences that share long prefixes (one prompt,
 * filled once, under many answers).  Queries, q_start, max_q, tree_mask, scale, out and lse as in
 * ridgefill_tree_attention; kv->lengths and its block tables are the sequences' own rows.  With
 * `prefix`, sequences group_start[g] .. group_start[g+1]-1 all see the lengths[g] rows of prefix g
 * before their own: one softmax over both.  A prefix's rows are read once for every block of its
 * matrix of queries and query heads that share a key head: of 256 rows, of 128 where n_q queries come to
 * 128 rows a group or less, of 16 where they come to 16 and to no more than 64 in all.  Sequences
 * before group_start[0] and from group_start[groups] on have no prefix.
 * ------------------------------------------------------------------------------ */
typedef struct rf_prefix {
  const int32_t* block_tables;  /* device int32 [groups][table_stride]: pages of the same pools */
  const int32_t* lengths;       /* device int32 [groups]: rows of each prefix, 0 .. max_len   */
  const int32_t* group_start;   /* device int32 [groups + 1], ascending, within 0 .. batch    */
  int64_t table_stride;         /* >= ceil(max_len / kv->page_size)                           */
  int32_t groups;               /* 1 .. 65535; groups * n_kv_heads <= 2^22                    */
  int32_t max_len;              /* 1 .. 2^30: the host's bound on the lengths                 */
} rf_prefix;

/*   prefix      NULL: sequences of their own rows alone, which over a bf16 cache is
 *               ridgefill_tree_attention
 *   cache       v_pages (and v_scales) may be NULL where out is
 *   n_q         with a prefix batch * n_q_heads * max_q <= 2^25
 *   ws          >= ridgefill_cache_attention_workspace_bytes(kv, prefix, n_q_heads, max_q, n_q), of
 *               which the pointers in kv and prefix are not read; 256-byte aligned; its first 256
 *               bytes hold the status
 * A group whose length or sequences are out of range, or whose queries are out of order or more
 * than max_q for each sequence, sets RF_E_ROWS, and its sequences are skipped.  So does a group that
 * begins, in sequences or in queries, before the end of one in front of it that has none of these
 * faults.  Where groups overlap, a sequence belongs to the first.  Precision and repeatability as in
 * ridgefill_tree_attention. */
size_t ridgefill_cache_attention_workspace_bytes(const rf_paged_batch* kv, const rf_prefix* prefix,
                                                 int32_t n_q_heads, int32_t max_q, int64_t n_q);
rf_status ridgefill_cache_attention(const rf_paged_batch* kv, const rf_prefix* prefix,
                                    const rf_cache* cache, const uint16_t* q, int32_t n_q_heads,
                                    int64_t q_stride, const int32_t* q_start, int64_t n_q,
                                    int32_t max_q, const uint64_t* tree_mask, float scale,
                                    uint16_t* out, int64_t out_stride, float* lse, void* ws,
                                    size_t ws_bytes, void* stream);

/* Waits for `stream`, then returns the device status word of a fill, solve or selection
 * workspace, or of a cache call's workspace or status word: RF_OK, RF_E_ROWS, RF_E_NOT_SPD,
 * RF_E_WORKSPACE for a solve on a calibration state whose header disagrees with the solve's
 * sizes or that a calibrate call marked bad, or RF_E_INVALID for a NaN score or weight.  Each
 * call clears that word on the stream before its own kernels run (the cache calls write it
 * whole), so the word reflects the last call only. */
rf_status ridgefill_read_status(void* ws, void* stream);

/* Waits for `stream`, then reports the conditioning of the last solve on this solve
 * workspace: *kappa_f = |C + alpha I|_F |(C + alpha I)^-1|_F (an upper bound on the
 * 2-norm condition number) and *parts = the bf16 parts per operand the map product used
 * (3: hi, mid, hi pairs, three products; 6: six products).  Both outputs are host pointers;
 * either may be NULL. */
rf_status ridgefill_solve_info(void* ws, double* kappa_f, int32_t* parts, void* stream);

/* ------------------------------------------------------------------------------
 * Kernel timing for measurement.  While enabled, every compute-kernel launch of the
 * library is bracketed by a pair of HIP events recorded on the caller's stream (no
 * synchronisation is added).  ridgefill_profile_read waits for the recorded events and
 * returns, for one kernel, the launches seen since the last reset and their summed
 * duration in milliseconds.  Host-side only; thread safe.
 * ------------------------------------------------------------------------------ */
typedef enum rf_kernel_id {
  RF_KERNEL_FILL_MAP = 0,      /* map GEMM: x_hat = A x_S + b, RMS partials, x_hat * w   */
  RF_KERNEL_FILL_KV = 1,       /* K/V GEMM: RMS scale, RoPE, paged store                 */
  RF_KERNEL_CALIB_MOMENTS = 2, /* calibration: sum x_S x_S^T (lower) and every x_l x_S^T */
  RF_KERNEL_CALIB_SUMS = 3,    /* calibration: column sums and row count                 */
  RF_KERNEL_SOLVE_MAP = 4,     /* solve: A_l = C_l (C + alpha I)^-1 product              */
  RF_KERNEL_FILL_NORM = 5,     /* folded fill: per-row |R x_S + r|^2 partials            */
  RF_KERNEL_COUNT = 6
} rf_kernel_id;
rf_status ridgefill_profile_enable(int32_t enable);
rf_status ridgefill_profile_read(int32_t kernel, int64_t* launches, double* total_ms);
rf_status ridgefill_profile_reset(void);

const char* ridgefill_status_string(rf_status s);
/* Description of the last non-OK status returned on this thread ("" if none). */
const char* ridgefill_last_error(void);

#ifdef __cplusplus
}
#endif
#endif /* RIDGEFILL_H */
