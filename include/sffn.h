/*
 * sffn.h - activation-sparse ReLU feedforward layer for AMD Instinct MI355X
 * (gfx950), C ABI.
 *
 * The layer is the feedforward block of "Sparser, Faster, Lighter
 * Transformer Language Models" (Cetin et al.):
 *
 *   gated      y = (ReLU(x W_g) * (x W_u)) W_d
 *   non-gated  y = ReLU(x W_1) W_2
 *
 * (gist.science explainer, "2. Methodology" B, inference kernels; appendix
 * Table 2 for the gated/non-gated shapes). The sparse forward packs the gate
 * activations into TwELL inside the gate GEMM's epilogue and then runs the
 * up and down projections only over each token's active neurons, without a
 * dense hidden tensor in memory (same section). TwELL is tile-wise ELLPACK:
 * each row's columns are cut into 1-D tiles of W columns and every
 * (row, tile) keeps a fixed-capacity list of (value, column) plus a count
 * ("2. Methodology" A; wispaper blog, "1. TwELL: Tile-wise ELLPACK").
 *
 * Conventions shared by every call:
 *   - Every call returns an sffn_status and never aborts or throws.
 *   - Device memory the library needs per call is the caller's workspace;
 *     its size (sffn_workspace_bytes) follows the sparse work: the ELL
 *     capacity K and the dense path's row capacity R (desc.dense_rows),
 *     never T x F. Data-dependent overflow of R (more rows on the dense
 *     path than it holds) is not an argument error: the dense path's rows
 *     are then not valid, and sffn_check() reports SFFN_E_CAPACITY.
 *   - Argument errors (null or misaligned pointers, bad sizes) are found on
 *     the host before anything is enqueued and return SFFN_E_ARG.
 *   - All device work is ordered on the caller's stream; no call
 *     synchronises the stream except sffn_check() and sffn_hybrid_check().
 *     sffn_backward forks part of its work to a second stream of the handle
 *     (created on first use, default priority) and joins it back through
 *     events before it returns; work enqueued on the caller's stream after
 *     the call sees all of its results.
 *   - Pointers are device pointers unless stated; every array is
 *     caller-owned and must be 16-byte aligned. The library never frees
 *     caller memory.
 *   - A handle is not thread-safe; use one handle per concurrently used
 *     stream.
 *   - T = 0 is a no-op that returns SFFN_OK.
 *   - Layouts (row-major, contiguous):
 *       x, dy        [T, d]            dtype of the descriptor
 *       w_gate, w_up [F, d]            neuron-major (row j = column j of
 *                                      the math d x F matrix, i.e. the
 *                                      nn.Linear weight layout)
 *       w_down       [F, d]            row j = neuron j's output weights
 *                                      (the math F x d matrix as is)
 *       y, dx        [T, d]            float32
 *       z            [T, F]            float32 gate pre-activations
 *   - "active" means strictly z > 0; slots inside a tile ascend by column.
 */
#ifndef SFFN_H
#define SFFN_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef int32_t sffn_status;
#define SFFN_OK             0
#define SFFN_E_ARG         -1  /* null/misaligned pointer, bad size or enum */
#define SFFN_E_UNSUPPORTED -2  /* shape outside the supported set, wrong GPU */
#define SFFN_E_HIP         -3  /* HIP runtime or launch error; see sffn_last_error */
#define SFFN_E_CAPACITY    -4  /* a caller buffer was too small (data dependent) */

/* element type of x, the weights and dy */
#define SFFN_F32  0
#define SFFN_BF16 1
/* element type of an expert layer's weights (microscaled 4-bit, below) */
#define SFFN_MXFP4 2
/* a form of the norm's result (microscaled 8-bit, below) */
#define SFFN_MXFP8 3

/* forward modes */
#define SFFN_SPARSE 0   /* gate GEMM + TwELL, sparse up/down, dense path for flagged rows */
#define SFFN_DENSE  1   /* plain dense layer: the same library's baseline */

/* operations, for sffn_workspace_bytes */
#define SFFN_OP_PACK           0
#define SFFN_OP_FORWARD_SPARSE 1
#define SFFN_OP_FORWARD_DENSE  2
#define SFFN_OP_HYBRID         3
#define SFFN_OP_FORWARD_TRAIN  4
#define SFFN_OP_BACKWARD       5
#define SFFN_OP_TRAIN_DENSE    6   /* sffn_forward_train_dense */
#define SFFN_OP_BACKWARD_DENSE 7   /* sffn_backward_dense */

typedef struct sffn_handle sffn_handle;

/*
 * Layer descriptor.
 *   d          model width; d % 64 == 0, bf16: d % 512 == 0 and d <= 4096,
 *              f32: d % 256 == 0 and d <= 2048 (SFFN_E_UNSUPPORTED otherwise)
 *   d_ff       F, the number of neurons; F % 128 == 0, F <= 65408 so a
 *              neuron id fits uint16
 *   gated      1 gated, 0 non-gated (w_up unused and must be NULL)
 *   tile       TwELL tile width W; 128 is the one supported width
 *   twell_cap  C, TwELL slots per (row, tile); 1 <= C <= 128
 *   ell_cap    K, the ELL capacity of the sparse path: a row with more
 *              than K active neurons, or with a TwELL tile holding more
 *              than C, takes the dense path (the Hybrid routing rule,
 *              "2. Methodology" A on the gist.science explainer). Training
 *              needs K >= 1. At inference K = 0 means n_t * C (only rows
 *              with an overflowing tile go dense); a K above n_t * C acts
 *              as n_t * C.
 *   dtype      SFFN_BF16 (bf16 inputs, fp32 accumulation) or SFFN_F32
 *              (fp32 inputs and fp32 arithmetic throughout)
 *   store_dtype  SFFN_F32 (0): the stored activations (TwELL values, ELL
 *              a and u, backup rows' a and u) are float32, the accumulator
 *              values. SFFN_BF16 (bf16 layers only): they are bf16, rounded
 *              once (to nearest, ties to even) where they are stored, which
 *              halves the format's value bytes; the layer then computes
 *              with the stored values, H = bf16(a) * bf16(u) (the dense
 *              path's rows too), and the backward reads them, so the
 *              roundings pass gradients unchanged.
 *   dense_above  mean active neurons per token (over the rows that stay
 *              sparse) above which sffn_choose_mode picks the dense layer;
 *              0 = the library's cost model of the two paths on MI355X
 *   updown     how the inference forward runs the up/down projection of
 *              the ELL rows: 0 (default) three launches with the model
 *              width cut into slices that each XCD's L2 holds (per-slice
 *              partial dot products, their sums h = a * u, the down
 *              projection); 1 (bf16 layers) one fused kernel without
 *              slices, u and y kept in registers (the single fused kernel
 *              of "2. Methodology" B on the gist.science explainer). The
 *              training forward always runs the sliced form.
 *   dense_rows R, the most rows one call computes on the dense path
 *              (rows routed away from the ELL at inference, backup rows in
 *              training); the workspace holds R dense rows. 0 means T
 *              (every row may go dense; the workspace then grows as T x F).
 *              More routed rows than R: see sffn_check.
 */
typedef struct sffn_desc {
  int32_t d;
  int32_t d_ff;
  int32_t gated;
  int32_t tile;
  int32_t twell_cap;
  int32_t ell_cap;
  int32_t dtype;
  int32_t dense_rows;
  int32_t store_dtype;
  float   dense_above;
  int32_t updown;
} sffn_desc;

/*
 * TwELL buffers (device, caller-owned). n_t = F / W.
 *   val       [T, n_t, C] float32   slot values, the gate pre-activation
 *                                   z[t, j] (> 0) as accumulated in fp32
 *                                   (bf16 bits, uint16, when
 *                                   desc.store_dtype is SFFN_BF16)
 *   idx       [T, n_t, C] uint16    slot neuron ids j (global)
 *                                   Slots s >= min(cnt, C) of a (row, tile)
 *                                   are not written and hold unspecified
 *                                   values.
 *   cnt       [T, n_t]    int32     true number of positives in the tile
 *                                   (not capped at C)
 *   row_flag  [T]         uint8     1 iff some tile of the row has cnt > C
 *   flagged   [T]         int32     the flagged rows in ascending order;
 *                                   the first *n_flagged entries are valid
 *   n_flagged [1]         int32     number of flagged rows
 * Rows whose tiles all fit (row_flag 0) are stored losslessly; a flagged
 * row keeps its first C slots per tile and the layer computes it densely.
 */
typedef struct sffn_twell {
  void*     val;
  uint16_t* idx;
  int32_t*  cnt;
  uint8_t*  row_flag;
  int32_t*  flagged;
  int32_t*  n_flagged;
} sffn_twell;

/*
 * Hybrid buffers (device, caller-owned): the training-side format of
 * "2. Methodology" A ("Hybrid Format for Training") on the gist.science
 * explainer and "2. The Hybrid Training Algorithm" on the wispaper blog.
 * A row goes to the dense backup iff its total count of positives exceeds
 * K (desc.ell_cap) or one of its TwELL tiles overflowed C; every other row
 * keeps its positives as ELL slots 0..ell_cnt-1 in ascending neuron order.
 *   ell_a      [T, K]   float32  a = z > 0 of each ELL slot
 *   ell_u      [T, K]   float32  u = x . W_u[j] of each ELL slot (gated
 *                                layers; written by sffn_forward_train)
 *              (ell_a, ell_u, bk_a and bk_u hold bf16 bits, uint16,
 *              when desc.store_dtype is SFFN_BF16)
 *   ell_idx    [T, K]   uint16   neuron ids
 *   ell_cnt    [T]      int32    slots used (0 for backup rows)
 *                                (slots >= ell_cnt are unspecified)
 *   slot       [T]      int32    backup slot of the row, -1 for ELL rows
 *   brow       [max_backup] int32  backup rows in ascending order
 *   n_backup   [1]      int32    true number of backup rows (may exceed
 *                                the capacity R' = min(max_backup,
 *                                desc.dense_rows): then the rows from
 *                                slot R' on were not computed and the
 *                                result is invalid; see sffn_hybrid_check)
 *   bk_a       [max_backup, F] float32  ReLU(z) rows of the backup rows
 *   bk_u       [max_backup, F] float32  u rows of the backup rows (gated)
 *   max_backup capacity of brow, bk_a and bk_u in rows
 */
typedef struct sffn_hybrid {
  void*     ell_a;
  void*     ell_u;
  uint16_t* ell_idx;
  int32_t*  ell_cnt;
  int32_t*  slot;
  int32_t*  brow;
  int32_t*  n_backup;
  void*     bk_a;
  void*     bk_u;
  int64_t   max_backup;
} sffn_hybrid;

/* Create a handle for the current HIP device. Validates the descriptor
 * (SFFN_E_ARG / SFFN_E_UNSUPPORTED) before touching the device; returns
 * SFFN_E_UNSUPPORTED when the current device is not gfx950 and SFFN_E_HIP
 * when no device can be queried. Allocates host memory and one block of
 * device memory of about 64 KiB (the handle's status word and counters,
 * zeroed here; freed by sffn_destroy). Per-kernel timing events and the
 * backward's second stream and its two events are created on demand, on
 * the device current at that call. Calls on the handle must be made with
 * the same device current. */
sffn_status sffn_create(const sffn_desc* desc, sffn_handle** out);

/* Destroy a handle (NULL is allowed). */
void sffn_destroy(sffn_handle* h);

/* Text of the last error recorded on the handle ("" if none). The string
 * lives until the next call on the handle. */
const char* sffn_last_error(const sffn_handle* h);

/* Static name of a status code. */
const char* sffn_status_string(sffn_status s);

/* Bytes of device workspace that operation op needs for T tokens. The
 * workspace is caller-allocated, at least 256-byte aligned, and its
 * contents need not be initialised. */
sffn_status sffn_workspace_bytes(const sffn_handle* h, int64_t T, int32_t op,
                                 size_t* bytes);

/* ReLU + TwELL pack of a given pre-activation tensor z [T, F] float32
 * (the format of "2. Methodology" A on the gist.science explainer, here as
 * a stand-alone kernel that reads z). Fills every field of *tw. The result
 * is a pure function of z (bit-exact, deterministic). */
sffn_status sffn_pack_twell(sffn_handle* h, const float* z, int64_t T,
                            const sffn_twell* tw, void* ws, size_t ws_bytes,
                            hipStream_t stream);

/* Gate pre-activations z = x W_g, [T, F] float32, computed by the same
 * MFMA main loop as the fused gate GEMM of sffn_forward (so packing this z
 * with sffn_pack_twell reproduces the forward's TwELL bit for bit). */
sffn_status sffn_gate_preact(sffn_handle* h, const void* x, const void* w_gate,
                             int64_t T, float* z, hipStream_t stream);

/*
 * Forward pass y [T, d] float32.
 *   mode SFFN_SPARSE: gate GEMM with ReLU + TwELL pack in its epilogue
 *     ("2. Methodology" B: gate projection), then the fused up/down
 *     projection over each unflagged row's active neurons (same section:
 *     fused up/down projection); flagged rows (a tile overflowed C) are
 *     computed by a dense path restricted to those rows, the dense backup
 *     of the Hybrid format used as a safety valve at inference. If tw is
 *     non-NULL the TwELL is written there, else into the workspace.
 *   mode SFFN_DENSE: the plain dense layer with the same kernels' GEMMs;
 *     for bf16 the hidden activations are rounded once to bf16 between the
 *     two GEMMs, as in a standard bf16 feedforward, and W_d is transposed
 *     into the workspace first (both operands of the down GEMM then read
 *     k-contiguous). tw must be NULL.
 * w_up must be NULL iff the layer is non-gated. The workspace must hold
 * sffn_workspace_bytes(op = SFFN_OP_FORWARD_SPARSE or _DENSE).
 * SPARSE: rows whose TwELL overflowed, or with more than K = desc.ell_cap
 * active neurons, take the dense path; when more than desc.dense_rows rows
 * do, the outputs of the dense path's rows are not valid (rows past the
 * capacity are not computed, and the saved pre-activations of overflowing
 * tiles may not all fit), the rows on the ELL path are unaffected, and the
 * next sffn_check returns SFFN_E_CAPACITY.
 */
sffn_status sffn_forward(sffn_handle* h, const void* x, const void* w_gate,
                         const void* w_up, const void* w_down, int64_t T,
                         float* y, const sffn_twell* tw, int32_t mode,
                         void* ws, size_t ws_bytes, hipStream_t stream);

/*
 * sffn_forward without a caller workspace, for callers that cannot
 * allocate device memory (code under HIP graph capture, tight serving
 * loops, harnesses that forbid hipMalloc). Same arguments, kernels and
 * results as sffn_forward; the workspace is instead a static device array
 * of the library (128 MiB on each GPU the library runs on, held until the
 * process ends). A call whose sffn_workspace_bytes exceeds 128 MiB
 * returns SFFN_E_ARG before anything is enqueued (at d = 2048, F = 5632,
 * C = 8, K = 64, dense_rows = 512 that is above T = 15815). The
 * call allocates nothing: no hipMalloc, hipFree or event creation
 * (per-kernel timing is skipped for it). The scratch array is shared by
 * every call on a GPU, from every handle: calls that overlap on one GPU
 * (on different streams) race, so the caller orders them. Its contents
 * need no initialisation.
 */
sffn_status sffn_forward_noalloc(sffn_handle* h, const void* x, const void* w_gate,
                                 const void* w_up, const void* w_down, int64_t T, float* y,
                                 const sffn_twell* tw, int32_t mode, hipStream_t stream);

/* TwELL -> Hybrid ("Hybrid Conversion", "2. Methodology" B on the
 * gist.science explainer): routes every row, fills ell_a, ell_idx, ell_cnt,
 * slot, brow and n_backup of *hy from *tw. When z [T, F] float32 is given,
 * the backup rows' bk_a rows are set to ReLU(z) (ell_u and bk_u are not
 * touched). The result is a pure function of the TwELL (and z). */
sffn_status sffn_hybrid_compact(sffn_handle* h, const sffn_twell* tw, const float* z,
                                int64_t T, const sffn_hybrid* hy, void* ws, size_t ws_bytes,
                                hipStream_t stream);

/* Training forward: y [T, d] float32 as sffn_forward(SFFN_SPARSE), and the
 * Hybrid of the step saved for sffn_backward: the TwELL of the gate GEMM
 * (into tw, or the workspace when tw is NULL) is converted with ELL
 * capacity K = desc.ell_cap (>= 1); ELL rows' up/down projections run over
 * their slots and save u per slot; backup rows run densely and save their
 * ReLU(z) and u rows in fp32 (backup rows on the matrix cores, sparse rows
 * on the vector units: "2. Methodology" B, training kernels). */
sffn_status sffn_forward_train(sffn_handle* h, const void* x, const void* w_gate,
                               const void* w_up, const void* w_down, int64_t T, float* y,
                               const sffn_twell* tw, const sffn_hybrid* hy, void* ws,
                               size_t ws_bytes, hipStream_t stream);

/*
 * Sparse backward over the Hybrid saved by sffn_forward_train ("2.
 * Methodology" B, training kernels: backpropagation, on the gist.science
 * explainer). With M = 1[z > 0]: dH = dy W_d^T (only where M = 1),
 * dU = dH * a, dZ = dH * u * M + l1_coeff * M (non-gated: dZ = dH * M +
 * l1_coeff * M); dx = dZ W_g^T + dU W_u^T; dW_g = x^T dZ, dW_u = x^T dU,
 * dW_d = (a * u)^T dy (non-gated: a^T dy). ELL rows run over their slots
 * (the slots are regrouped by neuron, in ascending row order, for dW);
 * backup rows run as dense GEMMs. Outputs are overwritten: dx [T, d],
 * dw_gate, dw_up (NULL iff non-gated), dw_down [F, d] neuron-major, all
 * float32; rows of never-active neurons are zero. dy has the descriptor's
 * dtype. The workspace holds min(T, desc.dense_rows) backup rows; rows
 * from slot min(max_backup, desc.dense_rows) on are not processed (the
 * training forward has then already flagged the overflow: see
 * sffn_hybrid_check and sffn_check). T = 0 stores zero weight gradients
 * (no workspace needed). With backup
 * rows the ELL rows' dx sums and the neuron-major regrouping run on the
 * handle's second stream, beside the backup rows' dW products, joined
 * before the dW sums.
 */
sffn_status sffn_backward(sffn_handle* h, const void* x, const void* w_gate, const void* w_up,
                          const void* w_down, const sffn_hybrid* hy, const void* dy, int64_t T,
                          float* dx, float* dw_gate, float* dw_up, float* dw_down, float l1_coeff,
                          void* ws, size_t ws_bytes, hipStream_t stream);

/* Per-layer choice between the sparse and the dense forward, made from
 * the layer's own TwELL (the pages attribute the speed-up to each layer's
 * activation sparsity, which differs from layer to layer: listing page,
 * Figure 6 and Figures 10-11; at 108 active per token the gain is small,
 * Table 5). Reads the counts and row flags of *tw (T rows, as a sparse
 * forward of the layer wrote them), synchronises the stream and sets *mode
 * to SFFN_DENSE when the mean active neurons per token over the rows whose
 * TwELL did not overflow exceeds the crossover (desc.dense_above, or when
 * that is 0 the library's cost model of the two paths on MI355X, which
 * also counts the overflowing rows' dense-path work), else SFFN_SPARSE.
 * mean_active and crossover (nullable) receive the two numbers. T = 0
 * gives SFFN_SPARSE. */
sffn_status sffn_choose_mode(sffn_handle* h, const sffn_twell* tw, int64_t T, int32_t* mode,
                             float* mean_active, float* crossover, hipStream_t stream);

/*
 * The same library's dense training step of the layer, the comparator of
 * the sparse step (sffn_forward_train + sffn_backward): a standard bf16
 * layer that keeps its hidden activations dense (listing page, Table 1:
 * training step of the dense models; gist.science explainer, "2.
 * Methodology" B for the layer and its backpropagation). bf16 layers only,
 * T a multiple of 64 (SFFN_E_UNSUPPORTED otherwise).
 * Forward: Z_s = bf16(x W_g), U_s = bf16(x W_u) (gated), H =
 * bf16(ReLU(Z_s) U_s) (non-gated: ReLU(Z_s)), y = H W_d (float32 [T, d]).
 * act (caller-owned, sffn_train_dense_act_bytes) receives Z_s [T, F], U_s
 * [T, F] (gated) and H [T, F], all bf16: the saved activations the
 * backward reads. The workspace is sffn_workspace_bytes(
 * SFFN_OP_TRAIN_DENSE) (W_d transposed, F x d bf16: both operands of the
 * down GEMM k-contiguous).
 */
sffn_status sffn_train_dense_act_bytes(const sffn_handle* h, int64_t T, size_t* bytes);
sffn_status sffn_forward_train_dense(sffn_handle* h, const void* x, const void* w_gate,
                                     const void* w_up, const void* w_down, int64_t T, float* y,
                                     void* act, void* ws, size_t ws_bytes, hipStream_t stream);
/* Backward of sffn_forward_train_dense from its act: with M = 1[Z_s > 0],
 * dH = dy W_d^T; dZ = bf16(dH U_s M + l1_coeff M) (non-gated: dH M +
 * l1_coeff M); dU = bf16(dH ReLU(Z_s)); dx = dZ W_g^T + dU W_u^T;
 * dW_g = x^T dZ, dW_u = x^T dU, dW_d = H^T dy. Outputs float32 and
 * overwritten, dW neuron-major [F, d] as in sffn_backward. The workspace is
 * sffn_workspace_bytes(SFFN_OP_BACKWARD_DENSE) (dH [T, F] fp32, dZ | dU
 * [T, 2F] and dZ, dU, H transposed, and W_g | W_u, x and dy transposed,
 * bf16). T = 0 stores zero weight gradients. */
sffn_status sffn_backward_dense(sffn_handle* h, const void* x, const void* w_gate,
                                const void* w_up, const void* w_down, const void* act,
                                const void* dy, int64_t T, float* dx, float* dw_gate,
                                float* dw_up, float* dw_down, float l1_coeff, void* ws,
                                size_t ws_bytes, hipStream_t stream);

/* Synchronise the stream and return SFFN_E_CAPACITY when *hy->n_backup
 * exceeds hy->max_backup or desc.dense_rows (when that is set), else
 * SFFN_OK (or SFFN_E_HIP). */
sffn_status sffn_hybrid_check(sffn_handle* h, const sffn_hybrid* hy, hipStream_t stream);

/* Synchronise the stream and report the first asynchronous error since
 * the last check (SFFN_E_HIP); else SFFN_E_CAPACITY when a call since the
 * last check routed more rows to the dense path than it could hold
 * (desc.dense_rows, or max_backup in training), so that some rows were not
 * computed; else SFFN_OK. The capacity report is cleared by the check. */
sffn_status sffn_check(sffn_handle* h, hipStream_t stream);

/*
 * Microscaled 4-bit floating point (MXFP4). A matrix of R rows and K
 * columns is kept with one power-of-two scale for every 32 consecutive
 * elements of a row; an element is the scale times a signed e2m1 value (0,
 * 0.5, 1, 1.5, 2, 3, 4 or 6). With Kp = K rounded up to 128:
 *   codes   [R, Kp / 2] bytes: element k of a row is in byte k / 2, the
 *           even element in the low nibble (bit 3 the sign); the elements
 *           from K on are 0
 *   scales  [Kp / 128, R, 4] bytes: byte b of (g, r) is the scale's
 *           exponent plus 127 for elements 128 g + 32 b .. + 31 of row r;
 *           255 makes those elements NaN. The bytes of blocks that lie
 *           from K on are 0: sffn_mx_quantize writes them so, and scales
 *           made elsewhere must have them so (a 255 there makes the row's
 *           products NaN)
 * sffn_mx_bytes gives the two sizes. The calls take no handle: they run on
 * the current device, on the caller's stream, allocate nothing and keep no
 * state, so calls on different streams may overlap. Sizes: R up to 2^27
 * (products: up to 2^21 rows in either operand), K up to 2^22; a size of 0
 * is valid (nothing is written; a product over K = 0 writes zeros). Codes
 * must be 16-byte and scales 4-byte aligned; float matrices need only their
 * elements' alignment.
 */
sffn_status sffn_mx_bytes(int64_t rows, int64_t cols, size_t* code_bytes, size_t* scale_bytes);

/* Quantise x (dtype SFFN_F32 or SFFN_BF16, [rows, cols], row stride ldx >=
 * cols elements). transposed = 0: codes and scales describe x, blocks along
 * its rows (R = rows, K = cols). transposed = 1: they describe x^T (R =
 * cols, K = rows): the form of a weight stored [F, d] whose product
 * contracts over F, such as w_down's. A block's exponent is that of its
 * largest magnitude less 2, at least -127; elements round to the nearest
 * value (ties to the even code) and saturate at 6. A block that holds an
 * infinity or a NaN becomes NaN as a whole. */
sffn_status sffn_mx_quantize(const void* x, int32_t dtype, int64_t rows, int64_t cols, int64_t ldx,
                             int32_t transposed, uint8_t* codes, uint8_t* scales,
                             hipStream_t stream);

/* The values the codes stand for, [rows, cols] of dtype (SFFN_F32 or
 * SFFN_BF16) with row stride ldo >= cols elements; exact. */
sffn_status sffn_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows,
                               int64_t cols, void* out, int32_t dtype, int64_t ldo,
                               hipStream_t stream);

/* out[m, n] = sum_k a[m, k] b[n, k] of two MXFP4 matrices with the same K:
 * a [M, K] (tokens), b [N, K] (an nn.Linear weight or any neuron-major
 * one). Products are exact, sums float32, out float32 or bf16 (out_dtype;
 * rounded once), [M, N] with row stride ldo >= N elements. Deterministic.
 * A float32 out with ldo = N = d_ff is what sffn_pack_twell takes as z. */
sffn_status sffn_mx_matmul(const uint8_t* a_codes, const uint8_t* a_scales, int64_t M,
                           const uint8_t* b_codes, const uint8_t* b_scales, int64_t N, int64_t K,
                           void* out, int32_t out_dtype, int64_t ldo, hipStream_t stream);

/*
 * Microscaled 8-bit floating point (MXFP8), the form of activations beside
 * 4-bit weights: as MXFP4, with one byte an element, a signed e4m3 value (up
 * to 448), codes [R, Kp] bytes, and the same scales. Sizes and alignments
 * are MXFP4's.
 */
sffn_status sffn_mx8_bytes(int64_t rows, int64_t cols, size_t* code_bytes, size_t* scale_bytes);

/* Quantise x as sffn_mx_quantize does (not transposed): a block's exponent
 * is that of its largest magnitude less 8, at least -127; elements round to
 * the nearest value (ties to the even code) and saturate at 448. */
sffn_status sffn_mx8_quantize(const void* x, int32_t dtype, int64_t rows, int64_t cols,
                              int64_t ldx, uint8_t* codes, uint8_t* scales, hipStream_t stream);

/* The values the codes stand for, as sffn_mx_dequantize. Exact as float32,
 * and as bf16 down to its subnormals. */
sffn_status sffn_mx8_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows,
                                int64_t cols, void* out, int32_t dtype, int64_t ldo,
                                hipStream_t stream);

/* sffn_mx_matmul for a in MXFP8 (tokens) and b in MXFP4 (weights). Products
 * are exact, sums float32. A NaN code of a (0x7F, 0xFF) makes its row NaN. */
sffn_status sffn_mx8_matmul(const uint8_t* a_codes, const uint8_t* a_scales, int64_t M,
                            const uint8_t* b_codes, const uint8_t* b_scales, int64_t N, int64_t K,
                            void* out, int32_t out_dtype, int64_t ldo, hipStream_t stream);

/*
 * What stands between two layers: the residual's addition and the
 * root-mean-square norm of the sum,
 *   s = x + residual (rounded to the residual's type),
 *   r = 1 / sqrt(mean(s^2) + eps),   y = s r w,
 * over rows of up to 16384 columns (SFFN_E_UNSUPPORTED above, and above 2^25
 * rows of up to 512 columns, 2^31 / n of more, n an eighth of the columns rounded
 * up to a power of two, at most 1024; the gradient's limit is 2^27 rows). The
 * result is formed in float32 where it is bf16 (whose range a row's squares may
 * leave), in 64 bits where it is float32 or MXFP8; the same call repeats bit for
 * bit, and a row's result does not depend on the other rows.
 * Every matrix is float32 or bf16 with contiguous rows, its own row stride
 * (>= cols elements) and no more than its elements' alignment.
 *   x             [rows, cols]
 *   residual      nullable: then s = x
 *   residual_out  [rows, cols] of residual_dtype: s (NULL iff residual is).
 *                 May be residual itself, or x; out may be x. In the place
 *                 of an operand a result has its type and, of more than one
 *                 row, its row stride; otherwise they have no byte in common
 *                 (SFFN_E_ARG), nor have the results.
 *   weight        w [cols], nullable: 1
 *   out           y: float32, bf16 (rounded once), or MXFP8 codes (16-byte
 *                 aligned; SFFN_MXFP8, ldo is not used) of the [rows, cols]
 *                 matrix, quantised from the float32 y
 *   out_scales    their scales (SFFN_MXFP8; else NULL)
 *   rstd          r [rows], nullable: the backward pass takes it (infinite
 *                 where r is above float32: a root mean square below 2^-128)
 */
typedef struct sffn_norm {
  const void* x;
  const void* residual;
  void* residual_out;
  const void* weight;
  void* out;
  uint8_t* out_scales;
  float* rstd;
  int64_t ldx;
  int64_t ldr;
  int64_t ldro;
  int64_t ldo;
  int32_t x_dtype;
  int32_t residual_dtype;
  int32_t weight_dtype;
  int32_t out_dtype;
} sffn_norm;

/* eps >= 0. n_rows (device int32, nullable): only the first *n_rows rows (at
 * most rows) count; results of the others are left as they were. No handle:
 * runs on the current device, on the stream, keeps no state. A size of 0 is
 * valid: nothing is written. */
sffn_status sffn_rms_norm(const sffn_norm* norm, int64_t rows, int64_t cols, float eps,
                          const int32_t* n_rows, hipStream_t stream);

/*
 * Its gradient: with xh = s r and g = dy w,
 *   ds      = r (g - xh mean(g xh)) + dstream,   the gradient of x and of
 *             residual alike
 *   dweight = sum over rows of dy xh
 * (the roundings of s and y count as the identity).
 *   dy, s    [rows, cols]; s is residual_out of the forward pass (x where
 *            there was no residual)
 *   dstream  nullable: the gradient that reaches s beside the norm's
 *   weight   nullable: 1
 *   rstd     [rows] float32 of the forward pass
 *   ds       [rows, cols], may be dy, s or dstream, then of the same type and,
 *            of more than one row, row stride; has no byte in common with any
 *            otherwise (SFFN_E_ARG)
 *   dweight  [cols] float32, nullable (NULL without a weight); written by
 *            rows == 0 too (zeros); not the weight's memory (SFFN_E_ARG), nor any
 *            other operand's
 * Sums are float32, of rows in an order that depends on the sizes alone. Every one
 * of the `rows` rows counts: after a forward pass with n_rows, whose s and rstd of
 * the other rows are left as they were, rows is that number.
 */
typedef struct sffn_norm_grad {
  const void* dy;
  const void* s;
  const void* dstream;
  const void* weight;
  const float* rstd;
  void* ds;
  float* dweight;
  int64_t lddy;
  int64_t lds;
  int64_t lddstream;
  int64_t ldds;
  int32_t dy_dtype;
  int32_t s_dtype;
  int32_t dstream_dtype;
  int32_t weight_dtype;
  int32_t ds_dtype;
} sffn_norm_grad;

/* The workspace (256-byte aligned; not shared by calls that overlap) is for
 * dweight and may be NULL without it, and where its size is 0 (small matrices). */
sffn_status sffn_rms_norm_backward_workspace_bytes(int64_t rows, int64_t cols, size_t* bytes);
sffn_status sffn_rms_norm_backward(const sffn_norm_grad* grad, int64_t rows, int64_t cols,
                                   void* ws, size_t ws_bytes, hipStream_t stream);

/*
 * The choice of a token's experts from the router's logits l [T, E]:
 *   scores   s = softmax(l) over the E experts, or (sigmoid = 1)
 *            s = 1 / (1 + exp(-l))
 *   c        s + bias, the bias [E] for balance (nullable)
 *   groups   of E / groups consecutive experts each; the score of one is the
 *            sum of its group_best (1 or 2) largest c, and only experts of the
 *            top_groups groups with the largest score are chosen from
 *   ids      the top_k experts with the largest c, in descending order (ties,
 *            of groups too: the lower index first)
 *   probs    scale s of the chosen experts, or (normalize = 1) scale s / (the
 *            sum of the chosen s); without the bias
 * Experts are compared in 64 bits, without a bias by their logits (which have
 * the scores' order). Logits may be -infinity (an expert that is masked, of
 * score 0, chosen only where nothing else is left); a token whose chosen
 * experts all have score 0 gets weights 0. A NaN or +infinity leaves a
 * token's indices valid and its weights unspecified, and other tokens alone.
 *   n_experts  E <= 1024, a multiple of groups
 *   top_k      k <= min(32, top_groups E / groups)
 *   groups     <= 64 (1: no groups); group_best <= E / groups
 *   scale      finite
 * (SFFN_E_ARG for sizes below 1, a bad flag or sizes that do not fit together,
 * SFFN_E_UNSUPPORTED beyond the limits.)
 */
typedef struct sffn_route_desc {
  int32_t n_experts;
  int32_t top_k;
  int32_t groups;
  int32_t top_groups;
  int32_t group_best;
  int32_t sigmoid;
  int32_t normalize;
  float scale;
} sffn_route_desc;

/* logits [T, E] of dtype with row stride ldl >= E, ids [T, k] int32, probs
 * [T, k] float32; T up to 2^25 (SFFN_E_UNSUPPORTED above). n_tokens as in
 * sffn_moe_forward. No handle, no workspace, no state. */
sffn_status sffn_route(const sffn_route_desc* desc, const void* logits, int32_t dtype, int64_t T,
                       int64_t ldl, const float* bias, const int32_t* n_tokens, int32_t* ids,
                       float* probs, hipStream_t stream);

/* The gradient of the logits [T, E] (dl_dtype, row stride lddl >= E, every
 * element written; it may be logits itself, of the same type and row stride, and
 * shares no byte with it otherwise: SFFN_E_ARG) from that of the weights, dprobs
 * [T, k] float32; the choice itself, and with it the bias, has none. logits and ids are the forward
 * pass's; an index outside 0 .. E - 1 counts as an expert that was not
 * chosen. */
sffn_status sffn_route_backward(const sffn_route_desc* desc, const float* dprobs,
                                const void* logits, int32_t dtype, int64_t T, int64_t ldl,
                                const int32_t* ids, const int32_t* n_tokens, void* dlogits,
                                int32_t dl_dtype, int64_t lddl, hipStream_t stream);

/*
 * A whole mixture-of-experts layer for few tokens (decoding batches). With
 * the router l = x W_r^T, the k = top_k experts e(0), e(1), .. of a token in
 * descending order of l (ties: the lower expert first) and p their softmax
 * weights,
 *   y = sum_r p_r (ReLU(x W_g,e(r)) * (x W_u,e(r))) W_d,e(r)     gated
 *   y = sum_r p_r ReLU(x W_1,e(r)) W_2,e(r)                      non-gated
 * Only the selected experts' weights are read, the up and down rows only of
 * neurons that are active (strictly z > 0, as everywhere here) for one of
 * the tokens. Logits are float64 sums in an order that depends on d alone, so
 * that a token's experts are the same in every call; the sums are exact
 * where the products of a logit (zeros aside) lie within a factor of 2^37 /
 * d of each other, and ties are those of the sums. Everything else is float32 (h
 * enters the down product with its 24 bits, in three bf16 parts). The same
 * call repeats bit for bit; a token's row may differ in its last bits when
 * the other tokens of the call are others.
 *   d          model width; d % 128 == 0, d <= 8192
 *   d_ff       F, neurons an expert; F % 32 == 0, F <= 65536
 *   n_experts  E <= 1024, E F <= 2^27
 *   top_k      k <= min(E, 32)
 *   gated      1 gated, 0 non-gated
 *   normalize  1: p is the softmax over the token's k experts; 0: over all
 *              E (the k weights then sum to less than 1)
 *   weights    SFFN_BF16 or SFFN_MXFP4 (of the experts; x and the router
 *              are bf16)
 * (SFFN_E_ARG for a size below 1 or a bad enum, SFFN_E_UNSUPPORTED outside
 * these ranges.)
 */
typedef struct sffn_moe_desc {
  int32_t d;
  int32_t d_ff;
  int32_t n_experts;
  int32_t top_k;
  int32_t gated;
  int32_t normalize;
  int32_t weights;
} sffn_moe_desc;

/*
 * Weights of an expert layer (device).
 *   router          [E, d] bf16
 *   gate, up, down  [E, F, d], row j of an expert belongs to neuron j (as
 *                   in the layer): bf16, or the codes of the [E F, d]
 *                   matrix (blocks along d) as sffn_mx_quantize makes them.
 *                   up is NULL iff non-gated; non-gated layers pass W_1 as
 *                   gate and W_2 as down.
 *   *_scales        the scales of those codes (SFFN_MXFP4; else NULL)
 * All 16-byte aligned (scales 4). Non-finite weights make the results of
 * every token of their expert unspecified.
 */
typedef struct sffn_moe_weights {
  const void* router;
  const void* gate;
  const void* up;
  const void* down;
  const uint8_t* gate_scales;
  const uint8_t* up_scales;
  const uint8_t* down_scales;
} sffn_moe_weights;

/* Most tokens of one call. */
#define SFFN_MOE_MAX_TOKENS 256

/* Bytes of workspace for T tokens (256-byte aligned, contents need no
 * initialisation, not shared by calls that overlap). */
sffn_status sffn_moe_workspace_bytes(const sffn_moe_desc* desc, int64_t T, size_t* bytes);

/* The layer's forward: x [T, d] bf16, y [T, d] float32, T <=
 * SFFN_MOE_MAX_TOKENS (SFFN_E_UNSUPPORTED above). ids [T, k] int32 and
 * probs [T, k] float32 (each nullable) receive the experts and their
 * weights by rank. n_tokens (device int32, nullable): only the first
 * *n_tokens rows (at most T) are tokens; the others are not read and their
 * rows of y, ids and probs are left as they were, so one captured graph
 * serves smaller batches. A NaN in a token's x makes its row NaN and no
 * other. No handle: runs on the current device, on the stream, keeps no
 * state. */
sffn_status sffn_moe_forward(const sffn_moe_desc* desc, const void* x, const sffn_moe_weights* w,
                             int64_t T, const int32_t* n_tokens, float* y, int32_t* ids,
                             float* probs, void* ws, size_t ws_bytes, hipStream_t stream);

/* The layer with experts that the caller has chosen (sffn_route, or any
 * other way) in place of its router's: y = sum_r probs_r expert_{ids_r}(x).
 * ids [T, k] int32, probs [T, k] float32 (any values); w->router must be NULL,
 * and desc.normalize is not used. An index outside 0 .. E - 1 adds nothing (a
 * pair that was dropped, or another rank's); one that a token has twice
 * counts with both weights. Workspace and the rest as in sffn_moe_forward. */
sffn_status sffn_moe_forward_chosen(const sffn_moe_desc* desc, const void* x,
                                    const sffn_moe_weights* w, int64_t T, const int32_t* n_tokens,
                                    const int32_t* ids, const float* probs, float* y, void* ws,
                                    size_t ws_bytes, hipStream_t stream);

/*
 * Per-kernel timing. While enabled, every kernel launch of the handle's
 * calls is bracketed by two HIP events recorded on the call's stream, so that each
 * interval holds one kernel id's launches alone. sffn_profile_read waits
 * for the recorded events, writes for each kernel id k < n the summed
 * milliseconds and the
 * number of launches since the last read (or since enabling), and resets
 * the sums. Disabling drops pending records. Kernel ids:
 */
#define SFFN_K_GATE_TWELL    0  /* gate GEMM with the ReLU + TwELL epilogue */
#define SFFN_K_FLAGS         1  /* overflow flags and flagged-row list */
#define SFFN_K_SPARSE_UP     2  /* sparse up projection: per-slice partial dots */
#define SFFN_K_FLAG_GATEUP   3  /* hidden rows of the dense path: bf16 up GEMM + combine
                                    from the gate's own outputs, fp32 gate/up GEMM + combine */
#define SFFN_K_FLAG_DOWN     4  /* down GEMM of the flagged rows (split-K) */
#define SFFN_K_SPLITK_REDUCE 5  /* split-K reduction into the flagged rows */
#define SFFN_K_DENSE_GATEUP  6  /* dense mode: gate/up GEMM */
#define SFFN_K_DENSE_DOWN    7  /* dense mode: down GEMM */
#define SFFN_K_PACK          8  /* stand-alone TwELL pack */
#define SFFN_K_GATE_PREACT   9  /* gate GEMM writing z */
#define SFFN_K_ROWS         10  /* per-row route + ELL compaction of the TwELL */
#define SFFN_K_SPARSE_DOWN  11  /* sparse down projection into y */
#define SFFN_K_BWD_SDDMM    12  /* backward: dy . W_d[j] per ELL slot (partial dots) */
#define SFFN_K_BWD_DX       13  /* backward: dZ, dU per slot and dx of ELL rows */
#define SFFN_K_BWD_TRANSPOSE 14 /* backward: ELL slots grouped by neuron */
#define SFFN_K_BWD_DW       15  /* backward: dW rows from the ELL slots */
#define SFFN_K_BWD_DENSE    16  /* backward: the backup rows' dense GEMMs */
#define SFFN_K_SPARSE_HSUM  17  /* sparse up projection: slice partials summed, h = a * u */
#define SFFN_K_TRAIN_DENSE_GATEUP 18  /* dense training step: gate/up GEMM saving Z, U, H^T */
#define SFFN_K_TRAIN_DENSE_DOWN   19  /* dense training step: down GEMM */
#define SFFN_K_BWD_DENSE_DH       20  /* dense backward: dH GEMM forming dZ, dU */
#define SFFN_K_BWD_DENSE_DX       21  /* dense backward: dx GEMMs */
#define SFFN_K_BWD_DENSE_DW       22  /* dense backward: dW GEMMs */
#define SFFN_K_FUSED_UPDOWN       23  /* inference up/down in one kernel (desc.updown = 1) */
#define SFFN_K_COUNT        24
sffn_status sffn_profile_enable(sffn_handle* h, int32_t enable);
sffn_status sffn_profile_read(sffn_handle* h, double* total_ms, int32_t* launches, int32_t n);
/* Static name of a kernel id ("" if out of range). */
const char* sffn_kernel_name(int32_t k);

#ifdef __cplusplus
}
#endif

#endif /* SFFN_H */
