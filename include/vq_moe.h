/*
 * vq_moe.h -- C ABI of the VQ-MoE expert-path library (libvqmoe.so).
 *
 * The library computes the hot path of vector-quantised (VQ) MoE checkpoints
 * on one NVIDIA B200 (sm_100a): expert weights are stored as packed
 * log2(K)-bit indices into a per-module codebook of K fp16 centroids of
 * d weights each, with one fp16 scale per (row, 64 weights), and dead
 * "skipzero" rows dropped. The kernels reconstruct the weights on the fly and
 * contract them with the activations of the tokens routed to each expert.
 *
 * Format (VQ model cards):
 *   - Qwen3.5-397B-A17B-VQ-2.6bpw card, "Methodology": one index per
 *     d-weight subvector into a per-tensor fp16 codebook, fp16 scale per
 *     (row, 64 weights).
 *   - Qwen3.5-397B-A17B-VQ-2.4bpw card, "Methodology": codes packed into
 *     uint32 words, row-local, 32-code blocks. The bit order inside a block
 *     is not printed; this library reads it as: code j of a row occupies
 *     bits [j*b, j*b+b) of the row's bit string, bit i of the string being
 *     bit (i % 32) of word i / 32 (least significant bit first).
 *   - same card, "Changelog 2026-10-01 (vq-skipzero)": dead output rows
 *     carry no codes or scales and output exact zeros.
 *
 * Conventions for every call:
 *   - Pointers marked "device" are CUDA device pointers the caller owns; the
 *     library never allocates, frees or retains them after the call returns.
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *     stream). Device calls are asynchronous on that stream and never
 *     synchronise the host; their results are valid once the stream has run.
 *   - The return value reports argument errors and launch failures
 *     synchronously. Nothing is launched when a call returns an error.
 *   - fp16 and bf16 values are passed as their uint16 bit patterns.
 */
#ifndef VQ_MOE_H
#define VQ_MOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum vq_status {
    VQ_OK = 0,
    VQ_ERR_ARG = 1,           /* NULL where a pointer is required, bad size or shape */
    VQ_ERR_ALIGN = 2,         /* a pointer is not aligned as documented */
    VQ_ERR_UNSUPPORTED = 3,   /* geometry (d, bits) or size the kernels do not implement */
    VQ_ERR_WORKSPACE = 4,     /* workspace NULL, misaligned or smaller than required */
    VQ_ERR_CUDA = 5,          /* a CUDA runtime call or kernel launch failed */
    VQ_ERR_DEVICE_CHECK = 6   /* a kernel recorded an error: it gave up a bounded wait, or
                                 vq_fit met an index out of range (see vq_moe_check) */
} vq_status;

/* Output element types. */
enum { VQ_F32 = 0, VQ_BF16 = 1 };

/*
 * One VQ module: the weights of one (layer, projection) for E experts that
 * share one codebook (reading of "per-tensor codebook": one codebook per
 * projection of a layer, shared by all of that layer's experts).
 *
 * Expert e's weight matrix is W_e [rows, cols] with
 *   W_e[r, c] = fp32(codebook[code_e(r, c / d)][c % d]) * fp32(scale_e[r, c / 64])
 *               (+ fp32(bias_e[r, c / 64]) for a module with biases)
 * where code_e(r, j) is the j-th b-bit code of row r. The bias is the
 * optional affine arm: the cards' fallback format "affine 3-bit, group 64"
 * (Qwen3.5-397B-A17B-VQ-2.4bpw card, Changelog 2026-09-20) is stated without
 * its formula; this library reads it as the group-wise affine form
 * w = s * q + b with an fp16 scale and an fp16 bias per (row, 64 weights),
 * which is d = 1 with the codebook C[q] = q plus the bias.
 *
 * Requirements: d in {1, 2, 4, 8}; cols a multiple of 64 and of 32*d (whole
 * 32-code blocks and whole scale groups); (d, bits) one of the implemented
 * geometries (vq_geometry_supported).
 */
typedef struct vq_module {
    int32_t E;        /* experts */
    int32_t rows;     /* output features of each expert */
    int32_t cols;     /* input features of each expert */
    int32_t d;        /* weights per code (subvector length) */
    int32_t bits;     /* code width b; the codebook has K = 2^bits entries */
    /* device, 16-byte aligned: packed codes of the live rows, expert-major,
     * live rows of one expert in increasing row order; each row is
     * vq_packed_words(1, cols / d, bits) uint32 words. */
    const uint32_t *codes;
    /* device, 2-byte aligned: fp16 scales [live rows, cols / 64], same row order. */
    const uint16_t *scales;
    /* device, 16-byte aligned: fp16 codebook [2^bits, d]. */
    const uint16_t *codebook;
    /* device or NULL: live-row bitmap [E, ceil(rows / 32)]; bit (r % 32) of
     * word r / 32 is 1 when row r of the expert is live. NULL: every row of
     * every expert is live and expert e's row r is packed row e*rows + r. */
    const uint32_t *live_bitmap;
    /* device, required when live_bitmap is set: [E, ceil(rows / 32)], the
     * packed-row index of the first live row at or after row 32*w of expert
     * e (vq_live_rank builds it). */
    const uint32_t *live_rank;
    /* number of packed rows in `codes` and `scales` (the extent the kernels
     * may read); required when live_bitmap is set, ignored (E * rows)
     * otherwise. */
    int64_t live_rows;
    /* device, 2-byte aligned, or NULL (no bias): fp16 biases [live rows,
     * cols / 64], the same layout as `scales`. */
    const uint16_t *biases;
} vq_module;

/* A SwiGLU MoE layer: y = sum_j w_j * down_e( silu(gate_e x) * up_e x ).
 * gate and up: rows = inter, cols = hidden; down: rows = hidden, cols = inter;
 * all three with the same E. Each has its own codebook and geometry. */
typedef struct vq_moe_layer {
    vq_module gate;
    vq_module up;
    vq_module down;
} vq_moe_layer;

/* Human-readable name of a status. Never NULL. */
const char *vq_status_str(vq_status s);

/* 1 when the kernels implement geometry (d, bits), else 0. */
int vq_geometry_supported(int32_t d, int32_t bits);

/* ------------------------------------------------------------ host packing */

/* uint32 words of `rows` packed rows of `ncode` codes of `bits` bits:
 * rows * (ncode / 32) * bits (a 32-code block is exactly `bits` words).
 * Returns 0 when ncode is not a positive multiple of 32 or bits not in 1..16. */
size_t vq_packed_words(int64_t rows, int32_t ncode, int32_t bits);

/* Host. Packs codes [E, rows, ncode] (uint16, values < 2^bits) into the
 * row-local LSB-first layout, keeping only live rows when live_bitmap (host,
 * [E, ceil(rows/32)]) is given (skipzero: live rows are byte-identical to a
 * full packing). out: host, out_words >= vq_packed_words(live rows, ncode,
 * bits). *rows_written receives the number of packed rows.
 * Errors: VQ_ERR_ARG (NULL, bad sizes, a code >= 2^bits, out too small). */
vq_status vq_pack(const uint16_t *codes, int32_t E, int32_t rows, int32_t ncode, int32_t bits,
                  const uint32_t *live_bitmap, uint32_t *out, size_t out_words, size_t *rows_written);

/* Host. Keeps the live rows of per-row fp16 scales [E, rows, ngroups]
 * (ngroups = cols / 64) in the same order as vq_pack. */
vq_status vq_pack_scales(const uint16_t *scales, int32_t E, int32_t rows, int32_t ngroups,
                         const uint32_t *live_bitmap, uint16_t *out, size_t out_elems,
                         size_t *rows_written);

/* Host. Builds live_rank [E, ceil(rows/32)] from a live bitmap (both host).
 * Bits at or beyond `rows` in the last word of an expert must be 0. */
vq_status vq_live_rank(const uint32_t *live_bitmap, int32_t E, int32_t rows, uint32_t *rank_out);

/* ------------------------------------------------------------ device calls */

/* Diagnostic. codes_out: device uint16 [rows, cols/d]: the codes of expert
 * `expert`'s rows; dead rows are filled with 0xFFFF. */
vq_status vq_unpack(const vq_module *m, int32_t expert, uint16_t *codes_out, void *stream);

/* Diagnostic. w_out: device fp32 [rows, cols]: the dequantised weights of
 * `expert` (exact: the fp16 x fp16 product is exact in fp32); dead rows +0. */
vq_status vq_dequant(const vq_module *m, int32_t expert, float *w_out, void *stream);

/* y[t, r] = sum_c W_expert[r, c] * x[t, c] for t < T, accumulated in fp32.
 * x: device bf16 [T, cols], 16-byte aligned. y: device [T, rows] of y_dtype
 * (VQ_F32 or VQ_BF16, round to nearest even). Dead rows give +0.
 * The contraction runs on tensor cores (the decode GEMV) with the codebook
 * entries and the activations in fp16. Every 64-column group of a token's
 * activations is multiplied by a power of two 2^k that puts its largest |x|
 * in [2^14, 2^15) before the fp16 rounding, so any finite bf16 input keeps
 * fp16's full precision (down to 2^-28 of the group's largest value) and
 * nothing overflows; the group's fp32 partial sum is multiplied by its fp32
 * scale and by 2^-k (exact). Results are accurate wherever y is a normal fp32
 * number. */
vq_status vq_gemv(const vq_module *m, int32_t expert, const uint16_t *x, int32_t T, void *y,
                  int32_t y_dtype, void *stream);

/* Bytes of workspace vq_gemm needs for T tokens of module m's shape; 0 on
 * invalid arguments. */
size_t vq_gemm_workspace_size(const vq_module *m, int32_t T);

/* The prefill path's tcgen05 GEMM for one expert (a dense building block with
 * the same arithmetic as vq_moe_prefill's expert GEMMs): for t < T,
 *   y0[t, r] = sum_c W0_expert[r, c] * x[t, c]     (module m0)
 *   y1[t, r] = sum_c W1_expert[r, c] * x[t, c]     (module m1, when not NULL)
 * m1, when given, must have m0's E, rows, cols, d and bits: the two share
 * each weight-tile pass, as a layer's gate and up projections do. The weight
 * tiles are decoded on chip to fp16 (fp16(centroid) x fp16(group scale),
 * rounded to nearest even) and contracted with the tokens' activations in
 * fp16 on the tensor cores, accumulated in fp32. Each token's activations are
 * multiplied by 2^k (largest |x| in [2^14, 2^15)) before their fp16 rounding
 * and the fp32 result by 2^-k. x: device bf16 [T, cols], 16-byte aligned.
 * y0, y1: device fp32 [T, rows], 16-byte aligned. workspace: device,
 * 256-byte aligned, vq_gemm_workspace_size(m0, T) bytes (its first word is the
 * error word that vq_moe_check reads). Requirements as vq_moe_prefill's for
 * each module (VQ_ERR_UNSUPPORTED otherwise). Errors: VQ_ERR_ARG (bad sizes,
 * expert out of range, m1 of another shape), VQ_ERR_ALIGN, VQ_ERR_WORKSPACE. */
vq_status vq_gemm(const vq_module *m0, const vq_module *m1, int32_t expert, const uint16_t *x, int32_t T,
                  float *y0, float *y1, void *workspace, size_t ws_bytes, void *stream);

/* Top-k routing and expert bucketing of T tokens: the MoE router of the VQ
 * model cards' layers (Qwen3.8-Flash-Next-VQ-4.4bpw card: 10 of 512 experts
 * per token; gemma-4-26b-a4b-it-VQ-6.2bpw card: 128 experts, top 8). The
 * cards print no tie or normalisation rule; the readings taken here follow.
 * logits: device fp32 [T, E]. Per token the top_k experts are taken in order
 * of larger logit first, ties to the smaller expert index, NaN last.
 * weights: renorm != 0 -> softmax over the selected logits; renorm == 0 ->
 * the full softmax over all E experts, evaluated at the selected ones.
 * Outputs (device): ids int32 [T, top_k]; weights fp32 [T, top_k];
 * offsets int32 [E + 1] (exclusive prefix sums of per-expert pair counts);
 * perm int32 [T * top_k]: pair indices p = t*top_k + j grouped by expert,
 * increasing p inside each expert's bucket.
 * Requires 1 <= top_k <= min(E, 32), E <= 4096, T * top_k < 2^31. */
vq_status vq_route(const float *logits, int32_t T, int32_t E, int32_t top_k, int32_t renorm,
                   int32_t *ids, float *weights, int32_t *offsets, int32_t *perm, void *stream);

/* Which MoE path a workspace is sized for. */
enum { VQ_MODE_DECODE = 0, VQ_MODE_PREFILL = 1 };

/* Bytes of workspace vq_moe_decode (mode VQ_MODE_DECODE) or vq_moe_prefill
 * (VQ_MODE_PREFILL) need for T tokens and top_k. 0 on invalid arguments. */
size_t vq_moe_workspace_size(const vq_moe_layer *L, int32_t T, int32_t top_k, int32_t mode);

/* MoE SwiGLU layer for decode-sized batches (a few tokens per expert). T = 0
 * launches nothing and returns VQ_OK; x, logits and y may then be NULL:
 *   y[t] = sum_j w[t, j] * W_down,e_j ( silu(W_gate,e_j x[t]) * (W_up,e_j x[t]) )
 * with (e_j, w[t, j]) from vq_route on `logits` (device fp32 [T, E]).
 * Range: the tensor cores take 16-bit fp16 operands, so each token's
 * activation row, and each (token, expert) row of the SwiGLU output h, is
 * multiplied by a power of two that puts its largest magnitude in
 * [2^14, 2^15) before its fp16 rounding; the fp32 results are multiplied back
 * exactly. Any finite bf16 input is therefore taken at fp16's full precision
 * (down to 2^-28 of its row's largest value) without overflow; g, u, h and y
 * are fp32, and results are accurate wherever those are normal fp32 numbers.
 * x: device bf16 [T, hidden], 16-byte aligned. y: device [T, hidden] of
 * y_dtype, 16-byte aligned. workspace: device, 256-byte aligned, at least
 * vq_moe_workspace_size(L, T, top_k, VQ_MODE_DECODE) bytes; it holds the
 * routing tables and the intermediate activations and may be reused by the
 * next call once this one has run. Sums over experts run in slot order j,
 * so results are deterministic. */
vq_status vq_moe_decode(const vq_moe_layer *L, const uint16_t *x, int32_t T, const float *logits,
                        int32_t top_k, int32_t renorm, void *y, int32_t y_dtype, void *workspace,
                        size_t ws_bytes, void *stream);

/* The same layer for prefill-sized batches (many tokens per expert): per
 * expert bucket a grouped GEMM on the tcgen05 tensor cores with the weight
 * tiles decoded on chip to fp16 (fp16(centroid) x fp16(group scale), rounded
 * to nearest even). Same arguments, result definition and range handling as
 * vq_moe_decode; workspace sized with VQ_MODE_PREFILL. Additionally requires,
 * for every module, a packed row that is a multiple of 16 bytes
 * ((cols / d / 32) * bits divisible by 4) and cols a multiple of 64 * CH,
 * CH being the smallest number of 64-column steps whose codes fill a whole
 * number of 16-byte units (VQ_ERR_UNSUPPORTED otherwise). */
vq_status vq_moe_prefill(const vq_moe_layer *L, const uint16_t *x, int32_t T, const float *logits,
                         int32_t top_k, int32_t renorm, void *y, int32_t y_dtype, void *workspace,
                         size_t ws_bytes, void *stream);

/* Prefill of a long prompt in chunks, so that scratch memory is bounded by
 * the chunk rather than the prompt (the Qwen3.8-Flash-Next-VQ-4.4bpw card
 * chunks its speculative prefill in 2048 tokens, and the GLM-5.3-Flash-VQ-2.7bpw
 * card tells serving loops to chunk the prefill at 2048). Tokens [c0, c0 + chunk) of x and logits
 * go through vq_moe_prefill into rows [c0, c0 + chunk) of y, one chunk after
 * another on `stream`; the last chunk takes the remaining tokens. Each
 * token's output depends only on its own x row and logits, so the result is
 * vq_moe_prefill's over all T tokens. The workspace is sized for one chunk:
 * vq_moe_workspace_size(L, min(T, chunk), top_k, VQ_MODE_PREFILL) bytes, and
 * is reused by every chunk. chunk < 1 returns VQ_ERR_ARG; other errors as
 * vq_moe_prefill (a chunk that fails stops the loop; earlier chunks stay
 * queued). */
vq_status vq_moe_prefill_chunked(const vq_moe_layer *L, const uint16_t *x, int32_t T, const float *logits,
                                 int32_t top_k, int32_t renorm, int32_t chunk, void *y, int32_t y_dtype,
                                 void *workspace, size_t ws_bytes, void *stream);

/* ---- Data-free VQ fit: the step that makes a module's codebook, codes and
 * scales from a bf16 weight tensor ----
 * The VQ model cards ("Methodology" of Qwen3.5-397B-A17B-VQ-2.6bpw,
 * Qwen3.8-Flash-Next-VQ-4.4bpw, GLM-5.3-Flash-VQ-2.7bpw) fit each tensor's codebook
 * in pure weight space: k-means / Lloyd over the weight subvectors of a drawn
 * subsample, no Hessian, activation statistics or calibration data; an fp16
 * scale per (row, 64 weights). For one tensor W (bf16, row-major
 * [rows, cols]; subvector i = row i / (cols/d), weights d*(i % (cols/d)) ..)
 * vq_fit computes:
 *   scales   fp16 [rows, cols/64]: the group's largest |w| (the cards give the
 *            scale's shape only; this is the reading taken),
 *   v        = w / scale per subvector, fp32 (0 where the scale is 0),
 *   `iters`  Lloyd steps over the subvectors sample[0..n_sample) from the
 *            centroids v[init[k]]: each point goes to its nearest centroid
 *            (fp32 squared distance, components summed in order with no fused
 *            multiply-add, ties to the lower index); a centroid with points
 *            becomes their exact mean rounded to fp32, one with none keeps its
 *            value,
 *   codebook fp16 [K, d]: the final centroids rounded to fp16,
 *   codes    uint16 [rows, cols/d]: every subvector's nearest codebook entry.
 * Pack codes with vq_pack for the expert path. All arrays are device memory;
 * sample and init hold subvector indices drawn by the caller. Requirements:
 * d in {1, 2, 4, 8}; cols a multiple of 64; 2 <= K <= 65536 and K*d <= 32768
 * (the centroids sit in shared memory); K <= n_sample <= 2^22; iters >= 0;
 * rows*cols/d < 2^31 (VQ_ERR_ARG otherwise); w, scales, codebook and codes
 * 16-byte aligned (VQ_ERR_ALIGN). An index outside [0, rows*cols/d) is
 * skipped and sets the workspace's error word (see vq_moe_check). Results are
 * deterministic: centroid sums are exact integers. Workspace:
 * vq_fit_workspace_size(K, d) bytes (0 for invalid K or d), 256-byte aligned,
 * owned by the caller. Asynchronous on `stream`. */
size_t vq_fit_workspace_size(int32_t K, int32_t d);
vq_status vq_fit(const uint16_t *w, int32_t rows, int32_t cols, int32_t d, int32_t K, const int32_t *sample,
                 int32_t n_sample, const int32_t *init, int32_t iters, uint16_t *scales, uint16_t *codebook,
                 uint16_t *codes, void *workspace, size_t ws_bytes, void *stream);

/* ---- The block around the experts ----
 * A MoE block is more than its routed experts: a norm makes x from the residual stream, the router's load has to
 * stay balanced when it is trained, dense 4-bit projections (a shared expert) run beside the experts, and the
 * block's output is normed, gated, scaled and added back. The calls below are those row-wise and dense parts. They
 * follow the conventions above; T = 0 launches nothing and returns VQ_OK (row pointers may then be NULL). */

/* A root-mean-square norm over rows of `hidden` elements: n(v)[c] = v[c] * rsqrt(mean(v^2) + eps) * (weight[c] +
 * weight_offset). weight: device [hidden] of weight_dtype (VQ_F32 or VQ_BF16); weight_offset is 1 for checkpoints
 * that store weight - 1, else 0. eps >= 0, finite. Sums of squares are fp32: a row whose sum of squares leaves
 * fp32's range gives what fp32 arithmetic gives (0 or NaN). An Inf or NaN stays in its own row. */
typedef struct vq_norm {
    int32_t hidden;
    int32_t weight_dtype;
    const void *weight;
    float eps;
    float weight_offset;
} vq_norm;

/* Row arrays of the norm calls: a device pointer, an element type (VQ_F32 or VQ_BF16) where both are taken, and
 * `ld`, the elements from one row to the next (>= hidden; any value when T = 1). Pointers are aligned to their
 * element; rows on 16-byte boundaries (pointers, and ld * element size) with hidden a multiple of 8 take the
 * vector kernels, others the scalar ones (same results up to the order of the row sums). hidden is 1 to 16384
 * (VQ_ERR_UNSUPPORTED beyond). Outputs must not overlap inputs unless said. Gradients of bf16 arrays are bf16;
 * weight gradients are fp32 [hidden]. All row arithmetic is fp32, each output rounded once. */

/* The norm that makes a block's input: x[t] = bf16(n(h[t])). h: [T, hidden] of h_dtype; x: bf16 [T, hidden]. */
vq_status vq_norm_pre(const vq_norm *n, const void *h, int32_t h_dtype, int64_t h_ld, int32_t T, uint16_t *x,
                      int64_t x_ld, void *stream);

/* Bytes of workspace the two norm backward calls need for T rows of `hidden`: 0 for one row (workspace may be NULL),
 * and on invalid sizes. */
size_t vq_norm_workspace_size(int32_t hidden, int32_t T);

/* Gradient of vq_norm_pre. dx: bf16 [T, hidden]; dres: NULL, or [T, hidden] of h_dtype, a gradient that reaches h
 * past the norm (the residual path) and is added. With r = rsqrt(mean(h^2) + eps) and g = (weight + offset) dx:
 *   dh = r g - r^3 h mean(g h) + dres        (h_dtype; may be dres itself, same ld)
 *   dweight = sum_t dx h r                   (fp32 [hidden], or NULL: not computed)
 * The sum over rows runs in a fixed order: equal calls give equal bits. T = 0 writes dweight = 0. workspace:
 * 256-byte aligned, vq_norm_workspace_size bytes; needed (VQ_ERR_WORKSPACE) only with dweight and more than one row.
 * Calls that may overlap on the GPU need workspaces of their own. */
vq_status vq_norm_pre_backward(const vq_norm *n, const void *h, int32_t h_dtype, int64_t h_ld, const uint16_t *dx,
                               int64_t dx_ld, const void *dres, int64_t dres_ld, int32_t T, void *dh, int64_t dh_ld,
                               float *dweight, void *workspace, size_t ws_bytes, void *stream);

/* A block's output joined to the residual stream, and the next block's norm, in one pass:
 *   u = n_post(y[t])                                (post NULL: u = y[t])
 *   h_out[t] = res_scale * h[t] + out_scale * sigmoid(gate[t]) * u       (gate NULL: factor 1)
 *   x_out[t] = bf16(n_next(h_out[t]))               (next NULL: not computed; of h_out as stored)
 * y: [T, hidden] of y_dtype (a layer's output). gate: logits of gate_dtype, gate_cols = 1 (one per token, element t *
 * gate_ld) or gate_cols = hidden (one per channel). h and h_out: h_dtype; h_out may be h itself (same ld). post and
 * next must have the same hidden as given. */
vq_status vq_norm_post(const vq_norm *post, const vq_norm *next, int32_t hidden, const void *y, int32_t y_dtype,
                       int64_t y_ld, const void *gate, int32_t gate_dtype, int32_t gate_cols, int64_t gate_ld,
                       const void *h, int32_t h_dtype, int64_t h_ld, float res_scale, float out_scale, int32_t T,
                       void *h_out, int64_t h_out_ld, uint16_t *x_out, int64_t x_out_ld, void *stream);

/* Gradient of vq_norm_post from y, gate and the stored h_out (needed with next, else may be NULL). dh_out: [T, hidden]
 * of h_dtype, or NULL (0): the gradient that reaches h_out past the next norm; dx_out: bf16, required with next, else
 * NULL. With dH = dh_out + (n_next's gradient of dx_out at h_out), s = sigmoid(gate), dv = out_scale * dH:
 *   dh = res_scale * dH                                   (h_dtype; may be dh_out itself, same ld; NULL: not wanted)
 *   dy = n_post's gradient of s * dv at y                 (y_dtype)
 *   dgate = s (1 - s) * dv * u, summed over the row when gate_cols = 1  (gate_dtype; NULL: not wanted)
 *   dpost = sum_t s dv y r_post,  dnext = sum_t dx_out h_out r_next     (fp32 [hidden]; each NULL: not wanted)
 * The rounding of h_out is taken as the identity. T = 0 writes zero weight gradients. workspace as in
 * vq_norm_pre_backward, needed only with dpost or dnext. */
vq_status vq_norm_post_backward(const vq_norm *post, const vq_norm *next, int32_t hidden, const void *y,
                                int32_t y_dtype, int64_t y_ld, const void *gate, int32_t gate_dtype, int32_t gate_cols,
                                int64_t gate_ld, const void *h_out, int32_t h_dtype, int64_t h_out_ld, float res_scale,
                                float out_scale, int32_t T, const void *dh_out, int64_t dh_out_ld,
                                const uint16_t *dx_out, int64_t dx_out_ld, void *dy, int64_t dy_ld, void *dgate,
                                int64_t dgate_ld, void *dh, int64_t dh_ld, float *dpost, float *dnext, void *workspace,
                                size_t ws_bytes, void *stream);

/* Bytes of workspace vq_balance_loss needs for T tokens: 0 up to 64 tokens (one CTA does it all; workspace may be NULL),
 * and on invalid sizes. */
size_t vq_balance_workspace_size(int32_t T, int32_t E);

/* The router's balance loss and the experts' load, over the tokens that count (mask NULL, or mask[t] != 0; mask:
 * device bytes [T]). logits: device fp32 [T, E], ids: device int32 [T, top_k], both as vq_route takes and gives
 * them; an id outside [0, E) is a dropped pair and is not counted, an id twice in a token counts twice.
 *   counts[e] = pairs routed to e, e < E;  counts[E] = V, the tokens that count       (int32 [E + 1])
 *   probs[e]  = (1 / V) sum_t softmax(logits[t])[e]                                   (fp32 [E]; 0 when V = 0)
 *   loss      = coef * sum_e (E counts[e] / (V top_k)) probs[e]                       (fp32 [1])
 * (coef when the load is even). A token whose logits are all -Inf has probability 0 everywhere; other Inf and NaN
 * follow IEEE. Masked rows are not read. Column sums run in a fixed order: equal calls give equal bits. Limits as
 * vq_route (E <= 4096, 1 <= top_k <= min(E, 32), T * top_k < 2^31). workspace: 256-byte aligned; calls that may
 * overlap on the GPU need workspaces of their own. T = 0 writes zeros (logits, ids and mask may then be NULL). */
vq_status vq_balance_loss(const float *logits, const int32_t *ids, const uint8_t *mask, int32_t T, int32_t E,
                          int32_t top_k, float coef, float *loss, int32_t *counts, float *probs, void *workspace,
                          size_t ws_bytes, void *stream);

/* Gradient of vq_balance_loss at the logits, the counts held fixed. counts: as written by vq_balance_loss for the
 * same mask; dloss: device fp32 [1], or NULL for 1.  With d[e] = E counts[e] / (V top_k):
 *   dlogits[t, e] = dloss * coef / V * p[t, e] * (d[e] - sum_e' p[t, e'] d[e'])     (fp32 [T, E])
 * Masked tokens, and all tokens when V = 0, get 0. dlogits may be logits itself. */
vq_status vq_balance_loss_backward(const float *logits, const int32_t *counts, const uint8_t *mask, int32_t T,
                                   int32_t E, int32_t top_k, float coef, const float *dloss, float *dlogits,
                                   void *stream);

/* A dense matrix of 4-bit integers with group scales, W [rows, cols]:
 *   W[r, c] = fp32(scale[r, c / group]) * (q[r, c] - 8)                                  without biases
 *   W[r, c] = fp32(scale[r, c / group]) * q[r, c] + fp32(bias[r, c / group])             with biases
 * group is 32, 64 or 128 and divides cols; rows and cols are 1 to 2^30. (The d = 1, 4-bit modules above look their
 * values up in a codebook and have groups of 64 only.) words, scales and biases are in the tile layout that vq_q4_pack
 * writes. */
typedef struct vq_q4_module {
    int32_t rows;
    int32_t cols;
    int32_t group;
    const uint32_t *words;     /* device, 16-byte aligned: vq_q4_packed_words(rows, cols) words */
    const uint16_t *scales;    /* device, 16-byte aligned: fp16, vq_q4_packed_scales(rows, cols, group) */
    const uint16_t *biases;    /* device, 16-byte aligned, or NULL: as scales */
} vq_q4_module;

/* Words, and fp16 scales (or biases), of a packed module: 16-row by 128-column tiles, the last ones padded with
 * codes, scales and biases of 0. 0 on invalid arguments. */
size_t vq_q4_packed_words(int32_t rows, int32_t cols);
size_t vq_q4_packed_scales(int32_t rows, int32_t cols, int32_t group);

/* Lays a module out for vq_q4_gemv, once, when it is loaded. codes: device uint32 [rows, cols / 8], row-major, code c
 * in bits 4 (c % 8) of word c / 8 (vq_pack's layout for 4 bits); scales, biases: device fp16 [rows, cols / group],
 * row-major, biases and biases_out NULL together. Outputs: device, 16-byte aligned, of the sizes above.
 * Tile (i, j) (rows 16 i, columns 128 j; j fastest) is 256 words: word ((b * 32) + l) * 4 + s, lane l = 4 g + c,
 * holds rows 16 i + g and 16 i + g + 8, columns k .. k + 3 with k = 128 j + 64 b + 32 (s / 2) + 8 c + 4 (s % 2): rotated
 * right by 4 m bits (m = 0 .. 3), it has the codes of row g + 8 (m % 2), columns k + 2 (m / 2) and k + 2 (m / 2) + 1 in
 * bits 3 to 6 and 19 to 22. A tile's scales are [8 (g)][128 / group][2 (rows g, g + 8)]. */
vq_status vq_q4_pack(const uint32_t *codes, const uint16_t *scales, const uint16_t *biases, int32_t rows, int32_t cols,
                     int32_t group, uint32_t *words_out, uint16_t *scales_out, uint16_t *biases_out, void *stream);

/* Matrix-vector products of T tokens with a packed 4-bit module (the dense, codebook-free sibling of vq_gemv):
 *   m1 NULL:  y[t, r] = sum_c W0[r, c] x[t, c]
 *   else:     y[t, r] = silu(sum_c W0[r, c] x[t, c]) * sum_c W1[r, c] x[t, c]      (a gate and up pair)
 * m1 has m0's rows, cols and group, and biases when m0 has them. x: device bf16 [T, cols], row stride x_ld >= cols
 * elements, 16-byte aligned, x_ld a multiple of 8 (T > 1). y: device [T, rows] of y_dtype, row stride y_ld >= rows,
 * aligned to its element. x enters the tensor cores unrounded as bf16 against the exact integers 16 + q; group sums
 * (24 sum x is taken off them), scales and the sum over groups are fp32 in a fixed order, and y is rounded once: the
 * error is a few 2^-24 of sum |scale| (16 + q) |x|, also where the weights' own sum is much smaller (a row of codes 8
 * is 0 within it, not exactly). Sums of (16 + q) |x| over a group have to stay in fp32's range. The
 * weights are streamed and decoded once for every 16 tokens, so that the time grows with T from there on: the call is
 * meant for decode-sized T (T > 16 * 65535: VQ_ERR_UNSUPPORTED). An
 * Inf or NaN in x gives Inf or NaN in its token's outputs. */
vq_status vq_q4_gemv(const vq_q4_module *m0, const vq_q4_module *m1, const uint16_t *x, int64_t x_ld, int32_t T,
                     void *y, int32_t y_dtype, int64_t y_ld, void *stream);

/* Diagnostic (synchronises `stream`). Every wait of the library's pipelined
 * kernels on an on-chip barrier is bounded; a kernel that gives up records a
 * nonzero word at offset 0 of the MoE workspace it ran with (the routing
 * kernel of each vq_moe_decode / vq_moe_prefill call clears it) and stops
 * without completing its outputs. vq_fit records the same word in its own
 * workspace for a sample or init index out of range (each call clears it). Returns VQ_ERR_DEVICE_CHECK when the word
 * of `workspace` is set after the work queued on `stream`, VQ_OK when not,
 * VQ_ERR_WORKSPACE for a NULL or misaligned workspace. */
vq_status vq_moe_check(const void *workspace, void *stream);

/* vq_moe_decode without a workspace argument, for callers that cannot
 * allocate device memory: code running inside a host framework that owns
 * every device allocation and allows no new ones on its serving path, or a
 * program that reaches this library through a thin C FFI without a CUDA
 * memory API. The paper has no counterpart; the layer computed is exactly
 * vq_moe_decode's, with the same arguments minus the workspace.
 *
 * Scratch: one 16 MiB file-scope device array inside the library. Every GPU
 * that loads the library holds it until the process exits. Calls whose
 * vq_moe_workspace_size(L, T, top_k, VQ_MODE_DECODE) exceeds 16 MiB return
 * VQ_ERR_WORKSPACE and launch nothing.
 * Set-up: the first call on a device looks up the array's device address
 * (cudaGetSymbolAddress, with that device current); make that first call
 * before any stream capture. The address is kept per device and looked up
 * again when the calling thread's context is not the one it was found in
 * (for instance after cudaDeviceReset).
 * Sharing: all calls on a device use the same array and it keeps the last
 * call's contents (no call needs it zeroed: each writes what it reads).
 * Calls that overlap on the GPU (other streams, other host threads) race on
 * it; serialise them. The library allocates nothing for this call. */
vq_status vq_moe_decode_noalloc(const vq_moe_layer *L, const uint16_t *x, int32_t T, const float *logits,
                                int32_t top_k, int32_t renorm, void *y, int32_t y_dtype, void *stream);

/* Bound on the polls of every barrier wait in the pipelined kernels that the
 * calling thread launches from now on (no counterpart on the pages; a
 * failure-detection hook). polls < 0 restores the default, 2^22 polls (each
 * may suspend the waiting thread briefly); 0 makes every wait give up at
 * once. A wait that gives up makes its CTA stop: it lets
 * the copies and tensor-core operations it issued complete, frees its tensor
 * memory, records a nonzero word in the workspace (see vq_moe_check) and
 * returns without completing its outputs. Nothing faults or hangs. Errors:
 * VQ_ERR_ARG when polls > 2^32 - 1. */
vq_status vq_set_wait_limit(int64_t polls);

/* Tracing (no counterpart on the pages; an observability hook for timing
 * each kernel stage with the caller's CUDA events). events: host array of
 * n_events cudaEvent_t handles (as void*) created by the caller, or NULL to
 * switch tracing off. While set, the calling thread's vq_moe_decode and
 * vq_moe_prefill record events[i] on their stream at stage boundary i:
 *   decode:  0 | route | 1 | gate/up GEMV | 2 | SwiGLU | 3 | down GEMV | 4 | combine | 5
 *   prefill: 0 | route | 1 | gather | 2 | gate/up GEMM | 3 | h scales + down GEMM | 4 | combine | 5
 * Boundaries beyond n_events are not recorded. The library does not own
 * the events. Errors: VQ_ERR_ARG when n_events < 0. */
vq_status vq_set_trace_events(void *const *events, int32_t n_events);

#ifdef __cplusplus
}
#endif

#endif /* VQ_MOE_H */
