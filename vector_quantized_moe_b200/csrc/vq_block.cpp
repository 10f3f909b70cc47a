// C ABI of the block around the experts (norms, balance loss, dense 4-bit
// products): argument validation and dispatch. See include/vq_moe.h.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "vq_balance.h"
#include "vq_internal.h"
#include "vq_norm.h"
#include "vq_q4.h"

using namespace vq;

namespace {

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

bool is_dtype(int32_t d) { return d == VQ_F32 || d == VQ_BF16; }

size_t elem(int32_t dtype) { return dtype == VQ_F32 ? 4 : 2; }

vq_status status(cudaError_t e) { return e == cudaSuccess ? VQ_OK : VQ_ERR_CUDA; }

vq_status check_norm(const vq_norm *n, int32_t hidden)
{
    if (!n->weight || !is_dtype(n->weight_dtype) || n->hidden != hidden || !(n->eps >= 0.f) || !std::isfinite(n->eps) ||
        !std::isfinite(n->weight_offset))
        return VQ_ERR_ARG;
    return aligned(n->weight, elem(n->weight_dtype)) ? VQ_OK : VQ_ERR_ALIGN;
}

NormDev norm_dev(const vq_norm *n)
{
    return n ? NormDev{n->weight, n->weight_dtype, n->eps, n->weight_offset} : NormDev{nullptr, VQ_F32, 0.f, 0.f};
}

// The row arrays of one call: validity, alignment, and whether all of them
// (and the weights) allow the 16-byte kernels.
struct Rows {
    int32_t hidden, T;
    vq_status st = VQ_OK;
    bool vec8;
    Rows(int32_t h, int32_t t) : hidden(h), T(t), vec8(h % 8 == 0) {}
    void add(const void *p, int32_t dtype, int64_t ld, int32_t cols)
    {
        if (st != VQ_OK)
            return;
        if (!is_dtype(dtype) || (T > 0 && !p) || (T > 1 && ld < cols))
            st = VQ_ERR_ARG;
        else if (!aligned(p, elem(dtype)))
            st = VQ_ERR_ALIGN;
        else if (cols > 1 && (!aligned(p, 16) || (T > 1 && (ld * (int64_t)elem(dtype)) % 16 != 0)))
            vec8 = false;
    }
    void weight(const vq_norm *n)
    {
        if (n && !aligned(n->weight, 16))
            vec8 = false;
    }
    void gradient(const float *d)   // a weight's: one row's kernel writes it itself
    {
        if (!aligned(d, 16))
            vec8 = false;
    }
};

vq_status check_hidden(int32_t hidden, int32_t T)
{
    if (hidden < 1 || T < 0)
        return VQ_ERR_ARG;
    return hidden > NORM_MAX_HIDDEN ? VQ_ERR_UNSUPPORTED : VQ_OK;
}

vq_status check_ws(const void *ws, size_t bytes, size_t need)
{
    return need == 0 || (ws && aligned(ws, 256) && bytes >= need) ? VQ_OK : VQ_ERR_WORKSPACE;
}

bool balance_sizes_ok(int32_t T, int32_t E, int32_t k)
{
    return T >= 0 && E >= 1 && E <= 4096 && k >= 1 && k <= std::min(E, 32) && (long)T * k < (1L << 31);
}

constexpr int32_t Q4_MAX_COLS = 1 << 30, Q4_MAX_T = 16 * 65535;   // 16 tokens to a CTA, grid.y

bool q4_sizes_ok(int32_t rows, int32_t cols, int32_t group)
{
    return rows >= 1 && rows <= (1 << 30) && cols >= 1 && cols <= Q4_MAX_COLS &&
           (group == 32 || group == 64 || group == 128) && cols % group == 0;
}

vq_status check_q4(const vq_q4_module *m)
{
    if (!m || !m->words || !m->scales || !q4_sizes_ok(m->rows, m->cols, m->group))
        return VQ_ERR_ARG;
    return aligned(m->words, 16) && aligned(m->scales, 16) && aligned(m->biases, 16) ? VQ_OK : VQ_ERR_ALIGN;
}

size_t q4_tiles(int32_t rows, int32_t cols) { return (((size_t)rows + 15) / 16) * (((size_t)cols + 127) / 128); }

}  // namespace

extern "C" {

vq_status vq_norm_pre(const vq_norm *n, const void *h, int32_t h_dtype, int64_t h_ld, int32_t T, uint16_t *x,
                      int64_t x_ld, void *stream)
{
    if (!n)
        return VQ_ERR_ARG;
    vq_status st = check_hidden(n->hidden, T);
    if (st == VQ_OK)
        st = check_norm(n, n->hidden);
    if (st != VQ_OK)
        return st;
    Rows r(n->hidden, T);
    r.add(h, h_dtype, h_ld, n->hidden);
    r.add(x, VQ_BF16, x_ld, n->hidden);
    r.weight(n);
    if (r.st != VQ_OK || T == 0)
        return r.st;
    NormPreArgs a{};
    a.n = norm_dev(n);
    a.h = h;
    a.x = x;
    a.h_ld = h_ld;
    a.x_ld = x_ld;
    a.T = T;
    a.H = n->hidden;
    a.inv_h = 1.f / (float)n->hidden;
    return status(launch_norm_pre(a, h_dtype, r.vec8, (cudaStream_t)stream));
}

size_t vq_norm_workspace_size(int32_t hidden, int32_t T)
{
    return check_hidden(hidden, T) == VQ_OK ? norm_workspace_bytes(hidden, T) : 0;
}

vq_status vq_norm_pre_backward(const vq_norm *n, const void *h, int32_t h_dtype, int64_t h_ld, const uint16_t *dx,
                               int64_t dx_ld, const void *dres, int64_t dres_ld, int32_t T, void *dh, int64_t dh_ld,
                               float *dweight, void *workspace, size_t ws_bytes, void *stream)
{
    if (!n)
        return VQ_ERR_ARG;
    vq_status st = check_hidden(n->hidden, T);
    if (st == VQ_OK)
        st = check_norm(n, n->hidden);
    if (st != VQ_OK)
        return st;
    Rows r(n->hidden, T);
    r.add(h, h_dtype, h_ld, n->hidden);
    r.add(dx, VQ_BF16, dx_ld, n->hidden);
    if (dres)
        r.add(dres, h_dtype, dres_ld, n->hidden);
    r.add(dh, h_dtype, dh_ld, n->hidden);
    r.weight(n);
    if (r.st != VQ_OK)
        return r.st;
    if (!aligned(dweight, 4))
        return VQ_ERR_ALIGN;
    r.gradient(dweight);
    if (dweight && (st = check_ws(workspace, ws_bytes, norm_workspace_bytes(n->hidden, T))) != VQ_OK)
        return st;
    NormPreBwdArgs a{};
    a.n = norm_dev(n);
    a.h = h;
    a.dres = dres;
    a.dx = dx;
    a.dh = dh;
    a.h_ld = h_ld;
    a.dx_ld = dx_ld;
    a.dres_ld = dres_ld;
    a.dh_ld = dh_ld;
    a.T = T;
    a.H = n->hidden;
    a.inv_h = 1.f / (float)n->hidden;
    return status(launch_norm_pre_bwd(a, h_dtype, r.vec8, dweight, static_cast<float *>(workspace),
                                      (cudaStream_t)stream));
}

// What vq_norm_post and its gradient check alike: the norms, the gate.
static vq_status check_post(const vq_norm *post, const vq_norm *next, int32_t hidden, int32_t T, const void *gate,
                            int32_t gate_dtype, int32_t gate_cols, int64_t gate_ld, float res_scale, float out_scale,
                            Rows &r)
{
    vq_status st = check_hidden(hidden, T);
    if (st == VQ_OK && post)
        st = check_norm(post, hidden);
    if (st == VQ_OK && next)
        st = check_norm(next, hidden);
    if (st != VQ_OK)
        return st;
    if (!std::isfinite(res_scale) || !std::isfinite(out_scale))
        return VQ_ERR_ARG;
    if (gate) {
        if (gate_cols != 1 && gate_cols != hidden)
            return VQ_ERR_ARG;
        r.add(gate, gate_dtype, gate_ld, gate_cols);
    }
    r.weight(post);
    r.weight(next);
    return r.st;
}

static int gate_mode(const void *gate, int32_t gate_cols)
{
    return !gate ? GATE_NONE : gate_cols == 1 ? GATE_TOKEN : GATE_CHANNEL;
}

vq_status vq_norm_post(const vq_norm *post, const vq_norm *next, int32_t hidden, const void *y, int32_t y_dtype,
                       int64_t y_ld, const void *gate, int32_t gate_dtype, int32_t gate_cols, int64_t gate_ld,
                       const void *h, int32_t h_dtype, int64_t h_ld, float res_scale, float out_scale, int32_t T,
                       void *h_out, int64_t h_out_ld, uint16_t *x_out, int64_t x_out_ld, void *stream)
{
    Rows r(hidden, T);
    vq_status st = check_post(post, next, hidden, T, gate, gate_dtype, gate_cols, gate_ld, res_scale, out_scale, r);
    if (st != VQ_OK)
        return st;
    r.add(y, y_dtype, y_ld, hidden);
    r.add(h, h_dtype, h_ld, hidden);
    r.add(h_out, h_dtype, h_out_ld, hidden);
    if (next)
        r.add(x_out, VQ_BF16, x_out_ld, hidden);
    else if (x_out)
        return VQ_ERR_ARG;
    if (r.st != VQ_OK || T == 0)
        return r.st;
    NormPostArgs a{};
    a.post = norm_dev(post);
    a.next = norm_dev(next);
    a.y = y;
    a.gate = gate;
    a.h = h;
    a.h_out = h_out;
    a.x = x_out;
    a.y_ld = y_ld;
    a.gate_ld = gate_ld;
    a.h_ld = h_ld;
    a.ho_ld = h_out_ld;
    a.x_ld = x_out_ld;
    a.gate_mode = gate_mode(gate, gate_cols);
    a.gate_dtype = gate_dtype;
    a.T = T;
    a.H = hidden;
    a.inv_h = 1.f / (float)hidden;
    a.res_scale = res_scale;
    a.out_scale = out_scale;
    return status(launch_norm_post(a, y_dtype, h_dtype, r.vec8, (cudaStream_t)stream));
}

vq_status vq_norm_post_backward(const vq_norm *post, const vq_norm *next, int32_t hidden, const void *y,
                                int32_t y_dtype, int64_t y_ld, const void *gate, int32_t gate_dtype, int32_t gate_cols,
                                int64_t gate_ld, const void *h_out, int32_t h_dtype, int64_t h_out_ld, float res_scale,
                                float out_scale, int32_t T, const void *dh_out, int64_t dh_out_ld,
                                const uint16_t *dx_out, int64_t dx_out_ld, void *dy, int64_t dy_ld, void *dgate,
                                int64_t dgate_ld, void *dh, int64_t dh_ld, float *dpost, float *dnext, void *workspace,
                                size_t ws_bytes, void *stream)
{
    Rows r(hidden, T);
    vq_status st = check_post(post, next, hidden, T, gate, gate_dtype, gate_cols, gate_ld, res_scale, out_scale, r);
    if (st != VQ_OK)
        return st;
    if ((dgate && !gate) || (dpost && !post) || (dnext && !next) || (dx_out && !next) || !is_dtype(h_dtype))
        return VQ_ERR_ARG;
    r.add(y, y_dtype, y_ld, hidden);
    if (next) {
        r.add(h_out, h_dtype, h_out_ld, hidden);
        r.add(dx_out, VQ_BF16, dx_out_ld, hidden);
    }
    if (dh_out)
        r.add(dh_out, h_dtype, dh_out_ld, hidden);
    r.add(dy, y_dtype, dy_ld, hidden);
    if (dgate)
        r.add(dgate, gate_dtype, dgate_ld, gate_cols);
    if (dh)
        r.add(dh, h_dtype, dh_ld, hidden);
    if (r.st != VQ_OK)
        return r.st;
    if (!aligned(dpost, 4) || !aligned(dnext, 4))
        return VQ_ERR_ALIGN;
    r.gradient(dpost);
    r.gradient(dnext);
    if ((dpost || dnext) && (st = check_ws(workspace, ws_bytes, norm_workspace_bytes(hidden, T))) != VQ_OK)
        return st;
    NormPostBwdArgs a{};
    a.post = norm_dev(post);
    a.next = norm_dev(next);
    a.y = y;
    a.gate = gate;
    a.h = h_out;
    a.dho = dh_out;
    a.dx = dx_out;
    a.dy = dy;
    a.dgate = dgate;
    a.dh = dh;
    a.y_ld = y_ld;
    a.gate_ld = gate_ld;
    a.h_ld = h_out_ld;
    a.dho_ld = dh_out_ld;
    a.dx_ld = dx_out_ld;
    a.dy_ld = dy_ld;
    a.dgate_ld = dgate_ld;
    a.dh_ld = dh_ld;
    a.gate_mode = gate_mode(gate, gate_cols);
    a.gate_dtype = gate_dtype;
    a.T = T;
    a.H = hidden;
    a.inv_h = 1.f / (float)hidden;
    a.res_scale = res_scale;
    a.out_scale = out_scale;
    return status(launch_norm_post_bwd(a, y_dtype, h_dtype, r.vec8, dpost, dnext, static_cast<float *>(workspace),
                                       (cudaStream_t)stream));
}

size_t vq_balance_workspace_size(int32_t T, int32_t E)
{
    return balance_sizes_ok(T, E, 1) ? balance_workspace_bytes(T, E) : 0;
}

vq_status vq_balance_loss(const float *logits, const int32_t *ids, const uint8_t *mask, int32_t T, int32_t E,
                          int32_t top_k, float coef, float *loss, int32_t *counts, float *probs, void *workspace,
                          size_t ws_bytes, void *stream)
{
    if (!balance_sizes_ok(T, E, top_k) || (T > 0 && (!logits || !ids)) || !loss || !counts || !probs ||
        !std::isfinite(coef))
        return VQ_ERR_ARG;
    if (!aligned(logits, 4) || !aligned(ids, 4) || !aligned(loss, 4) || !aligned(counts, 4) || !aligned(probs, 4))
        return VQ_ERR_ALIGN;
    const size_t need = balance_workspace_bytes(T, E);
    const vq_status st = check_ws(workspace, ws_bytes, need);
    if (st != VQ_OK)
        return st;
    BalanceArgs a{};
    a.logits = logits;
    a.ids = ids;
    a.mask = mask;
    a.loss = loss;
    a.probs = probs;
    a.counts = counts;
    a.T = T;
    a.E = E;
    a.k = top_k;
    a.coef = coef;
    return status(launch_balance(a, workspace, (cudaStream_t)stream));
}

vq_status vq_balance_loss_backward(const float *logits, const int32_t *counts, const uint8_t *mask, int32_t T,
                                   int32_t E, int32_t top_k, float coef, const float *dloss, float *dlogits,
                                   void *stream)
{
    if (!balance_sizes_ok(T, E, top_k) || (T > 0 && (!logits || !counts || !dlogits)) || !std::isfinite(coef))
        return VQ_ERR_ARG;
    if (!aligned(logits, 4) || !aligned(counts, 4) || !aligned(dloss, 4) || !aligned(dlogits, 4))
        return VQ_ERR_ALIGN;
    if (T == 0)
        return VQ_OK;
    BalanceBwdArgs a{};
    a.logits = logits;
    a.counts = counts;
    a.mask = mask;
    a.dloss = dloss;
    a.dlogits = dlogits;
    a.T = T;
    a.E = E;
    a.k = top_k;
    a.coef = coef;
    return status(launch_balance_bwd(a, (cudaStream_t)stream));
}

size_t vq_q4_packed_words(int32_t rows, int32_t cols)
{
    return q4_sizes_ok(rows, cols, 32) ? q4_tiles(rows, cols) * 256 : 0;
}

size_t vq_q4_packed_scales(int32_t rows, int32_t cols, int32_t group)
{
    return q4_sizes_ok(rows, cols, group) ? q4_tiles(rows, cols) * 16 * (128 / group) : 0;
}

vq_status vq_q4_pack(const uint32_t *codes, const uint16_t *scales, const uint16_t *biases, int32_t rows, int32_t cols,
                     int32_t group, uint32_t *words_out, uint16_t *scales_out, uint16_t *biases_out, void *stream)
{
    if (!codes || !scales || !words_out || !scales_out || !biases != !biases_out || !q4_sizes_ok(rows, cols, group))
        return VQ_ERR_ARG;
    if (!aligned(codes, 4) || !aligned(scales, 2) || !aligned(biases, 2) || !aligned(words_out, 16) ||
        !aligned(scales_out, 16) || !aligned(biases_out, 16))
        return VQ_ERR_ALIGN;
    return status(launch_q4_pack(codes, scales, biases, rows, cols, group, words_out, scales_out, biases_out,
                                 (cudaStream_t)stream));
}

vq_status vq_q4_gemv(const vq_q4_module *m0, const vq_q4_module *m1, const uint16_t *x, int64_t x_ld, int32_t T,
                     void *y, int32_t y_dtype, int64_t y_ld, void *stream)
{
    vq_status st = check_q4(m0);
    if (st == VQ_OK && m1)
        st = check_q4(m1);
    if (st != VQ_OK)
        return st;
    if (m1 && (m1->rows != m0->rows || m1->cols != m0->cols || m1->group != m0->group || !m1->biases != !m0->biases))
        return VQ_ERR_ARG;
    if (T < 0 || (T > 0 && (!x || !y)) || !is_dtype(y_dtype) || (T > 1 && (x_ld < m0->cols || y_ld < m0->rows)))
        return VQ_ERR_ARG;
    if (T > Q4_MAX_T)
        return VQ_ERR_UNSUPPORTED;
    if (!aligned(x, 16) || (T > 1 && x_ld % 8 != 0) || !aligned(y, elem(y_dtype)))
        return VQ_ERR_ALIGN;
    if (T == 0)
        return VQ_OK;
    Q4Args a{};
    for (int i = 0; i < 2; ++i) {
        const vq_q4_module *m = i && m1 ? m1 : m0;
        a.words[i] = m->words;
        a.scales[i] = m->scales;
        a.biases[i] = m->biases;
    }
    a.x = x;
    a.y = y;
    a.x_ld = x_ld;
    a.y_ld = y_ld;
    a.rows = m0->rows;
    a.cols = m0->cols;
    a.T = T;
    a.tiles = (m0->rows + 15) / 16;
    a.nsb = (m0->cols + 127) / 128;
    a.pair = m1 != nullptr;
    a.y_dtype = y_dtype;
    return status(launch_q4_gemv(a, m0->group, (cudaStream_t)stream));
}

}  // extern "C"
