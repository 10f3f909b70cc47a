// Block norms, backward. With n(v) = v r (w + off), r = rsqrt(mean(v^2) + eps),
// v^ = v r and g = (w + off) d for the output's gradient d:
//   dv = r (g - v^ mean(g v^)),   dw = sum over rows of d v^.
// norm_post's gradient chains two of them around the sigmoid gate: first at
// the stored row h' (the next norm), then at y (the post norm).
//
// Persistent CTAs take rows in turn; a thread keeps its columns' weight
// gradients in registers over all rows of its CTA, one partial row per CTA goes
// to the workspace, and a second kernel adds the partial rows in order.
#include <algorithm>

#include "vq_block.cuh"
#include "vq_norm.h"

namespace vq {
namespace {

constexpr int BWD_THREADS = 512;    // most threads per CTA: 128 registers each
constexpr int NORM_PARTS = 592;     // most partial rows (4 per SM of 148)

template <int VEC>
__device__ __forceinline__ int chunk_at(int i, int tid, int W) { return (tid + i * 32 * W) * VEC; }

template <typename HT, int VEC, int NV>
__global__ void __launch_bounds__(BWD_THREADS) vq_norm_pre_bwd_kernel(const NormPreBwdArgs a)
{
    __shared__ RowSum<2> rs;
    grid_dep_launch();
    grid_dep_wait();
    const int W = a.W, tid = threadIdx.x % (32 * W), R = blockDim.x / (32 * W);
    const int slot = blockIdx.x * R + threadIdx.x / (32 * W);
    float acc[NV][VEC];
    AnyChunk<VEC> wc[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = chunk_at<VEC>(i, tid, W);
        if (c < a.H)
            wc[i].load(a.n.weight, a.n.dtype, c);
#pragma unroll
        for (int j = 0; j < VEC; ++j)
            acc[i][j] = 0.f;
    }
    int turn = 0;
    // one row of W > 1 warps per CTA: all its warps take the same trips; rows of one warp meet at no barrier
    for (long row = slot; row < a.T; row += (long)gridDim.x * R) {
        const HT *h = static_cast<const HT *>(a.h) + row * a.h_ld;
        const HT *dres = static_cast<const HT *>(a.dres) + row * a.dres_ld;
        const uint16_t *dx = a.dx + row * a.dx_ld;
        HT *dh = static_cast<HT *>(a.dh) + row * a.dh_ld;
        Chunk<HT, VEC> hc[NV], rc[NV];
        Chunk<uint16_t, VEC> dc[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = chunk_at<VEC>(i, tid, W);
            if (c < a.H) {
                hc[i].load(h + c);
                dc[i].load(dx + c);
                if (a.dres)
                    rc[i].load(dres + c);
            }
        }
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (chunk_at<VEC>(i, tid, W) < a.H) {
                float v[VEC], d[VEC], w[VEC];
                hc[i].get(v);
                dc[i].get(d);
                wc[i].get(w, a.n.dtype);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    s[0] = fmaf(v[j], v[j], s[0]);
                    s[1] = fmaf(d[j] * (w[j] + a.n.offset), v[j], s[1]);
                }
            }
        row_sum(s, rs, W, turn);
        const float r = rsqrtf(s[0] * a.inv_h + a.n.eps);
        const float m = r * (s[1] * a.inv_h);   // mean(g v^)
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = chunk_at<VEC>(i, tid, W);
            if (c < a.H) {
                float v[VEC], d[VEC], w[VEC], o[VEC];
                hc[i].get(v);
                dc[i].get(d);
                wc[i].get(w, a.n.dtype);
                if (a.dres)
                    rc[i].get(o);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const float n = v[j] * r;
                    acc[i][j] = fmaf(d[j], n, acc[i][j]);
                    const float t = r * (d[j] * (w[j] + a.n.offset) - n * m);
                    o[j] = a.dres ? o[j] + t : t;
                }
                Chunk<HT, VEC> oc;
                oc.set(o);
                oc.store(dh + c);
            }
        }
    }
    if (!a.part)
        return;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = chunk_at<VEC>(i, tid, W);
        if (c < a.H)
#pragma unroll
            for (int j = 0; j < VEC; ++j)
                a.part[(long)slot * a.H + c + j] = acc[i][j];
    }
}

template <typename YT, typename HT, int VEC, int NV>
__global__ void __launch_bounds__(BWD_THREADS) vq_norm_post_bwd_kernel(const NormPostBwdArgs a)
{
    __shared__ RowSum<3> rs;
    grid_dep_launch();
    grid_dep_wait();
    const int W = a.W, tid = threadIdx.x % (32 * W), R = blockDim.x / (32 * W);
    const int slot = blockIdx.x * R + threadIdx.x / (32 * W);
    const bool post = a.post.weight != nullptr, next = a.next.weight != nullptr;
    float acc1[NV][VEC], acc2[NV][VEC];
    AnyChunk<VEC> w1[NV], w2[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = chunk_at<VEC>(i, tid, W);
        if (c < a.H) {
            if (post)
                w1[i].load(a.post.weight, a.post.dtype, c);
            if (next)
                w2[i].load(a.next.weight, a.next.dtype, c);
        }
#pragma unroll
        for (int j = 0; j < VEC; ++j)
            acc1[i][j] = acc2[i][j] = 0.f;
    }
    int turn = 0;
    for (long row = slot; row < a.T; row += (long)gridDim.x * R) {
        const YT *y = static_cast<const YT *>(a.y) + row * a.y_ld;
        const HT *h = static_cast<const HT *>(a.h) + row * a.h_ld;
        const HT *dho = static_cast<const HT *>(a.dho) + row * a.dho_ld;
        const uint16_t *dx = a.dx + row * a.dx_ld;
        Chunk<YT, VEC> yc[NV];
        Chunk<HT, VEC> hc[NV], gc[NV];
        Chunk<uint16_t, VEC> dc[NV];
        AnyChunk<VEC> zc[NV];
        float on = 1.f, off = 0.f;   // sigmoid(z), 1 - sigmoid(z)
        if (a.gate_mode == GATE_TOKEN) {
            AnyChunk<1> z;
            float v[1];
            z.load(a.gate, a.gate_dtype, row * a.gate_ld);
            z.get(v, a.gate_dtype);
            on = sigmoid(v[0]);
            off = sigmoid(-v[0]);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = chunk_at<VEC>(i, tid, W);
            if (c < a.H) {
                yc[i].load(y + c);
                if (next) {
                    hc[i].load(h + c);
                    dc[i].load(dx + c);
                }
                if (a.dho)
                    gc[i].load(dho + c);
                if (a.gate_mode == GATE_CHANNEL)
                    zc[i].load(a.gate, a.gate_dtype, row * a.gate_ld + c);
            }
        }
        // the sums that need nothing but the inputs: |h'|^2, sum g h' of the next norm, |y|^2
        float s[3] = {0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (chunk_at<VEC>(i, tid, W) < a.H) {
                float v[VEC], d[VEC], w[VEC];
                if (next) {
                    hc[i].get(v);
                    dc[i].get(d);
                    w2[i].get(w, a.next.dtype);
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        s[0] = fmaf(v[j], v[j], s[0]);
                        s[1] = fmaf(d[j] * (w[j] + a.next.offset), v[j], s[1]);
                    }
                }
                if (post) {
                    yc[i].get(v);
#pragma unroll
                    for (int j = 0; j < VEC; ++j)
                        s[2] = fmaf(v[j], v[j], s[2]);
                }
            }
        if (next || post)
            row_sum(s, rs, W, turn);
        const float r2 = rsqrtf(s[0] * a.inv_h + a.next.eps), m2 = r2 * (s[1] * a.inv_h);
        const float r1 = post ? rsqrtf(s[2] * a.inv_h + a.post.eps) : 1.f;
        float dH[NV][VEC];
        float q[2] = {0.f, 0.f};   // sum g y of the post norm, sum dv u of a token's gate
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = chunk_at<VEC>(i, tid, W);
            if (c < a.H) {
                float v[VEC], d[VEC], w[VEC];
                if (a.dho)
                    gc[i].get(dH[i]);
                else
#pragma unroll
                    for (int j = 0; j < VEC; ++j)
                        dH[i][j] = 0.f;
                if (next) {
                    hc[i].get(v);
                    dc[i].get(d);
                    w2[i].get(w, a.next.dtype);
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        const float n = v[j] * r2;
                        acc2[i][j] = fmaf(d[j], n, acc2[i][j]);
                        dH[i][j] += r2 * (d[j] * (w[j] + a.next.offset) - n * m2);
                    }
                }
                if (a.dh) {
#pragma unroll
                    for (int j = 0; j < VEC; ++j)
                        d[j] = a.res_scale * dH[i][j];
                    Chunk<HT, VEC> oc;
                    oc.set(d);
                    oc.store(static_cast<HT *>(a.dh) + row * a.dh_ld + c);
                }
                yc[i].get(v);
                if (post)
                    w1[i].get(w, a.post.dtype);
                float z[VEC];
                if (a.gate_mode == GATE_CHANNEL)
                    zc[i].get(z, a.gate_dtype);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    float du = a.out_scale * dH[i][j];                                    // dv
                    const float wj = post ? w[j] + a.post.offset : 1.f;
                    const float n = v[j] * r1;
                    q[1] = fmaf(du, n * wj, q[1]);                                        // dv u
                    if (a.gate_mode == GATE_CHANNEL) {
                        const float so = sigmoid(z[j]);
                        z[j] = du * (n * wj) * so * sigmoid(-z[j]);
                        du *= so;
                    } else {
                        du *= on;
                    }
                    acc1[i][j] = fmaf(du, n, acc1[i][j]);
                    du *= wj;                                                             // g
                    q[0] = fmaf(du, v[j], q[0]);
                    dH[i][j] = du;
                }
                if (a.gate_mode == GATE_CHANNEL && a.dgate) {
                    const long at = row * a.dgate_ld + c;
                    if (a.gate_dtype == VQ_F32) {
                        Chunk<float, VEC> oc;
                        oc.set(z);
                        oc.store(static_cast<float *>(a.dgate) + at);
                    } else {
                        Chunk<uint16_t, VEC> oc;
                        oc.set(z);
                        oc.store(static_cast<uint16_t *>(a.dgate) + at);
                    }
                }
            }
        }
        if (post || (a.gate_mode == GATE_TOKEN && a.dgate))
            row_sum(q, rs, W, turn);
        if (a.gate_mode == GATE_TOKEN && a.dgate && tid == 0) {
            const float dz = q[1] * on * off;
            const long at = row * a.dgate_ld;
            if (a.gate_dtype == VQ_F32)
                static_cast<float *>(a.dgate)[at] = dz;
            else
                static_cast<uint16_t *>(a.dgate)[at] = f32_to_bf16_bits(dz);
        }
        const float m1 = r1 * (q[0] * a.inv_h);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = chunk_at<VEC>(i, tid, W);
            if (c < a.H) {
                float v[VEC];
                yc[i].get(v);
#pragma unroll
                for (int j = 0; j < VEC; ++j)
                    v[j] = post ? r1 * (dH[i][j] - v[j] * r1 * m1) : dH[i][j];
                Chunk<YT, VEC> oc;
                oc.set(v);
                oc.store(static_cast<YT *>(a.dy) + row * a.dy_ld + c);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = chunk_at<VEC>(i, tid, W);
        if (c < a.H)
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                if (a.part1)
                    a.part1[(long)slot * a.H + c + j] = acc1[i][j];
                if (a.part2)
                    a.part2[(long)slot * a.H + c + j] = acc2[i][j];
            }
    }
}

// Column sums of the partial rows, in row order within each of 8 interleaved
// strands, then over the strands: d[c] = sum_p part[p][c]. blockIdx.y: which
// weight gradient.
__global__ void __launch_bounds__(256) vq_norm_dw_kernel(const float *p1, float *d1, const float *p2, float *d2,
                                                         int parts, int H)
{
    __shared__ float s[8][33];
    grid_dep_launch();
    grid_dep_wait();
    const float *p = blockIdx.y ? p2 : p1;
    float *d = blockIdx.y ? d2 : d1;
    if (!d)
        return;
    const int x = threadIdx.x & 31, yy = threadIdx.x >> 5, c = blockIdx.x * 32 + x;
    float v = 0.f;
    if (c < H) {
#pragma unroll 8
        for (int i = yy; i < parts; i += 8)
            v += p[(long)i * H + c];
    }
    s[yy][x] = v;
    __syncthreads();
    if (yy == 0 && c < H) {
#pragma unroll
        for (int i = 1; i < 8; ++i)
            v += s[i][x];
        d[c] = v;
    }
}

struct BwdShape {
    int W, R, nv, ctas, parts;
};

BwdShape bwd_shape(int H, int vec, int T)
{
    BwdShape s;
    const int chunks = (H + vec - 1) / vec;
    int nv = 1;
    while ((chunks + nv - 1) / nv > BWD_THREADS)
        nv = vec == 8 ? nv * 2 : nv == 1 ? 8 : 32;
    s.nv = nv;
    s.W = ((chunks + nv - 1) / nv + 31) / 32;
    s.R = s.W == 1 ? 4 : 1;
    s.ctas = std::max(1, (int)std::min(((long)T + s.R - 1) / s.R, (long)NORM_PARTS / s.R));
    s.parts = s.ctas * s.R;
    return s;
}

cudaError_t finish(const BwdShape &sh, int T, int H, const float *p1, float *d1, const float *p2, float *d2,
                   cudaStream_t s)
{
    if (!d1 && !d2)
        return cudaSuccess;
    return launch_after(vq_norm_dw_kernel, dim3((H + 31) / 32, 2), dim3(256), 0, s, p1, d1, p2, d2,
                        T > 0 ? sh.parts : 0, H);
}

template <typename HT>
cudaError_t pre_bwd(const NormPreBwdArgs &a, const BwdShape &sh, bool vec8, cudaStream_t s)
{
    const dim3 grid(sh.ctas), block(32 * sh.W * sh.R);
    if (vec8) {
        switch (sh.nv) {
        case 1: return launch_after(vq_norm_pre_bwd_kernel<HT, 8, 1>, grid, block, 0, s, a);
        case 2: return launch_after(vq_norm_pre_bwd_kernel<HT, 8, 2>, grid, block, 0, s, a);
        default: return launch_after(vq_norm_pre_bwd_kernel<HT, 8, 4>, grid, block, 0, s, a);
        }
    }
    switch (sh.nv) {
    case 1: return launch_after(vq_norm_pre_bwd_kernel<HT, 1, 1>, grid, block, 0, s, a);
    case 8: return launch_after(vq_norm_pre_bwd_kernel<HT, 1, 8>, grid, block, 0, s, a);
    default: return launch_after(vq_norm_pre_bwd_kernel<HT, 1, 32>, grid, block, 0, s, a);
    }
}

template <typename YT, typename HT>
cudaError_t post_bwd(const NormPostBwdArgs &a, const BwdShape &sh, bool vec8, cudaStream_t s)
{
    const dim3 grid(sh.ctas), block(32 * sh.W * sh.R);
    if (vec8) {
        switch (sh.nv) {
        case 1: return launch_after(vq_norm_post_bwd_kernel<YT, HT, 8, 1>, grid, block, 0, s, a);
        case 2: return launch_after(vq_norm_post_bwd_kernel<YT, HT, 8, 2>, grid, block, 0, s, a);
        default: return launch_after(vq_norm_post_bwd_kernel<YT, HT, 8, 4>, grid, block, 0, s, a);
        }
    }
    switch (sh.nv) {
    case 1: return launch_after(vq_norm_post_bwd_kernel<YT, HT, 1, 1>, grid, block, 0, s, a);
    case 8: return launch_after(vq_norm_post_bwd_kernel<YT, HT, 1, 8>, grid, block, 0, s, a);
    default: return launch_after(vq_norm_post_bwd_kernel<YT, HT, 1, 32>, grid, block, 0, s, a);
    }
}

}  // namespace

size_t norm_workspace_bytes(int H, int T)
{
    // bwd_shape's partial rows: at most NORM_PARTS, and at most 4 (one CTA of one-warp rows) over T
    return (size_t)2 * (size_t)std::min((long)NORM_PARTS, (long)std::max(T, 1) + 3) * (size_t)H * sizeof(float);
}

cudaError_t launch_norm_pre_bwd(const NormPreBwdArgs &args, int h_dtype, bool vec8, float *dw, float *ws, cudaStream_t s)
{
    NormPreBwdArgs a = args;
    const BwdShape sh = bwd_shape(a.H, vec8 ? 8 : 1, a.T);
    a.W = sh.W;
    a.part = dw ? ws : nullptr;
    if (a.T > 0) {
        const cudaError_t e = h_dtype == VQ_F32 ? pre_bwd<float>(a, sh, vec8, s) : pre_bwd<uint16_t>(a, sh, vec8, s);
        if (e != cudaSuccess)
            return e;
    }
    return finish(sh, a.T, a.H, a.part, dw, nullptr, nullptr, s);
}

cudaError_t launch_norm_post_bwd(const NormPostBwdArgs &args, int y_dtype, int h_dtype, bool vec8, float *dpost,
                                 float *dnext, float *ws, cudaStream_t s)
{
    NormPostBwdArgs a = args;
    const BwdShape sh = bwd_shape(a.H, vec8 ? 8 : 1, a.T);
    a.W = sh.W;
    a.part1 = dpost ? ws : nullptr;
    a.part2 = dnext ? ws + (size_t)sh.parts * a.H : nullptr;
    if (a.T > 0) {
        cudaError_t e;
        if (y_dtype == VQ_F32)
            e = h_dtype == VQ_F32 ? post_bwd<float, float>(a, sh, vec8, s) : post_bwd<float, uint16_t>(a, sh, vec8, s);
        else
            e = h_dtype == VQ_F32 ? post_bwd<uint16_t, float>(a, sh, vec8, s)
                                  : post_bwd<uint16_t, uint16_t>(a, sh, vec8, s);
        if (e != cudaSuccess)
            return e;
    }
    return finish(sh, a.T, a.H, a.part1, dpost, a.part2, dnext, s);
}

}  // namespace vq
