// Block norms, forward: the norm that makes a MoE block's input, and the join
// of the block's output with the residual stream (norm, sigmoid gate, two
// scales, and the next block's norm) in one pass over each row.
//
//   norm_pre:  x = bf16(h r (w + off)),  r = rsqrt(mean(h^2) + eps)
//   norm_post: u = y r1 (w1 + off1) (or y); h' = a h + b s(z) u; x' = norm of the stored h'
//
// A row stays in the registers of one CTA (or one warp) between the row sum
// and the output, so each array crosses HBM once; the time is that of the
// bytes for many rows and of one load, one or two row sums and one store for
// few.
#include "vq_block.cuh"
#include "vq_norm.h"

namespace vq {
namespace {

// Where a thread's i-th chunk of a row starts, for a row over W warps.
template <int VEC>
__device__ __forceinline__ int chunk_at(int i, int tid, int W) { return (tid + i * 32 * W) * VEC; }

template <typename HT, int VEC, int NV>
__global__ void __launch_bounds__(1024) vq_norm_pre_kernel(const NormPreArgs a)
{
    __shared__ RowSum<1> rs;
    grid_dep_launch();
    grid_dep_wait();
    const int W = a.W, tid = threadIdx.x % (32 * W);
    const long row = (long)blockIdx.x * (blockDim.x / (32 * W)) + threadIdx.x / (32 * W);
    if (row >= a.T)   // only in CTAs of one-warp rows, which never meet at a barrier
        return;
    const HT *h = static_cast<const HT *>(a.h) + row * a.h_ld;
    Chunk<HT, VEC> hc[NV];
    AnyChunk<VEC> wc[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = chunk_at<VEC>(i, tid, W);
        if (c < a.H)
            hc[i].load(h + c);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = chunk_at<VEC>(i, tid, W);
        if (c < a.H)
            wc[i].load(a.n.weight, a.n.dtype, c);
    }
    float ss[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (chunk_at<VEC>(i, tid, W) < a.H) {
            float v[VEC];
            hc[i].get(v);
#pragma unroll
            for (int j = 0; j < VEC; ++j)
                ss[0] = fmaf(v[j], v[j], ss[0]);
        }
    }
    int turn = 0;
    row_sum(ss, rs, W, turn);
    const float r = rsqrtf(ss[0] * a.inv_h + a.n.eps);
    uint16_t *x = a.x + row * a.x_ld;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = chunk_at<VEC>(i, tid, W);
        if (c < a.H) {
            float v[VEC], w[VEC];
            hc[i].get(v);
            wc[i].get(w, a.n.dtype);
#pragma unroll
            for (int j = 0; j < VEC; ++j)
                v[j] = v[j] * r * (w[j] + a.n.offset);
            Chunk<uint16_t, VEC> o;
            o.set(v);
            o.store(x + c);
        }
    }
}

template <typename YT, typename HT, int VEC, int NV>
__global__ void __launch_bounds__(1024) vq_norm_post_kernel(const NormPostArgs a)
{
    __shared__ RowSum<1> rs;
    grid_dep_launch();
    grid_dep_wait();
    const int W = a.W, tid = threadIdx.x % (32 * W);
    const long row = (long)blockIdx.x * (blockDim.x / (32 * W)) + threadIdx.x / (32 * W);
    if (row >= a.T)
        return;
    const YT *y = static_cast<const YT *>(a.y) + row * a.y_ld;
    const HT *h = static_cast<const HT *>(a.h) + row * a.h_ld;
    Chunk<YT, VEC> yc[NV];
    Chunk<HT, VEC> hc[NV];
    AnyChunk<VEC> w1[NV], w2[NV], zc[NV];
    float gate = 1.f;
    if (a.gate_mode == GATE_TOKEN) {
        AnyChunk<1> z;
        float v[1];
        z.load(a.gate, a.gate_dtype, row * a.gate_ld);
        z.get(v, a.gate_dtype);
        gate = sigmoid(v[0]);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = chunk_at<VEC>(i, tid, W);
        if (c < a.H) {
            yc[i].load(y + c);
            hc[i].load(h + c);
            if (a.gate_mode == GATE_CHANNEL)
                zc[i].load(a.gate, a.gate_dtype, row * a.gate_ld + c);
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = chunk_at<VEC>(i, tid, W);
        if (c < a.H) {
            if (a.post.weight)
                w1[i].load(a.post.weight, a.post.dtype, c);
            if (a.next.weight)
                w2[i].load(a.next.weight, a.next.dtype, c);
        }
    }
    int turn = 0;
    float r1 = 1.f;
    if (a.post.weight) {
        float ss[1] = {0.f};
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (chunk_at<VEC>(i, tid, W) < a.H) {
                float v[VEC];
                yc[i].get(v);
#pragma unroll
                for (int j = 0; j < VEC; ++j)
                    ss[0] = fmaf(v[j], v[j], ss[0]);
            }
        row_sum(ss, rs, W, turn);
        r1 = rsqrtf(ss[0] * a.inv_h + a.post.eps);
    }
    float ss[1] = {0.f};
    HT *ho = static_cast<HT *>(a.h_out) + row * a.ho_ld;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = chunk_at<VEC>(i, tid, W);
        if (c < a.H) {
            float u[VEC], v[VEC], t[VEC];
            yc[i].get(u);
            hc[i].get(v);
            if (a.post.weight) {
                w1[i].get(t, a.post.dtype);
#pragma unroll
                for (int j = 0; j < VEC; ++j)
                    u[j] = u[j] * r1 * (t[j] + a.post.offset);
            }
            if (a.gate_mode == GATE_CHANNEL) {
                zc[i].get(t, a.gate_dtype);
#pragma unroll
                for (int j = 0; j < VEC; ++j)
                    u[j] *= sigmoid(t[j]);
            } else {
#pragma unroll
                for (int j = 0; j < VEC; ++j)
                    u[j] *= gate;
            }
#pragma unroll
            for (int j = 0; j < VEC; ++j)
                v[j] = a.res_scale * v[j] + a.out_scale * u[j];
            hc[i].set(v);   // the row as stored: what the next norm sees
            hc[i].store(ho + c);
            hc[i].get(v);
#pragma unroll
            for (int j = 0; j < VEC; ++j)
                ss[0] = fmaf(v[j], v[j], ss[0]);
        }
    }
    if (!a.next.weight)
        return;
    row_sum(ss, rs, W, turn);
    const float r2 = rsqrtf(ss[0] * a.inv_h + a.next.eps);
    uint16_t *x = a.x + row * a.x_ld;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = chunk_at<VEC>(i, tid, W);
        if (c < a.H) {
            float v[VEC], w[VEC];
            hc[i].get(v);
            w2[i].get(w, a.next.dtype);
#pragma unroll
            for (int j = 0; j < VEC; ++j)
                v[j] = v[j] * r2 * (w[j] + a.next.offset);
            Chunk<uint16_t, VEC> o;
            o.set(v);
            o.store(x + c);
        }
    }
}

// Warps per row, and rows per CTA: rows of one warp share a CTA of 4 warps.
struct RowShape {
    int W, R, nv;
};

RowShape row_shape(int H, int vec, int T)
{
    RowShape s;
    const int chunks = (H + vec - 1) / vec;
    const int wide = vec == 8 ? 2 : 16;                       // most chunks per thread
    int nv = 1;
    while (nv < wide && (chunks + nv - 1) / nv > 1024)
        nv = nv == 1 && vec == 1 ? 4 : nv * (vec == 8 ? 2 : 4);
    s.nv = nv;
    s.W = ((chunks + nv - 1) / nv + 31) / 32;
    s.R = s.W == 1 ? 4 : 1;
    (void)T;
    return s;
}

template <typename HT>
cudaError_t pre_launch(NormPreArgs a, bool vec8, cudaStream_t s)
{
    const RowShape sh = row_shape(a.H, vec8 ? 8 : 1, a.T);
    a.W = sh.W;
    const dim3 grid((unsigned)(((long)a.T + sh.R - 1) / sh.R)), block(32 * sh.W * sh.R);
    if (vec8)
        return sh.nv == 1 ? launch_after(vq_norm_pre_kernel<HT, 8, 1>, grid, block, 0, s, a)
                          : launch_after(vq_norm_pre_kernel<HT, 8, 2>, grid, block, 0, s, a);
    switch (sh.nv) {
    case 1: return launch_after(vq_norm_pre_kernel<HT, 1, 1>, grid, block, 0, s, a);
    case 4: return launch_after(vq_norm_pre_kernel<HT, 1, 4>, grid, block, 0, s, a);
    default: return launch_after(vq_norm_pre_kernel<HT, 1, 16>, grid, block, 0, s, a);
    }
}

template <typename YT, typename HT>
cudaError_t post_launch(NormPostArgs a, bool vec8, cudaStream_t s)
{
    const RowShape sh = row_shape(a.H, vec8 ? 8 : 1, a.T);
    a.W = sh.W;
    const dim3 grid((unsigned)(((long)a.T + sh.R - 1) / sh.R)), block(32 * sh.W * sh.R);
    if (vec8)
        return sh.nv == 1 ? launch_after(vq_norm_post_kernel<YT, HT, 8, 1>, grid, block, 0, s, a)
                          : launch_after(vq_norm_post_kernel<YT, HT, 8, 2>, grid, block, 0, s, a);
    switch (sh.nv) {
    case 1: return launch_after(vq_norm_post_kernel<YT, HT, 1, 1>, grid, block, 0, s, a);
    case 4: return launch_after(vq_norm_post_kernel<YT, HT, 1, 4>, grid, block, 0, s, a);
    default: return launch_after(vq_norm_post_kernel<YT, HT, 1, 16>, grid, block, 0, s, a);
    }
}

}  // namespace

cudaError_t launch_norm_pre(const NormPreArgs &a, int h_dtype, bool vec8, cudaStream_t s)
{
    return h_dtype == VQ_F32 ? pre_launch<float>(a, vec8, s) : pre_launch<uint16_t>(a, vec8, s);
}

cudaError_t launch_norm_post(const NormPostArgs &a, int y_dtype, int h_dtype, bool vec8, cudaStream_t s)
{
    if (y_dtype == VQ_F32)
        return h_dtype == VQ_F32 ? post_launch<float, float>(a, vec8, s) : post_launch<float, uint16_t>(a, vec8, s);
    return h_dtype == VQ_F32 ? post_launch<uint16_t, float>(a, vec8, s) : post_launch<uint16_t, uint16_t>(a, vec8, s);
}

}  // namespace vq
