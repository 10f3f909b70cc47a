// Block norms, forward: the norm that makes a MoE block's input, and the join
// of the block's output with the residual stream (norm, sigmoid gate, two
// scales, and the next block's norm) in one pass over each row.
//
//   norm_pre:  x = bf16(h r (w + off)),  r = rsqrt(mean(h^2) + eps)
//   norm_post: u = y r1 (w1 + off1) (or y); h' = a h + b s(z) u; x' = norm of the stored h'
//
// A row stays in the registers of one CTA (or one warp) between the row sum
// and the output, so each array crosses HBM once. Many rows: persistent CTAs
// with the next rows on their way. 4096 x 4096 bf16 with both norms takes 27.3
// us for 134 MB (4.9 TB/s, 0.75 of the copy rate), 4096 x 6144 36.5 us (0.84), 16384 x
// 512 13.9 us (0.74); a CTA per row from registers took 43 us for the first. norm_pre 4096
// x 4096 takes 12.9 us (0.80), 65536 x 256 12.6 us (0.82).
// What is left is latency: two row sums per row with 16 to 24 warps on an SM,
// which issue 2.1 instructions a cycle between them. The warps are as many as registers
// allow: both weights of a thread's columns stay in them as fp32 (32 of 89 to 120 with two
// chunks). Weights in shared memory, as the gradient has them, were not tried here. With
// four chunks (hidden over 12288) norm_post spills 60 to 110 bytes a thread: 1024 x 16384
// 49 us (0.53). Few rows: one load, one or two row sums and one store, 1.9 us (1 x 4096, pre)
// to 4.1 us (16 x 6144, post), the launch included.
#include <algorithm>

#include "vq_block.cuh"
#include "vq_norm.h"

namespace vq {
namespace {

// ---------------------------------------------------------------- any rows, element by element
//
// Rows off the 16-byte boundaries (odd widths, windows of wider arrays): a
// warp's loads and stores are contiguous elements, a row's fp32 values wait in
// shared memory between the passes, and several CTAs on an SM overlap. 1024 x 4099:
// norm_pre 11.4 us, norm_post (fp32 y) 26.7 us, where the bytes take 2.6 and 6.4: an access
// moves 2 or 4 bytes a lane, and nothing of a CTA's next row is on its way while it works on one.

template <typename HT>
__global__ void __launch_bounds__(ROW_THREADS) vq_norm_pre_scalar_kernel(const NormPreArgs a)
{
    __shared__ RowSum<1> rs;
    extern __shared__ float rows_f32[];
    grid_dep_launch();
    grid_dep_wait();
    const RowTeam team(a.W);
    const int step = 32 * team.W;
    float *u = rows_f32 + team.rg * a.H;
    int turn = 0;
    for (long row = (long)blockIdx.x * team.R + team.rg; row < a.T; row += (long)gridDim.x * team.R) {
        const HT *h = static_cast<const HT *>(a.h) + row * a.h_ld;
        float ss[1] = {0.f};
        for (int e0 = team.tid; e0 < a.H; e0 += BATCH * step) {
            float v[BATCH];
            batch(v, h, e0, step, a.H);
#pragma unroll
            for (int i = 0; i < BATCH; ++i)
                if (e0 + i * step < a.H) {
                    u[e0 + i * step] = v[i];
                    ss[0] = fmaf(v[i], v[i], ss[0]);
                }
        }
        row_sum(ss, rs, team, turn);
        const float r = rsqrtf(ss[0] * a.inv_h + a.n.eps);
        uint16_t *x = a.x + row * a.x_ld;
        for (int e0 = team.tid; e0 < a.H; e0 += BATCH * step) {
            float w[BATCH], v[BATCH];
            batch_any(w, a.n.weight, a.n.dtype, 0, e0, step, a.H);
            batch(v, u, e0, step, a.H);
#pragma unroll
            for (int i = 0; i < BATCH; ++i)
                if (e0 + i * step < a.H)
                    put(x[e0 + i * step], v[i] * r * (w[i] + a.n.offset));
        }
    }
}

template <typename YT, typename HT>
__global__ void __launch_bounds__(ROW_THREADS) vq_norm_post_scalar_kernel(const NormPostArgs a)
{
    __shared__ RowSum<1> rs;
    extern __shared__ float rows_f32[];
    grid_dep_launch();
    grid_dep_wait();
    const RowTeam team(a.W);
    const int step = 32 * team.W;
    float *u = rows_f32 + team.rg * a.H;
    int turn = 0;
    for (long row = (long)blockIdx.x * team.R + team.rg; row < a.T; row += (long)gridDim.x * team.R) {
        const YT *y = static_cast<const YT *>(a.y) + row * a.y_ld;
        const HT *h = static_cast<const HT *>(a.h) + row * a.h_ld;
        HT *ho = static_cast<HT *>(a.h_out) + row * a.ho_ld;
        float f = a.out_scale;   // the branch's factor, but for the weight and a channel's gate
        if (a.gate_mode == GATE_TOKEN)
            f *= sigmoid(weight_at(a.gate, a.gate_dtype, row * a.gate_ld));
        if (a.post.weight) {
            float ss[1] = {0.f};
            for (int e0 = team.tid; e0 < a.H; e0 += BATCH * step) {
                float v[BATCH];
                batch(v, y, e0, step, a.H);
#pragma unroll
                for (int i = 0; i < BATCH; ++i)
                    if (e0 + i * step < a.H) {
                        u[e0 + i * step] = v[i];
                        ss[0] = fmaf(v[i], v[i], ss[0]);
                    }
            }
            row_sum(ss, rs, team, turn);
            f *= rsqrtf(ss[0] * a.inv_h + a.post.eps);
        }
        float ss[1] = {0.f};
        for (int e0 = team.tid; e0 < a.H; e0 += BATCH * step) {
            float v[BATCH], w[BATCH], z[BATCH], r[BATCH];
            batch(r, h, e0, step, a.H);
            if (a.post.weight) {
                batch(v, u, e0, step, a.H);
                batch_any(w, a.post.weight, a.post.dtype, 0, e0, step, a.H);
            } else {
                batch(v, y, e0, step, a.H);
            }
            if (a.gate_mode == GATE_CHANNEL)
                batch_any(z, a.gate, a.gate_dtype, row * a.gate_ld, e0, step, a.H);
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                const int e = e0 + i * step;
                if (e >= a.H)
                    break;
                v[i] *= f;
                if (a.post.weight)
                    v[i] *= w[i] + a.post.offset;
                if (a.gate_mode == GATE_CHANNEL)
                    v[i] *= sigmoid(z[i]);
                HT o;
                put(o, fmaf(a.res_scale, r[i], v[i]));
                ho[e] = o;   // the row as stored: what the next norm sees
                u[e] = element(o);
                ss[0] = fmaf(element(o), element(o), ss[0]);
            }
        }
        if (!a.next.weight)
            continue;
        row_sum(ss, rs, team, turn);
        const float r = rsqrtf(ss[0] * a.inv_h + a.next.eps);
        uint16_t *x = a.x + row * a.x_ld;
        for (int e0 = team.tid; e0 < a.H; e0 += BATCH * step) {
            float w[BATCH], v[BATCH];
            batch_any(w, a.next.weight, a.next.dtype, 0, e0, step, a.H);
            batch(v, u, e0, step, a.H);
#pragma unroll
            for (int i = 0; i < BATCH; ++i)
                if (e0 + i * step < a.H)
                    put(x[e0 + i * step], v[i] * r * (w[i] + a.next.offset));
        }
    }
}

// ---------------------------------------------------------------- rows on 16-byte boundaries
//
// Persistent CTAs, two or more on an SM; each copies its next rows into shared
// memory while it works on one. A thread's columns are the same in every row,
// so the weights stay in its registers.

template <typename HT, int NV>
__global__ void __launch_bounds__(ROW_THREADS) vq_norm_pre_kernel(const NormPreArgs a, int S)
{
    __shared__ RowSum<1> rs;
    extern __shared__ __align__(16) unsigned char ring[];
    constexpr int PH = PIECES<HT>, P = NV * PH;
    const RowTeam team(a.W);
    const int W = team.W, tid = team.tid, R = team.R, stride = gridDim.x * R;
    const long row0 = (long)blockIdx.x * R + team.rg;
    const uint32_t step = blockDim.x * 16, base = (uint32_t)__cvta_generic_to_shared(ring) + threadIdx.x * 16;
    const int hop = 256 * W;   // elements from a thread's chunk to its next
    const HT *h = static_cast<const HT *>(a.h) + row0 * a.h_ld + tid * 8;
    uint16_t *x = a.x + row0 * a.x_ld + tid * 8;
    bool in[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i)
        in[i] = chunk_at(i, tid, W) < a.H;
    long ahead = row0;   // the row the next copy is for
    auto fetch = [&](int s) {
        if (ahead < a.T) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (in[i])
                    ring_copy(base + (s * P + i * PH) * step, step, h + i * hop);
            h += stride * a.h_ld;
            ahead += stride;
        }
        copy_commit();
    };
    grid_dep_launch();
    grid_dep_wait();
    for (int s = 0; s < S - 1; ++s)
        fetch(s);
    float2 w[NV][4];
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (in[i])
            load_weight(a.n.weight, a.n.dtype, a.n.offset, chunk_at(i, tid, W), w[i]);
    int turn = 0, s = 0;
    for (long row = row0; row < a.T; row += stride) {
        if (S == 1) {
            fetch(0);
            copy_wait(0);
        } else {
            copy_wait(S - 2);
            fetch(s == 0 ? S - 1 : s - 1);
        }
        const uint32_t at = base + s * P * step;
        s = s == S - 1 ? 0 : s + 1;
        float2 v[NV][4], sq = splat(0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (in[i]) {
                ring_get<HT>(at + i * PH * step, step, v[i]);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    sq = fma2(v[i][j], v[i][j], sq);
            }
        float ss[1] = {sq.x + sq.y};
        row_sum(ss, rs, team, turn);
        const float r = rsqrtf(ss[0] * a.inv_h + a.n.eps);
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (in[i]) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    v[i][j] = mul2(mul2(v[i][j], splat(r)), w[i][j]);
                Chunk<uint16_t, 8> o;
                o.set(v[i]);
                o.store(x + i * hop);
            }
        x += stride * a.x_ld;
    }
}

template <typename YT, typename HT, int NV>
__global__ void __launch_bounds__(ROW_THREADS) vq_norm_post_kernel(const NormPostArgs a, int S)
{
    __shared__ RowSum<1> rs;
    extern __shared__ __align__(16) unsigned char ring[];
    // pieces of a stage: y, h, per-channel gates
    constexpr int PY = PIECES<YT>, PH = PIECES<HT>, OH = NV * PY, OZ = OH + NV * PH;
    const bool post = a.post.weight != nullptr, next = a.next.weight != nullptr;
    const int pz = a.gate_mode != GATE_CHANNEL ? 0 : a.gate_dtype == VQ_F32 ? 2 : 1, P = OZ + NV * pz;
    const RowTeam team(a.W);
    const int W = team.W, tid = team.tid, R = team.R, stride = gridDim.x * R;
    const long row0 = (long)blockIdx.x * R + team.rg;
    const uint32_t step = blockDim.x * 16, base = (uint32_t)__cvta_generic_to_shared(ring) + threadIdx.x * 16;
    const int hop = 256 * W;   // elements from a thread's chunk to its next
    const YT *y = static_cast<const YT *>(a.y) + row0 * a.y_ld + tid * 8;
    const HT *h = static_cast<const HT *>(a.h) + row0 * a.h_ld + tid * 8;
    HT *ho = static_cast<HT *>(a.h_out) + row0 * a.ho_ld + tid * 8;
    uint16_t *x = a.x + row0 * a.x_ld + tid * 8;
    bool in[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i)
        in[i] = chunk_at(i, tid, W) < a.H;
    long ahead = row0;   // the row the next copy is for
    auto fetch = [&](int s) {
        if (ahead < a.T) {
            const uint32_t at = base + s * P * step;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (in[i]) {
                    ring_copy(at + i * PY * step, step, y + i * hop);
                    ring_copy(at + (OH + i * PH) * step, step, h + i * hop);
                    if (pz)
                        ring_copy_any(at + (OZ + i * pz) * step, step, a.gate, a.gate_dtype,
                                      ahead * a.gate_ld + tid * 8 + i * hop);
                }
            y += stride * a.y_ld;
            h += stride * a.h_ld;
            ahead += stride;
        }
        copy_commit();
    };
    grid_dep_launch();
    grid_dep_wait();
    for (int s = 0; s < S - 1; ++s)
        fetch(s);
    float2 w1[NV][4], w2[NV][4];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            w1[i][j] = w2[i][j] = splat(1.f);
        if (in[i]) {
            if (post)
                load_weight(a.post.weight, a.post.dtype, a.post.offset, chunk_at(i, tid, W), w1[i]);
            if (next)
                load_weight(a.next.weight, a.next.dtype, a.next.offset, chunk_at(i, tid, W), w2[i]);
        }
    }
    int turn = 0, s = 0;
    for (long row = row0; row < a.T; row += stride) {
        float f = a.out_scale;   // the branch's factor, but for the weight and a channel's gate
        if (a.gate_mode == GATE_TOKEN) {
            AnyChunk<1> z;
            float v[1];
            z.load(a.gate, a.gate_dtype, row * a.gate_ld);
            z.get(v, a.gate_dtype);
            f *= sigmoid(v[0]);
        }
        if (S == 1) {
            fetch(0);
            copy_wait(0);
        } else {
            copy_wait(S - 2);
            fetch(s == 0 ? S - 1 : s - 1);
        }
        const uint32_t at = base + s * P * step;
        s = s == S - 1 ? 0 : s + 1;
        float2 u[NV][4], sq = splat(0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (in[i]) {
                ring_get<YT>(at + i * PY * step, step, u[i]);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    sq = fma2(u[i][j], u[i][j], sq);
            }
        if (post) {
            float ss[1] = {sq.x + sq.y};
            row_sum(ss, rs, team, turn);
            f *= rsqrtf(ss[0] * a.inv_h + a.post.eps);
        }
        sq = splat(0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (in[i]) {
                float2 v[4];
                ring_get<HT>(at + (OH + i * PH) * step, step, v);
                if (pz) {
                    float2 z[4];
                    ring_get_any(at + (OZ + i * pz) * step, step, a.gate_dtype, z);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        u[i][j] = mul2(u[i][j], make_float2(sigmoid(z[j].x), sigmoid(z[j].y)));
                }
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    v[j] = fma2(mul2(u[i][j], splat(f)), w1[i][j], mul2(v[j], splat(a.res_scale)));
                Chunk<HT, 8> o;
                o.set(v);   // the row as stored: what the next norm sees
                o.store(ho + i * hop);
                o.get(u[i]);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    sq = fma2(u[i][j], u[i][j], sq);
            }
        ho += stride * a.ho_ld;
        if (next) {
            float ss[1] = {sq.x + sq.y};
            row_sum(ss, rs, team, turn);
            const float r2 = rsqrtf(ss[0] * a.inv_h + a.next.eps);
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (in[i]) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        u[i][j] = mul2(mul2(u[i][j], splat(r2)), w2[i][j]);
                    Chunk<uint16_t, 8> o;
                    o.set(u[i]);
                    o.store(x + i * hop);
                }
            x += stride * a.x_ld;
        }
    }
}

template <typename HT>
cudaError_t pre_launch(NormPreArgs a, bool vec8, cudaStream_t s)
{
    int regs[4];
    const cudaError_t e = ring_regs<vq_norm_pre_kernel<HT, 1>, vq_norm_pre_kernel<HT, 2>, vq_norm_pre_kernel<HT, 3>,
                                    vq_norm_pre_kernel<HT, 4>>(regs);
    if (e != cudaSuccess)
        return e;
    const NormShape sh = norm_shape(a.H, a.T, sizeof(HT), 0, regs, 2, 2, 0);
    if (vec8 && sh.S > 0) {
        a.W = sh.W;
        switch (sh.nv) {
        case 1: return launch_rows<vq_norm_pre_kernel<HT, 1>>(sh, s, a);
        case 2: return launch_rows<vq_norm_pre_kernel<HT, 2>>(sh, s, a);
        case 3: return launch_rows<vq_norm_pre_kernel<HT, 3>>(sh, s, a);
        default: return launch_rows<vq_norm_pre_kernel<HT, 4>>(sh, s, a);
        }
    }
    const NormShape sc = scalar_shape(a.H, a.T, 1, 0);
    a.W = sc.W;
    return launch_smem<vq_norm_pre_scalar_kernel<HT>, SCALAR_SMEM>(dim3(sc.ctas), dim3(32 * sc.W * sc.R), sc.smem, s, a);
}

template <typename YT, typename HT>
cudaError_t post_launch(NormPostArgs a, bool vec8, cudaStream_t s)
{
    const int gate = a.gate_mode != GATE_CHANNEL ? 0 : a.gate_dtype == VQ_F32 ? 4 : 2;
    int regs[4];
    const cudaError_t e = ring_regs<vq_norm_post_kernel<YT, HT, 1>, vq_norm_post_kernel<YT, HT, 2>,
                                    vq_norm_post_kernel<YT, HT, 3>, vq_norm_post_kernel<YT, HT, 4>>(regs);
    if (e != cudaSuccess)
        return e;
    const NormShape sh = norm_shape(a.H, a.T, sizeof(YT) + sizeof(HT) + gate, 0, regs, 2, 3, 0);
    if (vec8 && sh.S > 0) {
        a.W = sh.W;
        switch (sh.nv) {
        case 1: return launch_rows<vq_norm_post_kernel<YT, HT, 1>>(sh, s, a);
        case 2: return launch_rows<vq_norm_post_kernel<YT, HT, 2>>(sh, s, a);
        case 3: return launch_rows<vq_norm_post_kernel<YT, HT, 3>>(sh, s, a);
        default: return launch_rows<vq_norm_post_kernel<YT, HT, 4>>(sh, s, a);
        }
    }
    const NormShape sc = scalar_shape(a.H, a.T, 1, 0);
    a.W = sc.W;
    return launch_smem<vq_norm_post_scalar_kernel<YT, HT>, SCALAR_SMEM>(dim3(sc.ctas), dim3(32 * sc.W * sc.R), sc.smem, s, a);
}

}  // namespace

NormShape scalar_shape(int H, int T, int floats, int max_ctas)
{
    NormShape s{};
    s.W = H <= 128 ? 1 : H <= 256 ? 2 : H <= 512 ? 4 : H <= 8192 ? 8 : 16;
    s.R = std::max(1, 8 / s.W);
    s.smem = (size_t)s.R * H * floats * sizeof(float);
    const int per_sm = (int)std::max<size_t>(1, std::min<size_t>(s.W == 16 ? 3 : 6, SCALAR_SMEM / (s.smem + 2048)));
    long ctas = std::min(((long)T + s.R - 1) / s.R, 148L * per_sm);
    if (max_ctas)
        ctas = std::min<long>(ctas, max_ctas);
    s.ctas = (int)std::max(1L, ctas);
    return s;
}

NormShape norm_shape(int H, int T, int bytes, int fixed, const int (&regs)[4], int nv, int max_nv,
                     int max_ctas)
{
    NormShape s;
    const int chunks = (H + 7) / 8;
    const bool stream = T > 2 * 148;
    // With at most a row or two per SM a row takes as many threads as it can use. Rows that stream take the kernel's nv
    // chunks a thread (the row sums and the addresses cost by the warp), more up to its max_nv before they take over
    // 256 threads, and share a CTA of 8 warps when they are narrow. Measured (us) with 1, 2, 3 and 4 chunks: post 4096 x
    // 4096 29.1, 27.8, 28.3, 33.6; pre backward 38.5, 31.1, 31.3, 27.3; post backward 100, 81, 134, 105.
    s.nv = !stream ? (chunks + ROW_THREADS - 1) / ROW_THREADS
           : chunks <= 512 ? std::min(nv, (chunks + 31) / 32)
           : chunks <= 256 * max_nv ? (chunks + 255) / 256
                                    : (chunks + ROW_THREADS - 1) / ROW_THREADS;
    s.W = ((chunks + s.nv - 1) / s.nv + 31) / 32;
    s.R = s.W == 1 || stream ? std::max(1, 8 / s.W) : 1;
    const size_t row = (size_t)32 * s.W * 8 * s.nv, keep = row * fixed, room = NORM_SMEM;
    // with weights in shared memory: rows side by side share them, up to ROW_THREADS threads
    if (fixed && stream)
        while (2 * s.R * 32 * s.W <= ROW_THREADS && 2 * 2 * s.R * row * bytes + keep <= room)
            s.R *= 2;
    const int block = 32 * s.W * s.R;
    const size_t stage = row * s.R * bytes;
    s.S = s.ctas = 0;
    s.smem = 0;
    if (stage + keep > room)
        return s;
    // two rows ahead where they fit, then as many CTAs as registers and shared memory allow
    int per_sm = std::max(1, std::min(16, 65536 / (regs[s.nv - 1] * block)));
    while (per_sm > 1 && per_sm * (2 * stage + keep + 2048) > room)
        --per_sm;
    s.S = (int)std::min<size_t>(4, (room / per_sm - keep - (per_sm > 1 ? 2048 : 0)) / stage);
    long ctas = std::min(((long)T + s.R - 1) / s.R, 148L * per_sm);
    if (max_ctas)
        ctas = std::min<long>(ctas, max_ctas);
    s.ctas = (int)std::max(1L, ctas);
    // no more stages than a CTA has rows
    const long rows = ((long)T + (long)s.ctas * s.R - 1) / ((long)s.ctas * s.R);
    s.S = (int)std::min<long>(s.S, std::max(1L, rows));
    s.smem = s.S * stage + keep;
    return s;
}

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
