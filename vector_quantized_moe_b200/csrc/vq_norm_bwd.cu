// Block norms, backward. With n(v) = v r (w + off), r = rsqrt(mean(v^2) + eps),
// v^ = v r and g = (w + off) d for the output's gradient d:
//   dv = r (g - v^ mean(g v^)),   dw = sum over rows of d v^.
// norm_post's gradient chains two of them around the sigmoid gate: first at
// the stored row h' (the next norm), then at y (the post norm).
//
// Persistent CTAs take rows in turn; a thread keeps its columns' weight
// gradients in registers over all rows of its CTA, one partial row per CTA goes
// to the workspace, and a second kernel adds the partial rows in order. No
// statistics are saved: the row sums that need only the inputs (|h'|^2, g h',
// |y|^2) come out of one pass, so recomputing them adds no barrier.
//
// Measured: norm_pre's 4096 x 6144 bf16 with a residual gradient 37.9 us for 201 MB
// (5.3 TB/s, 0.81 of the copy rate); norm_post's 2047 x 4096 with both norms and a
// gate per channel 47.6 us for 168 MB (3.5 TB/s, 0.54). The second holds 128 registers a
// thread (two weight gradients), so an SM has 16 warps, at two rows a time; it
// is bound by their latency between the two row sums (1.8 instructions a
// cycle), not by HBM. Wider rows have one CTA of one row on an SM, 12 warps at
// 6144: 4096 x 6144 (fp32 y) 121 us (0.51). With three and four chunks (hidden over 8192) it
// spills 130 to 660 bytes a thread: 1024 x 12288 83 us (0.37), 1024 x 16384 306 us (0.13).
#include <algorithm>

#include "vq_block.cuh"
#include "vq_norm.h"

namespace vq {
namespace {

constexpr int NORM_PARTS = 592;     // most partial rows: 4 CTAs on each of 148 SMs

// ---------------------------------------------------------------- any rows, element by element
//
// A thread's columns are the same in every row, so the weight gradients' sums
// wait in shared memory without a barrier. Arrays are read again in each pass
// (from L1 or L2), 2 or 4 bytes a lane. 1024 x 4099: norm_pre's 32 us, norm_post's (fp32 y)
// 77 us, where the bytes take 5.1 and 10.3.

// A CTA's partial row: its side-by-side rows' sums (the first floats of each row's share) added in order.
__device__ __forceinline__ void write_part_scalar(float *part, const float *acc, int share, int R, int H)
{
    __syncthreads();
    for (int e = threadIdx.x; e < H; e += blockDim.x) {
        float v = acc[e];
        for (int r = 1; r < R; ++r)
            v += acc[(size_t)r * share + e];
        part[(long)blockIdx.x * H + e] = v;
    }
}

template <typename HT>
__global__ void __launch_bounds__(ROW_THREADS) vq_norm_pre_bwd_scalar_kernel(const NormPreBwdArgs a)
{
    __shared__ RowSum<2> rs;
    extern __shared__ float sums[];   // [R][H]
    grid_dep_launch();
    grid_dep_wait();
    const RowTeam team(a.W);
    const int step = 32 * team.W;
    float *acc = sums + team.rg * a.H;
    for (int e = team.tid; e < a.H; e += step)
        acc[e] = 0.f;
    int turn = 0;
    for (long row = (long)blockIdx.x * team.R + team.rg; row < a.T; row += (long)gridDim.x * team.R) {
        const HT *h = static_cast<const HT *>(a.h) + row * a.h_ld;
        const HT *dres = static_cast<const HT *>(a.dres) + row * a.dres_ld;
        const uint16_t *dx = a.dx + row * a.dx_ld;
        HT *dh = static_cast<HT *>(a.dh) + row * a.dh_ld;
        float q[2] = {0.f, 0.f};   // |h|^2, sum g h
        for (int e0 = team.tid; e0 < a.H; e0 += BATCH * step) {
            float v[BATCH], d[BATCH], w[BATCH];
            batch(v, h, e0, step, a.H);
            batch(d, dx, e0, step, a.H);
            batch_any(w, a.n.weight, a.n.dtype, 0, e0, step, a.H);
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {   // elements past the row are zeros
                q[0] = fmaf(v[i], v[i], q[0]);
                q[1] = fmaf(d[i] * (w[i] + a.n.offset), v[i], q[1]);
            }
        }
        row_sum(q, rs, team, turn);
        const float r = rsqrtf(q[0] * a.inv_h + a.n.eps);
        const float rm = r * (r * (q[1] * a.inv_h));   // r mean(g v^)
        for (int e0 = team.tid; e0 < a.H; e0 += BATCH * step) {
            float v[BATCH], d[BATCH], w[BATCH], o[BATCH];
            batch(v, h, e0, step, a.H);
            batch(d, dx, e0, step, a.H);
            batch_any(w, a.n.weight, a.n.dtype, 0, e0, step, a.H);
            if (a.dres)
                batch(o, dres, e0, step, a.H);
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                const int e = e0 + i * step;
                if (e >= a.H)
                    break;
                const float n = v[i] * r, t = fmaf(-n, rm, r * (d[i] * (w[i] + a.n.offset)));
                acc[e] = fmaf(d[i], n, acc[e]);
                put(dh[e], a.dres ? o[i] + t : t);
            }
        }
    }
    if (a.part)
        write_part_scalar(a.part, sums, a.H, team.R, a.H);
}

template <typename YT, typename HT>
__global__ void __launch_bounds__(ROW_THREADS) vq_norm_post_bwd_scalar_kernel(const NormPostBwdArgs a)
{
    __shared__ RowSum<3> rs;
    extern __shared__ float sums[];   // [R][3][H]: the two weight gradients, and a row's values between the passes
    grid_dep_launch();
    grid_dep_wait();
    const RowTeam team(a.W);
    const int step = 32 * team.W;
    const bool post = a.post.weight != nullptr, next = a.next.weight != nullptr;
    float *acc1 = sums + (size_t)team.rg * 3 * a.H, *acc2 = acc1 + a.H, *g = acc2 + a.H;
    for (int e = team.tid; e < a.H; e += step)
        acc1[e] = acc2[e] = 0.f;
    int turn = 0;
    for (long row = (long)blockIdx.x * team.R + team.rg; row < a.T; row += (long)gridDim.x * team.R) {
        const YT *y = static_cast<const YT *>(a.y) + row * a.y_ld;
        const HT *h = static_cast<const HT *>(a.h) + row * a.h_ld;
        const HT *dho = static_cast<const HT *>(a.dho) + row * a.dho_ld;
        const uint16_t *dx = a.dx + row * a.dx_ld;
        YT *dy = static_cast<YT *>(a.dy) + row * a.dy_ld;
        HT *dh = static_cast<HT *>(a.dh) + row * a.dh_ld;
        float on = 1.f, off = 0.f;   // sigmoid(z), 1 - sigmoid(z)
        if (a.gate_mode == GATE_TOKEN)
            sigmoids(weight_at(a.gate, a.gate_dtype, row * a.gate_ld), on, off);
        float q[3] = {0.f, 0.f, 0.f};   // |h'|^2, sum g h' of the next norm, |y|^2
        if (next || post) {
            for (int e0 = team.tid; e0 < a.H; e0 += BATCH * step) {
                float v[BATCH], d[BATCH], w[BATCH];
                if (next) {
                    batch(v, h, e0, step, a.H);
                    batch(d, dx, e0, step, a.H);
                    batch_any(w, a.next.weight, a.next.dtype, 0, e0, step, a.H);
#pragma unroll
                    for (int i = 0; i < BATCH; ++i) {   // elements past the row are zeros
                        q[0] = fmaf(v[i], v[i], q[0]);
                        q[1] = fmaf(d[i] * (w[i] + a.next.offset), v[i], q[1]);
                    }
                }
                if (post) {
                    batch(v, y, e0, step, a.H);
#pragma unroll
                    for (int i = 0; i < BATCH; ++i)
                        q[2] = fmaf(v[i], v[i], q[2]);
                }
            }
            row_sum(q, rs, team, turn);
        }
        const float r2 = rsqrtf(q[0] * a.inv_h + a.next.eps), rm2 = r2 * (r2 * (q[1] * a.inv_h));
        const float r1 = post ? rsqrtf(q[2] * a.inv_h + a.post.eps) : 1.f;
        float t[2] = {0.f, 0.f};   // sums: g y^ of the post norm, dv u of a token's gate
        for (int e0 = team.tid; e0 < a.H; e0 += BATCH * step) {
            float dH[BATCH], v[BATCH], w[BATCH], z[BATCH], hv[BATCH], d[BATCH], w2[BATCH];
            batch(v, y, e0, step, a.H);
            if (a.dho)
                batch(dH, dho, e0, step, a.H);
            if (next) {
                batch(hv, h, e0, step, a.H);
                batch(d, dx, e0, step, a.H);
                batch_any(w2, a.next.weight, a.next.dtype, 0, e0, step, a.H);
            }
            if (post)
                batch_any(w, a.post.weight, a.post.dtype, 0, e0, step, a.H);
            if (a.gate_mode == GATE_CHANNEL)
                batch_any(z, a.gate, a.gate_dtype, row * a.gate_ld, e0, step, a.H);
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                const int e = e0 + i * step;
                if (e >= a.H)
                    break;
                float s = a.dho ? dH[i] : 0.f;
                if (next) {
                    const float n = hv[i] * r2;
                    acc2[e] = fmaf(d[i], n, acc2[e]);
                    s += fmaf(-n, rm2, r2 * (d[i] * (w2[i] + a.next.offset)));
                }
                if (a.dh)
                    put(dh[e], a.res_scale * s);
                const float dv = a.out_scale * s, n = v[i] * r1, wj = post ? w[i] + a.post.offset : 1.f;
                float zon = on, zoff;
                if (a.gate_mode == GATE_CHANNEL) {
                    sigmoids(z[i], zon, zoff);
                    if (a.dgate) {
                        const float dz = dv * (n * wj) * zon * zoff;
                        const long to = row * a.dgate_ld + e;
                        if (a.gate_dtype == VQ_F32)
                            static_cast<float *>(a.dgate)[to] = dz;
                        else
                            put(static_cast<uint16_t *>(a.dgate)[to], dz);
                    }
                }
                const float du = dv * zon;
                acc1[e] = fmaf(du, n, acc1[e]);
                g[e] = du * wj;
                t[0] = fmaf(du * wj, n, t[0]);
                t[1] = fmaf(dv, n * wj, t[1]);
            }
        }
        const bool token = a.gate_mode == GATE_TOKEN && a.dgate;
        if (post || token)
            row_sum(t, rs, team, turn);
        if (token && team.tid == 0) {
            const float dz = t[1] * on * off;
            const long to = row * a.dgate_ld;
            if (a.gate_dtype == VQ_F32)
                static_cast<float *>(a.dgate)[to] = dz;
            else
                put(static_cast<uint16_t *>(a.dgate)[to], dz);
        }
        const float rm1 = r1 * (t[0] * a.inv_h);   // r1 mean(g y^)
        for (int e0 = team.tid; e0 < a.H; e0 += BATCH * step) {
            float v[BATCH], o[BATCH];
            batch(o, g, e0, step, a.H);
            if (post)
                batch(v, y, e0, step, a.H);
#pragma unroll
            for (int i = 0; i < BATCH; ++i)
                if (e0 + i * step < a.H)
                    put(dy[e0 + i * step], post ? fmaf(-(v[i] * r1), rm1, r1 * o[i]) : o[i]);
        }
    }
    if (a.part1)
        write_part_scalar(a.part1, sums, 3 * a.H, team.R, a.H);
    if (a.part2)
        write_part_scalar(a.part2, sums + a.H, 3 * a.H, team.R, a.H);
}

// ---------------------------------------------------------------- rows on 16-byte boundaries, copied ahead

// A CTA's weight gradient: the sums of its side-by-side rows added in order
// into one partial row. side: H floats of shared memory.
template <int NV>
__device__ __forceinline__ void write_part(float *part, float2 (&acc)[NV][4], float *side, int tid, int W, int H)
{
    const int R = blockDim.x / (32 * W), rg = threadIdx.x / (32 * W);
    for (int r = 1; r < R; ++r) {
        __syncthreads();
        if (rg == r)
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (chunk_at(i, tid, W) < H) {
                    Chunk<float, 8> o;
                    o.set(acc[i]);
                    o.store(side + chunk_at(i, tid, W));
                }
        __syncthreads();
        if (rg == 0)
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (chunk_at(i, tid, W) < H) {
                    Chunk<float, 8> o;
                    float2 v[4];
                    o.load(side + chunk_at(i, tid, W));
                    o.get(v);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        acc[i][j] = add2(acc[i][j], v[j]);
                }
    }
    if (rg == 0)
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = chunk_at(i, tid, W);
            if (c < H) {
                Chunk<float, 8> o;
                o.set(acc[i]);
                o.store(part + (long)blockIdx.x * H + c);
            }
        }
}

template <typename HT, int NV>
__global__ void __launch_bounds__(ROW_THREADS) vq_norm_pre_bwd_kernel(const NormPreBwdArgs a, int S)
{
    __shared__ RowSum<2> rs;
    extern __shared__ __align__(16) unsigned char ring[];
    constexpr int PH = PIECES<HT>, OX = NV * PH, OR = OX + NV;   // pieces: h, dx, dres
    const bool res = a.dres != nullptr;
    const int P = OR + (res ? NV * PH : 0);
    const RowTeam team(a.W);
    const int W = team.W, tid = team.tid, R = team.R, stride = gridDim.x * R;
    const long row0 = (long)blockIdx.x * R + team.rg;
    const uint32_t step = blockDim.x * 16, base = (uint32_t)__cvta_generic_to_shared(ring) + threadIdx.x * 16;
    const int hop = 256 * W;   // elements from a thread's chunk to its next
    const HT *h = static_cast<const HT *>(a.h) + row0 * a.h_ld + tid * 8;
    const HT *dres = static_cast<const HT *>(a.dres) + row0 * a.dres_ld + tid * 8;
    const uint16_t *dx = a.dx + row0 * a.dx_ld + tid * 8;
    HT *dh = static_cast<HT *>(a.dh) + row0 * a.dh_ld + tid * 8;
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
                    ring_copy(at + i * PH * step, step, h + i * hop);
                    ring_copy(at + (OX + i) * step, step, dx + i * hop);
                    if (res)
                        ring_copy(at + (OR + i * PH) * step, step, dres + i * hop);
                }
            h += stride * a.h_ld;
            dx += stride * a.dx_ld;
            dres += stride * a.dres_ld;
            ahead += stride;
        }
        copy_commit();
    };
    grid_dep_launch();
    grid_dep_wait();
    for (int s = 0; s < S - 1; ++s)
        fetch(s);
    float2 acc[NV][4], w[NV][4];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (in[i])
            load_weight(a.n.weight, a.n.dtype, a.n.offset, chunk_at(i, tid, W), w[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            acc[i][j] = splat(0.f);
    }
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
        float2 q0 = splat(0.f), q1 = q0;   // |h|^2, sum g h
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (in[i]) {
                float2 v[4], d[4];
                ring_get<HT>(at + i * PH * step, step, v);
                ring_get<uint16_t>(at + (OX + i) * step, step, d);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    q0 = fma2(v[j], v[j], q0);
                    q1 = fma2(mul2(d[j], w[i][j]), v[j], q1);
                }
            }
        float q[2] = {q0.x + q0.y, q1.x + q1.y};
        row_sum(q, rs, team, turn);
        const float r = rsqrtf(q[0] * a.inv_h + a.n.eps);
        const float rm = r * (r * (q[1] * a.inv_h));   // r mean(g v^)
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (in[i]) {
                float2 v[4], d[4], o[4];
                ring_get<HT>(at + i * PH * step, step, v);
                ring_get<uint16_t>(at + (OX + i) * step, step, d);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    o[j] = splat(0.f);
                if (res)
                    ring_get<HT>(at + (OR + i * PH) * step, step, o);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 n = mul2(v[j], splat(r));
                    acc[i][j] = fma2(d[j], n, acc[i][j]);
                    o[j] = add2(o[j], fma2(n, splat(-rm), mul2(mul2(d[j], w[i][j]), splat(r))));   // r (g - v^ mean(g v^))
                }
                Chunk<HT, 8> oc;
                oc.set(o);
                oc.store(dh + i * hop);
            }
        dh += stride * a.dh_ld;
    }
    if (a.part)
        write_part(a.part, acc, reinterpret_cast<float *>(ring), tid, W, a.H);
}

// The weights of a thread's columns sit in shared memory behind the ring: with
// two weight gradients a thread has no registers for them.
template <typename YT, typename HT, int NV>
__global__ void __launch_bounds__(ROW_THREADS) vq_norm_post_bwd_kernel(const NormPostBwdArgs a, int S)
{
    __shared__ RowSum<3> rs;
    extern __shared__ __align__(16) unsigned char ring[];
    const bool post = a.post.weight != nullptr, next = a.next.weight != nullptr, has = a.dho != nullptr;
    // pieces of a stage: y, dh_out, h_out and dx_out (with the next norm), per-channel gates
    constexpr int PY = PIECES<YT>, PH = PIECES<HT>, OG = NV * PY;
    const int OH = OG + (has ? NV * PH : 0), OX = OH + (next ? NV * PH : 0), OZ = OX + (next ? NV : 0);
    const int pz = a.gate_mode != GATE_CHANNEL ? 0 : a.gate_dtype == VQ_F32 ? 2 : 1, P = OZ + NV * pz;
    const RowTeam team(a.W);
    const int W = team.W, tid = team.tid, R = team.R, stride = gridDim.x * R;
    const long row0 = (long)blockIdx.x * R + team.rg;
    const uint32_t step = blockDim.x * 16, base = (uint32_t)__cvta_generic_to_shared(ring) + threadIdx.x * 16;
    // the weights, one copy for all rows side by side
    const uint32_t wstep = 32 * W * 16;
    const uint32_t at1 = (uint32_t)__cvta_generic_to_shared(ring) + S * P * step + tid * 16;
    const int p1 = !post ? 0 : a.post.dtype == VQ_F32 ? 2 : 1, p2 = a.next.dtype == VQ_F32 ? 2 : 1;
    const uint32_t at2 = at1 + p1 * NV * wstep;
    const int hop = 256 * W;   // elements from a thread's chunk to its next
    const YT *y = static_cast<const YT *>(a.y) + row0 * a.y_ld + tid * 8;
    const HT *h = static_cast<const HT *>(a.h) + row0 * a.h_ld + tid * 8;
    const HT *dho = static_cast<const HT *>(a.dho) + row0 * a.dho_ld + tid * 8;
    const uint16_t *dx = a.dx + row0 * a.dx_ld + tid * 8;
    YT *dy = static_cast<YT *>(a.dy) + row0 * a.dy_ld + tid * 8;
    HT *dh = static_cast<HT *>(a.dh) + row0 * a.dh_ld + tid * 8;
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
                    if (has)
                        ring_copy(at + (OG + i * PH) * step, step, dho + i * hop);
                    if (next) {
                        ring_copy(at + (OH + i * PH) * step, step, h + i * hop);
                        ring_copy(at + (OX + i) * step, step, dx + i * hop);
                    }
                    if (pz)
                        ring_copy_any(at + (OZ + i * pz) * step, step, a.gate, a.gate_dtype,
                                      ahead * a.gate_ld + tid * 8 + i * hop);
                }
            y += stride * a.y_ld;
            h += stride * a.h_ld;
            dho += stride * a.dho_ld;
            dx += stride * a.dx_ld;
            ahead += stride;
        }
        copy_commit();
    };
    grid_dep_launch();
    grid_dep_wait();
    float2 acc1[NV][4], acc2[NV][4];
#pragma unroll
    for (int i = 0; i < NV; ++i) {   // the weights come with the first row's copies
        if (in[i] && post)
            ring_copy_any(at1 + p1 * i * wstep, wstep, a.post.weight, a.post.dtype, chunk_at(i, tid, W));
        if (in[i] && next)
            ring_copy_any(at2 + p2 * i * wstep, wstep, a.next.weight, a.next.dtype, chunk_at(i, tid, W));
#pragma unroll
        for (int j = 0; j < 4; ++j)
            acc1[i][j] = acc2[i][j] = splat(0.f);
    }
    for (int s = 0; s < S - 1; ++s)
        fetch(s);
    auto weight = [&](uint32_t at, const NormDev &n, float2 (&w)[4]) {
        ring_get_any(at, wstep, n.dtype, w);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            w[j] = add2(w[j], splat(n.offset));
    };
    int turn = 0, s = 0;
    for (long row = row0; row < a.T; row += stride) {
        float on = 1.f, off = 0.f;   // sigmoid(z), 1 - sigmoid(z)
        if (a.gate_mode == GATE_TOKEN) {
            AnyChunk<1> z;
            float v[1];
            z.load(a.gate, a.gate_dtype, row * a.gate_ld);
            z.get(v, a.gate_dtype);
            sigmoids(v[0], on, off);
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
        // the sums that need nothing but the inputs: |h'|^2, sum g h' of the next norm, |y|^2
        float2 q0 = splat(0.f), q1 = q0, q2 = q0;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (in[i]) {
                float2 v[4], d[4], w[4];
                if (next) {
                    ring_get<HT>(at + (OH + i * PH) * step, step, v);
                    ring_get<uint16_t>(at + (OX + i) * step, step, d);
                    weight(at2 + p2 * i * wstep, a.next, w);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        q0 = fma2(v[j], v[j], q0);
                        q1 = fma2(mul2(d[j], w[j]), v[j], q1);
                    }
                }
                if (post) {
                    ring_get<YT>(at + i * PY * step, step, v);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        q2 = fma2(v[j], v[j], q2);
                }
            }
        float q[3] = {q0.x + q0.y, q1.x + q1.y, q2.x + q2.y};
        if (next || post)
            row_sum(q, rs, team, turn);
        const float r2 = rsqrtf(q[0] * a.inv_h + a.next.eps), rm2 = r2 * (r2 * (q[1] * a.inv_h));
        const float r1 = post ? rsqrtf(q[2] * a.inv_h + a.post.eps) : 1.f;
        float2 dH[NV][4], t0 = splat(0.f);   // t0: sum g y of the post norm (channel gates), or sum dv u
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (in[i]) {
                float2 v[4], w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    dH[i][j] = splat(0.f);
                if (has)
                    ring_get<HT>(at + (OG + i * PH) * step, step, dH[i]);
                if (next) {
                    float2 d[4];
                    ring_get<HT>(at + (OH + i * PH) * step, step, v);
                    ring_get<uint16_t>(at + (OX + i) * step, step, d);
                    weight(at2 + p2 * i * wstep, a.next, w);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 n = mul2(v[j], splat(r2));
                        acc2[i][j] = fma2(d[j], n, acc2[i][j]);
                        dH[i][j] = add2(dH[i][j], fma2(n, splat(-rm2), mul2(mul2(d[j], w[j]), splat(r2))));
                    }
                }
                if (a.dh) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        v[j] = mul2(dH[i][j], splat(a.res_scale));
                    Chunk<HT, 8> oc;
                    oc.set(v);
                    oc.store(dh + i * hop);
                }
                ring_get<YT>(at + i * PY * step, step, v);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    w[j] = splat(1.f);
                if (post)
                    weight(at1 + p1 * i * wstep, a.post, w);
                if (pz) {
                    float2 z[4];
                    ring_get_any(at + (OZ + i * pz) * step, step, a.gate_dtype, z);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float2 zon, zoff;
                        sigmoids(z[j].x, zon.x, zoff.x);
                        sigmoids(z[j].y, zon.y, zoff.y);
                        const float2 du = mul2(mul2(dH[i][j], splat(a.out_scale)), zon), n = mul2(v[j], splat(r1));
                        dH[i][j] = mul2(du, w[j]);                              // g
                        z[j] = mul2(mul2(dH[i][j], n), zoff);                   // dv u s (1 - s)
                        acc1[i][j] = fma2(du, n, acc1[i][j]);
                        t0 = fma2(dH[i][j], v[j], t0);
                    }
                    if (a.dgate) {
                        const long to = row * a.dgate_ld + tid * 8 + i * hop;
                        if (a.gate_dtype == VQ_F32) {
                            Chunk<float, 8> oc;
                            oc.set(z);
                            oc.store(static_cast<float *>(a.dgate) + to);
                        } else {
                            Chunk<uint16_t, 8> oc;
                            oc.set(z);
                            oc.store(static_cast<uint16_t *>(a.dgate) + to);
                        }
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 du = mul2(dH[i][j], splat(a.out_scale)), n = mul2(v[j], splat(r1));   // dv
                        acc1[i][j] = fma2(mul2(du, splat(on)), n, acc1[i][j]);
                        const float2 dn = mul2(du, w[j]);
                        t0 = fma2(dn, n, t0);                                   // dv u
                        dH[i][j] = mul2(dn, splat(on));                         // g
                    }
                }
            }
        dh += stride * a.dh_ld;
        const bool token = a.gate_mode == GATE_TOKEN && a.dgate;
        float t[1] = {t0.x + t0.y};
        if (post || token)
            row_sum(t, rs, team, turn);
        if (token && tid == 0) {
            const float dz = t[0] * on * off;
            const long to = row * a.dgate_ld;
            if (a.gate_dtype == VQ_F32)
                static_cast<float *>(a.dgate)[to] = dz;
            else
                static_cast<uint16_t *>(a.dgate)[to] = f32_to_bf16_bits(dz);
        }
        // r1 mean(g y^): from sum g y, or from sum dv u = sum (g / on) y^
        const float rm1 = r1 * ((pz ? r1 : on) * t[0] * a.inv_h);
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (in[i]) {
                if (post) {
                    float2 v[4];
                    ring_get<YT>(at + i * PY * step, step, v);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        dH[i][j] = fma2(mul2(v[j], splat(r1)), splat(-rm1), mul2(dH[i][j], splat(r1)));
                }
                Chunk<YT, 8> oc;
                oc.set(dH[i]);
                oc.store(dy + i * hop);
            }
        dy += stride * a.dy_ld;
    }
    if (a.part1)
        write_part(a.part1, acc1, reinterpret_cast<float *>(ring), tid, W, a.H);
    if (a.part2)
        write_part(a.part2, acc2, reinterpret_cast<float *>(ring), tid, W, a.H);
}

// Column sums of the partial rows: 32 columns and 32 interleaved strands of
// rows per CTA, each strand in row order, then over the strands in order.
// blockIdx.y: which weight gradient.
__global__ void __launch_bounds__(1024) vq_norm_dw_kernel(const float *p1, float *d1, const float *p2, float *d2,
                                                          int parts, int H)
{
    __shared__ float s[32][33];
    grid_dep_launch();
    grid_dep_wait();
    const float *p = blockIdx.y ? p2 : p1;
    float *d = blockIdx.y ? d2 : d1;
    const int x = threadIdx.x & 31, strand = threadIdx.x >> 5, c = blockIdx.x * 32 + x;
    float v = 0.f;
    if (c < H) {
#pragma unroll 4
        for (int i = strand; i < parts; i += 32)
            v += p[(long)i * H + c];
    }
    s[strand][x] = v;
    __syncthreads();
    // warp w adds the strands of column w
    v = warp_total(s[x][strand]);
    if (x == 0 && blockIdx.x * 32 + strand < H)
        d[blockIdx.x * 32 + strand] = v;
}

cudaError_t finish(int parts, int H, const float *p1, float *d1, const float *p2, float *d2, cudaStream_t s)
{
    if (!d1 && !d2)
        return cudaSuccess;
    if (!d1)
        p1 = p2, d1 = d2, d2 = nullptr;
    return launch_after(vq_norm_dw_kernel, dim3((H + 31) / 32, d2 ? 2 : 1), dim3(1024), 0, s, p1, d1, p2, d2, parts, H);
}

// Both launch and say how many partial rows they leave.
template <typename HT>
cudaError_t pre_bwd(NormPreBwdArgs a, bool vec8, int &parts, cudaStream_t s)
{
    int regs[4];
    const cudaError_t e = ring_regs<vq_norm_pre_bwd_kernel<HT, 1>, vq_norm_pre_bwd_kernel<HT, 2>,
                                    vq_norm_pre_bwd_kernel<HT, 3>, vq_norm_pre_bwd_kernel<HT, 4>>(regs);
    if (e != cudaSuccess)
        return e;
    NormShape sh = norm_shape(a.H, a.T, sizeof(HT) * (a.dres ? 2 : 1) + 2, 0, regs, 4, 4, NORM_PARTS);
    if (vec8 && sh.S > 0) {
        a.W = sh.W;
        parts = sh.ctas;
        switch (sh.nv) {
        case 1: return launch_rows<vq_norm_pre_bwd_kernel<HT, 1>>(sh, s, a);
        case 2: return launch_rows<vq_norm_pre_bwd_kernel<HT, 2>>(sh, s, a);
        case 3: return launch_rows<vq_norm_pre_bwd_kernel<HT, 3>>(sh, s, a);
        default: return launch_rows<vq_norm_pre_bwd_kernel<HT, 4>>(sh, s, a);
        }
    }
    sh = scalar_shape(a.H, a.T, 1, NORM_PARTS);
    a.W = sh.W;
    parts = sh.ctas;
    return launch_smem<vq_norm_pre_bwd_scalar_kernel<HT>, SCALAR_SMEM>(dim3(sh.ctas), dim3(32 * sh.W * sh.R), sh.smem, s, a);
}

template <typename YT, typename HT>
cudaError_t post_bwd(NormPostBwdArgs a, bool vec8, int &parts, cudaStream_t s)
{
    const int gate = a.gate_mode != GATE_CHANNEL ? 0 : a.gate_dtype == VQ_F32 ? 4 : 2;
    auto w = [](const NormDev &n) { return !n.weight ? 0 : n.dtype == VQ_F32 ? 4 : 2; };
    int regs[4];
    const cudaError_t e = ring_regs<vq_norm_post_bwd_kernel<YT, HT, 1>, vq_norm_post_bwd_kernel<YT, HT, 2>,
                                    vq_norm_post_bwd_kernel<YT, HT, 3>, vq_norm_post_bwd_kernel<YT, HT, 4>>(regs);
    if (e != cudaSuccess)
        return e;
    NormShape sh = norm_shape(a.H, a.T, sizeof(YT) + (a.dho ? sizeof(HT) : 0) + (a.next.weight ? sizeof(HT) + 2 : 0) + gate,
                              w(a.post) + w(a.next), regs, 2, 2, NORM_PARTS);
    if (vec8 && sh.S > 0) {
        a.W = sh.W;
        parts = sh.ctas;
        switch (sh.nv) {
        case 1: return launch_rows<vq_norm_post_bwd_kernel<YT, HT, 1>>(sh, s, a);
        case 2: return launch_rows<vq_norm_post_bwd_kernel<YT, HT, 2>>(sh, s, a);
        case 3: return launch_rows<vq_norm_post_bwd_kernel<YT, HT, 3>>(sh, s, a);
        default: return launch_rows<vq_norm_post_bwd_kernel<YT, HT, 4>>(sh, s, a);
        }
    }
    sh = scalar_shape(a.H, a.T, 3, NORM_PARTS);
    a.W = sh.W;
    parts = sh.ctas;
    return launch_smem<vq_norm_post_bwd_scalar_kernel<YT, HT>, SCALAR_SMEM>(dim3(sh.ctas), dim3(32 * sh.W * sh.R), sh.smem, s, a);
}

}  // namespace

size_t norm_workspace_bytes(int H, int T)
{
    // One row's CTA writes the weight gradients itself. For more rows the second launch (about 1 us) costs less than rows
    // in turn in one CTA (norm_post, 6144 wide, 2 and 4 rows: 11.2 and 19.7 us against 9.6) or the partial rows added
    // through the shared memory of a cluster of 8 (4, 16, 32 rows: 10.6, 13.9, 22.6 us against 9.7, 9.8, 10.0).
    if (T <= 1)
        return 0;
    // at most NORM_PARTS partial rows of each weight, and no more than rows
    return (size_t)2 * (size_t)std::min(NORM_PARTS, T) * (size_t)H * sizeof(float);
}

cudaError_t launch_norm_pre_bwd(const NormPreBwdArgs &args, int h_dtype, bool vec8, float *dw, float *ws, cudaStream_t s)
{
    NormPreBwdArgs a = args;
    const bool one = a.T == 1;
    a.part = !dw ? nullptr : one ? dw : ws;
    int parts = 0;
    if (a.T > 0) {
        const cudaError_t e = h_dtype == VQ_F32 ? pre_bwd<float>(a, vec8, parts, s) : pre_bwd<uint16_t>(a, vec8, parts, s);
        if (e != cudaSuccess)
            return e;
    }
    return one ? cudaSuccess : finish(parts, a.H, a.part, dw, nullptr, nullptr, s);
}

cudaError_t launch_norm_post_bwd(const NormPostBwdArgs &args, int y_dtype, int h_dtype, bool vec8, float *dpost,
                                 float *dnext, float *ws, cudaStream_t s)
{
    NormPostBwdArgs a = args;
    const bool one = a.T == 1;
    // the second half of the workspace holds dnext's partial rows
    a.part1 = !dpost ? nullptr : one ? dpost : ws;
    a.part2 = !dnext ? nullptr : one ? dnext : ws + norm_workspace_bytes(a.H, a.T) / (2 * sizeof(float));
    int parts = 0;
    if (a.T > 0) {
        cudaError_t e;
        if (y_dtype == VQ_F32)
            e = h_dtype == VQ_F32 ? post_bwd<float, float>(a, vec8, parts, s) : post_bwd<float, uint16_t>(a, vec8, parts, s);
        else
            e = h_dtype == VQ_F32 ? post_bwd<uint16_t, float>(a, vec8, parts, s)
                                  : post_bwd<uint16_t, uint16_t>(a, vec8, parts, s);
        if (e != cudaSuccess)
            return e;
    }
    return one ? cudaSuccess : finish(parts, a.H, a.part1, dpost, a.part2, dnext, s);
}

}  // namespace vq
