// The router's balance loss, the experts' load, and the loss's gradient.
//
// With V tokens that count (mask), N = V k pairs, p = softmax(logits):
//   d[e] = E counts[e] / N,  P[e] = (1/V) sum_t p[t, e],  loss = coef sum_e d[e] P[e]
//   dlogits[t, e] = dloss coef / V p[t, e] (d[e] - sum p[t, .] d)
// Since sum p = 1, d may be shifted by any constant in the gradient: d - 1 is
// taken (0 for an even load), which keeps the difference's leading digits.
//
// One warp takes a token: its E logits sit in the lanes' registers (E <= 1024;
// wider rows are re-read), each lane keeps the column sums of its experts over
// its tokens in registers. Few tokens: one CTA does it all. More: CTAs write
// partial sums and counts, and one cluster of CTAs adds them in order.
//
// Measured: 32768 x 512, loss 18 us + 5 us for the partial rows, gradient 23 us, 45.2 us
// together; reading the logits twice and writing the gradient is 31 us at the
// copy rate. 4096 x 256 12.1 us and 16 x 512 5.9 us, both of them the launches. With the next row
// loaded ahead and the pairs counted on the way 45.2 us, without 68.
#include <algorithm>

#include "vq_block.cuh"
#include "vq_balance.h"

namespace vq {
namespace {

constexpr int BAL_WARPS = 16;            // warps per CTA
constexpr int BAL_WIDE_WARPS = 8;        // the same for rows beyond BAL_REG_E: one row of sums per warp fits shared memory
constexpr int BWD_WARPS = 8;             // warps per CTA of the gradient
constexpr int BAL_ONE_CTA = 64;          // most tokens of the one-CTA form
constexpr int BAL_PARTS = 296;           // most partial rows: 2 CTAs on each of 148 SMs (at most FIN_THREADS)
constexpr int BAL_CLUSTER = 8;           // CTAs that add the partial rows
constexpr int BAL_REG_E = 1024;          // widest row held in registers

// Largest of the warp's values (one instruction on sm_100a; NaN is passed over).
__device__ __forceinline__ float warp_max(float v)
{
    float m;
    asm volatile("redux.sync.max.f32 %0, %1, 0xFFFFFFFF;" : "=f"(m) : "f"(v));
    return m;
}

// exp(l - top) as 2^((l - top) log2e). A row of -Inf (top = -Inf) is taken off 0 and gives 0; NaN stays NaN.
__device__ __forceinline__ float base_of(float top) { return top == -INFINITY ? 0.f : top; }
__device__ __forceinline__ float soft(float l, float base)
{
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"((l - base) * 1.4426950408889634f));
    return e;
}

// The expert in register i of a lane: VEC consecutive experts per lane and 32-lane sweep.
template <int VEC>
__device__ __forceinline__ int expert_at(int i, int lane) { return (i / VEC * 32 + lane) * VEC + i % VEC; }

// One row in the lanes' registers (PER experts each; -Inf beyond E).
template <int PER, int VEC>
__device__ __forceinline__ void load_row(const float *l, int E, int lane, float (&v)[PER])
{
#pragma unroll
    for (int i = 0; i < PER; i += VEC) {
        const int e = expert_at<VEC>(i, lane);
        if constexpr (VEC == 4) {
            float4 t = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
            if (e < E)
                t = *reinterpret_cast<const float4 *>(l + e);
            v[i] = t.x, v[i + 1] = t.y, v[i + 2] = t.z, v[i + 3] = t.w;
        } else {
            v[i] = e < E ? l[e] : -INFINITY;
        }
    }
}

// v <- exp(v - max); returns 1 / sum (0 for a row of -Inf). NaN spreads over the row by the sum.
template <int PER>
__device__ __forceinline__ float soften(float (&v)[PER])
{
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < PER; ++i)
        top = fmaxf(top, v[i]);
    const float base = base_of(warp_max(top));
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        v[i] = soft(v[i], base);
        s += v[i];
    }
    s = warp_total(s);
    return s == 0.f ? 0.f : 1.f / s;
}

// The first token at or after t, in steps of `step`, that counts.
__device__ __forceinline__ long next_live(const uint8_t *mask, long t, long end, int step)
{
    while (mask && t < end && !mask[t])
        t += step;
    return t;
}

// Rows wider than 512 experts leave no registers for a row loaded ahead.
template <int PER>
constexpr bool AHEAD = PER <= 16;

// The expert of lane j's pair of token t (j < k), -1 for none.
__device__ __forceinline__ int pair_of(const BalanceArgs &a, long t, int lane)
{
    return lane < a.k ? a.ids[t * a.k + lane] : -1;
}

// Counts a token's pairs, and the token, into cnt[0..E] (shared). Integer sums: their order does not matter.
__device__ __forceinline__ void count_token(int *cnt, int E, int e, int lane)
{
    if ((unsigned)e < (unsigned)E)
        atomicAdd(&cnt[e], 1);
    if (lane == 0)
        atomicAdd(&cnt[E], 1);
}

// Column sums of warp-held rows: tokens t0 + warp, + NW, ...; acc[i] is
// expert_at(i)'s; the tokens' pairs are counted on the way. The next row's
// loads are under way while one is summed.
template <int PER, int VEC, int NW>
__device__ __forceinline__ void sum_rows(const BalanceArgs &a, long t0, long t1, int warp, int lane, int *cnt,
                                         float (&acc)[PER])
{
#pragma unroll
    for (int i = 0; i < PER; ++i)
        acc[i] = 0.f;
    float v[PER], next[AHEAD<PER> ? PER : 1];
    int e = -1, e_next = -1;
    long t = next_live(a.mask, t0 + warp, t1, NW);
    if (t < t1) {
        load_row<PER, VEC>(a.logits + t * a.E, a.E, lane, v);
        e = pair_of(a, t, lane);
    }
    while (t < t1) {
        const long u = next_live(a.mask, t + NW, t1, NW);
        if (u < t1) {
            if constexpr (AHEAD<PER>)
                load_row<PER, VEC>(a.logits + u * a.E, a.E, lane, next);
            e_next = pair_of(a, u, lane);
        }
        const float inv = soften(v);
#pragma unroll
        for (int i = 0; i < PER; ++i)
            acc[i] = fmaf(v[i], inv, acc[i]);
        count_token(cnt, a.E, e, lane);
        if constexpr (AHEAD<PER>) {
#pragma unroll
            for (int i = 0; i < PER; ++i)
                v[i] = next[i];
        } else if (u < t1) {
            load_row<PER, VEC>(a.logits + u * a.E, a.E, lane, v);
        }
        e = e_next;
        t = u;
    }
}

// 1 / (V k), for d[e] = counts[e] E / (V k). The gradient's d[e] - 1 is
// (counts[e] E - V k) / (V k) with an exact integer numerator.
__device__ __forceinline__ float per_pair(int V, int k) { return V ? (float)(1.0 / ((double)V * (double)k)) : 0.f; }
__device__ __forceinline__ float share(int count, int E, float pp) { return (float)((long)count * E) * pp; }
__device__ __forceinline__ float excess(int count, int E, int V, int k, float pp)
{
    return (float)((long)count * E - (long)V * k) * pp;
}

// PER == 0: rows wider than BAL_REG_E, column sums in shared memory, one row of E per warp.
template <int PER, int VEC>
__global__ void __launch_bounds__((PER > 0 ? BAL_WARPS : BAL_WIDE_WARPS) * 32, PER > 0 && AHEAD<PER> ? 2 : 1)
    vq_balance_kernel(const BalanceArgs a, int per_cta, int one)
{
    constexpr int NW = PER > 0 ? BAL_WARPS : BAL_WIDE_WARPS, THREADS = NW * 32;
    extern __shared__ float sm[];
    float *sums = sm;                                             // [NW][E]
    int *cnt = reinterpret_cast<int *>(sm + (size_t)NW * a.E);    // [E + 1]
    __shared__ float red[NW];
    grid_dep_launch();
    grid_dep_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, E = a.E;
    const long t0 = min((long)a.T, (long)blockIdx.x * per_cta), t1 = min((long)a.T, t0 + per_cta);
    for (int e = threadIdx.x; e <= E; e += THREADS)
        cnt[e] = 0;
    __syncthreads();
    if constexpr (PER > 0) {
        float acc[PER];
        sum_rows<PER, VEC, NW>(a, t0, t1, warp, lane, cnt, acc);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = expert_at<VEC>(i, lane);
            if (e < E)
                sums[warp * E + e] = acc[i];
        }
    } else {
        for (int e = lane; e < E; e += 32)
            sums[warp * E + e] = 0.f;
        for (long t = t0 + warp; t < t1; t += NW) {
            if (a.mask && !a.mask[t])
                continue;
            count_token(cnt, E, pair_of(a, t, lane), lane);
            const float *l = a.logits + t * E;
            float top = -INFINITY, s = 0.f;
            for (int e = lane; e < E; e += 32)
                top = fmaxf(top, l[e]);
            const float base = base_of(warp_max(top));
            for (int e = lane; e < E; e += 32)
                s += soft(l[e], base);
            s = warp_total(s);
            const float inv = s == 0.f ? 0.f : 1.f / s;
            for (int e = lane; e < E; e += 32)
                sums[warp * E + e] = fmaf(soft(l[e], base), inv, sums[warp * E + e]);
        }
    }
    __syncthreads();
    if (!one) {
        for (int e = threadIdx.x; e <= E; e += THREADS) {
            a.part_counts[(long)blockIdx.x * (E + 1) + e] = cnt[e];
            if (e < E) {
                float v = 0.f;
#pragma unroll
                for (int w = 0; w < NW; ++w)
                    v += sums[w * E + e];
                a.part_sums[(long)blockIdx.x * E + e] = v;
            }
        }
        return;
    }
    const int V = cnt[E];
    const float pp = per_pair(V, a.k);
    float loss = 0.f;
    for (int e = threadIdx.x; e <= E; e += THREADS) {
        a.counts[e] = cnt[e];
        if (e < E) {
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w)
                v += sums[w * E + e];
            v = V ? v / (float)V : 0.f;
            a.probs[e] = v;
            loss = fmaf(share(cnt[e], E, pp), v, loss);
        }
    }
    loss = warp_total(loss);
    if (lane == 0)
        red[warp] = loss;
    __syncthreads();
    if (threadIdx.x == 0) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w)
            v += red[w];
        *a.loss = a.coef * v;
    }
}

// Adds the CTAs' partial rows: a cluster of BAL_CLUSTER CTAs, each with a
// slice of the experts; the first CTA adds the slices' loss terms through the
// cluster's shared memory.
constexpr int FIN_THREADS = 1024;
__global__ void __cluster_dims__(BAL_CLUSTER, 1, 1) __launch_bounds__(FIN_THREADS)
    vq_balance_finish_kernel(const BalanceArgs a, int parts)
{
    __shared__ float fs[FIN_THREADS], term, red[FIN_THREADS / 32];
    __shared__ int is[FIN_THREADS], valid[FIN_THREADS / 32];
    grid_dep_launch();
    grid_dep_wait();
    const int E = a.E, rank = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
    // a thread: one expert of the CTA's slice (at most 512), one of `strands` interleaved strands of partial rows
    const int per = (E + BAL_CLUSTER - 1) / BAL_CLUSTER, width = per <= 32 ? 32 : per <= 64 ? 64 : per <= 128 ? 128 : per <= 256 ? 256 : 512;
    const int strands = FIN_THREADS / width, x = tid & (width - 1), e = rank * per + x;
    const bool mine = x < per && e < E;
    float s = 0.f;
    int c = 0;
    if (mine) {
#pragma unroll 4
        for (int p = tid / width; p < parts; p += strands) {
            s += a.part_sums[(long)p * E + e];
            c += a.part_counts[(long)p * (E + 1) + e];
        }
    }
    fs[tid] = s;
    is[tid] = c;
    // the tokens that count, by every CTA for itself
    const int v = __reduce_add_sync(0xFFFFFFFFu, tid < parts ? a.part_counts[(long)tid * (E + 1) + E] : 0);
    if (lane == 0)
        valid[tid >> 5] = v;
    __syncthreads();
    const int V = __reduce_add_sync(0xFFFFFFFFu, valid[lane]);
    const float pp = per_pair(V, a.k);
    float loss = 0.f;
    if (tid < width && mine) {
        for (int i = 1; i < strands; ++i) {
            s += fs[i * width + tid];
            c += is[i * width + tid];
        }
        s = V ? s / (float)V : 0.f;
        a.probs[e] = s;
        a.counts[e] = c;
        loss = share(c, E, pp) * s;
    }
    loss = warp_total(loss);
    if (lane == 0)
        red[tid >> 5] = loss;
    __syncthreads();
    loss = red[lane];
    if (tid < 32) {
        loss = warp_total(loss);
        if (tid == 0)
            term = loss;
    }
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
    if (rank == 0 && tid == 0) {
        a.counts[E] = V;
        float t = 0.f;
        for (int r = 0; r < BAL_CLUSTER; ++r) {
            uint32_t at;
            float x;
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(&term)), "r"(r));
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(at));
            t += x;
        }
        *a.loss = a.coef * t;
    }
    // no CTA leaves while its term may still be read
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// T = 0: nothing counted.
__global__ void vq_balance_empty_kernel(const BalanceArgs a)
{
    grid_dep_launch();
    grid_dep_wait();
    for (int e = threadIdx.x; e <= a.E; e += blockDim.x) {
        a.counts[e] = 0;
        if (e < a.E)
            a.probs[e] = 0.f;
    }
    if (threadIdx.x == 0)
        *a.loss = 0.f;
}

// ---------------------------------------------------------------- gradient

template <int PER, int VEC>
__global__ void __launch_bounds__(BWD_WARPS * 32) vq_balance_bwd_kernel(const BalanceBwdArgs a)
{
    grid_dep_launch();
    grid_dep_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, E = a.E;
    const int V = a.counts[E];
    const float scale = V ? (a.dloss ? *a.dloss : 1.f) * a.coef / (float)V : 0.f;
    const float pp = per_pair(V, a.k);
    const int step = gridDim.x * BWD_WARPS;
    constexpr int N = PER > 0 ? PER : 1;
    float d[N], next[PER > 0 && AHEAD<PER> ? PER : 1];
    auto counts = [&](long t) { return V && (!a.mask || a.mask[t]); };
    long t = (long)blockIdx.x * BWD_WARPS + warp;
    bool live = t < a.T && counts(t);
    if constexpr (PER > 0) {
        if constexpr (AHEAD<PER>)
            if (live)
                load_row<PER, VEC>(a.logits + t * E, E, lane, next);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = expert_at<VEC>(i, lane);
            d[i] = e < E ? excess(a.counts[e], E, V, a.k, pp) : 0.f;
        }
    }
    for (; t < a.T; t += step) {
        const float *l = a.logits + t * E;
        float *o = a.dlogits + t * E;
        if constexpr (PER > 0) {
            float v[PER];
            const bool now = live;
            if constexpr (AHEAD<PER>) {
#pragma unroll
                for (int i = 0; i < PER; ++i)
                    v[i] = next[i];
                live = t + step < a.T && counts(t + step);
                if (live)
                    load_row<PER, VEC>(l + (long)step * E, E, lane, next);
            } else {
                if (now)
                    load_row<PER, VEC>(l, E, lane, v);
                live = t + step < a.T && counts(t + step);
            }
            float dot = 0.f, inv = 0.f;
            if (now) {
                inv = soften(v);
#pragma unroll
                for (int i = 0; i < PER; ++i)
                    dot = fmaf(v[i], d[i], dot);
                dot = warp_total(dot) * inv;
                inv *= scale;
            }
#pragma unroll
            for (int i = 0; i < PER; ++i)
                v[i] = now ? v[i] * inv * (d[i] - dot) : 0.f;
#pragma unroll
            for (int i = 0; i < PER; i += VEC) {
                const int e = expert_at<VEC>(i, lane);
                if (e < E) {
                    if constexpr (VEC == 4)
                        *reinterpret_cast<float4 *>(o + e) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                    else
                        o[e] = v[i];
                }
            }
        } else {
            if (!counts(t)) {
                for (int e = lane; e < E; e += 32)
                    o[e] = 0.f;
                continue;
            }
            float top = -INFINITY, s = 0.f, dot = 0.f;
            for (int e = lane; e < E; e += 32)
                top = fmaxf(top, l[e]);
            const float base = base_of(warp_max(top));
            for (int e = lane; e < E; e += 32) {
                const float p = soft(l[e], base);
                s += p;
                dot = fmaf(p, excess(a.counts[e], E, V, a.k, pp), dot);
            }
            s = warp_total(s);
            const float inv = s == 0.f ? 0.f : 1.f / s;
            dot = warp_total(dot) * inv;
            for (int e = lane; e < E; e += 32)
                o[e] = soft(l[e], base) * (inv * scale) * (excess(a.counts[e], E, V, a.k, pp) - dot);
        }
    }
}

size_t balance_smem(int E) { return ((size_t)(E <= BAL_REG_E ? BAL_WARPS : BAL_WIDE_WARPS) * E + E + 1) * 4; }

template <int PER, int VEC>
cudaError_t fwd(const BalanceArgs &a, int ctas, int per_cta, int one, cudaStream_t s)
{
    const size_t smem = balance_smem(a.E);
    if (smem > 48 * 1024) {
        static std::atomic<uint64_t> allowed{0};
        const int most = PER > 0 ? (BAL_WARPS * BAL_REG_E + BAL_REG_E + 1) * 4 : (BAL_WIDE_WARPS * 4096 + 4097) * 4;
        const cudaError_t e = allow_smem((const void *)vq_balance_kernel<PER, VEC>, most, allowed);
        if (e != cudaSuccess)
            return e;
    }
    return launch_after(vq_balance_kernel<PER, VEC>, dim3(ctas), dim3((PER > 0 ? BAL_WARPS : BAL_WIDE_WARPS) * 32), smem, s, a, per_cta, one);
}

template <int PER, int VEC>
cudaError_t bwd(const BalanceBwdArgs &a, cudaStream_t s)
{
    // persistent warps: 3 CTAs of 8 on an SM
    const int ctas = (int)std::min(((long)a.T + BWD_WARPS - 1) / BWD_WARPS, 3L * 148);
    return launch_after(vq_balance_bwd_kernel<PER, VEC>, dim3(ctas), dim3(BWD_WARPS * 32), 0, s, a);
}

}  // namespace

size_t balance_workspace_bytes(int T, int E)
{
    if (T <= BAL_ONE_CTA)
        return 0;
    return align_up((size_t)BAL_PARTS * E * 4, 256) + align_up((size_t)BAL_PARTS * (E + 1) * 4, 256);
}

cudaError_t launch_balance(const BalanceArgs &args, void *ws, cudaStream_t s)
{
    BalanceArgs a = args;
    if (a.T == 0)
        return launch_after(vq_balance_empty_kernel, dim3(1), dim3(256), 0, s, a);
    const int one = a.T <= BAL_ONE_CTA;
    if (!one) {
        a.part_sums = static_cast<float *>(ws);
        a.part_counts = ws_at<int32_t>(ws, align_up((size_t)BAL_PARTS * a.E * 4, 256));
    }
    const int per_cta = one ? a.T : std::max(BAL_WARPS, (int)(((long)a.T + BAL_PARTS - 1) / BAL_PARTS));
    const int ctas = (int)(((long)a.T + per_cta - 1) / per_cta);
    const bool v4 = a.E % 4 == 0 && (uintptr_t)a.logits % 16 == 0;
    cudaError_t e;
    if (a.E <= 128)
        e = v4 ? fwd<4, 4>(a, ctas, per_cta, one, s) : fwd<4, 1>(a, ctas, per_cta, one, s);
    else if (a.E <= 256)
        e = v4 ? fwd<8, 4>(a, ctas, per_cta, one, s) : fwd<8, 1>(a, ctas, per_cta, one, s);
    else if (a.E <= 512)
        e = v4 ? fwd<16, 4>(a, ctas, per_cta, one, s) : fwd<16, 1>(a, ctas, per_cta, one, s);
    else if (a.E <= BAL_REG_E)
        e = v4 ? fwd<32, 4>(a, ctas, per_cta, one, s) : fwd<32, 1>(a, ctas, per_cta, one, s);
    else
        e = fwd<0, 1>(a, ctas, per_cta, one, s);
    if (e != cudaSuccess || one)
        return e;
    return launch_after(vq_balance_finish_kernel, dim3(BAL_CLUSTER), dim3(FIN_THREADS), 0, s, a, ctas);
}

cudaError_t launch_balance_bwd(const BalanceBwdArgs &a, cudaStream_t s)
{
    const bool v4 = a.E % 4 == 0 && (uintptr_t)a.logits % 16 == 0 && (uintptr_t)a.dlogits % 16 == 0;
    if (a.E <= 128)
        return v4 ? bwd<4, 4>(a, s) : bwd<4, 1>(a, s);
    if (a.E <= 256)
        return v4 ? bwd<8, 4>(a, s) : bwd<8, 1>(a, s);
    if (a.E <= 512)
        return v4 ? bwd<16, 4>(a, s) : bwd<16, 1>(a, s);
    if (a.E <= BAL_REG_E)
        return v4 ? bwd<32, 4>(a, s) : bwd<32, 1>(a, s);
    return bwd<0, 1>(a, s);
}

}  // namespace vq
