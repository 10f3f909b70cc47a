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
#include <algorithm>

#include "vq_block.cuh"
#include "vq_balance.h"

namespace vq {
namespace {

constexpr int BAL_WARPS = 16;            // warps per CTA
constexpr int BAL_WIDE_WARPS = 8;        // the same for rows beyond BAL_REG_E: one row of sums per warp fits shared memory
constexpr int BAL_ONE_CTA = 64;          // most tokens of the one-CTA form
constexpr int BAL_PARTS = 148;           // most partial rows
constexpr int BAL_CLUSTER = 8;           // CTAs that add the partial rows
constexpr int BAL_REG_E = 1024;          // widest row held in registers

__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1)
        v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
}

// exp(l - top); a row of -Inf (top = -Inf) is taken as 0. NaN stays NaN.
__device__ __forceinline__ float soft(float l, float top)
{
    return top == -INFINITY ? (l != l ? l : 0.f) : expf(l - top);
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
    top = warp_max(top);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        v[i] = soft(v[i], top);
        s += v[i];
    }
    s = warp_total(s);
    return s == 0.f ? 0.f : 1.f / s;
}

// Column sums of warp-held rows: tokens t0 + warp, + warps, ...; acc[i] is expert_at(i)'s.
template <int PER, int VEC, int NW>
__device__ __forceinline__ void sum_rows(const BalanceArgs &a, long t0, long t1, int warp, int lane, float (&acc)[PER])
{
#pragma unroll
    for (int i = 0; i < PER; ++i)
        acc[i] = 0.f;
    for (long t = t0 + warp; t < t1; t += NW) {
        if (a.mask && !a.mask[t])
            continue;
        float v[PER];
        load_row<PER, VEC>(a.logits + t * a.E, a.E, lane, v);
        const float inv = soften(v);
#pragma unroll
        for (int i = 0; i < PER; ++i)
            acc[i] = fmaf(v[i], inv, acc[i]);
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

// Counts a CTA's pairs and valid tokens into cnt[0..E] (shared, zeroed here).
__device__ __forceinline__ void count_pairs(const BalanceArgs &a, long t0, long t1, int *cnt)
{
    for (int e = threadIdx.x; e <= a.E; e += blockDim.x)
        cnt[e] = 0;
    __syncthreads();
    const int k = a.k;
    for (long p = t0 * k + threadIdx.x; p < t1 * k; p += blockDim.x) {
        const long t = p / k;
        if (a.mask && !a.mask[t])
            continue;
        const int e = a.ids[p];
        if ((unsigned)e < (unsigned)a.E)
            atomicAdd(&cnt[e], 1);
        if (p == t * k)
            atomicAdd(&cnt[a.E], 1);
    }
    __syncthreads();
}

// PER == 0: rows wider than BAL_REG_E, column sums in shared memory, one row of E per warp.
template <int PER, int VEC>
__global__ void __launch_bounds__((PER > 0 ? BAL_WARPS : BAL_WIDE_WARPS) * 32)
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
    count_pairs(a, t0, t1, cnt);
    if constexpr (PER > 0) {
        float acc[PER];
        sum_rows<PER, VEC, NW>(a, t0, t1, warp, lane, acc);
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
            const float *l = a.logits + t * E;
            float top = -INFINITY, s = 0.f;
            for (int e = lane; e < E; e += 32)
                top = fmaxf(top, l[e]);
            top = warp_max(top);
            for (int e = lane; e < E; e += 32)
                s += soft(l[e], top);
            s = warp_total(s);
            const float inv = s == 0.f ? 0.f : 1.f / s;
            for (int e = lane; e < E; e += 32)
                sums[warp * E + e] = fmaf(soft(l[e], top), inv, sums[warp * E + e]);
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
    __shared__ float fs[FIN_THREADS];
    __shared__ int is[FIN_THREADS];
    __shared__ float term;
    grid_dep_launch();
    grid_dep_wait();
    const int E = a.E, rank = blockIdx.x, tid = threadIdx.x;
    // the tokens that count, by every CTA for itself
    int v = 0;
    for (int p = tid; p < parts; p += FIN_THREADS)
        v += a.part_counts[(long)p * (E + 1) + E];
    is[tid] = v;
    __syncthreads();
    for (int o = FIN_THREADS / 2; o; o >>= 1) {
        if (tid < o)
            is[tid] += is[tid + o];
        __syncthreads();
    }
    const int V = is[0];
    const float pp = per_pair(V, a.k);
    __syncthreads();
    const int per = (E + BAL_CLUSTER - 1) / BAL_CLUSTER, e0 = rank * per, e1 = min(E, e0 + per);
    float loss = 0.f;
    // 32 experts at a time, 32 strands of partial rows each
    for (int b = e0; b < e1; b += 32) {
        const int e = b + (tid & 31);
        float s = 0.f;
        int c = 0;
        if (e < e1)
            for (int p = tid >> 5; p < parts; p += 32) {
                s += a.part_sums[(long)p * E + e];
                c += a.part_counts[(long)p * (E + 1) + e];
            }
        fs[tid] = s;
        is[tid] = c;
        __syncthreads();
        if (tid < 32 && e < e1) {
            s = 0.f;
            c = 0;
            for (int i = 0; i < 32; ++i) {
                s += fs[i * 32 + tid];
                c += is[i * 32 + tid];
            }
            s = V ? s / (float)V : 0.f;
            a.probs[e] = s;
            a.counts[e] = c;
            loss = fmaf(share(c, E, pp), s, loss);
        }
        __syncthreads();
    }
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
__global__ void __launch_bounds__(BAL_WARPS * 32) vq_balance_bwd_kernel(const BalanceBwdArgs a)
{
    grid_dep_launch();
    grid_dep_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, E = a.E;
    const int V = a.counts[E];
    const float scale = V ? (a.dloss ? *a.dloss : 1.f) * a.coef / (float)V : 0.f;
    const float pp = per_pair(V, a.k);
    const int step = gridDim.x * BAL_WARPS;
    constexpr int N = PER > 0 ? PER : 1;
    float d[N];
    if constexpr (PER > 0) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = expert_at<VEC>(i, lane);
            d[i] = e < E ? excess(a.counts[e], E, V, a.k, pp) : 0.f;
        }
    }
    for (long t = (long)blockIdx.x * BAL_WARPS + warp; t < a.T; t += step) {
        const float *l = a.logits + t * E;
        float *o = a.dlogits + t * E;
        const bool live = V && (!a.mask || a.mask[t]);
        if constexpr (PER > 0) {
            float v[PER];
            float dot = 0.f, inv = 0.f;
            if (live) {
                load_row<PER, VEC>(l, E, lane, v);
                inv = soften(v);
#pragma unroll
                for (int i = 0; i < PER; ++i)
                    dot = fmaf(v[i], d[i], dot);
                dot = warp_total(dot) * inv;
                inv *= scale;
            }
#pragma unroll
            for (int i = 0; i < PER; ++i)
                v[i] = live ? v[i] * inv * (d[i] - dot) : 0.f;
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
            if (!live) {
                for (int e = lane; e < E; e += 32)
                    o[e] = 0.f;
                continue;
            }
            float top = -INFINITY, s = 0.f, dot = 0.f;
            for (int e = lane; e < E; e += 32)
                top = fmaxf(top, l[e]);
            top = warp_max(top);
            for (int e = lane; e < E; e += 32) {
                const float p = soft(l[e], top);
                s += p;
                dot = fmaf(p, excess(a.counts[e], E, V, a.k, pp), dot);
            }
            s = warp_total(s);
            const float inv = s == 0.f ? 0.f : 1.f / s;
            dot = warp_total(dot) * inv;
            for (int e = lane; e < E; e += 32)
                o[e] = soft(l[e], top) * (inv * scale) * (excess(a.counts[e], E, V, a.k, pp) - dot);
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
    const int ctas = (int)std::min(((long)a.T + BAL_WARPS - 1) / BAL_WARPS, 8L * 148);
    return launch_after(vq_balance_bwd_kernel<PER, VEC>, dim3(ctas), dim3(BAL_WARPS * 32), 0, s, a);
}

}  // namespace

size_t balance_workspace_bytes(int T, int E)
{
    return align_up((size_t)BAL_PARTS * E * 4, 256) + align_up((size_t)BAL_PARTS * (E + 1) * 4, 256);
}

cudaError_t launch_balance(const BalanceArgs &args, void *ws, cudaStream_t s)
{
    BalanceArgs a = args;
    if (a.T == 0)
        return launch_after(vq_balance_empty_kernel, dim3(1), dim3(256), 0, s, a);
    a.part_sums = static_cast<float *>(ws);
    a.part_counts = ws_at<int32_t>(ws, align_up((size_t)BAL_PARTS * a.E * 4, 256));
    const int one = a.T <= BAL_ONE_CTA;
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
