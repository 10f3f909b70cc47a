// Arguments of the block-norm kernels (vq_norm.cu, vq_norm_bwd.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "vq_internal.h"
#ifdef __CUDACC__
#include "vq_block.cuh"
#endif

namespace vq {

constexpr int NORM_MAX_HIDDEN = 16384;

// A norm's parameters; weight NULL: no norm.
struct NormDev {
    const void *weight;
    int dtype;
    float eps, offset;
};

enum { GATE_NONE = 0, GATE_TOKEN = 1, GATE_CHANNEL = 2 };

#ifdef __CUDACC__
// Single elements: fp32 or bf16, and of a type known at run time.
__device__ __forceinline__ float element(float v) { return v; }
__device__ __forceinline__ float element(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
__device__ __forceinline__ void put(float &o, float v) { o = v; }
__device__ __forceinline__ void put(uint16_t &o, float v) { o = __bfloat16_as_ushort(__float2bfloat16_rn(v)); }
// A batch of a thread's elements e, e + step, ...: loaded before any of the batch is stored, since an output may be
// the input itself and the compiler then keeps every load behind the stores before it.
constexpr int BATCH = 4;
template <typename T>
__device__ __forceinline__ void batch(float (&v)[BATCH], const T *p, int e, int step, int H)
{
#pragma unroll
    for (int i = 0; i < BATCH; ++i)
        v[i] = e + i * step < H ? element(p[e + i * step]) : 0.f;
}
__device__ __forceinline__ void batch_any(float (&v)[BATCH], const void *p, int dtype, long at, int e, int step, int H)
{
    if (dtype == VQ_F32)
        batch(v, static_cast<const float *>(p) + at, e, step, H);
    else
        batch(v, static_cast<const uint16_t *>(p) + at, e, step, H);
}
__device__ __forceinline__ float weight_at(const void *p, int dtype, long i)
{
    return dtype == VQ_F32 ? static_cast<const float *>(p)[i] : element(static_cast<const uint16_t *>(p)[i]);
}

// 2^x and 1 / x of the special function unit (ex2.approx, rcp.approx: a few 2^-24 off; results below 2^-126 are 0).
__device__ __forceinline__ float ex2_ftz(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_ftz(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// sigmoid(z), off by a few 2^-24 times max(1, |z|), as a rounding of z is.
__device__ __forceinline__ float sigmoid(float z) { return rcp_ftz(1.f + ex2_ftz(-1.4426950408889634f * z)); }

// sigmoid(z) and sigmoid(-z) from one exponential and one reciprocal of a number in [1, 2].
__device__ __forceinline__ void sigmoids(float z, float &on, float &off)
{
    const float e = ex2_ftz(-1.4426950408889634f * fabsf(z)), s = rcp_ftz(1.f + e), r = e * s;
    on = z < 0.f ? r : s;
    off = z < 0.f ? s : r;
}
#endif

struct NormPreArgs {
    NormDev n;
    const void *h;
    uint16_t *x;
    int64_t h_ld, x_ld;
    int T, H, W;          // W: warps per row
    float inv_h;          // 1 / H
};

struct NormPostArgs {
    NormDev post, next;
    const void *y, *gate, *h;
    void *h_out;
    uint16_t *x;
    int64_t y_ld, gate_ld, h_ld, ho_ld, x_ld;
    int gate_mode, gate_dtype;
    int T, H, W;
    float inv_h, res_scale, out_scale;
};

struct NormPreBwdArgs {
    NormDev n;
    const void *h, *dres;      // dres NULL: none
    const uint16_t *dx;
    void *dh;
    int64_t h_ld, dx_ld, dres_ld, dh_ld;
    float *part;               // [parts][H] partial weight gradients; NULL: not wanted
    int T, H, W;
    float inv_h;
};

struct NormPostBwdArgs {
    NormDev post, next;
    const void *y, *gate, *h, *dho;   // dho NULL: zero
    const uint16_t *dx;
    void *dy, *dgate, *dh;            // dgate, dh NULL: not wanted
    int64_t y_ld, gate_ld, h_ld, dho_ld, dx_ld, dy_ld, dgate_ld, dh_ld;
    float *part1, *part2;             // [parts][H] each; NULL: not wanted
    int gate_mode, gate_dtype;
    int T, H, W;
    float inv_h, res_scale, out_scale;
};

// How a launch of the ring kernels covers the rows: W warps a row, R rows side
// by side in a CTA, nv chunks of 8 elements a thread, S rows of shared memory
// (S - 1 copied ahead), `ctas` persistent CTAs. S = 0: a row does not fit.
struct NormShape {
    int W, R, nv, S, ctas;
    size_t smem;
};
constexpr int NORM_SMEM = 222 * 1024;      // shared memory of an SM given to the rings
// bytes: of input an element copied ahead; fixed: bytes an element kept for the whole launch; regs: registers a
// thread of the kernel with nv chunks (regs[nv - 1]), which bound the CTAs that an SM holds; nv, max_nv: chunks a
// thread takes when rows stream, and the most it has registers for; max_ctas: 0, or the most CTAs.
NormShape norm_shape(int H, int T, int bytes, int fixed, const int (&regs)[4], int nv, int max_nv, int max_ctas);

#ifdef __CUDACC__
// Where a thread's i-th chunk of a row starts, for a row over W warps.
__device__ __forceinline__ int chunk_at(int i, int tid, int W) { return (tid + i * 32 * W) * 8; }

// Registers a thread of the kernels with 1 to 4 chunks, as allocated (in units of 8), asked for once.
template <auto K1, auto K2, auto K3, auto K4>
cudaError_t ring_regs(int (&regs)[4])
{
    static std::atomic<int> known[4];
    const void *kernels[4] = {(const void *)K1, (const void *)K2, (const void *)K3, (const void *)K4};
    for (int i = 0; i < 4; ++i) {
        regs[i] = known[i].load(std::memory_order_relaxed);
        if (regs[i] == 0) {
            cudaFuncAttributes f;
            const cudaError_t e = cudaFuncGetAttributes(&f, kernels[i]);
            if (e != cudaSuccess)
                return e;
            regs[i] = (f.numRegs + 7) / 8 * 8;
            known[i].store(regs[i], std::memory_order_relaxed);
        }
    }
    return cudaSuccess;
}

// Launches a ring kernel over the shape's rows.
template <auto K, typename Args>
cudaError_t launch_rows(const NormShape &sh, cudaStream_t s, const Args &a)
{
    return launch_smem<K, NORM_SMEM>(dim3(sh.ctas), dim3(32 * sh.W * sh.R), sh.smem, s, a, sh.S);
}
#endif

// The same for the element-by-element kernels: about 256 threads a CTA, `floats` fp32 values an element in shared
// memory for each of its rows side by side.
constexpr int SCALAR_SMEM = 224 * 1024;
NormShape scalar_shape(int H, int T, int floats, int max_ctas);

// vec8: every row (pointers and strides) on 16-byte boundaries and H a multiple of 8.
cudaError_t launch_norm_pre(const NormPreArgs &a, int h_dtype, bool vec8, cudaStream_t s);
cudaError_t launch_norm_post(const NormPostArgs &a, int y_dtype, int h_dtype, bool vec8, cudaStream_t s);

// The backward launches sum the weight gradients over the rows in `ws`
// (norm_workspace_bytes; none for one row) and finish them in d1 / d2 (each may be NULL).
size_t norm_workspace_bytes(int H, int T);
cudaError_t launch_norm_pre_bwd(const NormPreBwdArgs &a, int h_dtype, bool vec8, float *dw, float *ws, cudaStream_t s);
cudaError_t launch_norm_post_bwd(const NormPostBwdArgs &a, int y_dtype, int h_dtype, bool vec8, float *dpost,
                                 float *dnext, float *ws, cudaStream_t s);

}  // namespace vq
