// Device helpers shared by the kernels of the block around the experts (norms,
// balance loss, 4-bit products): chunks of a row in registers, sums over a
// row's warps, and launches with programmatic stream serialisation.
#pragma once

#include <cuda_runtime.h>

#include <atomic>

#include "vq_device.cuh"
#include "vq_internal.h"

namespace vq {

// Launch that may start its prologue while the previous kernel on the stream
// drains; every kernel launched so calls grid_dep_wait() before it touches
// memory that earlier work may have written.
template <typename K, typename... Args>
cudaError_t launch_after(K kernel, dim3 grid, dim3 block, size_t smem, cudaStream_t s, Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Raises a kernel's dynamic shared-memory limit to `bytes`, once per device:
// `done` (one per kernel, always the same bytes) remembers the devices.
inline cudaError_t allow_smem(const void *kernel, int bytes, std::atomic<uint64_t> &done)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit)
        return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess)
        done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// ---------------------------------------------------------------- chunks of a row
//
// VEC consecutive elements of a row: 8 with 16-byte accesses, or 1.

template <typename T, int VEC>
struct Chunk;

template <>
struct Chunk<uint16_t, 8> {   // bf16
    uint4 r;
    __device__ __forceinline__ void load(const uint16_t *p) { r = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void get(float (&v)[8]) const
    {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    __device__ __forceinline__ void set(const float (&v)[8])
    {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&b);
        }
        r = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ __forceinline__ void store(uint16_t *p) const { *reinterpret_cast<uint4 *>(p) = r; }
};

template <>
struct Chunk<float, 8> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p)
    {
        a = reinterpret_cast<const float4 *>(p)[0];
        b = reinterpret_cast<const float4 *>(p)[1];
    }
    __device__ __forceinline__ void get(float (&v)[8]) const
    {
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
    __device__ __forceinline__ void set(const float (&v)[8])
    {
        a = make_float4(v[0], v[1], v[2], v[3]);
        b = make_float4(v[4], v[5], v[6], v[7]);
    }
    __device__ __forceinline__ void store(float *p) const
    {
        reinterpret_cast<float4 *>(p)[0] = a;
        reinterpret_cast<float4 *>(p)[1] = b;
    }
};

template <>
struct Chunk<uint16_t, 1> {
    uint16_t r;
    __device__ __forceinline__ void load(const uint16_t *p) { r = *p; }
    __device__ __forceinline__ void get(float (&v)[1]) const { v[0] = bf16_to_f32(r); }
    __device__ __forceinline__ void set(const float (&v)[1]) { r = f32_to_bf16_bits(v[0]); }
    __device__ __forceinline__ void store(uint16_t *p) const { *p = r; }
};

template <>
struct Chunk<float, 1> {
    float r;
    __device__ __forceinline__ void load(const float *p) { r = *p; }
    __device__ __forceinline__ void get(float (&v)[1]) const { v[0] = r; }
    __device__ __forceinline__ void set(const float (&v)[1]) { r = v[0]; }
    __device__ __forceinline__ void store(float *p) const { *p = r; }
};

// A chunk whose type is known at run time (norm weights, per-channel gates):
// loaded raw, converted on use, so that the loads of several chunks overlap.
template <int VEC>
struct AnyChunk {
    Chunk<float, VEC> f;       // fp32 source
    Chunk<uint16_t, VEC> h;    // bf16 source
    __device__ __forceinline__ void load(const void *p, int dtype, long i)
    {
        if (dtype == VQ_F32)
            f.load(static_cast<const float *>(p) + i);
        else
            h.load(static_cast<const uint16_t *>(p) + i);
    }
    __device__ __forceinline__ void get(float (&v)[VEC], int dtype) const
    {
        if (dtype == VQ_F32)
            f.get(v);
        else
            h.get(v);
    }
};

// ---------------------------------------------------------------- sums

__device__ __forceinline__ float warp_total(float v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1)
        v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// Sums of N values over the W warps of a row (one row per CTA when W > 1).
// Two buffers in turn: a warp may start the next sum while another still
// reads this one.
template <int N>
struct RowSum {
    float buf[2][N][32];
};

template <int N, int M>
__device__ __forceinline__ void row_sum(float (&v)[N], RowSum<M> &s, int W, int &turn)
{
    static_assert(N <= M, "buffer too small");
#pragma unroll
    for (int i = 0; i < N; ++i)
        v[i] = warp_total(v[i]);
    if (W == 1)
        return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < N; ++i)
            s.buf[turn][i][warp] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i)
        v[i] = warp_total(lane < W ? s.buf[turn][i][lane] : 0.f);
    turn ^= 1;
}

}  // namespace vq
