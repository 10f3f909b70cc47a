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

// Launches kernel K with `smem` <= MOST bytes of dynamic shared memory.
template <auto K, int MOST, typename... Args>
cudaError_t launch_smem(dim3 grid, dim3 block, size_t smem, cudaStream_t s, Args... args)
{
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem((const void *)K, MOST, done);
    return e != cudaSuccess ? e : launch_after(K, grid, block, smem, s, args...);
}

// ---------------------------------------------------------------- pairs
//
// Two fp32 operations per instruction (fma.rn.f32x2 and its kin): the row
// kernels are bound by instruction issue before they are by HBM.

__device__ __forceinline__ float2 splat(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }

// ---------------------------------------------------------------- chunks of a row
//
// VEC consecutive elements of a row: 8 with 16-byte accesses, as four fp32 pairs, or 1 (read only).

template <typename T, int VEC>
struct Chunk;

template <>
struct Chunk<uint16_t, 8> {   // bf16
    uint4 r;
    __device__ __forceinline__ void load(const uint16_t *p) { r = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void store(uint16_t *p) const { *reinterpret_cast<uint4 *>(p) = r; }
    __device__ __forceinline__ void get(float2 (&v)[4]) const
    {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
    }
    __device__ __forceinline__ void set(const float2 (&v)[4])
    {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[i].x, v[i].y);
            w[i] = *reinterpret_cast<const uint32_t *>(&b);
        }
        r = make_uint4(w[0], w[1], w[2], w[3]);
    }
};

template <>
struct Chunk<float, 8> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p)
    {
        a = reinterpret_cast<const float4 *>(p)[0];
        b = reinterpret_cast<const float4 *>(p)[1];
    }
    __device__ __forceinline__ void store(float *p) const
    {
        reinterpret_cast<float4 *>(p)[0] = a;
        reinterpret_cast<float4 *>(p)[1] = b;
    }
    __device__ __forceinline__ void get(float2 (&v)[4]) const
    {
        v[0] = make_float2(a.x, a.y), v[1] = make_float2(a.z, a.w);
        v[2] = make_float2(b.x, b.y), v[3] = make_float2(b.z, b.w);
    }
    __device__ __forceinline__ void set(const float2 (&v)[4])
    {
        a = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
        b = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
    }
};

template <>
struct Chunk<uint16_t, 1> {
    uint16_t r;
    __device__ __forceinline__ void load(const uint16_t *p) { r = *p; }
    __device__ __forceinline__ void get(float (&v)[1]) const { v[0] = bf16_to_f32(r); }
};

template <>
struct Chunk<float, 1> {
    float r;
    __device__ __forceinline__ void load(const float *p) { r = *p; }
    __device__ __forceinline__ void get(float (&v)[1]) const { v[0] = r; }
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
    template <typename V>
    __device__ __forceinline__ void get(V &v, int dtype) const
    {
        if (dtype == VQ_F32)
            f.get(v);
        else
            h.get(v);
    }
};

// A chunk of a norm's weight as fp32, offset added.
__device__ __forceinline__ void load_weight(const void *p, int dtype, float offset, int c, float2 (&w)[4])
{
    AnyChunk<8> k;
    k.load(p, dtype, c);
    k.get(w, dtype);
#pragma unroll
    for (int j = 0; j < 4; ++j)
        w[j] = add2(w[j], splat(offset));
}

// ---------------------------------------------------------------- asynchronous copies
//
// A thread's own ring of 16-byte pieces in shared memory: piece k of a stage
// is `step` bytes (16 x threads) after piece k - 1, so a warp's accesses are
// contiguous. Each thread copies and reads only its own pieces, so a copy
// needs no barrier, only the thread's own wait.

__device__ __forceinline__ void copy16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// Waits until at most `pending` (0 to 2) of this thread's groups are in flight.
__device__ __forceinline__ void copy_wait(int pending)
{
    if (pending == 2)
        asm volatile("cp.async.wait_group 2;" ::: "memory");
    else if (pending == 1)
        asm volatile("cp.async.wait_group 1;" ::: "memory");
    else
        asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// An ordinary load, so that the compiler may place it (the waits above are its only fences).
__device__ __forceinline__ uint4 lds128(uint32_t at)
{
    return *static_cast<const uint4 *>(__cvta_shared_to_generic(at));
}

// Pieces of a chunk of 8 elements.
template <typename T>
constexpr int PIECES = sizeof(T) / 2;

template <typename T>
__device__ __forceinline__ void ring_copy(uint32_t at, uint32_t step, const T *p)
{
    copy16(at, p);
    if constexpr (PIECES<T> == 2)
        copy16(at + step, p + 4);
}

template <typename T>
__device__ __forceinline__ void ring_get(uint32_t at, uint32_t step, float2 (&v)[4])
{
    Chunk<T, 8> c;
    if constexpr (PIECES<T> == 2) {
        const uint4 a = lds128(at), b = lds128(at + step);
        c.a = make_float4(__uint_as_float(a.x), __uint_as_float(a.y), __uint_as_float(a.z), __uint_as_float(a.w));
        c.b = make_float4(__uint_as_float(b.x), __uint_as_float(b.y), __uint_as_float(b.z), __uint_as_float(b.w));
    } else {
        c.r = lds128(at);
    }
    c.get(v);
}

// The same for an array whose type is known at run time.
__device__ __forceinline__ void ring_copy_any(uint32_t at, uint32_t step, const void *p, int dtype, long i)
{
    if (dtype == VQ_F32)
        ring_copy(at, step, static_cast<const float *>(p) + i);
    else
        ring_copy(at, step, static_cast<const uint16_t *>(p) + i);
}

__device__ __forceinline__ void ring_get_any(uint32_t at, uint32_t step, int dtype, float2 (&v)[4])
{
    if (dtype == VQ_F32)
        ring_get<float>(at, step, v);
    else
        ring_get<uint16_t>(at, step, v);
}

// ---------------------------------------------------------------- sums

__device__ __forceinline__ float warp_total(float v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1)
        v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// One step of a sum of two values over a warp at once: after it, lanes whose
// bit `bit` is 0 work on a, the others on b.
__device__ __forceinline__ float fold(float a, float b, int bit, int lane)
{
    const bool up = lane & bit;
    return (up ? b : a) + __shfl_xor_sync(0xFFFFFFFFu, up ? a : b, bit);
}

template <int FROM>
__device__ __forceinline__ float warp_total_from(float v)
{
#pragma unroll
    for (int o = FROM; o; o >>= 1)
        v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// Sums of N <= 3 values over the W <= 16 warps of a row, in a fixed order; rows side
// by side in a CTA meet at barriers of their own. Several values share the warp's shuffles: 5, 5 and
// 6 for 1, 2 and 3 values. Two buffers in turn: a warp may start the next sum
// while another still reads this one.
constexpr int ROW_THREADS = 512;           // most threads a row, and a CTA of rows
template <int N>
struct RowSum {
    float buf[2][N][ROW_THREADS / 32];
};

// A thread's place among the W warps of its row, R rows side by side in the CTA.
struct RowTeam {
    int W, R, tid, rg, warp;   // tid: thread of the row; rg: row of the CTA; warp: warp of the row
    __device__ __forceinline__ explicit RowTeam(int w)
        : W(w), R(blockDim.x / (32 * w)), tid(threadIdx.x % (32 * w)), rg(threadIdx.x / (32 * w)), warp(tid >> 5) {}
};

template <int N, int M>
__device__ __forceinline__ void row_sum(float (&v)[N], RowSum<M> &s, const RowTeam &m, int &turn)
{
    static_assert(N <= M && N <= 3, "sums");
    const int lane = threadIdx.x & 31, W = m.W, first = m.rg * W;
    float x;        // lanes 0, 16, 8: totals of v[0], v[1], v[2]
    if constexpr (N == 1)
        x = warp_total_from<16>(v[0]);
    else if constexpr (N == 2)
        x = warp_total_from<8>(fold(v[0], v[1], 16, lane));
    else
        x = warp_total_from<4>(fold(fold(v[0], v[1], 16, lane), fold(v[2], 0.f, 16, lane), 8, lane));
    if (W == 1) {
        v[0] = __shfl_sync(0xFFFFFFFFu, x, 0);
        if constexpr (N > 1)
            v[1] = __shfl_sync(0xFFFFFFFFu, x, 16);
        if constexpr (N > 2)
            v[2] = __shfl_sync(0xFFFFFFFFu, x, 8);
        return;
    }
    if (lane == 0)
        s.buf[turn][0][first + m.warp] = x;
    if (N > 1 && lane == 16)
        s.buf[turn][N > 1 ? 1 : 0][first + m.warp] = x;
    if (N > 2 && lane == 8)
        s.buf[turn][N > 2 ? 2 : 0][first + m.warp] = x;
    if (m.R == 1)
        __syncthreads();
    else
        asm volatile("bar.sync %0, %1;" ::"r"(1 + m.rg), "r"(32 * W) : "memory");
    const int l = lane & 15;
    if constexpr (N == 1) {
        v[0] = warp_total_from<8>(l < W ? s.buf[turn][0][first + l] : 0.f);
    } else {
        x = warp_total_from<8>(l < W ? s.buf[turn][lane >> 4][first + l] : 0.f);
        v[0] = __shfl_sync(0xFFFFFFFFu, x, 0);
        v[1] = __shfl_sync(0xFFFFFFFFu, x, 16);
        if constexpr (N > 2)
            v[2] = warp_total_from<8>(l < W ? s.buf[turn][2][first + l] : 0.f);
    }
    turn ^= 1;
}

}  // namespace vq
