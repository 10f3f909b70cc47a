// Dense 4-bit matrix-vector products with group scales.
//
//   y[t, r] = sum_g ( s[r, g] sum_{c in g} (q[r, c] - 8) x[t, c]  +  (b[r, g] + 8 s[r, g]) sum_{c in g} x[t, c] )
// (the second term with biases only). The integers q - 8 are exact in bf16, so
// the inner sums run on the tensor cores (mma m16n8k16: 16 rows of W against 8
// tokens) with x unrounded and fp32 accumulators; scales and the sum over
// groups are fp32. A group's sum of x comes out of the same instruction
// against a row of ones, in the lanes that need it.
//
// The weights dominate the bytes (0.5 byte each, read once), so the layout is
// the lanes' own: one 16-byte load per lane is four mma A operands of a 16 x 64
// block, a warp's load 512 contiguous bytes. A nibble pair becomes a bf16 pair
// with one mask-or (0x4300 | q is 128 + q) and one subtraction of 136, 11
// instructions per 8 weights.
//
// A warp takes R row tiles at one column tile at a time, so that its x
// fragments serve R tiles; the CTA's warps take column tiles in turn and add
// their sums through shared memory in warp order.
#include <algorithm>

#include "vq_block.cuh"
#include "vq_norm.h"
#include "vq_q4.h"

namespace vq {
namespace {

constexpr uint32_t BF16_ONES = 0x3F803F80u;

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The four bf16 pairs q - 8 of a packed word.
__device__ __forceinline__ void decode(uint32_t w, uint32_t (&a)[4])
{
    const __nv_bfloat162 off = __halves2bfloat162(__ushort_as_bfloat16(0x4308), __ushort_as_bfloat16(0x4308));   // 136
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t v = ((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
        const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&v), off);
        a[i] = *reinterpret_cast<const uint32_t *>(&d);
    }
}

// A lane's scale (or bias) pairs of a column tile: NG pairs (rows g, g + 8), 4 NG bytes.
template <int NG>
__device__ __forceinline__ void load_pairs(const uint16_t *p, uint32_t (&v)[NG])
{
    if constexpr (NG == 4) {
        const uint4 t = ldg_u128(p);
        v[0] = t.x, v[1] = t.y, v[2] = t.z, v[3] = t.w;
    } else if constexpr (NG == 2) {
        const uint2 t = ldg_u64(reinterpret_cast<const uint32_t *>(p));
        v[0] = t.x, v[1] = t.y;
    } else {
        v[0] = ldg_u32(reinterpret_cast<const uint32_t *>(p));
    }
}

__device__ __forceinline__ float2 half_pair(uint32_t v)
{
    return __half22float2(*reinterpret_cast<const __half2 *>(&v));
}

// R: row tiles per warp (of a pair: R / 2 of each module); NT: 8-token tiles.
template <int R, int NT, int G, bool BIAS>
__global__ void __launch_bounds__(256) vq_q4_gemv_kernel(const Q4Args a)
{
    constexpr int NG = 128 / G;           // groups per column tile
    constexpr int SPANS = G / 32;         // 32-column spans per group
    extern __shared__ float sums[];       // [warps][R * NT * 4][32]
    grid_dep_launch();
    grid_dep_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const int g = lane >> 2, c = lane & 3;
    const int t0 = blockIdx.y * (8 * NT);
    const int per = a.pair ? R / 2 : R;   // row tiles of a module per CTA
    const uint32_t *wp[R];
    const uint16_t *sp[R], *bp[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        // tiles past the last repeat it; their sums are not stored
        const int m = a.pair ? r & 1 : 0, i = a.pair ? r >> 1 : r;
        const long tile = min((long)blockIdx.x * per + i, (long)a.tiles - 1);
        wp[r] = a.words[m] + tile * a.nsb * 256 + lane * 4;
        sp[r] = a.scales[m] + (tile * a.nsb * 8 + g) * (2 * NG);
        bp[r] = BIAS ? a.biases[m] + (tile * a.nsb * 8 + g) * (2 * NG) : nullptr;
    }
    const uint16_t *xp[NT];
    bool live[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        live[n] = t0 + 8 * n + g < a.T;
        xp[n] = a.x + (live[n] ? (long)(t0 + 8 * n + g) * a.x_ld : 0) + 8 * c;
    }
    float acc[R][NT][4];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc[r][n][j] = 0.f;

    for (int sb = warp; sb < a.nsb; sb += warps) {
        uint4 w[R][2];
        uint32_t sc[R][NG], bi[R][NG];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            w[r][0] = ldg_u128(wp[r] + (long)sb * 256);
            w[r][1] = ldg_u128(wp[r] + (long)sb * 256 + 128);
            load_pairs<NG>(sp[r] + (long)sb * (16 * NG), sc[r]);
            if constexpr (BIAS)
                load_pairs<NG>(bp[r] + (long)sb * (16 * NG), bi[r]);
        }
        float part[R][NT][4], xs[NT][4];
#pragma unroll
        for (int p = 0; p < 4; ++p) {   // 32-column spans
            if (p % SPANS == 0) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
#pragma unroll
                    for (int r = 0; r < R; ++r)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            part[r][n][j] = 0.f;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        xs[n][j] = 0.f;
                }
            }
            const int k0 = sb * 128 + p * 32;
            uint4 xv[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n)
                xv[n] = live[n] && k0 < a.cols ? ldg_u128(xp[n] + k0) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const uint4 q = w[r][p >> 1];
                    const uint32_t word = (p & 1) ? (h ? q.w : q.z) : (h ? q.y : q.x);
                    uint32_t A[4];
                    decode(word, A);
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        mma_bf16(part[r][n], A, h ? xv[n].z : xv[n].x, h ? xv[n].w : xv[n].y);
                }
                if constexpr (BIAS) {
                    const uint32_t A[4] = {BF16_ONES, BF16_ONES, BF16_ONES, BF16_ONES};
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        mma_bf16(xs[n], A, h ? xv[n].z : xv[n].x, h ? xv[n].w : xv[n].y);
                }
            }
            if (p % SPANS == SPANS - 1) {
                const int grp = p / SPANS;
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float2 s = half_pair(sc[r][grp]);
                    float2 b = make_float2(0.f, 0.f);
                    if constexpr (BIAS) {
                        b = half_pair(bi[r][grp]);
                        b = make_float2(fmaf(8.f, s.x, b.x), fmaf(8.f, s.y, b.y));
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        acc[r][n][0] = fmaf(s.x, part[r][n][0], acc[r][n][0]);
                        acc[r][n][1] = fmaf(s.x, part[r][n][1], acc[r][n][1]);
                        acc[r][n][2] = fmaf(s.y, part[r][n][2], acc[r][n][2]);
                        acc[r][n][3] = fmaf(s.y, part[r][n][3], acc[r][n][3]);
                        if constexpr (BIAS) {
                            acc[r][n][0] = fmaf(b.x, xs[n][0], acc[r][n][0]);
                            acc[r][n][1] = fmaf(b.x, xs[n][1], acc[r][n][1]);
                            acc[r][n][2] = fmaf(b.y, xs[n][2], acc[r][n][2]);
                            acc[r][n][3] = fmaf(b.y, xs[n][3], acc[r][n][3]);
                        }
                    }
                }
            }
        }
    }

    constexpr int V = R * NT * 4;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                sums[(warp * V + (r * NT + n) * 4 + j) * 32 + lane] = acc[r][n][j];
    __syncthreads();
    // outputs, rows fastest: (token, row of the CTA's tiles)
    for (int o = threadIdx.x; o < per * 16 * 8 * NT; o += blockDim.x) {
        const int rr = o % (per * 16), t = o / (per * 16);
        const int i = rr >> 4, row16 = rr & 15, n = t >> 3, t8 = t & 7;
        const int at = ((n * 4) + (row16 >> 3) * 2 + (t8 & 1)) * 32 + (row16 & 7) * 4 + (t8 >> 1);
        const long row = ((long)blockIdx.x * per + i) * 16 + row16;
        const int token = t0 + t;
        if (row >= a.rows || token >= a.T)
            continue;
        float v[2] = {0.f, 0.f};
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            if (m && !a.pair)
                break;
            const int r = a.pair ? 2 * i + m : i;
            for (int w = 0; w < warps; ++w)
                v[m] += sums[(w * V + r * NT * 4) * 32 + at];
        }
        const float out = a.pair ? v[0] * sigmoid(v[0]) * v[1] : v[0];
        const long yi = (long)token * a.y_ld + row;
        if (a.y_dtype == VQ_F32)
            static_cast<float *>(a.y)[yi] = out;
        else
            static_cast<uint16_t *>(a.y)[yi] = f32_to_bf16_bits(out);
    }
}

// Row-major codes and scales into the tile layout: a thread per output word,
// then per output scale.
__global__ void __launch_bounds__(256) vq_q4_pack_kernel(const uint32_t *codes, const uint16_t *scales,
                                                         const uint16_t *biases, int rows, int cols, int group,
                                                         int tiles, int nsb, uint32_t *words_out,
                                                         uint16_t *scales_out, uint16_t *biases_out)
{
    grid_dep_launch();
    grid_dep_wait();
    const long nw = (long)tiles * nsb * 256, step = (long)gridDim.x * blockDim.x;
    for (long o = (long)blockIdx.x * blockDim.x + threadIdx.x; o < nw; o += step) {
        const int s = o & 3, lane = (o >> 2) & 31, b = (o >> 7) & 1;
        const long tile = (o >> 8) / nsb, sb = (o >> 8) % nsb;
        const int k = (int)(sb * 128 + b * 64 + (s >> 1) * 32 + (lane & 3) * 8 + (s & 1) * 4);
        uint32_t out = 0;
#pragma unroll
        for (int hi = 0; hi < 2; ++hi) {
            const long row = tile * 16 + (lane >> 2) + 8 * hi;
            if (row < rows && k < cols) {
                const uint32_t w = codes[row * (cols / 8) + (k >> 3)] >> ((k & 4) * 4);   // columns k .. k + 3
#pragma unroll
                for (int pr = 0; pr < 2; ++pr) {   // columns k + 2 pr and k + 2 pr + 1
                    const int m = hi + 2 * pr;
                    out |= ((w >> (8 * pr)) & 15u) << (4 * m);
                    out |= ((w >> (8 * pr + 4)) & 15u) << (16 + 4 * m);
                }
            }
        }
        words_out[o] = out;
    }
    const int ng = 128 / group, ngroups = cols / group;
    const long ns = (long)tiles * nsb * 16 * ng;
    for (long o = (long)blockIdx.x * blockDim.x + threadIdx.x; o < ns; o += step) {
        const int hi = o & 1, gi = (int)((o >> 1) % ng), gr = (int)((o >> 1) / ng % 8);
        const long t = (o >> 1) / ng / 8, tile = t / nsb, sb = t % nsb;
        const long row = tile * 16 + gr + 8 * hi, grp = sb * ng + gi;
        const bool in = row < rows && grp < ngroups;
        scales_out[o] = in ? scales[row * ngroups + grp] : (uint16_t)0;
        if (biases)
            biases_out[o] = in ? biases[row * ngroups + grp] : (uint16_t)0;
    }
}

template <int R, int NT, int G, bool BIAS>
cudaError_t run(const Q4Args &a, cudaStream_t s)
{
    const int per = a.pair ? R / 2 : R;
    const int warps = std::min(8, a.nsb);
    const size_t smem = (size_t)warps * R * NT * 4 * 32 * 4;   // at most 32 KB
    const dim3 grid((a.tiles + per - 1) / per, (a.T + 8 * NT - 1) / (8 * NT));
    return launch_after(vq_q4_gemv_kernel<R, NT, G, BIAS>, grid, dim3(32 * warps), smem, s, a);
}

template <int G, bool BIAS>
cudaError_t pick(const Q4Args &a, cudaStream_t s)
{
    const int nt = a.T <= 8 ? 1 : a.T <= 16 ? 2 : 4;
    const int tiles = a.tiles * (a.pair ? 2 : 1);
    const int r = nt < 4 && tiles >= 4 * 4 * 148 ? 4 : a.pair || tiles >= 2 * 2 * 148 ? 2 : 1;
    switch (r * 8 + nt) {
    case 9: return run<1, 1, G, BIAS>(a, s);
    case 10: return run<1, 2, G, BIAS>(a, s);
    case 12: return run<1, 4, G, BIAS>(a, s);
    case 17: return run<2, 1, G, BIAS>(a, s);
    case 18: return run<2, 2, G, BIAS>(a, s);
    case 20: return run<2, 4, G, BIAS>(a, s);
    case 33: return run<4, 1, G, BIAS>(a, s);
    default: return run<4, 2, G, BIAS>(a, s);
    }
}

}  // namespace

cudaError_t launch_q4_gemv(const Q4Args &a, int group, cudaStream_t s)
{
    const bool b = a.biases[0] != nullptr;
    switch (group) {
    case 32: return b ? pick<32, true>(a, s) : pick<32, false>(a, s);
    case 64: return b ? pick<64, true>(a, s) : pick<64, false>(a, s);
    default: return b ? pick<128, true>(a, s) : pick<128, false>(a, s);
    }
}

cudaError_t launch_q4_pack(const uint32_t *codes, const uint16_t *scales, const uint16_t *biases, int rows, int cols,
                           int group, uint32_t *words_out, uint16_t *scales_out, uint16_t *biases_out, cudaStream_t s)
{
    const int tiles = (int)(((long)rows + 15) / 16), nsb = (int)(((long)cols + 127) / 128);
    const long blocks = (long)tiles * nsb;   // 256 words each
    return launch_after(vq_q4_pack_kernel, dim3((unsigned)std::min(blocks, 148L * 64)), dim3(256), 0, s, codes, scales,
                        biases, rows, cols, group, tiles, nsb, words_out, scales_out, biases_out);
}

}  // namespace vq
