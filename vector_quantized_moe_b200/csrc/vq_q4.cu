// Dense 4-bit matrix-vector products with group scales.
//
//   y[t, r] = sum_g ( s[r, g] sum_{c in g} (q[r, c] - 8) x[t, c]  +  (b[r, g] + 8 s[r, g]) sum_{c in g} x[t, c] )
// (the second term with biases only). The integers are exact in bf16, so the
// inner sums run on the tensor cores (mma m16n8k16: 16 rows of W against 8
// tokens) with x unrounded and fp32 accumulators; scales and the sum over
// groups are fp32. What the tensor cores get is 16 + q: a code moved into the
// upper mantissa bits of 16.0 needs one shift and one mask-or per pair of
// weights and no subtraction. 24 times a group's sum of x comes off its sum in
// fp32; the sum of x comes out of the same instruction against ones, in the
// lanes that need it. The offset makes the sums of a group about 5 times
// larger than those of q - 8, so their fp32 rounding counts that much more
// (measured against 64 bits: 3e-7 of the result's norm, a plain fp32 product
// 3e-7).
//
// The weights dominate the bytes (0.5 byte each, read once), so the layout is
// the lanes' own: one 16-byte load per lane is four mma A operands of a 16 x 64
// block, a warp's load 512 contiguous bytes.
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

// d (+)= a b, from zero when `first`.
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, bool first)
{
    if (first)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
            "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
            "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The four bf16 pairs 16 + q of a packed word: rotated by 4 i, code i of each
// half sits in the upper four mantissa bits of 16.0 (0x4180).
__device__ __forceinline__ void decode(uint32_t w, uint32_t (&a)[4])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t v = i == 3 ? __funnelshift_r(w, w, 12) : w >> (4 * i);
        asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(a[i]) : "r"(v), "r"(0x00780078u), "r"(0x41804180u));   // v & mask | 16.0
    }
}

__device__ __forceinline__ float2 half_pair(uint32_t v)
{
    return __half22float2(*reinterpret_cast<const __half2 *>(&v));
}

// Most warps per CTA (and per row group): the kernels' registers decide.
template <int R, int NT>
constexpr int MAX_WARPS = R == 4 ? 4 : R == 2 && NT < 4 ? 16 : 8;
constexpr long Q4_WANT_WARPS = 148 * 16;   // 16 warps on every SM

// CTAs of that size an SM holds at least.
template <int R, int NT>
constexpr int MIN_CTAS = R == 4 ? 4 : NT == 4 || MAX_WARPS<R, NT> == 16 ? 1 : NT == 2 ? 2 : 3;

// Bytes of one pipeline stage of a warp: R tiles' words, their scale (and bias)
// pairs.
template <int R, int G, bool BIAS>
constexpr int STAGE_BYTES = R * (1024 + 32 * (128 / G) * (BIAS ? 2 : 1));
// Stages per warp: enough bytes in flight per SM with two CTAs resident.
template <int R>
constexpr int STAGES = R == 4 ? 2 : R == 2 ? 4 : 6;

template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src)
{
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}

template <int NG>
__device__ __forceinline__ void lds_pairs(uint32_t at, uint32_t (&v)[NG])
{
    if constexpr (NG == 4) {
        const uint4 t = lds128(at);
        v[0] = t.x, v[1] = t.y, v[2] = t.z, v[3] = t.w;
    } else if constexpr (NG == 2) {
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "r"(at));
    } else {
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v[0]) : "r"(at));
    }
}

// R: row tiles per warp (of a pair: R / 2 of each module); NT: 8-token tiles.
// ks of the CTA's warps share a row group of R tiles and take its column tiles
// in turn.
template <int R, int NT, int G, bool BIAS>
__global__ void __launch_bounds__(32 * MAX_WARPS<R, NT>, MIN_CTAS<R, NT>) vq_q4_gemv_kernel(const Q4Args a, int ks)
{
    constexpr int NG = 128 / G;           // groups of columns per column tile
    constexpr int SPANS = G / 32;         // 32-column spans per group
    constexpr int D = STAGES<R>, SB = STAGE_BYTES<R, G, BIAS>, V = R * NT * 4;
    extern __shared__ __align__(128) unsigned char ring[];   // [warps][D][SB]; later the warps' sums [warps][V][32]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, c = lane & 3;
    const int t0 = blockIdx.y * (8 * NT);
    const int per = a.pair ? R / 2 : R;   // row tiles of a module per row group
    const int kw = warp & (ks - 1);
    const int grp = blockIdx.x * (blockDim.x / 32 / ks) + warp / ks;

    // a lane's place in its row group's tiles; tiles past the last repeat it (their sums are not stored)
    const uint32_t base = (uint32_t)__cvta_generic_to_shared(ring) + warp * (D * SB);
    const uint32_t *wp[R];
    const uint16_t *sp[R], *bp[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const bool up = a.pair && (r & 1);
        const long at = min((long)grp * per + (a.pair ? r >> 1 : r), (long)a.tiles - 1) * a.nsb + kw;
        wp[r] = (up ? a.words[1] : a.words[0]) + at * 256 + lane * 4;
        sp[r] = (up ? a.scales[1] : a.scales[0]) + (at * 8 + g) * (2 * NG);
        bp[r] = BIAS ? (up ? a.biases[1] : a.biases[0]) + (at * 8 + g) * (2 * NG) : nullptr;
    }
    auto fetch = [&](int sb, int stage) {
        if (sb < a.nsb) {
            const uint32_t at = base + stage * SB;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                copy_async<16>(at + r * 1024 + lane * 16, wp[r]);
                copy_async<16>(at + r * 1024 + 512 + lane * 16, wp[r] + 128);
                wp[r] += ks * 256;
                if (c == 0) {
                    copy_async<4 * NG>(at + R * 1024 + (r * 8 + g) * (4 * NG), sp[r]);
                    if constexpr (BIAS)
                        copy_async<4 * NG>(at + R * 1024 + ((R + r) * 8 + g) * (4 * NG), bp[r]);
                }
                sp[r] += ks * (16 * NG);
                if constexpr (BIAS)
                    bp[r] += ks * (16 * NG);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // x fragments of a column tile (of a span for 32 tokens). Tokens past the last read token 0 again (their results
    // are not stored), spans past the last column its last span (their scales are 0).
    const uint16_t *xp[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n)
        xp[n] = a.x + (t0 + 8 * n + g < a.T ? (long)(t0 + 8 * n + g) * a.x_ld : 0) + 8 * c;
    uint4 xv[NT < 4 ? 4 : 1][NT];
    auto load_x = [&](int sb, int p, uint4 (&v)[NT]) {
        const int k = min(sb * 128 + p * 32, a.cols - 32);
#pragma unroll
        for (int n = 0; n < NT; ++n)
            v[n] = ldg_u128(xp[n] + k);
    };
    float acc[R][NT][4];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc[r][n][j] = 0.f;

    grid_dep_launch();
    grid_dep_wait();
#pragma unroll
    for (int i = 0; i < D - 1; ++i)
        fetch(kw + i * ks, i);
    int stage = 0;
    for (int sb = kw; sb < a.nsb; sb += ks) {
        if constexpr (NT < 4) {
#pragma unroll
            for (int p = 0; p < 4; ++p)
                load_x(sb, p, xv[p]);
        }
        asm volatile("cp.async.wait_group %0;" ::"n"(D - 2) : "memory");
        __syncwarp();   // the stage's scales came through other lanes, and all lanes are done with the stage refilled next
        fetch(sb + (D - 1) * ks, stage == 0 ? D - 1 : stage - 1);
        const uint32_t at = base + stage * SB;
        stage = stage == D - 1 ? 0 : stage + 1;
        uint32_t sc[R][NG], bi[R][NG];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            lds_pairs<NG>(at + R * 1024 + (r * 8 + g) * (4 * NG), sc[r]);
            if constexpr (BIAS)
                lds_pairs<NG>(at + R * 1024 + ((R + r) * 8 + g) * (4 * NG), bi[r]);
        }
        float part[R][NT][4], xs[NT][4];
        uint4 w[R];
#pragma unroll
        for (int p = 0; p < 4; ++p) {   // 32-column spans
            if ((p & 1) == 0) {
#pragma unroll
                for (int r = 0; r < R; ++r)
                    w[r] = lds128(at + r * 1024 + (p >> 1) * 512 + lane * 16);
            }
            if constexpr (NT == 4)
                load_x(sb, p, xv[0]);
            constexpr int XP = NT < 4 ? 1 : 0;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const bool first = p % SPANS == 0 && h == 0;   // a group's sums start from zero
                const uint32_t ones[4] = {BF16_ONES, BF16_ONES, BF16_ONES, BF16_ONES};
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const uint4 &x = xv[XP * p][n];
                    mma_bf16(xs[n], ones, h ? x.z : x.x, h ? x.w : x.y, first);
                }
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const uint32_t word = (p & 1) ? (h ? w[r].w : w[r].z) : (h ? w[r].y : w[r].x);
                    uint32_t A[4];
                    decode(word, A);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const uint4 &x = xv[XP * p][n];
                        mma_bf16(part[r][n], A, h ? x.z : x.x, h ? x.w : x.y, first);
                    }
                }
            }
            if (p % SPANS == SPANS - 1) {
                const int gi = p / SPANS;
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float2 s = half_pair(sc[r][gi]);
                    float2 b = make_float2(0.f, 0.f);
                    if constexpr (BIAS) {
                        b = half_pair(bi[r][gi]);
                        b = make_float2(fmaf(8.f, s.x, b.x), fmaf(8.f, s.y, b.y));
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float q = fmaf(-24.f, xs[n][j & 1], part[r][n][j]);   // sum (q - 8) x
                            acc[r][n][j] = fmaf(j < 2 ? s.x : s.y, q, acc[r][n][j]);
                            if constexpr (BIAS)
                                acc[r][n][j] = fmaf(j < 2 ? b.x : b.y, xs[n][j & 1], acc[r][n][j]);
                        }
                }
            }
        }
    }

    if (ks > 1) {
        float *sums = reinterpret_cast<float *>(ring);
        // every copy has landed (the last turns' groups are empty) and every warp is done with its ring
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    sums[(warp * V + (r * NT + n) * 4 + j) * 32 + lane] = acc[r][n][j];
        __syncthreads();
        // the values are spread over the row group's warps, each adds its own in warp order; of a pair, the warp that
        // stores a value needs both modules' sums
        const float *s = sums + (size_t)(warp - kw) * V * 32;
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int v = ((a.pair ? r >> 1 : r) * NT + n) * 4 + j;
                    if ((v & (ks - 1)) == kw) {
                        float t = 0.f;
                        for (int w = 0; w < ks; ++w)
                            t += s[(w * V + (r * NT + n) * 4 + j) * 32 + lane];
                        acc[r][n][j] = t;
                    }
                }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if (a.pair && (r & 1))
            continue;
        const int i = a.pair ? r >> 1 : r;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int v = (i * NT + n) * 4 + j;
                const long row = ((long)grp * per + i) * 16 + g + 8 * (j >> 1);
                const int token = t0 + 8 * n + 2 * c + (j & 1);
                if ((v & (ks - 1)) != kw || row >= a.rows || token >= a.T)
                    continue;
                float out = acc[r][n][j];
                if constexpr (R > 1)
                    if (a.pair)
                        out = out * sigmoid(out) * acc[r | 1][n][j];
                const long yi = (long)token * a.y_ld + row;
                if (a.y_dtype == VQ_F32)
                    static_cast<float *>(a.y)[yi] = out;
                else
                    static_cast<uint16_t *>(a.y)[yi] = f32_to_bf16_bits(out);
            }
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
                    const uint32_t both = ((w >> (8 * pr)) & 15u) | ((w >> (8 * pr + 4)) & 15u) << 16;
                    out |= __funnelshift_l(both, both, 3 + 4 * m);
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
    const long groups = (a.tiles + per - 1) / per;
    // warps per row group: enough warps for the GPU, but no more than there are column tiles
    int ks = 1;
    while (ks < MAX_WARPS<R, NT> && 2 * ks <= a.nsb && groups * ks < Q4_WANT_WARPS)
        ks *= 2;
    const int warps = std::max(4, ks);
    constexpr int PER_WARP = std::max(STAGES<R> * STAGE_BYTES<R, G, BIAS>, R * NT * 4 * 32 * 4);
    static_assert(MAX_WARPS<R, NT> * PER_WARP <= 227 * 1024);
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t e = allow_smem((const void *)vq_q4_gemv_kernel<R, NT, G, BIAS>, MAX_WARPS<R, NT> * PER_WARP, allowed);
    if (e != cudaSuccess)
        return e;
    const dim3 grid((unsigned)((groups + warps / ks - 1) / (warps / ks)), (a.T + 8 * NT - 1) / (8 * NT));
    return launch_after(vq_q4_gemv_kernel<R, NT, G, BIAS>, grid, dim3(32 * warps), warps * PER_WARP, s, a, ks);
}

template <int G, bool BIAS>
cudaError_t pick(const Q4Args &a, cudaStream_t s)
{
    const int nt = a.T <= 8 ? 1 : a.T <= 16 ? 2 : 4;
    const long tiles = (long)a.tiles * (a.pair ? 2 : 1);
    // more row tiles per warp once R tiles a group still give every SM its warps (8 per group)
    const int r = nt < 4 && tiles * 8 >= 4 * Q4_WANT_WARPS ? 4 : a.pair || tiles * 8 >= 2 * Q4_WANT_WARPS ? 2 : 1;
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
