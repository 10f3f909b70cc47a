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
// larger than those of q - 8, so their fp32 rounding counts that much more. Against 64
// bits, relative to the result's norm: 131072 x 4096, tokens of mean 0, 2.1e-7 (a plain fp32
// product 3.3e-7); tokens with a common offset of 1 to 100, 2e-7 to 7e-7 (plain: 4e-8 to 1.1e-7).
//
// The weights dominate the bytes (0.5 byte each, read once), so the layout is
// the lanes' own: one 16-byte load per lane is four mma A operands of a 16 x 64
// block, a warp's load 512 contiguous bytes.
//
// A warp takes R row tiles at one column tile at a time, so that its x
// fragments serve R tiles; the CTA's warps take column tiles in turn and add
// their sums through shared memory in warp order.
//
// Measured (GPU time): 131072 x 4096, 8 tokens 53.1 us for 281 MB (5.3 TB/s, 0.81 of the
// copy rate; the copies alone, without decoding and mma, take 45 us); bound by
// the ALU pipe (65% busy: three shifts and four mask-ors per word, 7 per 8
// weights, at half rate) and the latency of 16 warps on an SM. 6144 x 6144, 1 token 8.4
// us for 21 MB, 2 x 2040 x 6144, 16 tokens 9.0 us: 3 to 6 turns of a warp at 0.9 to 1.2 us and
// 2 to 4 us of start and end. The subtraction of 8 as an instruction: 171
// instructions a 16 x 128 tile instead of 126. Shifts as high multiplies on
// the FMA pipe: 73 us. Persistent CTAs that copy ahead across row groups: 64 us.
// Every 16 tokens more decode all weights once more: 16384 x 4096, 16 tokens 17.6 us, 32
// tokens 30.2 us.
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
        asm(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
            "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
    else
        asm(
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

// Most warps per CTA (and per row group), and CTAs of that size an SM holds at least: the kernels' registers decide.
template <int R, int NT>
constexpr int MAX_WARPS = R == 4 ? 4 : R == 2 ? 16 : 8;
template <int R, int NT>
constexpr int MIN_CTAS = R == 4 ? 4 : R == 2 ? 1 : NT == 1 ? 3 : 2;

// Bytes of one pipeline stage of a warp: R tiles' words and their scale (and
// bias) pairs; with x in the ring, 256 more for every live token.
template <int R, int G, bool BIAS>
constexpr int STAGE_BYTES = R * (1024 + 32 * (128 / G) * (BIAS ? 2 : 1));

// Whether x goes through the ring too. A warp of four row tiles has enough to
// do to hide its x loads (from L1, shared with its neighbours); with fewer,
// each turn would wait for them.
template <int R>
constexpr bool X_RING = R < 4;

// Warps an SM should hold.
template <int R, int NT>
constexpr int SM_WARPS = R == 1 && NT == 1 ? 24 : 16;
constexpr int Q4_SMEM = 222 * 1024;   // shared memory of an SM given to the rings

template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src)
{
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}

__device__ __forceinline__ void sts128(uint32_t at, uint4 v)
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

template <int NG>
__device__ __forceinline__ void lds_pairs(uint32_t at, uint32_t (&v)[NG])
{
    const void *p = __cvta_shared_to_generic(at);
    if constexpr (NG == 4) {
        const uint4 t = *static_cast<const uint4 *>(p);
        v[0] = t.x, v[1] = t.y, v[2] = t.z, v[3] = t.w;
    } else if constexpr (NG == 2) {
        const uint2 t = *static_cast<const uint2 *>(p);
        v[0] = t.x, v[1] = t.y;
    } else {
        v[0] = *static_cast<const uint32_t *>(p);
    }
}

// R: row tiles per warp (of a pair: R / 2 of each module); NT: 8-token tiles.
// ks of the CTA's warps share a row group of R tiles and take its column tiles
// in turn; S stages of SB bytes a warp, S - 1 of them copied ahead.
template <int R, int NT, int G, bool BIAS>
__global__ void __launch_bounds__(32 * MAX_WARPS<R, NT>, MIN_CTAS<R, NT>) vq_q4_gemv_kernel(const Q4Args a, int ks, int S, int SB)
{
    constexpr int NG = 128 / G;           // groups of columns per column tile
    constexpr int SPANS = G / 32;         // 32-column spans per group
    constexpr int V = R * NT * 4, XS = STAGE_BYTES<R, G, BIAS>;   // XS: where a stage's x starts
    extern __shared__ __align__(128) unsigned char ring[];   // [warps][S][SB]; later the warps' sums [warps][V][32]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, c = lane & 3;
    const int t0 = blockIdx.y * (8 * NT), live = min(8 * NT, a.T - t0);
    const int per = a.pair ? R / 2 : R;   // row tiles of a module per row group
    const int kw = warp & (ks - 1);
    const int grp = blockIdx.x * (blockDim.x / 32 / ks) + warp / ks;

    // a lane's place in its row group's tiles; tiles past the last repeat it (their sums are not stored)
    const uint32_t base = (uint32_t)__cvta_generic_to_shared(ring) + warp * (S * SB);
    auto tile_at = [&](int r) {
        return min((long)grp * per + (a.pair ? r >> 1 : r), (long)a.tiles - 1) * a.nsb + kw;
    };
    const uint32_t *wp[R];
#pragma unroll
    for (int r = 0; r < R; ++r)
        wp[r] = (a.pair && (r & 1) ? a.words[1] : a.words[0]) + tile_at(r) * 256 + lane * 4;
    // scales: the lanes of column c copy tile c's, the next R columns its biases (a second copy where R is 4)
    const int cr = c & (R - 1);
    const bool cup = a.pair && (cr & 1), scale_lane = c < R, bias_lane = BIAS && R < 4 && c >= R && c < 2 * R;
    const long scale_at = (tile_at(cr) * 8 + g) * (2 * NG);
    const uint16_t *sp = (bias_lane ? (cup ? a.biases[1] : a.biases[0]) : (cup ? a.scales[1] : a.scales[0])) + scale_at;
    const uint16_t *bp = BIAS && R == 4 ? (cup ? a.biases[1] : a.biases[0]) + scale_at : nullptr;
    const uint32_t sdst = R * 1024 + (((bias_lane ? R : 0) + cr) * 8 + g) * (4 * NG);
    auto fetch = [&](int sb, int stage) {
        if (sb < a.nsb) {
            const uint32_t at = base + stage * SB;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                copy_async<16>(at + r * 1024 + lane * 16, wp[r]);
                copy_async<16>(at + r * 1024 + 512 + lane * 16, wp[r] + 128);
                wp[r] += ks * 256;
            }
            if (scale_lane || bias_lane)
                copy_async<4 * NG>(at + sdst, sp);
            sp += ks * (16 * NG);
            if constexpr (BIAS && R == 4) {
                copy_async<4 * NG>(at + sdst + R * 8 * (4 * NG), bp);
                bp += ks * (16 * NG);
            }
            if constexpr (X_RING<R>) {
                // 16 chunks of 8 columns a token, odd tokens with their 64-byte halves swapped so that two tokens'
                // reads meet in no bank; chunks past the last column stay what they were (their scales are 0)
                for (int i = lane; i < live * 16; i += 32) {
                    const int n = i >> 4, k = i & 15;
                    if (sb * 128 + k * 8 < a.cols)
                        copy_async<16>(at + XS + n * 256 + (k ^ (n & 1) * 4) * 16,
                                       a.x + (t0 + n) * a.x_ld + sb * 128 + k * 8);
                }
            }
        }
        copy_commit();
    };
    // x fragments. Tokens past the last read token 0 again (their results are not stored), spans past the last column
    // something finite: the last span again, or what the ring holds.
    const uint16_t *xp[NT];
    uint32_t xat[NT], xhalf[NT];   // spans p: xat + 128 (p / 2), + xhalf for even p, + 64 - xhalf for odd p
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int m = 8 * n + g < live ? 8 * n + g : 0;
        xp[n] = a.x + (t0 + m) * a.x_ld + 8 * c;
        xat[n] = XS + m * 256 + c * 16;
        xhalf[n] = (m & 1) * 64;
    }
    uint4 xv[X_RING<R> ? 1 : 4][NT];
    auto load_x = [&](int sb, int p, uint4 (&v)[NT]) {
        const int k = min(sb * 128 + p * 32, a.cols - 32);
#pragma unroll
        for (int n = 0; n < NT; ++n)
            v[n] = load_u128(xp[n] + k);
    };
    if constexpr (X_RING<R>) {   // chunks that no copy fills hold zeros
        if (a.cols % 128)
            for (int i = lane; i < S * (live * 16); i += 32)
                sts128(base + (i / (live * 16)) * SB + XS + (i % (live * 16)) * 16, make_uint4(0, 0, 0, 0));
        __syncwarp();
    }
    float2 acc[R][NT][2];   // rows g and g + 8, tokens 2 c and 2 c + 1
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int n = 0; n < NT; ++n)
            acc[r][n][0] = acc[r][n][1] = splat(0.f);

    // while the work before this launch ends: the first weights into L2 (a hint; they are read after the wait). 6144 x
    // 6144 out of HBM: 9.25 -> 8.7 us. Grids of several rounds (R = 4) have their own CTAs to overlap: 54.4 -> 55.8 us.
    if (R < 4 && lane == 0) {
#pragma unroll
        for (int r = 0; r < R; ++r)
            for (int i = 0; i < S && kw + i * ks < a.nsb; ++i)
                asm volatile("cp.async.bulk.prefetch.L2.global [%0], 1024;" ::"l"(wp[r] + i * ks * 256) : "memory");
    }
    grid_dep_launch();
    grid_dep_wait();
    for (int i = 0; i < S - 1; ++i)
        fetch(kw + i * ks, i);
    int stage = 0;
    for (int sb = kw; sb < a.nsb; sb += ks) {
        if constexpr (!X_RING<R>) {
#pragma unroll
            for (int p = 0; p < 4; ++p)
                load_x(sb, p, xv[p]);
        }
        copy_wait(S - 2);
        __syncwarp();   // scales and x came through other lanes, and all lanes are done with the stage refilled next
        fetch(sb + (S - 1) * ks, stage == 0 ? S - 1 : stage - 1);
        const uint32_t at = base + stage * SB;
        stage = stage == S - 1 ? 0 : stage + 1;
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
            constexpr int XP = X_RING<R> ? 0 : 1;
            if constexpr (X_RING<R>) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    xv[0][n] = lds128(at + xat[n] + (p >> 1) * 128 + ((p & 1) ? 64 - xhalf[n] : xhalf[n]));
            }
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
                    // s sum (q - 8) x + b' sum x with b' = 0 or b + 8 s, as s sum (16 + q) x + (b' - 24 s) sum x
                    const float2 s = half_pair(sc[r][gi]);
                    float2 b = make_float2(-24.f * s.x, -24.f * s.y);
                    if constexpr (BIAS) {
                        b = half_pair(bi[r][gi]);
                        b = make_float2(fmaf(-16.f, s.x, b.x), fmaf(-16.f, s.y, b.y));
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const float2 x = make_float2(xs[n][0], xs[n][1]);
                        acc[r][n][0] = fma2(splat(b.x), x, fma2(splat(s.x), make_float2(part[r][n][0], part[r][n][1]), acc[r][n][0]));
                        acc[r][n][1] = fma2(splat(b.y), x, fma2(splat(s.y), make_float2(part[r][n][2], part[r][n][3]), acc[r][n][1]));
                    }
                }
            }
        }
    }

    float out[R][NT][4];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                out[r][n][j] = (j & 1) ? acc[r][n][j >> 1].y : acc[r][n][j >> 1].x;
    if (ks > 1) {
        float *sums = reinterpret_cast<float *>(ring);
        // every copy has landed (the last turns' groups are empty) and every warp is done with its ring
        copy_wait(0);
        __syncthreads();
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    sums[(warp * V + (r * NT + n) * 4 + j) * 32 + lane] = out[r][n][j];
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
                        out[r][n][j] = t;
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
                float o = out[r][n][j];
                if constexpr (R > 1)
                    if (a.pair)
                        o = o * sigmoid(o) * out[r | 1][n][j];
                const long yi = (long)token * a.y_ld + row;
                if (a.y_dtype == VQ_F32)
                    static_cast<float *>(a.y)[yi] = o;
                else
                    static_cast<uint16_t *>(a.y)[yi] = f32_to_bf16_bits(o);
            }
    }
}

// Row-major codes and scales into the tile layout: a thread per lane of a 16 x
// 64 block (4 words from two rows), then per output scale.
__global__ void __launch_bounds__(256) vq_q4_pack_kernel(const uint32_t *codes, const uint16_t *scales,
                                                         const uint16_t *biases, int rows, int cols, int group,
                                                         int tiles, int nsb, uint32_t *words_out,
                                                         uint16_t *scales_out, uint16_t *biases_out)
{
    grid_dep_launch();
    grid_dep_wait();
    const long nq = (long)tiles * nsb * 64, step = (long)gridDim.x * blockDim.x;
    for (long o = (long)blockIdx.x * blockDim.x + threadIdx.x; o < nq; o += step) {
        const int lane = o & 31, b = (o >> 5) & 1;
        const long tile = (o >> 6) / nsb, sb = (o >> 6) - tile * nsb;
        const long k = sb * 128 + b * 64 + (lane & 3) * 8, row = tile * 16 + (lane >> 2);
        uint32_t w[2][2];   // [span][row g, g + 8]: 8 codes each
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int hi = 0; hi < 2; ++hi)
                w[p][hi] = row + 8 * hi < rows && k + 32 * p < cols ? codes[(row + 8 * hi) * (cols / 8) + (k >> 3) + 4 * p] : 0;
        uint32_t out[4] = {0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int m = 0; m < 4; ++m) {   // row g + 8 (m % 2), columns 4 (s % 2) + 2 (m / 2) and the next
                const uint32_t v = w[s >> 1][m & 1] >> (16 * (s & 1) + 8 * (m >> 1));
                const uint32_t both = (v & 15u) | ((v >> 4) & 15u) << 16;
                out[s] |= __funnelshift_l(both, both, 3 + 4 * m);
            }
        reinterpret_cast<uint4 *>(words_out)[o] = make_uint4(out[0], out[1], out[2], out[3]);
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
cudaError_t run(const Q4Args &a, int ks, cudaStream_t s)
{
    const int per = a.pair ? R / 2 : R, groups = (a.tiles + per - 1) / per;
    const int warps = std::max(4, ks);
    const int sb = STAGE_BYTES<R, G, BIAS> + (X_RING<R> ? std::min(a.T, 8 * NT) * 256 : 0);
    const int stages = R == 4 ? 2 : std::max(2, std::min(4, Q4_SMEM / (std::max(SM_WARPS<R, NT>, warps) * sb)));
    const size_t smem = (size_t)warps * std::max(stages * sb, R * NT * 4 * 32 * 4);
    // two stages of the most warps fit
    static_assert(MAX_WARPS<R, NT> * 2 * (STAGE_BYTES<R, G, BIAS> + (X_RING<R> ? 8 * NT * 256 : 0)) <= Q4_SMEM);
    const dim3 grid((groups + warps / ks - 1) / (warps / ks), (a.T + 8 * NT - 1) / (8 * NT));
    return launch_smem<vq_q4_gemv_kernel<R, NT, G, BIAS>, Q4_SMEM>(grid, dim3(32 * warps), smem, s, a, ks, stages, sb);
}

// The row tiles per warp and the warps per row group with the least estimated
// time. CTAs run in rounds of what an SM holds; a round takes its warps' turns
// (a column tile each) and a start and end of about 4 us; a turn takes 0.9 us
// (1.2 us for 16 tokens), its latency, or its instructions at 4750 per us and
// SM. Measured over 12 shapes, the choice is within 10% of the best split of
// each, e.g. (us, R x ks) 6144 x 6144, 1 token: 1 x 8 8.5, 2 x 8 8.9, 4 x 4
// 12.7; 4096 x 16384, 1 token: 2 x 16 12.6, 1 x 8 20; 131072 x 4096, 8 tokens:
// 4 x 2 54, 4 x 1 59, 2 x 2 69; 16384 x 4096, 16 tokens: 2 x 4 18, 1 x 8 23.
// Four row tiles of 16 tokens do not fit the registers.
struct Q4Split {
    int R, ks;
};

Q4Split q4_split(const Q4Args &a, int nt)
{
    Q4Split best{1, 1};
    double least = -1;
    for (int r = a.pair ? 2 : 1; r <= (nt == 1 ? 4 : 2); r *= 2)
        for (int k = 1; k <= (r == 4 ? 4 : r == 2 ? 16 : 8) && k <= a.nsb; k *= 2) {
            const int per = a.pair ? r / 2 : r, w = std::max(4, k);
            const long groups = (a.tiles + per - 1) / per;
            const long ctas = (groups + w / k - 1) / (w / k) * ((a.T + 8 * nt - 1) / (8 * nt));
            const long fits = (r == 1 && nt == 1 ? 24 : 16) / w, on_sm = (ctas + 147) / 148;
            const double instr = nt == 1 ? 60 + 111 * r : 100 + 175 * r, turns = (a.nsb + k - 1) / k;
            auto round = [&](long n) {   // n CTAs on an SM
                return n ? turns * std::max(nt == 1 ? 0.9 : 1.2, n * w * instr / 4750) + 4 : 0.;
            };
            const double us = (on_sm / fits) * round(fits) + round(on_sm % fits);
            if (least < 0 || us < least)
                least = us, best = {r, k};
        }
    return best;
}

template <int G, bool BIAS>
cudaError_t pick(const Q4Args &a, cudaStream_t s)
{
    const int nt = a.T <= 8 ? 1 : 2;
    const Q4Split q = q4_split(a, nt);
    switch (q.R * 2 + nt) {
    case 3: return run<1, 1, G, BIAS>(a, q.ks, s);
    case 4: return run<1, 2, G, BIAS>(a, q.ks, s);
    case 5: return run<2, 1, G, BIAS>(a, q.ks, s);
    case 6: return run<2, 2, G, BIAS>(a, q.ks, s);
    default: return run<4, 1, G, BIAS>(a, q.ks, s);
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
    const long blocks = ((long)tiles * nsb + 3) / 4;   // 64 lanes a tile
    return launch_after(vq_q4_pack_kernel, dim3((unsigned)std::min(blocks, 148L * 64)), dim3(256), 0, s, codes, scales,
                        biases, rows, cols, group, tiles, nsb, words_out, scales_out, biases_out);
}

}  // namespace vq
