// The 4-bit product kernel; q4_g32.cu, q4_g64.cu and q4_g128.cu instantiate it, one group
// size each, so that they compile beside one another.
//
// Mathematics.  y[b, m] = sum over groups of scale * sum_k (code - z) x[b, k].  The inner
// sums are tensor-core products (mma m16n8k16, fp16 in, fp32 sums) of 16 weight rows by 8
// batch rows, so batches of 1 to 8 cost the same:
//  - a code c, masked in place, is already an fp16 number: bits 0-3 are the subnormal
//    c * 2^-24, bits 4-7 are c * 2^-20.  Eight codes become four operand registers with four
//    ands and one shift, and no arithmetic;
//  - x, which has 8 significant bits, is fp16 too, times the power of two that brings its
//    row's largest value to [2^14, 2^15): exact down to 2^-29 of that value (columns that
//    meet bits 4-7 are also divided by 16: 2^-25), with an absolute error below 2^-39
//    (2^-35) of it beneath;
//  - the zero point leaves the sum as -z * sum_k x[b, k] of the group, in fp32.  Its
//    magnitude is about that of the sum (codes lie in 0..15), so the difference loses about
//    one bit of fp32's 24.
// Both, times the group's scale, are added to the row's sum in fp32.  (262144 x 1536 with 8
// rows ends 4.6e-7 of the outputs' size off in the mean, products in fp32 alone 1.3e-7.)
//
// What bounds it.  HBM up to 8 batch rows: 4.25 bits a weight with groups of 64; 262144 x
// 1536 with 8 rows takes 39.1 us behind another launch, 5.7 TB/s, the same loads and stores
// without the products about 2 us less.  Above, the products and what feeds them: 50 us at
// 16 rows, 83 at 32; 50021 x 2592 with 23 rows takes 38 us with the tensor pipe 35 % busy,
// one round of tiles a warp and x in two chunks.  Unpacking to bf16 with a subtraction of the
// zero point took 23 integer instructions for every 8 here (61 us at 8 rows).
#pragma once

#include <algorithm>

#include "lm_ops.h"

namespace mtp {

template <int GROUP> cudaError_t launch_q4_group(const Q4Params &p, cudaStream_t s);

namespace {

struct Q4Plan {
    int tiles;      // tiles of 16 rows in all
    int chunk;      // columns of x in shared memory at a time, a multiple of kCols
};

constexpr int kCols = 256;   // columns of a step: 4 blocks of 64

// Bytes of a tile's scales and zero points in a step, and of a ring slot.
template <int GROUP> constexpr int kScales = 8 * (kCols / GROUP) * 4;
template <int GROUP> constexpr int kZeros = kScales<GROUP> / 2;
template <int GROUP, bool ZEROS, int TILES> constexpr int kStage = TILES * (2048 + kScales<GROUP> + (ZEROS ? kZeros<GROUP> : 0));

// Byte b of v (below 16) as a float: or-ed into 2^23, whose last place is 1.
template <int B> __device__ __forceinline__ float byte_value(uint32_t v)
{
    return __uint_as_float(__byte_perm(v, 0x4b000000u, 0x7650 + B)) - 8388608.f;
}

// NT: batch rows / 8; GROUP: columns of a group; ZEROS: zero points; W: warps; S: slots of a
// warp's ring; TILES: row tiles of a warp that share one read of x.
template <int NT, int GROUP, bool ZEROS, int W, int S, int TILES>
__global__ void __launch_bounds__(W * 32, 1) k_q4_matvec(Q4Params p, Q4Plan plan)
{
    constexpr int WORDS = GROUP / 32;      // words of a lane in a group
    constexpr int SG = kCols / GROUP;      // groups of a step
    constexpr int STAGE = kStage<GROUP, ZEROS, TILES>, SCALES = kScales<GROUP>, ZPS = kZeros<GROUP>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float s_factor[NT * 8];
    __shared__ float2 s_inverse[NT * 8];   // its inverse times 2^24, as two factors that keep sums within fp32's range
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    const int b0 = blockIdx.y * NT * 8;
    const uint8_t *ring = smem + warp * S * STAGE;
    const uint32_t ring_s = (uint32_t)__cvta_generic_to_shared(ring) + lane * 16;
    uint4 *xs = (uint4 *)(smem + W * S * STAGE);                          // [word][NT][lane, see below]
    float *xw = (float *)(xs + plan.chunk / 32 * NT * 32);                   // [word][NT * 8] sums of 32 columns
    const int blocks = p.blocks, all_steps = (p.K + kCols - 1) / kCols;

    // Tiles of this CTA; x in chunks of columns.  With TILES = 2 a warp's work is a list of
    // rounds (two tiles each), each over all chunks; every warp of the CTA runs the same rounds
    // and chunks.  With TILES = 1 the CTA has at most a tile for each warp.  Up to 16 batch rows
    // (TWO) each chunk's steps of all tiles, one tile after the other, are shared evenly: a warp
    // has steps of tile t0 (of the CTA's) and perhaps of the next (21488 x 3392, 9 tiles a CTA, 5
    // rows: 10.5 us, 11.8 with a power of two of warps for each tile).  Above, where a second tile's
    // sums would not stay in registers (2048 x 4096, 32 rows: 16.5 us, without 14.8), `parts`
    // warps share each tile's steps.
    constexpr bool SPREAD = TILES == 1, TWO = SPREAD && NT <= 2;
    const int c_lo = (int)((long long)plan.tiles * blockIdx.x / gridDim.x);
    const int c_n = (int)((long long)plan.tiles * (blockIdx.x + 1) / gridDim.x) - c_lo;
    int parts = 1;
    if (SPREAD && !TWO)
        while (c_n * parts * 2 <= W) parts *= 2;
    const int t0 = SPREAD && !TWO ? warp / parts : c_n * warp / W;
    const int t_lo = c_lo + t0, t_hi = c_lo + c_n * (warp + 1) / W;   // the latter with TILES = 2
    const int rounds = SPREAD ? 1 : ((c_n + W - 1) / W + TILES - 1) / TILES;
    const int chunk_steps = plan.chunk / kCols, chunks = (p.K + plan.chunk - 1) / plan.chunk;
    // this warp's steps of chunk c: from step *k of tile t0 on, *n of them; the chunk ends at *end
    auto share = [&](int c, int *k, int *n, int *end) {
        const int first = c * chunk_steps, steps = min(chunk_steps, all_steps - first);
        int lo = 0, hi = steps;
        if (TWO)
            lo = c_n * steps * warp / W - t0 * steps, hi = c_n * steps * (warp + 1) / W - t0 * steps;
        else if (SPREAD)
            lo = steps * (warp % parts) / parts, hi = t0 < c_n ? steps * (warp % parts + 1) / parts : lo;
        *k = first + lo, *n = hi - lo, *end = first + steps;
    };

    // loads run ahead of the products through the same list
    int l_tile = t_lo, l_chunk = 0, l_k, l_n, l_end;
    share(0, &l_k, &l_n, &l_end);
    if (!SPREAD && t_lo >= t_hi) l_n = 0, l_chunk = chunks;
    auto load = [&](int slot) {
        while (l_n == 0) {   // the next chunk or round with steps of this warp
            if (l_chunk == chunks) return;
            if (++l_chunk == chunks) {
                if (SPREAD || (l_tile += TILES) >= t_hi) return;
                l_chunk = 0;
            }
            if (TWO) l_tile = t_lo;
            share(l_chunk, &l_k, &l_n, &l_end);
        }
        const int n = min(blocks - l_k * 4, 4);
        const uint32_t dst = ring_s + slot * STAGE;
#pragma unroll
        for (int r = 0; r < TILES; ++r) {
            if (!SPREAD && l_tile + r >= t_hi) break;
            const uint8_t *src = p.codes + ((long long)(l_tile + r) * blocks + l_k * 4) * 512 + lane * 16;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < n) cp_async16(dst + r * 2048 + i * 512, src + i * 512);
            const long long at = (long long)(l_tile + r) * all_steps + l_k;
            if (lane < SCALES / 16) cp_async16(dst + TILES * 2048 + r * SCALES, p.scales + at * SCALES + lane * 16);
            if (ZEROS && lane < ZPS / 16)
                cp_async16(dst + TILES * (2048 + SCALES) + r * ZPS, p.zeros + at * ZPS + lane * 16);
        }
        --l_n;
        if (++l_k == l_end && TWO) l_k = l_chunk * chunk_steps, ++l_tile;
    };
    let_next_start();
    wait_for_previous();
#pragma unroll
    for (int i = 0; i < S - 1; ++i) {
        load(i);
        cp_async_commit();
    }

    // A warp takes batch rows warp, warp + W, ..., eight loads of a lane in flight (2048
    // columns).  x of a chunk is staged in the operand's order: the 16 bytes of lane (g, t) lie
    // at lane (g ^ (word % 8), t), which spreads a row's words over the banks.  Beside it the
    // sums of a group's columns, in the place of its first word.
    auto load_x = [&](uint4 (&u)[8], int n, int k0, int left) {   // columns k0 + lane * 8 + i * 256
        const uint16_t *x = p.x + (b0 + n) * p.ld_x + k0;
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = i * 256 + lane * 8 < left ? ld_ro16(x + i * 256 + lane * 8) : make_uint4(0, 0, 0, 0);
    };
    auto put_x = [&](const uint4 (&u)[8], int n, int w0, int words, float f) {   // words w0 + i * 8 + g
        uint4 *dst = xs + n / 8 * 32 + ((n % 8 ^ g) * 4 + t);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int word = w0 + i * 8 + g;
            if (w0 + i * 8 >= words) break;   // words is a multiple of 8
            const float v0 = bf_lo(u[i].x) * f, v1 = bf_hi(u[i].x) * f, v2 = bf_lo(u[i].y) * f, v3 = bf_hi(u[i].y) * f;
            const float v4 = bf_lo(u[i].z) * f, v5 = bf_hi(u[i].z) * f, v6 = bf_lo(u[i].w) * f, v7 = bf_hi(u[i].w) * f;
            dst[word * NT * 32] = make_uint4(half_pair(v0, v4), half_pair(v1 * 0.0625f, v5 * 0.0625f), half_pair(v2, v6),
                                             half_pair(v3 * 0.0625f, v7 * 0.0625f));
            float sum = ((v0 + v4) + (v1 + v5)) + ((v2 + v6) + (v3 + v7));
#pragma unroll
            for (int o = 1; o < 4 * WORDS; o *= 2) sum += __shfl_xor_sync(~0u, sum, o);
            if (lane % (4 * WORDS) == 0) xw[word * NT * 8 + n] = sum * ((ZEROS ? -1.f : -8.f) / 16777216.f);
        }
    };
    auto words_of = [&](int c) { return min(plan.chunk, all_steps * kCols - c * plan.chunk) / 32; };
    auto stage_x = [&](int c, int n, int w0) {   // the row's words of a chunk from w0 on
        for (; w0 < words_of(c); w0 += 64) {
            uint4 u[8];
            load_x(u, n, c * plan.chunk + w0 * 32, b0 + n < p.B ? p.K - c * plan.chunk - w0 * 32 : 0);
            put_x(u, n, w0, words_of(c), s_factor[n]);
        }
    };
    // each row's largest value and its power of two, and the first chunk
    for (int n = warp; n < NT * 8; n += W) {
        const int left = b0 + n < p.B ? p.K : 0;
        uint4 u[8];
        load_x(u, n, 0, left);
        uint32_t top = 0;
        auto largest = [&](const uint4 (&v)[8]) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                top = __vmaxu2(top, __vmaxu2(__vmaxu2(v[i].x & 0x7fff7fffu, v[i].y & 0x7fff7fffu),
                                             __vmaxu2(v[i].z & 0x7fff7fffu, v[i].w & 0x7fff7fffu)));
        };
        largest(u);
        for (int k = 2048; k < left; k += 2048) {
            uint4 v[8];
            load_x(v, n, k, left - k);
            largest(v);
        }
        top = __reduce_max_sync(~0u, max(top >> 16, top & 0xffffu));
        const uint32_t e = fp16_factor_field(top);
        const float f = __uint_as_float(e << 23);
        if (lane == 0) {
            s_factor[n] = f;
            // a row that holds a NaN or an infinity gives NaN
            const float inverse = top >= 0x7f80u ? __uint_as_float(0x7fffffffu) : fp16_factor_inverse(e);
            s_inverse[n] = inverse < 1.f ? make_float2(inverse * 16777216.f, 1.f) : make_float2(16777216.f, inverse);
        }
        __syncwarp();
        put_x(u, n, 0, words_of(0), f);
        stage_x(0, n, 64);
    }
    __syncthreads();

    constexpr int ACCS = TILES == 2 || TWO ? 2 : 1;
    float acc[ACCS][NT][4];   // of the tiles at hand: both, or the one that is computed and the other
#pragma unroll
    for (int r = 0; r < ACCS; ++r)
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[r][n][0] = acc[r][n][1] = acc[r][n][2] = acc[r][n][3] = 0.f;

    auto store = [&](float y, int m, int n) {
        if (m >= p.M || b0 + n >= p.B) return;
        y = y * s_inverse[n].x * s_inverse[n].y;
        if (p.softcap > 0.f) y = p.softcap * tanhf(y / p.softcap);
        if (p.bf16_out)
            ((uint16_t *)p.out)[(b0 + n) * p.ld_out + m] = bf16_bits(y);
        else
            ((float *)p.out)[(b0 + n) * p.ld_out + m] = y;
    };

    int slot = 0;
    for (int round = 0; round < rounds; ++round) {
        const int tile = t_lo + round * TILES, live = min(t_hi - tile, TILES);
        for (int c = 0; c < chunks; ++c) {
            if (round + c > 0 && chunks > 1) {
                __syncthreads();
                for (int n = warp; n < NT * 8; n += W) stage_x(c, n, 0);
                __syncthreads();
            }
            int k, n_steps, end;
            share(c, &k, &n_steps, &end);
            if (!SPREAD && live <= 0) n_steps = 0;
#pragma unroll 1
            for (int part = 0; part < (TWO ? 2 : 1); ++part) {
                const int k_hi = TWO ? min(end, k + n_steps) : k + n_steps;
                n_steps -= k_hi - k;
                for (; k < k_hi; ++k) {
                    cp_async_wait<S - 2>();
                    __syncwarp();   // the step is there for every lane, and the slot of the one before is free
                    load(slot == 0 ? S - 1 : slot - 1);
                    cp_async_commit();
                    const uint8_t *codes = ring + slot * STAGE + lane * 16;
                    const uint8_t *scales = ring + slot * STAGE + TILES * 2048 + g * SG * 4;
                    const uint8_t *zeros = ring + slot * STAGE + TILES * (2048 + SCALES) + g * SG * 2;
                    slot = slot == S - 1 ? 0 : slot + 1;
                    const int word0 = k * (kCols / 32) - c * (plan.chunk / 32);
                    const uint4 *xk = xs + word0 * NT * 32;
                    const float *sk = xw + word0 * NT * 8 + t * 2;
                    // No branch in here: a tile that is not there and columns beyond K are computed
                    // too, the one on whatever the slot holds (and not stored), the others on
                    // zeros of x with scales of zero.
#pragma unroll
                    for (int j = 0; j < SG; ++j) {
                        float d[TILES][NT][4];
#pragma unroll
                        for (int w = j * WORDS; w < (j + 1) * WORDS; ++w) {
                            uint4 x[NT];
#pragma unroll
                            for (int n = 0; n < NT; ++n) x[n] = xk[(w * NT + n) * 32 + ((g ^ w) * 4 + t)];
#pragma unroll
                            for (int r = 0; r < TILES; ++r) {
                                // words of rows g and g + 8: a block holds two words of each
                                const uint4 block = *(const uint4 *)(codes + r * 2048 + w / 2 * 512);
                                const uint32_t lo = w % 2 ? block.z : block.x, hi = w % 2 ? block.w : block.y;
                                const uint32_t lo8 = lo >> 8, hi8 = hi >> 8;
#pragma unroll
                                for (int n = 0; n < NT; ++n) {
                                    if (w == j * WORDS)
                                        mma_f16_first(d[r][n], lo & 0x000f000fu, hi & 0x000f000fu, lo & 0x00f000f0u, hi & 0x00f000f0u, x[n].x, x[n].y);
                                    else
                                        mma_f16(d[r][n], lo & 0x000f000fu, hi & 0x000f000fu, lo & 0x00f000f0u, hi & 0x00f000f0u, x[n].x, x[n].y);
                                }
#pragma unroll
                                for (int n = 0; n < NT; ++n)
                                    mma_f16(d[r][n], lo8 & 0x000f000fu, hi8 & 0x000f000fu, lo8 & 0x00f000f0u, hi8 & 0x00f000f0u, x[n].z, x[n].w);
                            }
                        }
                        float2 sum[NT];
#pragma unroll
                        for (int n = 0; n < NT; ++n) sum[n] = *(const float2 *)(sk + (j * WORDS * NT + n) * 8);
#pragma unroll
                        for (int r = 0; r < TILES; ++r) {
                            const uint32_t s2 = *(const uint32_t *)(scales + r * SCALES + j * 4);
                            const float s_lo = bf_lo(s2), s_hi = bf_hi(s2);
                            float z_lo = s_lo, z_hi = s_hi;   // 8 is in the sums of x
                            if (ZEROS) {
                                const uint32_t z = *(const uint16_t *)(zeros + r * ZPS + j * 2);
                                z_lo *= byte_value<0>(z), z_hi *= byte_value<1>(z);
                            }
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                fma_pair(acc[r][n][0], acc[r][n][1], s_lo, d[r][n][0], d[r][n][1]);
                                fma_pair(acc[r][n][2], acc[r][n][3], s_hi, d[r][n][2], d[r][n][3]);
                                fma_pair(acc[r][n][0], acc[r][n][1], z_lo, sum[n].x, sum[n].y);
                                fma_pair(acc[r][n][2], acc[r][n][3], z_hi, sum[n].x, sum[n].y);
                            }
                        }
                    }
                }
                if (TWO) {   // the rest is of the next tile
                    k = c * chunk_steps;
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float other = acc[0][n][e];
                            acc[0][n][e] = acc[ACCS - 1][n][e], acc[ACCS - 1][n][e] = other;
                        }
                }
            }
        }
        if (!SPREAD) {
#pragma unroll
            for (int r = 0; r < TILES; ++r) {
                if (r >= live) break;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        store(acc[r][n][e], (tile + r) * 16 + g + e / 2 * 8, n * 8 + t * 2 + e % 2);
                        acc[r][n][e] = 0.f;
                    }
            }
        }
    }
    if (!SPREAD) return;

    // each tile's sums, added in the order of the warps; they take the rings' place
    cp_async_wait<0>();
    __syncthreads();
    float4 *sums = (float4 *)smem;   // [warp][its tiles][NT][lane]
#pragma unroll
    for (int r = 0; r < ACCS; ++r)
#pragma unroll
        for (int n = 0; n < NT; ++n)
            sums[((warp * ACCS + r) * NT + n) * 32 + lane] = make_float4(acc[r][n][0], acc[r][n][1], acc[r][n][2], acc[r][n][3]);
    __syncthreads();
    for (int i = warp; i < c_n * NT; i += W) {
        const int tile = i / NT, n = i - tile * NT;
        const int w_lo = TWO ? tile * W / c_n : tile * parts, w_hi = TWO ? ((tile + 1) * W - 1) / c_n : w_lo + parts - 1;
        float y[4] = {};
#pragma unroll 4
        for (int w = w_lo; w <= w_hi; ++w) {
            const int r = TWO ? tile - c_n * w / W : 0;   // 0 or 1
            const float4 v = sums[((w * ACCS + r) * NT + n) * 32 + lane];
            y[0] += v.x, y[1] += v.y, y[2] += v.z, y[3] += v.w;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) store(y[e], (c_lo + tile) * 16 + g + e / 2 * 8, n * 8 + t * 2 + e % 2);
    }
}

// Columns of x that fit beside the rings of W warps of S slots.
template <int NT, int GROUP, bool ZEROS, int W, int S, int TILES> constexpr int q4_room()
{
    constexpr long long left = 227 * 1024 - NT * 96 - (long long)W * S * kStage<GROUP, ZEROS, TILES>;
    static_assert(left >= NT * 544 * kCols / 32, "a step of x fits");
    static_assert(TILES == 2 || S * kStage<GROUP, ZEROS, TILES> >= 2 * NT * 512, "the warps' sums fit the rings");
    return (int)(left / (NT * 544) * 32 / kCols * kCols);   // 512 + 32 bytes per 32 columns and 8 rows
}

template <int NT, int GROUP, bool ZEROS, int W, int S, int TILES> cudaError_t launch_q4_warps(const Q4Params &p, Q4Plan plan, cudaStream_t s)
{
    // all of x in shared memory, or in chunks that every CTA goes through for each round
    plan.chunk = std::min((p.K + kCols - 1) / kCols * kCols, q4_room<NT, GROUP, ZEROS, W, S, TILES>());
    const size_t smem = (size_t)W * S * kStage<GROUP, ZEROS, TILES> + (size_t)plan.chunk / 32 * NT * 544;
    cudaError_t e = allow_smem((const void *)k_q4_matvec<NT, GROUP, ZEROS, W, S, TILES>, smem);
    if (e != cudaSuccess) return e;
    const dim3 grid(std::min(sm_count(), plan.tiles), (p.B + NT * 8 - 1) / (NT * 8));
    return launch_dependent(k_q4_matvec<NT, GROUP, ZEROS, W, S, TILES>, grid, dim3(W * 32), smem, s, p, plan);
}

// 12 warps of two tiles where a CTA has more than 16 tiles, else 16 of one, which compute no
// tile that is not there (8192 x 4096, 32 rows: 21.4 us, with 8 warps of two 39.4; 16384 x
// 4096, one row: 9.7 and 15.0; 38000 x 2048, 8 rows, 16 tiles a CTA: 9.8, with 12 warps of two
// 11.1).  262144 x 1536, 8 rows: 12 warps 39.2, 16 warps of two 41.2 us; 50021 x 2592, 23 rows:
// 37.8 with 12, 55.9 with 8, 49.0 with 16.  Three slots if x fits beside them (262144 x 1536, 8
// rows: 40.8 with two; at 16 rows two would be ahead, 48.8 against 50.0).  With x in chunks 8
// warps are ahead up to 8 batch rows (65536 x 8192: 64.8 against 85.8 us), 12 above (90000 x
// 4096, 32 rows: 104.8 against 122.6).
template <int NT, int GROUP, bool ZEROS> cudaError_t launch_q4(const Q4Params &p, cudaStream_t s)
{
    Q4Plan plan{};
    plan.tiles = p.M / 16 + (p.M % 16 != 0);
    const int sms = sm_count(), per_cta = (plan.tiles + sms - 1) / sms;
    if (per_cta > 16) {
        if (p.K <= q4_room<NT, GROUP, ZEROS, 12, 3, 2>()) return launch_q4_warps<NT, GROUP, ZEROS, 12, 3, 2>(p, plan, s);
        if (NT > 1 || p.K <= q4_room<NT, GROUP, ZEROS, 12, 2, 2>())
            return launch_q4_warps<NT, GROUP, ZEROS, 12, 2, 2>(p, plan, s);
        if constexpr (NT == 1) return launch_q4_warps<NT, GROUP, ZEROS, 8, 3, 2>(p, plan, s);
    }
    return launch_q4_warps<NT, GROUP, ZEROS, 16, 3, 1>(p, plan, s);
}

template <int NT, int GROUP> cudaError_t launch_q4_zeros(const Q4Params &p, cudaStream_t s)
{
    return p.zeros ? launch_q4<NT, GROUP, true>(p, s) : launch_q4<NT, GROUP, false>(p, s);
}

}  // namespace

template <int GROUP> cudaError_t launch_q4_group(const Q4Params &p, cudaStream_t s)
{
    // the batch in equal slabs of at most 32 rows
    const int eights = (p.B + 7) / 8, slabs = (eights + 3) / 4, nt = (eights + slabs - 1) / slabs;
    return nt == 1   ? launch_q4_zeros<1, GROUP>(p, s)
           : nt == 2 ? launch_q4_zeros<2, GROUP>(p, s)
           : nt == 3 ? launch_q4_zeros<3, GROUP>(p, s)
                     : launch_q4_zeros<4, GROUP>(p, s);
}

}  // namespace mtp
