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
//  - the zero point leaves the sum through its start: -z * sum_k x[b, k] of the group, in
//    fp32.  Its magnitude is about that of the sum (codes lie in 0..15), so the difference
//    loses about one bit of fp32's 24.
// The group's sum times its scale is then added to the row's sum in fp32.
//
// What bounds it.  HBM for batches up to 16: 4.25 bits a weight with groups of 64.  The
// tensor pipe takes 8 cycles per 1024 weights and 8 batch rows (measured), HBM 21, so
// from 24 rows on the products bound it.  The integer pipe, the next one, takes 10 per 1024
// weights; unpacking to bf16 with a subtraction of the zero point took 23 and that kernel
// 61 us for 262144 x 1536 in groups of 64 and 8 rows.
#pragma once

#include <algorithm>

#include "lm_ops.h"

namespace mtp {

template <int GROUP> cudaError_t launch_q4_group(const Q4Params &p, cudaStream_t s);

namespace {

struct Q4Plan {
    int tiles;      // tiles of 16 rows in all
    int parts;      // warps that share a row's columns
    int chunk;      // columns of x in shared memory at a time, a multiple of kCols or >= K
};

constexpr int kTiles = 2;    // row tiles of a warp that share one read of x
constexpr int kCols = 256;   // columns of a step: 4 blocks of 64
constexpr int kSlots = 2;    // of a warp's ring
constexpr int kStage = kTiles * 2048;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// acc += s * d on a pair, with one instruction.
__device__ __forceinline__ void fma_pair(float &acc0, float &acc1, float s, float d0, float d1)
{
    asm("{\n .reg .b64 a, b, c;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %4};\n mov.b64 c, {%0, %1};\n"
        " fma.rn.f32x2 c, a, b, c;\n mov.b64 {%0, %1}, c;\n}\n"
        : "+f"(acc0), "+f"(acc1)
        : "f"(d0), "f"(d1), "f"(s));
}

__device__ __forceinline__ uint32_t half_pair(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// NT: batch rows / 8; GROUP: columns of a group; ZEROS: zero points; W: warps.
template <int NT, int GROUP, bool ZEROS, int W>
__global__ void __launch_bounds__(W * 32, 1) k_q4_matvec(Q4Params p, Q4Plan plan)
{
    constexpr int WORDS = GROUP / 32;      // words of a lane in a group
    constexpr int SG = kCols / GROUP;      // groups of a step
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float s_factor[NT * 8], s_inverse[NT * 8];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    const int b0 = blockIdx.y * NT * 8;
    uint8_t *ring = smem + warp * kSlots * kStage + lane * 16;
    const uint32_t ring_s = (uint32_t)__cvta_generic_to_shared(ring);
    uint4 *xs = (uint4 *)(smem + W * kSlots * kStage);                    // [word][NT][lane]
    const int chunk = min(plan.chunk, p.K);
    float *xw = (float *)(xs + chunk / 32 * NT * 32);                     // [word][NT * 8] sums of 32 columns
    const int blocks = p.blocks, all_steps = (p.K + kCols - 1) / kCols;

    // tiles of this CTA, then of this warp.  Its work is a list of rounds (kTiles tiles each),
    // each over all chunks of x; every warp of the CTA runs the same rounds and chunks.
    const int c_lo = (int)((long long)plan.tiles * blockIdx.x / gridDim.x);
    const int c_n = (int)((long long)plan.tiles * (blockIdx.x + 1) / gridDim.x) - c_lo;
    const int row_groups = W / plan.parts, rg = warp / plan.parts, part = warp % plan.parts;
    const int t_lo = c_lo + c_n * rg / row_groups, t_hi = c_lo + c_n * (rg + 1) / row_groups;
    const int rounds = ((c_n + row_groups - 1) / row_groups + kTiles - 1) / kTiles;
    const int chunk_steps = plan.chunk / kCols, chunks = (p.K + plan.chunk - 1) / plan.chunk;
    // steps [lo, hi) of chunk c that are this warp's
    auto share = [&](int c, int *lo, int *hi) {
        const int first = c * chunk_steps, n = min(chunk_steps, all_steps - first);
        *lo = first + n * part / plan.parts;
        *hi = first + n * (part + 1) / plan.parts;
    };

    // loads run ahead of the products through the same list, codes into the ring, scales
    // (and zero points) of rows g and g + 8 for the step's groups into registers
    uint32_t n_sc[kTiles][SG], n_zp[kTiles][SG / 2];
    int l_tile = t_lo, l_chunk = 0, l_k, l_hi;
    share(0, &l_k, &l_hi);
    auto load = [&](int slot) {
        while (l_tile < t_hi && l_k >= l_hi) {   // the next chunk or round with steps of this warp
            if (++l_chunk == chunks) l_chunk = 0, l_tile += kTiles;
            share(l_chunk, &l_k, &l_hi);
        }
        if (l_tile >= t_hi) return;
        const int n = min(blocks - l_k * 4, 4);
#pragma unroll
        for (int r = 0; r < kTiles; ++r) {
            if (l_tile + r >= t_hi) break;
            const uint8_t *src = p.codes + ((long long)(l_tile + r) * blocks + l_k * 4) * 512 + lane * 16;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < n) cp_async16(ring_s + slot * kStage + r * 2048 + i * 512, src + i * 512);
            const long long at = ((long long)(l_tile + r) * all_steps + l_k) * 8 + g;
            if (SG == 2) {
                const uint2 v = __ldg((const uint2 *)p.scales + at);
                n_sc[r][0] = v.x, n_sc[r][1] = v.y;
            } else {
#pragma unroll
                for (int j = 0; j < SG; j += 4) {
                    const uint4 v = __ldg((const uint4 *)p.scales + at * (SG / 4) + j / 4);
                    n_sc[r][j % SG] = v.x, n_sc[r][(j + 1) % SG] = v.y, n_sc[r][(j + 2) % SG] = v.z, n_sc[r][(j + 3) % SG] = v.w;
                }
            }
            if (ZEROS)
#pragma unroll
                for (int j = 0; j < SG / 2; ++j) n_zp[r][j] = __ldg((const uint32_t *)p.zeros + at * (SG / 2) + j);
        }
        ++l_k;
    };
    load(0);
    cp_async_commit();

    // each batch row's power of two
    for (int n = warp; n < NT * 8; n += W) {
        uint32_t top = 0;
        if (b0 + n < p.B)
            for (int k = lane * 8; k < p.K; k += 256) {
                const uint4 v = ld_ro16(p.x + (b0 + n) * p.ld_x + k);
                top = __vmaxu2(top, __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu), __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu)));
            }
        top = max(top >> 16, top & 0xffffu);
        top = __reduce_max_sync(~0u, top);
        if (lane == 0) {
            const uint32_t e = top == 0 ? 127u : min(254u, 268u - (top >> 7));   // exponent field of the factor
            s_factor[n] = __uint_as_float(e << 23);
            // a row that holds a NaN or an infinity gives NaN
            s_inverse[n] = top >= 0x7f80u ? __uint_as_float(0x7fffffffu) : __uint_as_float(e == 254u ? 0x00400000u : (254u - e) << 23);
        }
    }
    __syncthreads();

    float acc[kTiles][NT][4];
#pragma unroll
    for (int r = 0; r < kTiles; ++r)
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[r][n][0] = acc[r][n][1] = acc[r][n][2] = acc[r][n][3] = 0.f;

    auto store = [&](float y, int m, int n) {
        if (m >= p.M || b0 + n >= p.B) return;
        y = y * 16777216.f * s_inverse[n];
        if (p.softcap > 0.f) y = p.softcap * tanhf(y / p.softcap);
        if (p.bf16_out)
            ((uint16_t *)p.out)[(b0 + n) * p.ld_out + m] = bf16_bits(y);
        else
            ((float *)p.out)[(b0 + n) * p.ld_out + m] = y;
    };

    int slot = 0;
    for (int round = 0; round < rounds; ++round) {
        const int tile = t_lo + round * kTiles, live = min(t_hi - tile, kTiles);
        for (int c = 0; c < chunks; ++c) {
            if (chunks > 1 || round == 0) {
                // x of the chunk in the operand's order; its sums by 32 columns, then by group
                const int k0 = c * plan.chunk, words = min(chunk, p.K - k0) / 32;
                if (chunks > 1) __syncthreads();
                for (int i = threadIdx.x; i < words * NT * 32; i += W * 32) {
                    const int n = i / 32 % NT * 8 + lane / 4;
                    float v[8] = {};
                    if (b0 + n < p.B) {
                        const uint4 u = ld_ro16(p.x + (b0 + n) * p.ld_x + k0 + i / (32 * NT) * 32 + t * 8);
                        const float f = s_factor[n];
                        v[0] = bf_lo(u.x) * f, v[1] = bf_hi(u.x) * f, v[2] = bf_lo(u.y) * f, v[3] = bf_hi(u.y) * f;
                        v[4] = bf_lo(u.z) * f, v[5] = bf_hi(u.z) * f, v[6] = bf_lo(u.w) * f, v[7] = bf_hi(u.w) * f;
                    }
                    xs[i] = make_uint4(half_pair(v[0], v[4]), half_pair(v[1] * 0.0625f, v[5] * 0.0625f), half_pair(v[2], v[6]),
                                       half_pair(v[3] * 0.0625f, v[7] * 0.0625f));
                    float sum = ((v[0] + v[4]) + (v[1] + v[5])) + ((v[2] + v[6]) + (v[3] + v[7]));
                    sum += __shfl_xor_sync(~0u, sum, 1);
                    sum += __shfl_xor_sync(~0u, sum, 2);
                    if (t == 0) xw[i / 32 * 8 + g] = sum * ((ZEROS ? -1.f : -8.f) / 16777216.f);
                }
                __syncthreads();
                if (WORDS > 1) {   // the first word's place takes the group's sum
                    for (int i = threadIdx.x; i < words / WORDS * NT * 8; i += W * 32) {
                        float *at = xw + i / (NT * 8) * (WORDS * NT * 8) + i % (NT * 8);
                        float sum = at[0];
#pragma unroll
                        for (int w = 1; w < WORDS; ++w) sum += at[w * NT * 8];
                        at[0] = sum;
                    }
                    __syncthreads();
                }
            }
            int k, k_hi;
            share(c, &k, &k_hi);
            if (live <= 0) k = k_hi;
            for (; k < k_hi; ++k) {
                cp_async_wait<0>();   // a lane reads only what it copied itself
                uint32_t sc[kTiles][SG], zp[kTiles][SG / 2];
#pragma unroll
                for (int r = 0; r < kTiles; ++r) {
#pragma unroll
                    for (int j = 0; j < SG; ++j) sc[r][j] = n_sc[r][j];
#pragma unroll
                    for (int j = 0; j < SG / 2; ++j) zp[r][j] = n_zp[r][j];
                }
                load(slot ^ 1);
                cp_async_commit();
                const uint8_t *codes = ring + slot * kStage;
                slot ^= 1;
                const int word0 = k * (kCols / 32) - c * (plan.chunk / 32);
#pragma unroll
                for (int j = 0; j < SG; ++j) {
                    if (k * SG + j >= p.G) break;
                    uint4 x[WORDS][NT];
                    float2 sum[NT];
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        sum[n] = *(const float2 *)(xw + ((word0 + j * WORDS) * NT + n) * 8 + t * 2);
#pragma unroll
                        for (int w = 0; w < WORDS; ++w) x[w][n] = xs[((word0 + j * WORDS + w) * NT + n) * 32 + lane];
                    }
#pragma unroll
                    for (int r = 0; r < kTiles; ++r) {
                        if (r >= live) break;
                        const float s_lo = bf_lo(sc[r][j]), s_hi = bf_hi(sc[r][j]);
                        float d[NT][4];
                        if (ZEROS) {
                            const uint32_t z = zp[r][j / 2] >> (j % 2 * 16);
                            const float z_lo = (float)(z & 15u), z_hi = (float)(z >> 8 & 15u);
#pragma unroll
                            for (int n = 0; n < NT; ++n)
                                d[n][0] = z_lo * sum[n].x, d[n][1] = z_lo * sum[n].y, d[n][2] = z_hi * sum[n].x, d[n][3] = z_hi * sum[n].y;
                        } else {
#pragma unroll
                            for (int n = 0; n < NT; ++n) d[n][0] = d[n][2] = sum[n].x, d[n][1] = d[n][3] = sum[n].y;
                        }
#pragma unroll
                        for (int w = 0; w < WORDS; ++w) {
                            // words of rows g and g + 8: a block holds two words of each
                            const uint4 block = *(const uint4 *)(codes + r * 2048 + (j * WORDS + w) / 2 * 512);
                            const uint2 q = (j * WORDS + w) % 2 ? make_uint2(block.z, block.w) : make_uint2(block.x, block.y);
                            const uint32_t qx8 = q.x >> 8, qy8 = q.y >> 8;
#pragma unroll
                            for (int n = 0; n < NT; ++n)
                                mma_f16(d[n], q.x & 0x000f000fu, q.y & 0x000f000fu, q.x & 0x00f000f0u, q.y & 0x00f000f0u, x[w][n].x, x[w][n].y);
#pragma unroll
                            for (int n = 0; n < NT; ++n)
                                mma_f16(d[n], qx8 & 0x000f000fu, qy8 & 0x000f000fu, qx8 & 0x00f000f0u, qy8 & 0x00f000f0u, x[w][n].z, x[w][n].w);
                        }
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            fma_pair(acc[r][n][0], acc[r][n][1], s_lo, d[n][0], d[n][1]);
                            fma_pair(acc[r][n][2], acc[r][n][3], s_hi, d[n][2], d[n][3]);
                        }
                    }
                }
            }
        }
        if (plan.parts == 1) {
#pragma unroll
            for (int r = 0; r < kTiles; ++r) {
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
    if (plan.parts == 1) return;

    // the parts of each row are added in their order; a row group has one tile here.  The
    // sums take the rings' place.
    cp_async_wait<0>();
    __syncthreads();
    float4 *sums = (float4 *)smem;   // [warp][NT][lane]
    const int tiles = t_hi - t_lo;
#pragma unroll
    for (int n = 0; n < NT; ++n) sums[(warp * NT + n) * 32 + lane] = make_float4(acc[0][n][0], acc[0][n][1], acc[0][n][2], acc[0][n][3]);
    __syncthreads();
    for (int n = part; n < tiles * NT; n += plan.parts) {
        float y[4] = {};
        for (int q = 0; q < plan.parts; ++q) {
            const float4 v = sums[((rg * plan.parts + q) * NT + n) * 32 + lane];
            y[0] += v.x, y[1] += v.y, y[2] += v.z, y[3] += v.w;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) store(y[e], t_lo * 16 + g + e / 2 * 8, n * 8 + t * 2 + e % 2);
    }
}

template <int NT, int GROUP, bool ZEROS> cudaError_t launch_q4(const Q4Params &p, cudaStream_t s)
{
    // 16 warps leave 128 registers a thread, which holds the sums of 16 batch rows
    constexpr int W = NT <= 2 ? 16 : 12;
    constexpr size_t most = 227 * 1024 - NT * 64, ring = W * kSlots * kStage;
    static_assert(ring >= W * NT * 512, "the sums fit the rings");
    Q4Plan plan{};
    plan.tiles = p.M / 16 + (p.M % 16 != 0);
    const int sms = sm_count(), per_cta = (plan.tiles + sms - 1) / sms;
    // few tiles per CTA: its warps share the rows' columns instead, as long as each then has
    // one tile at most
    plan.parts = 1;
    while (W % (plan.parts * 2) == 0 && per_cta * plan.parts * 2 <= W && plan.parts < 16) plan.parts *= 2;
    // all of x in shared memory, or in chunks that every CTA goes through for each round
    const size_t per_word = NT * (512 + 32);
    plan.chunk = (p.K + kCols - 1) / kCols * kCols;
    if (p.K / 32 * per_word > most - ring) plan.chunk = (int)((most - ring) / per_word) * 32 / kCols * kCols;
    const size_t smem = ring + (size_t)std::min(plan.chunk, p.K) / 32 * per_word;
    cudaError_t e = allow_smem((const void *)k_q4_matvec<NT, GROUP, ZEROS, W>, smem);
    if (e != cudaSuccess) return e;
    const dim3 grid(std::min(sms, plan.tiles), (p.B + NT * 8 - 1) / (NT * 8));
    k_q4_matvec<NT, GROUP, ZEROS, W><<<grid, W * 32, smem, s>>>(p, plan);
    return cudaGetLastError();
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
