// The 4-bit product kernel; q4_g32.cu, q4_g64.cu and q4_g128.cu instantiate it, one group
// size each, so that they compile beside one another.
#pragma once

#include <algorithm>

#include "lm_ops.h"

namespace mtp {

struct Q4Plan {
    int tiles;        // tiles of 16 rows in all
    int parts;        // warps that share a row's columns
    int x_bytes;      // shared memory of x (0: read from global memory)
};

template <int GROUP> cudaError_t launch_q4_group(const Q4Params &p, cudaStream_t s);

namespace {

// k_q4_matvec.  The sums are tensor-core products (mma m16n8k16, bf16 in, fp32 sums): 16
// weight rows by 8 batch rows, so batches of 1 to 8 cost the same.  A code enters as the
// exact bf16 integer code - z, so one group's products are exact in fp32; the group's sum
// is then multiplied by its scale in fp32 and added to the row's sum.
//
// A warp owns up to kTiles tiles of 16 rows and streams their codes in steps of kCols
// columns through a ring of its own in shared memory (16-byte cp.async; no barrier is
// shared between warps).  ldmatrix hands lane (g, t) the four bytes t of 16 bytes of rows
// g and g + 8: 8 columns, which a mask and an or turn into four pairs of bf16 128 + code
// (pair i holds columns i and i + 4), and a subtraction of 128 + z into the operand.  x is
// staged once per CTA in the order of that operand, 16 bytes per lane.
constexpr int kTiles = 4;                   // row tiles of a warp that share one read of x
constexpr int kCols = 128;                  // columns of a step
constexpr int kRows = 16 * kTiles;
constexpr int kCodeBytes = kRows * kCols / 2;
constexpr int kScaleBytes = kRows * 16;     // an aligned window of 16 bytes per row
constexpr int kZeroBytes = kRows * 8;       // an aligned window of 8 bytes per row

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// The first `bytes` of N bytes; the rest of the destination is zeroed.
template <int N> __device__ __forceinline__ void cp_async_part(uint32_t dst, const void *src, int bytes)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix2(uint32_t &r0, uint32_t &r1, uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0, %1}, [%2];" : "=r"(r0), "=r"(r1) : "r"(addr) : "memory");
}

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Codes i and i + 4 of a word, less the zero point, as two bf16 integers: or-ing a code
// into bf16 128 (whose last place is 1) adds it; the difference is exact.
template <int I> __device__ __forceinline__ uint32_t weight_pair(uint32_t word, uint32_t zero128)
{
    uint32_t v = ((word >> (4 * I)) & 0x000f000fu) | 0x43004300u, r;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(zero128));
    return r;
}

// Columns (0, 4), (1, 5), (2, 6), (3, 7) of eight.
__device__ __forceinline__ uint4 x_pairs(uint4 v)
{
    return make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632), __byte_perm(v.y, v.w, 0x5410),
                      __byte_perm(v.y, v.w, 0x7632));
}

// acc += s * d on a pair, with one instruction.
__device__ __forceinline__ void fma_pair(float &acc0, float &acc1, float s, float d0, float d1)
{
    asm("{\n .reg .b64 a, b, c;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %4};\n mov.b64 c, {%0, %1};\n"
        " fma.rn.f32x2 c, a, b, c;\n mov.b64 {%0, %1}, c;\n}\n"
        : "+f"(acc0), "+f"(acc1)
        : "f"(d0), "f"(d1), "f"(s));
}

constexpr int kSlots = 2;   // of a warp's ring

// NT: batch rows / 8; GROUP: columns of a group; ZEROS: zero points; XS: x in shared memory
// (else read from global memory through L1); W: warps.
template <int NT, int GROUP, bool ZEROS, bool XS, int W>
__global__ void __launch_bounds__(W * 32, 1) k_q4_matvec(Q4Params p, Q4Plan plan)
{
    constexpr int WORDS = GROUP / 32;         // words of a lane in a group
    constexpr int GROUPS = kCols / GROUP;     // groups of a step
    constexpr int STAGE = kCodeBytes + kScaleBytes + (ZEROS ? kZeroBytes : 0);
    constexpr int WIN = GROUPS > 1 ? 2 : 1;   // pieces of a row's window of scales or zero points
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    const int b0 = blockIdx.y * NT * 8;
    const uint4 *xs = (const uint4 *)smem + lane;
    uint8_t *ring = smem + plan.x_bytes + warp * kSlots * STAGE;
    const uint32_t ring_s = (uint32_t)__cvta_generic_to_shared(ring);

    // tiles of this CTA, then of this warp; columns of this warp in steps
    const int c_lo = (int)((long long)plan.tiles * blockIdx.x / gridDim.x);
    const int c_n = (int)((long long)plan.tiles * (blockIdx.x + 1) / gridDim.x) - c_lo;
    const int row_groups = W / plan.parts, rg = warp / plan.parts, part = warp % plan.parts;
    const int t_lo = c_lo + c_n * rg / row_groups, t_hi = c_lo + c_n * (rg + 1) / row_groups;
    const int steps_row = (p.K + kCols - 1) / kCols;
    const int k_lo = steps_row * part / plan.parts, k_hi = steps_row * (part + 1) / plan.parts;
    const int steps = (t_hi - t_lo + kTiles - 1) / kTiles * (k_hi - k_lo);

    // the next step to load: its tiles and columns, its rows that exist, where the lane's
    // codes begin, and the scales and zero points of the tiles' first row
    int l_tile = t_lo - kTiles, l_k = k_hi - 1, l_rows = 0, s_left = 0, z_left = 0;
    const uint8_t *l_codes = nullptr, *l_scales = nullptr, *l_zeros = nullptr;
    const long long stride8 = 8 * p.ld_codes;
    const uint32_t code_dst = ring_s + lane / 4 * 64 + ((lane % 4) ^ (lane / 8 & 3)) * 16;
    auto load = [&](int slot) {
        if (++l_k == k_hi) {
            l_k = k_lo;
            l_tile += kTiles;
            const long long row0 = (long long)l_tile * 16, rows_left = p.M - row0;
            l_rows = (int)min((long long)min((t_hi - l_tile) * 16, kRows), rows_left);
            l_codes = p.codes + (row0 + lane / 4) * p.ld_codes + l_k * (kCols / 2) + lane % 4 * 16;
            l_scales = (const uint8_t *)p.scales + row0 * p.G * 2;
            s_left = (int)min(rows_left * p.G * 2, 1ll << 30);
            if (ZEROS) l_zeros = p.zeros + row0 * p.G, z_left = (int)min(rows_left * p.G, 1ll << 30);
        }
        const uint32_t off = slot * STAGE;
        const bool in = l_k * (kCols / 2) + lane % 4 * 16 < p.K / 2;
        const uint8_t *src = l_codes;
#pragma unroll
        for (int i = 0; i < kRows / 8; ++i) {
            // the swizzle's (row >> 1) & 3 does not depend on i
            if (in && i * 8 + lane / 4 < l_rows) cp_async16(code_dst + off + i * 512, src);
            src += stride8;
        }
        l_codes += kCols / 2;
        const int g0 = l_k * GROUPS;
#pragma unroll
        for (int i = 0; i < kRows * WIN / 32; ++i) {
            const int r = (i * 32 + lane) / WIN, j = (i * 32 + lane) % WIN, w = ((r * p.G + g0) * 2 & ~7) + j * 8;
            if (r < l_rows && w < s_left)
                cp_async_part<8>(ring_s + off + kCodeBytes + r * 16 + j * 8, l_scales + w, min(8, s_left - w));
        }
        if (ZEROS) {
#pragma unroll
            for (int i = 0; i < kRows * WIN / 32; ++i) {
                const int r = (i * 32 + lane) / WIN, j = (i * 32 + lane) % WIN, w = (r * p.G + g0 & ~3) + j * 4;
                if (r < l_rows && w < z_left)
                    cp_async_part<4>(ring_s + off + kCodeBytes + kScaleBytes + r * 8 + j * 4, l_zeros + w, min(4, z_left - w));
            }
        }
    };
    if (steps > 0) load(0);
    cp_async_commit();

    if (XS) {
        // x in the operand's order: [word of 32 columns][8 batch rows][lane]
        uint4 *dst = (uint4 *)smem;
        for (int i = threadIdx.x; i < p.K / 32 * NT * 32; i += W * 32) {
            const int l = i % 32, n = b0 + i / 32 % NT * 8 + l / 4, k = i / (32 * NT) * 32 + l % 4 * 8;
            dst[i] = n < p.B ? x_pairs(ld_ro16(p.x + n * p.ld_x + k)) : make_uint4(0, 0, 0, 0);
        }
        __syncthreads();
    }

    float acc[kTiles][NT][4];
#pragma unroll
    for (int r = 0; r < kTiles; ++r)
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[r][n][0] = acc[r][n][1] = acc[r][n][2] = acc[r][n][3] = 0.f;

    auto store = [&](float y, int m, int n) {
        if (m >= p.M || n >= p.B) return;
        if (p.softcap > 0.f) y = p.softcap * tanhf(y / p.softcap);
        if (p.bf16_out)
            ((uint16_t *)p.out)[n * p.ld_out + m] = bf16_bits(y);
        else
            ((float *)p.out)[n * p.ld_out + m] = y;
    };

    int tile = t_lo, k = k_lo;
    const int g_mod = g * p.G;                        // (row * G) mod 4 is the same for all of a lane's rows
    const uint32_t m_row = lane % 16 * 64, m_swz = lane % 16 / 2 & 3;
    for (int i = 0; i < steps; ++i) {
        const int slot = i % kSlots;
        cp_async_wait<0>();
        __syncwarp();   // step i is there for every lane, and the slot of step i - 1 is free
        if (i + 1 < steps) load((i + 1) % kSlots);
        cp_async_commit();
        const int live = min(t_hi - tile, kTiles), g0 = k * GROUPS;
        const uint32_t codes = ring_s + slot * STAGE + m_row;
        const uint8_t *sc = ring + slot * STAGE + kCodeBytes + g * 16 + (g_mod + g0 & 3) * 2;
        const uint8_t *zp = ring + slot * STAGE + kCodeBytes + kScaleBytes + g * 8 + (g_mod + g0 & 3);
#pragma unroll
        for (int j = 0; j < GROUPS; ++j) {
            if (g0 + j >= p.G) break;
            uint4 x[WORDS][NT];
#pragma unroll
            for (int w = 0; w < WORDS; ++w)
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const int word = (g0 + j) * WORDS + w;
                    if (XS) {
                        x[w][n] = xs[(word * NT + n) * 32];
                    } else {
                        const int row = b0 + n * 8 + g;
                        x[w][n] = row < p.B ? x_pairs(ld_ro16(p.x + row * p.ld_x + word * 32 + t * 8)) : make_uint4(0, 0, 0, 0);
                    }
                }
#pragma unroll
            for (int r = 0; r < kTiles; ++r) {
                if (r >= live) break;
                const float s_lo = bf16_value(*(const uint16_t *)(sc + r * 256 + j * 2));
                const float s_hi = bf16_value(*(const uint16_t *)(sc + r * 256 + 128 + j * 2));
                uint32_t z_lo = 0x43084308u, z_hi = 0x43084308u;
                if (ZEROS) {
                    z_lo = (zp[r * 128 + j] & 15u) * 0x10001u | 0x43004300u;
                    z_hi = (zp[r * 128 + 64 + j] & 15u) * 0x10001u | 0x43004300u;
                }
                uint32_t word[WORDS][2];
                const uint32_t at = codes + r * 1024;
                if (WORDS == 1) {
                    ldmatrix2(word[0][0], word[0][1], at + (j ^ m_swz) * 16);
                } else {
#pragma unroll
                    for (int w = 0; w < WORDS; w += 2) {
                        uint32_t q[4];
                        ldmatrix4(q, at + ((j * WORDS + w + lane / 16) ^ m_swz) * 16);
                        word[w][0] = q[0], word[w][1] = q[1], word[(w + 1) % WORDS][0] = q[2], word[(w + 1) % WORDS][1] = q[3];
                    }
                }
                float d[NT][4];
#pragma unroll
                for (int n = 0; n < NT; ++n) d[n][0] = d[n][1] = d[n][2] = d[n][3] = 0.f;
#pragma unroll
                for (int w = 0; w < WORDS; ++w) {
                    const uint32_t a = word[w][0], b = word[w][1];
                    const uint32_t a0 = weight_pair<0>(a, z_lo), a1 = weight_pair<0>(b, z_hi), a2 = weight_pair<1>(a, z_lo),
                                   a3 = weight_pair<1>(b, z_hi), a4 = weight_pair<2>(a, z_lo), a5 = weight_pair<2>(b, z_hi),
                                   a6 = weight_pair<3>(a, z_lo), a7 = weight_pair<3>(b, z_hi);
#pragma unroll
                    for (int n = 0; n < NT; ++n) mma_16816(d[n], a0, a1, a2, a3, x[w][n].x, x[w][n].y);
#pragma unroll
                    for (int n = 0; n < NT; ++n) mma_16816(d[n], a4, a5, a6, a7, x[w][n].z, x[w][n].w);
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    fma_pair(acc[r][n][0], acc[r][n][1], s_lo, d[n][0], d[n][1]);
                    fma_pair(acc[r][n][2], acc[r][n][3], s_hi, d[n][2], d[n][3]);
                }
            }
        }
        if (++k == k_hi) {
            k = k_lo;
            if (plan.parts == 1) {
#pragma unroll
                for (int r = 0; r < kTiles; ++r) {
                    if (r >= live) break;
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            store(acc[r][n][e], (tile + r) * 16 + g + e / 2 * 8, b0 + n * 8 + t * 2 + e % 2);
                            acc[r][n][e] = 0.f;
                        }
                }
                tile += kTiles;
            }
        }
    }
    if (plan.parts == 1) return;

    // the parts of each row are added in their order; a row group has at most kTiles tiles
    // here, so that each warp holds one unit.  The sums take the rings' place.
    __syncthreads();
    float4 *sums = (float4 *)(smem + plan.x_bytes);   // [warp][tile][NT][lane]
    const int tiles = t_hi - t_lo;
#pragma unroll
    for (int r = 0; r < kTiles; ++r) {
        if (r >= tiles) break;
#pragma unroll
        for (int n = 0; n < NT; ++n)
            sums[((warp * kTiles + r) * NT + n) * 32 + lane] = make_float4(acc[r][n][0], acc[r][n][1], acc[r][n][2], acc[r][n][3]);
    }
    __syncthreads();
    for (int i = part; i < tiles * NT; i += plan.parts) {
        const int r = i / NT, n = i % NT;
        float y[4] = {};
        for (int q = 0; q < plan.parts; ++q) {
            const float4 v = sums[(((rg * plan.parts + q) * kTiles + r) * NT + n) * 32 + lane];
            y[0] += v.x, y[1] += v.y, y[2] += v.z, y[3] += v.w;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) store(y[e], (t_lo + r) * 16 + g + e / 2 * 8, b0 + n * 8 + t * 2 + e % 2);
    }
}

constexpr size_t kSmemMost = 227 * 1024;

template <int W> size_t q4_ring(bool zeros)
{
    return (size_t)W * kSlots * (kCodeBytes + kScaleBytes + (zeros ? kZeroBytes : 0));
}

template <int NT, int GROUP, bool ZEROS, bool XS, int W> cudaError_t launch_q4(const Q4Params &p, cudaStream_t s)
{
    static_assert(W * kSlots * (kCodeBytes + kScaleBytes) >= W * kTiles * NT * 512, "the sums fit the rings");
    Q4Plan plan{};
    plan.tiles = (p.M + 15) / 16;
    plan.x_bytes = XS ? NT * 16 * p.K : 0;
    const int sms = sm_count(), per_cta = (plan.tiles + sms - 1) / sms;
    // few tiles per CTA: its warps share the rows' columns instead
    plan.parts = 1;
    while (plan.parts < 8 && per_cta * plan.parts * 2 <= W) plan.parts *= 2;
    if (W % plan.parts) plan.parts = 4;
    const size_t smem = plan.x_bytes + q4_ring<W>(ZEROS);
    cudaError_t e = allow_smem((const void *)k_q4_matvec<NT, GROUP, ZEROS, XS, W>, smem);
    if (e != cudaSuccess) return e;
    const dim3 grid(std::min(sms, plan.tiles), (p.B + NT * 8 - 1) / (NT * 8));
    k_q4_matvec<NT, GROUP, ZEROS, XS, W><<<grid, W * 32, smem, s>>>(p, plan);
    return cudaGetLastError();
}

template <int NT, int GROUP, bool ZEROS> cudaError_t launch_q4_x(const Q4Params &p, cudaStream_t s)
{
    constexpr int W = NT <= 2 ? 16 : 12;
    const size_t x = (size_t)NT * 16 * p.K;
    if (x + q4_ring<W>(ZEROS) <= kSmemMost) return launch_q4<NT, GROUP, ZEROS, true, W>(p, s);
    if (x + q4_ring<8>(ZEROS) <= kSmemMost) return launch_q4<NT, GROUP, ZEROS, true, 8>(p, s);
    return launch_q4<NT, GROUP, ZEROS, false, W>(p, s);
}

template <int NT, int GROUP> cudaError_t launch_q4_zeros(const Q4Params &p, cudaStream_t s)
{
    return p.zeros ? launch_q4_x<NT, GROUP, true>(p, s) : launch_q4_x<NT, GROUP, false>(p, s);
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
