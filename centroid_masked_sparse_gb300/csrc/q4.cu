// Products with 4-bit weights: out[b, m] = sum_k (code[m, k] - z) * scale * x[b, k], and the
// rounding of a bf16 matrix to that form.
#include <algorithm>

#include "lm_ops.h"

namespace mtp {

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
constexpr int kWarps = 8;
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

struct Q4Plan {
    int tiles;        // tiles of 16 rows in all
    int parts;        // warps that share a row's columns
    int stage_bytes;  // of one ring slot
    int x_bytes;
};

// NT: batch rows / 8; GROUP: columns of a group; S: ring slots; XS: x in shared memory
// (else read from global memory through L1).
template <int NT, int GROUP, int S, bool XS>
__global__ void __launch_bounds__(kWarps * 32) k_q4_matvec(Q4Params p, Q4Plan plan)
{
    constexpr int WORDS = GROUP / 32;         // words of a lane in a group
    constexpr int GROUPS = kCols / GROUP;     // groups of a step
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    const int b0 = blockIdx.y * NT * 8;
    const uint4 *xs = (const uint4 *)smem;
    uint8_t *ring = smem + plan.x_bytes + warp * S * plan.stage_bytes;
    const uint32_t ring_s = (uint32_t)__cvta_generic_to_shared(ring);

    // tiles of this CTA, then of this warp; steps of this warp
    const int c_lo = (int)((long long)plan.tiles * blockIdx.x / gridDim.x);
    const int c_n = (int)((long long)plan.tiles * (blockIdx.x + 1) / gridDim.x) - c_lo;
    const int row_groups = kWarps / plan.parts, rg = warp / plan.parts, part = warp % plan.parts;
    const int t_lo = c_lo + c_n * rg / row_groups, t_hi = c_lo + c_n * (rg + 1) / row_groups;
    const int steps_row = (p.K + kCols - 1) / kCols;
    const int k_lo = steps_row * part / plan.parts, k_n = steps_row * (part + 1) / plan.parts - k_lo;
    const int steps = (t_hi - t_lo + kTiles - 1) / kTiles * k_n;
    const uint8_t *scales = (const uint8_t *)p.scales, *scales_end = scales + 2ll * p.M * p.G;
    const uint8_t *zeros_end = p.zeros + (long long)p.M * p.G;

    // step i of the warp: tiles from t_lo + i / k_n * kTiles, columns (k_lo + i % k_n) * kCols
    int l_tile = t_lo, l_k = 0;   // of the next step to load
    auto load = [&](int slot) {
        const int rows = min(min((t_hi - l_tile) * 16, kRows), p.M - l_tile * 16);
        const long long row0 = (long long)l_tile * 16;
        const int byte0 = (k_lo + l_k) * (kCols / 2), g0 = (k_lo + l_k) * GROUPS;
        const uint32_t dst = ring_s + slot * plan.stage_bytes;
        const uint8_t *src = p.codes + (row0 + lane / 4) * p.ld_codes + byte0 + lane % 4 * 16;
        const bool in = byte0 + lane % 4 * 16 < p.K / 2;
#pragma unroll
        for (int i = 0; i < kRows / 8; ++i) {
            const int r = i * 8 + lane / 4;
            if (in && r < rows) cp_async16(dst + r * 64 + ((lane % 4) ^ (r >> 1 & 3)) * 16, src + i * 8 * p.ld_codes);
        }
        // 8-byte words of the window that holds the row's scales: one is enough for one group
        constexpr int N = GROUPS > 1 ? 2 : 1;
#pragma unroll
        for (int i = 0; i < kRows * N / 32; ++i) {
            const int r = (i * 32 + lane) / N, j = (i * 32 + lane) % N;
            const uint8_t *w = scales + (((row0 + r) * p.G + g0) * 2 & ~7ll) + j * 8;
            if (r < rows && w < scales_end)
                cp_async_part<8>(dst + kCodeBytes + r * 16 + j * 8, w, (int)min(8ll, (long long)(scales_end - w)));
        }
        if (p.zeros) {
#pragma unroll
            for (int i = 0; i < kRows * N / 32; ++i) {
                const int r = (i * 32 + lane) / N, j = (i * 32 + lane) % N;
                const uint8_t *w = p.zeros + ((row0 + r) * p.G + g0 & ~3ll) + j * 4;
                if (r < rows && w < zeros_end)
                    cp_async_part<4>(dst + kCodeBytes + kScaleBytes + r * 8 + j * 4, w,
                                     (int)min(4ll, (long long)(zeros_end - w)));
            }
        }
        if (++l_k == k_n) l_k = 0, l_tile += kTiles;
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i) {
        if (i < steps) load(i);
        cp_async_commit();
    }

    if (XS) {
        // x in the operand's order: [word of 32 columns][8 batch rows][lane]
        uint4 *dst = (uint4 *)smem;
        for (int i = threadIdx.x; i < p.K / 32 * NT * 32; i += kWarps * 32) {
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

    int tile = t_lo, k = 0;
    for (int i = 0, slot = 0; i < steps; ++i) {
        cp_async_wait<S - 2>();
        __syncwarp();   // step i is there for every lane, and the slot of step i - 1 is free
        if (i + S - 1 < steps) load(slot == 0 ? S - 1 : slot - 1);
        cp_async_commit();
        const int live = min(t_hi - tile, kTiles), g0 = (k_lo + k) * GROUPS;
        const uint32_t codes = ring_s + slot * plan.stage_bytes;
        const uint8_t *sc = ring + slot * plan.stage_bytes + kCodeBytes, *zp = sc + kScaleBytes;
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
                        x[w][n] = xs[(word * NT + n) * 32 + lane];
                    } else {
                        const int row = b0 + n * 8 + g;
                        x[w][n] = row < p.B ? x_pairs(ld_ro16(p.x + row * p.ld_x + word * 32 + t * 8)) : make_uint4(0, 0, 0, 0);
                    }
                }
#pragma unroll
            for (int r = 0; r < kTiles; ++r) {
                if (r >= live) break;
                // this lane's rows, the places of their scales in the windows
                const int lo = r * 16 + g, hi = lo + 8;
                const long long at_lo = ((long long)tile * 16 + lo) * p.G + g0, at_hi = at_lo + 8ll * p.G;
                const float s_lo = bf16_value(*(const uint16_t *)(sc + lo * 16 + (at_lo & 3) * 2 + j * 2));
                const float s_hi = bf16_value(*(const uint16_t *)(sc + hi * 16 + (at_hi & 3) * 2 + j * 2));
                uint32_t z_lo = 8, z_hi = 8;
                if (p.zeros) {
                    z_lo = zp[lo * 8 + (at_lo & 3) + j] & 15;
                    z_hi = zp[hi * 8 + (at_hi & 3) + j] & 15;
                }
                z_lo = z_lo * 0x10001u | 0x43004300u;
                z_hi = z_hi * 0x10001u | 0x43004300u;
                uint32_t word[WORDS][2];
                const int row = r * 16 + lane % 16;
                const uint32_t at = codes + row * 64;
                if (WORDS == 1) {
                    ldmatrix2(word[0][0], word[0][1], at + (j ^ (row >> 1 & 3)) * 16);
                } else {
#pragma unroll
                    for (int w = 0; w < WORDS; w += 2) {
                        uint32_t q[4];
                        ldmatrix4(q, at + ((j * WORDS + w + lane / 16) ^ (row >> 1 & 3)) * 16);
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
                    acc[r][n][0] = fmaf(s_lo, d[n][0], acc[r][n][0]);
                    acc[r][n][1] = fmaf(s_lo, d[n][1], acc[r][n][1]);
                    acc[r][n][2] = fmaf(s_hi, d[n][2], acc[r][n][2]);
                    acc[r][n][3] = fmaf(s_hi, d[n][3], acc[r][n][3]);
                }
            }
        }
        slot = slot == S - 1 ? 0 : slot + 1;
        if (++k == k_n) {
            k = 0;
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
    cp_async_wait<0>();
    __syncthreads();
    float4 *sums = (float4 *)(smem + plan.x_bytes);   // [warp][tile][NT][lane]
#pragma unroll
    for (int r = 0; r < kTiles; ++r)
#pragma unroll
        for (int n = 0; n < NT; ++n)
            sums[((warp * kTiles + r) * NT + n) * 32 + lane] = make_float4(acc[r][n][0], acc[r][n][1], acc[r][n][2], acc[r][n][3]);
    __syncthreads();
    for (int i = part; i < (t_hi - t_lo) * NT; i += plan.parts) {
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

// One warp per group; reads of neighbouring warps are neighbouring columns.
__global__ void __launch_bounds__(256)
k_q4_quantize(const uint16_t *w, long long ld_w, long long groups, int G, int group, uint8_t *codes, long long ld_codes,
              uint16_t *scales, uint8_t *zeros)
{
    const long long at = (long long)blockIdx.x * 8 + threadIdx.x / 32;
    const int lane = threadIdx.x % 32;
    if (at >= groups) return;
    const long long m = at / G;
    const int g = (int)(at % G);
    const uint16_t *row = w + m * ld_w + (long long)g * group;
    // a lane holds columns 2 * lane and 2 * lane + 1 of each 64
    float v[4];
    float low = 0.f, high = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int k = i / 2 * 64 + lane * 2 + i % 2;
        v[i] = k < group ? bf16_value(__ldg(row + k)) : 0.f;
        low = fminf(low, v[i]);
        high = fmaxf(high, v[i]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        low = fminf(low, __shfl_xor_sync(~0u, low, o));
        high = fmaxf(high, __shfl_xor_sync(~0u, high, o));
    }
    const uint16_t bits = bf16_bits(zeros ? __fdiv_rn(high - low, 15.f) : __fdiv_rn(fmaxf(-low, high), 7.f));
    const float scale = bf16_value(bits);
    const float zero = !zeros ? 8.f : scale > 0.f ? fminf(fmaxf(rintf(__fdiv_rn(-low, scale)), 0.f), 15.f) : 0.f;
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        const int k = i / 2 * 64 + lane * 2;
        if (k >= group) break;
        uint32_t c[2];
#pragma unroll
        for (int j = 0; j < 2; ++j)
            c[j] = (uint32_t)fminf(fmaxf((scale > 0.f ? rintf(__fdiv_rn(v[i + j], scale)) : 0.f) + zero, 0.f), 15.f);
        codes[m * ld_codes + ((long long)g * group + k) / 2] = (uint8_t)(c[0] | c[1] << 4);
    }
    if (lane == 0) {
        scales[at] = bits;
        if (zeros) zeros[at] = (uint8_t)zero;
    }
}

}  // namespace

namespace {

constexpr size_t kSmemMost = 227 * 1024;

template <int NT, int GROUP, int S, bool XS> cudaError_t launch_q4(const Q4Params &p, Q4Plan plan, cudaStream_t s)
{
    const int sms = sm_count(), per_cta = (plan.tiles + sms - 1) / sms;
    // few tiles per CTA: its warps share the rows' columns instead
    plan.parts = per_cta >= kWarps ? 1 : per_cta >= 4 ? 2 : per_cta >= 2 ? 4 : 8;
    const size_t smem = plan.x_bytes + (size_t)kWarps * S * plan.stage_bytes;
    cudaError_t e = allow_smem((const void *)k_q4_matvec<NT, GROUP, S, XS>, smem);
    if (e != cudaSuccess) return e;
    const dim3 grid(std::min(sms, plan.tiles), (p.B + NT * 8 - 1) / (NT * 8));
    k_q4_matvec<NT, GROUP, S, XS><<<grid, kWarps * 32, smem, s>>>(p, plan);
    return cudaGetLastError();
}

template <int NT, int S, bool XS> cudaError_t launch_q4_group(const Q4Params &p, const Q4Plan &plan, cudaStream_t s)
{
    return p.group == 32   ? launch_q4<NT, 32, S, XS>(p, plan, s)
           : p.group == 64 ? launch_q4<NT, 64, S, XS>(p, plan, s)
                           : launch_q4<NT, 128, S, XS>(p, plan, s);
}

template <int S, bool XS> cudaError_t launch_q4_batch(int nt, const Q4Params &p, const Q4Plan &plan, cudaStream_t s)
{
    return nt == 1   ? launch_q4_group<1, S, XS>(p, plan, s)
           : nt == 2 ? launch_q4_group<2, S, XS>(p, plan, s)
           : nt == 3 ? launch_q4_group<3, S, XS>(p, plan, s)
                     : launch_q4_group<4, S, XS>(p, plan, s);
}

}  // namespace

cudaError_t launch_q4_matvec(const Q4Params &p, cudaStream_t s)
{
    Q4Plan plan{};
    plan.tiles = (p.M + 15) / 16;
    plan.stage_bytes = kCodeBytes + kScaleBytes + (p.zeros ? kZeroBytes : 0);
    // the batch in equal slabs of at most 32 rows
    const int eights = (p.B + 7) / 8, slabs = (eights + 3) / 4, nt = (eights + slabs - 1) / slabs;
    plan.x_bytes = nt * 16 * p.K;
    const size_t slot = (size_t)kWarps * plan.stage_bytes;
    if (plan.x_bytes + 4 * slot <= kSmemMost) return launch_q4_batch<4, true>(nt, p, plan, s);
    if (plan.x_bytes + 2 * slot <= kSmemMost) return launch_q4_batch<2, true>(nt, p, plan, s);
    plan.x_bytes = 0;
    return launch_q4_batch<4, false>(nt, p, plan, s);
}

cudaError_t launch_q4_quantize(const uint16_t *w, long long ld_w, int M, int K, int group, uint8_t *codes,
                               long long ld_codes, uint16_t *scales, uint8_t *zeros, cudaStream_t s)
{
    const int G = K / group;
    const long long groups = (long long)M * G;
    const long long blocks = (groups + 7) / 8;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    k_q4_quantize<<<(unsigned)blocks, 256, 0, s>>>(w, ld_w, groups, G, group, codes, ld_codes, scales, zeros);
    return cudaGetLastError();
}

}  // namespace mtp
