// Products with 4-bit weights: out[b, m] = sum_k (code[m, k] - z) * scale * x[b, k], and the
// rounding of a bf16 matrix to that form.
#include "lm_ops.h"

namespace mtp {

namespace {

// One warp per output row; a lane takes 16 bytes of codes (32 columns, one group at most)
// at a time and sums their products per group before it multiplies by the scale.
__global__ void __launch_bounds__(256) k_q4_matvec(Q4Params p)
{
    const int m = blockIdx.x * 8 + threadIdx.x / 32, lane = threadIdx.x % 32;
    const int b0 = blockIdx.y * 8, nb = min(8, p.B - b0);
    if (m >= p.M) return;
    float acc[8] = {};
    for (int k = lane * 32; k < p.K; k += 32 * 32) {
        const uint4 w4 = ld_ro16(p.codes + m * p.ld_codes + k / 2);
        const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
        const long long g = (long long)m * p.G + k / p.group;
        const float scale = bf16_value(__ldg(p.scales + g));
        const int zero = p.zeros ? __ldg(p.zeros + g) & 15 : 8;
        for (int b = 0; b < nb; ++b) {
            const uint16_t *x = p.x + (b0 + b) * p.ld_x + k;
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < 32; ++i)
                sum = fmaf((float)((int)(w[i / 8] >> (i % 8 * 4) & 15) - zero), bf16_value(__ldg(x + i)), sum);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j == b) acc[j] = fmaf(scale, sum, acc[j]);
        }
    }
#pragma unroll
    for (int b = 0; b < 8; ++b) {
        float y = warp_sum(acc[b]);
        if (b >= nb || lane) continue;
        if (p.softcap > 0.f) y = p.softcap * tanhf(y / p.softcap);
        const long long at = (long long)(b0 + b) * p.ld_out + m;
        if (p.bf16_out)
            ((uint16_t *)p.out)[at] = bf16_bits(y);
        else
            ((float *)p.out)[at] = y;
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

cudaError_t launch_q4_matvec(const Q4Params &p, cudaStream_t s)
{
    k_q4_matvec<<<dim3((p.M + 7) / 8, (p.B + 7) / 8), 256, 0, s>>>(p);
    return cudaGetLastError();
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
