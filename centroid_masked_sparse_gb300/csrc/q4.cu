// Products with 4-bit weights (their kernel: q4_kernel.cuh), and the rounding of a bf16
// matrix to that form.
#include <algorithm>

#include "lm_ops.h"

namespace mtp {

namespace {

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

// One thread per four bytes of the packed codes, then per (row, group) of scales and zero points.
__global__ void __launch_bounds__(256) k_q4_pack(Q4PackParams p)
{
    const long long words = (long long)p.tiles * p.blocks * 128, step = (long long)gridDim.x * blockDim.x;
    for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < words; i += step) {
        const int j = (int)(i % 4), lane = (int)(i / 4 % 32);
        const long long block = i / 128, tile = block / p.blocks;
        const long long row = tile * 16 + lane / 4 + j % 2 * 8;
        const int byte = (int)(block % p.blocks) * 32 + j / 2 * 16 + lane % 4 * 4;
        uint32_t v = 0;
        if (row < p.M && byte < p.K / 2)
#pragma unroll
            for (int b = 0; b < 4; ++b) v |= (uint32_t)p.codes[row * p.ld_codes + byte + b] << (8 * b);
        ((uint32_t *)p.out_codes)[i] = v;
    }
    const int sg = 256 / p.group, steps = (p.K + 255) / 256;
    const long long groups = (long long)p.tiles * steps * 8 * sg;
    for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < groups; i += step) {
        const int j = (int)(i % sg), g = (int)(i / sg % 8);
        const long long ts = i / sg / 8, tile = ts / steps;
        const long long at = ts % steps * sg + j;
        uint32_t s = 0, z = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const long long row = tile * 16 + g + h * 8;
            if (row >= p.M || at >= p.G) continue;
            s |= (uint32_t)p.scales[row * p.G + at] << (16 * h);
            if (p.zeros) z |= (uint32_t)(p.zeros[row * p.G + at] & 15) << (8 * h);
        }
        ((uint32_t *)p.out_scales)[i] = s;
        if (p.zeros) ((uint16_t *)p.out_zeros)[i] = (uint16_t)z;
    }
}

// Blocks of 256 threads; returns this launch's own status, whatever an earlier call has left.
template <typename... KArgs, typename... Args> cudaError_t launch_plain(void (*kernel)(KArgs...), unsigned grid, cudaStream_t s, Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace

Q4Layout q4_layout(int M, int K, int group, bool zeros)
{
    Q4Layout L{};
    const size_t tiles = ((size_t)M + 15) / 16, groups = tiles * ((K + 255) / 256) * 8 * (256 / group);
    auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    L.scales = up(tiles * ((K + 63) / 64) * 512);
    L.zeros = L.scales + up(groups * 4);
    L.total = L.zeros + (zeros ? up(groups * 2) : 0);
    return L;
}

cudaError_t launch_q4_pack(const Q4PackParams &p, cudaStream_t s)
{
    const long long words = (long long)p.tiles * p.blocks * 128;
    return launch_plain(k_q4_pack, (unsigned)std::min((words + 255) / 256, 32ll * sm_count()), s, p);
}

template <int GROUP> cudaError_t launch_q4_group(const Q4Params &p, cudaStream_t s);   // q4_kernel.cuh

cudaError_t launch_q4_matvec(const Q4Params &p, cudaStream_t s)
{
    return p.group == 32 ? launch_q4_group<32>(p, s) : p.group == 64 ? launch_q4_group<64>(p, s) : launch_q4_group<128>(p, s);
}

cudaError_t launch_q4_quantize(const uint16_t *w, long long ld_w, int M, int K, int group, uint8_t *codes,
                               long long ld_codes, uint16_t *scales, uint8_t *zeros, cudaStream_t s)
{
    const int G = K / group;
    const long long groups = (long long)M * G;
    const long long blocks = (groups + 7) / 8;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    return launch_plain(k_q4_quantize, (unsigned)blocks, s, w, ld_w, groups, G, group, codes, ld_codes, scales, zeros);
}

}  // namespace mtp
