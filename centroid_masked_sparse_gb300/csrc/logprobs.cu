// Log probabilities of given tokens, entropy and largest alternatives of rows of logits,
// and the gradient of the former two.
//
// k_token_logprobs.  One pass over a row, shared by the CTAs of a cluster.  With c = log2(e)
// / temperature, a thread keeps s = sum 2^(x c - R) and t = sum 2^(x c - R) (x c - R) of its
// logits x, where R is the integer above its largest x c: then x c - R is one fused
// multiply-add with one rounding, R is exact and so are the powers of two that join the
// threads' sums; ln sum e^x = (R + log2 s) ln 2, entropy = (log2 s - t / s) ln 2.  A row
// whose largest |x c| is 2^22 or more (all logits at the type's lowest value, say), or a
// temperature of 2^64 or more, is read again with its maximum m and terms of (x - m) c.
//
// The alternatives: each of the W warps finds the ceil(n / W)-th largest of its threads'
// largest logits; the lowest of these is a bound that at least n logits reach, and few do.
// A thread has kept the largest logit of each of 32 groups of its tiles; only groups that
// reach the bound are read once more (a few hundred vectors), and what reaches it goes into a
// buffer of (logit, id) keys, which are ranked by counting.  Where the buffer does not hold
// them all (ties by the thousand), all vectors are read again in rounds that it holds, with
// sorted lists of 32 a warp between them.
//
// What bounds it: HBM for fp32; for bf16 neither that nor the issue slots alone.  320 rows of
// 262144 take 41.9 us with 20 alternatives, 4.0 TB/s, and 33.9 with none, 5 TB/s; two logits
// take 21.4 and 17.5 instructions (13 of them the sums, the maximum and the rank, on packed
// pairs), which fill 0.62 of the slots; what is missing is loads in flight, at 24 warps per SM
// and, for 8 us, searches beside which a CTA reads next to nothing.  In fp32 60 us, 5.6 TB/s.
// One row takes 9.2 us, all latency: a third of it its own reading, the rest the search and the
// joins of eight CTAs.
#include <algorithm>
#include <type_traits>

#include "lm_ops.h"

namespace mtp {

namespace {

constexpr int kGradThreads = 256;
constexpr int kVecs = 4;          // 16-byte vectors of a thread in a tile
constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.69314718055994531f;
constexpr float kFar = 4194304.f; // |x c| from which R would not be exact
constexpr float kFlat = 0x1p-64f; // 1 / temperature below which `low` (see there) would have a weight

typedef unsigned long long u64;

__device__ __forceinline__ u64 pair(float a, float b)
{
    u64 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 unpair(u64 v)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ u64 fma2(u64 a, u64 b, u64 c)
{
    u64 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ u64 mul2(u64 a, u64 b)
{
    u64 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ u64 add2(u64 a, u64 b)
{
    u64 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// max that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ float is_above(float a, float b)   // 1 or 0
{
    float r;
    asm("set.gt.f32.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// A word of logits: one fp32 or two bf16.
template <bool BF16> struct Logits;
template <> struct Logits<false> {
    typedef float type;
    static constexpr int VEC = 4;
    static __device__ __forceinline__ uint32_t masked() { return 0xff800000u; }
    static __device__ __forceinline__ float value(float v) { return v; }
};
template <> struct Logits<true> {
    typedef uint16_t type;
    static constexpr int VEC = 8;
    static __device__ __forceinline__ uint32_t masked() { return 0xff80ff80u; }
    static __device__ __forceinline__ float value(uint16_t v) { return bf16_value(v); }
};
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// Element e of a vector of logits.
template <bool BF16> __device__ __forceinline__ float element(const uint4 &v, int e)
{
    const uint32_t w = BF16 ? (e / 2 == 0 ? v.x : e / 2 == 1 ? v.y : e / 2 == 2 ? v.z : v.w)
                            : (e == 0 ? v.x : e == 1 ? v.y : e == 2 ? v.z : v.w);
    return BF16 ? (e % 2 ? bf_hi(w) : bf_lo(w)) : __uint_as_float(w);
}

// What stands in for lower logits: their terms are 0 all the same (for factors from kFlat on,
// below which a second reading takes the terms), and it keeps 0 * -inf out.  A bf16 number, so
// that no logit of that type lies between it and what it is rounded to.
__device__ __forceinline__ float lowest(float factor)
{
    return __uint_as_float(__float_as_uint(-1e30f / fmaxf(factor, 1.f)) & 0xffff0000u);
}

// The warp's 32 keys in falling order, and the largest 32 of two such lists.
template <typename K> __device__ __forceinline__ K exchange(K v, int lane, int step, bool up)
{
    const K other = __shfl_xor_sync(~0u, v, step);
    return ((lane & step) != 0) == up ? max(v, other) : min(v, other);
}
template <typename K> __device__ __forceinline__ K warp_sort(K v, int lane)
{
#pragma unroll
    for (int size = 2; size <= 32; size *= 2)
#pragma unroll
        for (int step = size / 2; step > 0; step /= 2) v = exchange(v, lane, step, size < 32 && (lane & size) != 0);
    return v;
}
template <typename K> __device__ __forceinline__ K warp_merge(K a, K b, int lane)
{
    K v = max(a, __shfl_sync(~0u, b, 31 - lane));
#pragma unroll
    for (int step = 16; step > 0; step /= 2) v = exchange(v, lane, step, false);
    return v;
}

// Shared memory is what the loads in flight leave of L1, so the keys take the groups' place.
constexpr int kGroups = 32, kOvers = 64;

template <int W> struct TopState {
    static constexpr int kKeys = W * 32 * 8;   // what one vector of every thread may bring
    union {
        unsigned short group[kGroups][W * 32];  // the threads' largest logits by groups of tiles: bf16, rounded up
        u64 cand[kKeys];
    };
    u64 lists[W][32];
    u64 best[32];                      // the largest so far, falling
    unsigned short over[W][kOvers];    // a warp's groups that reach the bound: group * threads + thread
    uint32_t bounds[W];
    int have, many;                    // keys in cand (or more, if it is full); whether an `over` was too short
};

// The largest 32 of all warps' lists, falling: warp 0's result, and after a barrier lists[0].
template <int W, typename K> __device__ __forceinline__ K merge_lists(K (*lists)[32], K mine, int warp, int lane)
{
    lists[warp][lane] = mine;
#pragma unroll
    for (int half = W / 2; half > 0; half /= 2) {
        __syncthreads();
        if (warp < half) lists[warp][lane] = mine = warp_merge(mine, lists[warp + half][lane], lane);
    }
    return mine;
}

// Takes the buffer's keys into `best`.  Every thread calls it, with the buffer at rest.
template <int W> __device__ __forceinline__ void reduce_buffer(TopState<W> &top, int warp, int lane)
{
    const int have = top.have;
    u64 mine = warp == 0 ? top.best[lane] : 0ull;
    for (int at = warp * 32; at < have; at += W * 32)
        mine = warp_merge(mine, warp_sort(at + lane < have ? top.cand[at + lane] : 0ull, lane), lane);
    mine = merge_lists<W>(top.lists, mine, warp, lane);
    if (warp == 0) {
        top.best[lane] = mine;
        if (lane == 0) top.have = 0;
    }
    __syncthreads();
}

// The largest value of the type below v (any but -inf).
template <bool BF16> __device__ __forceinline__ float value_below(float v)
{
    const uint32_t u = __float_as_uint(v), step = BF16 ? 0x10000u : 1u;
    return __uint_as_float(v == 0.f ? 0x80000000u + step : v > 0.f ? u - step : u + step);
}

// The smallest bf16 from v up; for a NaN any value.
__device__ __forceinline__ unsigned short bf16_up(float v)
{
    const uint32_t u = __float_as_uint(v);
    return (unsigned short)((u + (u >> 31 ? 0u : 0xffffu)) >> 16);
}

struct Sums {
    float r, s, t, most;   // reference (an integer, or 0 for all), sums, largest logit
    int before;            // tokens before the given one
};

// The warp's sums, in every lane.
__device__ __forceinline__ Sums warp_join(Sums a)
{
    Sums j;
    // references below +-kFar are integers; one beyond makes the row's second reading, or a NaN
    const int r = (int)fminf(fmaxf(a.r, -2.f * kFar), 2.f * kFar), top = __reduce_max_sync(~0u, r);
    const float f = exp2_fast((float)(r - top));
    j.r = (float)top;
    j.s = warp_sum(f * a.s);
    j.t = warp_sum(f * fmaf((float)(r - top), a.s, a.t));
    j.most = ord_value(__reduce_max_sync(~0u, ord_key(a.most)));
    j.before = __reduce_add_sync(~0u, a.before);
    return j;
}

template <bool BF16, bool TOP, int W>
__global__ void __launch_bounds__(W * 32, 32 / W) k_token_logprobs(LogprobParams p)
{
    typedef Logits<BF16> L;
    typedef typename L::type T;
    constexpr int TH = W * 32, VEC = L::VEC;   // threads; logits of a vector
    __shared__ Sums s_warp[W], s_cta, s_row;
    __shared__ __align__(16) unsigned char s_top[TOP ? sizeof(TopState<W>) : 16];
    TopState<W> &top = *(TopState<W> *)s_top;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int csize = (int)cluster_size(), crank = (int)cluster_rank(), row = blockIdx.x / csize;
    const T *x = (const T *)p.logits + row * p.ld;
    const float c = p.factor * kLog2e;
    const float low = lowest(p.factor);
    const uint32_t low2 = (__float_as_uint(low) >> 16) * 0x10001u;

    // The row as scalars up to a 16-byte boundary, vectors, and scalars behind the last; the
    // first CTA takes the scalars before, the last one those behind, and each its vectors.
    const int head = min(p.vocab, (int)((16 - ((uintptr_t)x & 15)) % 16 / sizeof(T)));
    const int all = (p.vocab - head) / VEC, tail = head + all * VEC;
    const int v_lo = (int)((long long)all * crank / csize), vecs = (int)((long long)all * (crank + 1) / csize) - v_lo;
    const T *base = x + head + (long long)v_lo * VEC;
    const int id0 = head + v_lo * VEC;
    const uint4 *at_load = (const uint4 *)base + threadIdx.x;
    const int tiles = (vecs + kVecs * TH - 1) / (kVecs * TH), whole = vecs / (kVecs * TH);   // the last one may be short
    auto load = [&](int tile, uint4 (&v)[kVecs]) {
        if (tile < whole) {
#pragma unroll
            for (int j = 0; j < kVecs; ++j) v[j] = ld_ro16(at_load + j * TH);
        } else {
#pragma unroll
            for (int j = 0; j < kVecs; ++j)
                v[j] = (tile * kVecs + j) * TH + threadIdx.x < vecs ? ld_ro16(at_load + j * TH)
                                                                   : make_uint4(L::masked(), L::masked(), L::masked(), L::masked());
        }
        at_load += kVecs * TH;
    };
    wait_for_previous();
    const int given = p.tokens ? __ldg(p.tokens + row) : -1;
    uint4 next[kVecs];
    load(0, next);
    const bool has = given >= 0 && given < p.vocab;
    const float mine = has ? L::value(x[given]) : 0.f;
    if (TOP) {
        if (threadIdx.x < 32) top.best[threadIdx.x] = 0;
        if (threadIdx.x == 0) top.have = top.many = 0;
        __syncthreads();
    }

    float r = -kFar, most = -INFINITY;
    u64 s2 = 0, t2 = 0;   // pairs of sums
    int before = 0;
    auto raise = [&](float to) {   // the reference is at least `to` from here on
        const float up = ceilf(to);
        if (up > r) {
            const float f = exp2_fast(r - up), d = up - r;
            s2 = mul2(s2, pair(f, f));
            t2 = fma2(t2, pair(f, f), mul2(s2, pair(-d, -d)));
            r = up;
        }
    };
    auto add = [&](float a, float b) {   // two logits, or one and `low`
        const u64 d = fma2(pair(a, b), pair(c, c), pair(-r, -r));
        const float2 u = unpair(d);
        const u64 e = pair(exp2_fast(u.x), exp2_fast(u.y));
        s2 = add2(s2, e);
        t2 = fma2(e, d, t2);
    };
    u64 count2 = 0;   // logits above `over`, as floats (below 2^24 a thread)
    auto terms = [&](const uint4 (&v)[kVecs], auto counting, float over) {
        auto two = [&](float a, float b) {
            add(a, b);
            if (decltype(counting)::value) count2 = add2(count2, pair(is_above(a, over), is_above(b, over)));
        };
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            if (BF16) {
                const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t u = max_nan_bf16x2(w[i], low2);
                    two(bf_lo(u), bf_hi(u));
                }
            } else {
                two(max_nan(__uint_as_float(v[j].x), low), max_nan(__uint_as_float(v[j].y), low));
                two(max_nan(__uint_as_float(v[j].z), low), max_nan(__uint_as_float(v[j].w), low));
            }
        }
    };
    auto one = [&](int id, float v) {   // a scalar before or behind the vectors
        most = fmaxf(most, v);
        raise(v * c);
        add(max_nan(v, low), low);
        before += v > mine || (v == mine && id < given);
    };
    const bool before_it = crank == 0 && threadIdx.x < head, behind_it = crank == csize - 1 && threadIdx.x < p.vocab - tail;

    const int group_tiles = max(1, (tiles + kGroups - 1) / kGroups);
    int groups = 0, in_group = 0;
    float of_group = -INFINITY;
    for (int tile = 0; tile < tiles; ++tile) {
        uint4 v[kVecs];
#pragma unroll
        for (int j = 0; j < kVecs; ++j) v[j] = next[j];
        load(tile + 1, next);
        const int first = id0 + tile * kVecs * TH * VEC;   // the tile's ids
        float high;   // the thread's largest of the tile
        if (BF16) {
            uint32_t m = max_bf16x2(max_bf16x2(v[0].x, v[0].y), max_bf16x2(v[0].z, v[0].w));
#pragma unroll
            for (int j = 1; j < kVecs; ++j) m = max_bf16x2(m, max_bf16x2(max_bf16x2(v[j].x, v[j].y), max_bf16x2(v[j].z, v[j].w)));
            high = fmaxf(bf_lo(m), bf_hi(m));
        } else {
            high = -INFINITY;
#pragma unroll
            for (int j = 0; j < kVecs; ++j)
#pragma unroll
                for (int e = 0; e < VEC; ++e) high = fmaxf(high, element<BF16>(v[j], e));
        }
        most = fmaxf(most, high);
        raise(high * c);
        if (TOP) {
            of_group = fmaxf(of_group, high);
            if (++in_group == group_tiles) {
                top.group[groups++][threadIdx.x] = bf16_up(of_group);
                of_group = -INFINITY, in_group = 0;
            }
        }
        // Logits that come before the given one: not below it at lower ids, above it at higher
        // ones; a warp without one that reaches it (near the top: most) does not count.
        const long long last = first + (long long)kVecs * TH * VEC;
        const bool count = p.rank && has, here = count && ((first <= given && given < last) || mine <= low);
        if (count && !here && __any_sync(~0u, high >= mine))
            terms(v, std::true_type{}, given >= last ? value_below<BF16>(mine) : mine);   // v >= mine is v > the value below
        else
            terms(v, std::false_type{}, 0.f);
        if (here) {
#pragma unroll
            for (int j = 0; j < kVecs; ++j)
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const int id = first + (j * TH + threadIdx.x) * VEC + e;
                    const float u = element<BF16>(v[j], e);
                    before += (tile * kVecs + j) * TH + threadIdx.x < vecs && (u > mine || (u == mine && id < given));
                }
        }
    }
    before += (int)(unpair(count2).x + unpair(count2).y);
    const float v_before = before_it ? L::value(x[threadIdx.x]) : 0.f, v_behind = behind_it ? L::value(x[tail + threadIdx.x]) : 0.f;
    if (before_it) one(threadIdx.x, v_before);
    if (behind_it) one(tail + threadIdx.x, v_behind);

    if (TOP) {
        const uint32_t mark = most == -INFINITY ? 0u : ord_key(most);
        {
            uint32_t rest = mark, nth = 0;
            for (int k = 0; k < (p.top + W - 1) / W; ++k) {
                nth = __reduce_max_sync(~0u, rest);
                if (lane == __ffs(__ballot_sync(~0u, rest == nth)) - 1) rest = 0;
            }
            if (lane == 0) top.bounds[warp] = nth;
        }
        __syncthreads();
        uint32_t bound = top.bounds[0];
#pragma unroll
        for (int w = 1; w < W; ++w) bound = min(bound, top.bounds[w]);
        // what reaches this is above -inf
        const float reach = bound ? ord_value(bound) : -3.402823466e38f;
        auto push = [&](float v, int id, u64 least) {
            const u64 key = argmax_key(v, id);
            if (key <= least) return;
            const int at = atomicAdd(&top.have, 1);
            if (at < TopState<W>::kKeys) top.cand[at] = key;
        };
        auto look = [&](const uint4 &v, int at, u64 least) {
            float high;
            if (BF16) {
                const uint32_t m = max_bf16x2(max_bf16x2(v.x, v.y), max_bf16x2(v.z, v.w));
                high = fmaxf(bf_lo(m), bf_hi(m));
            } else {
                high = fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
            }
            if (!(high >= reach)) return;
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                if (element<BF16>(v, e) >= reach) push(element<BF16>(v, e), id0 + at * VEC + e, least);
        };
        auto look_at_scalars = [&] {
            if (before_it && v_before >= reach) push(v_before, threadIdx.x, 0);
            if (behind_it && v_behind >= reach) push(v_behind, tail + threadIdx.x, 0);
        };
        if (in_group) top.group[groups++][threadIdx.x] = bf16_up(of_group);
        // The groups that reach it: each thread's as bits, then one of every thread at a time.
        const int each = group_tiles * kVecs;   // vectors of a group
        uint32_t reached = 0;
        if (__any_sync(~0u, most >= reach)) {
#pragma unroll
            for (int k = 0; k < kGroups; ++k)
                if (k < groups) reached |= (uint32_t)(bf_lo(top.group[k][threadIdx.x]) >= reach) << k;
        }
        int overs = 0;
        for (uint32_t some; (some = __ballot_sync(~0u, reached != 0)) != 0; reached &= reached - 1) {
            const int at = overs + __popc(some & ((1u << lane) - 1));
            if (reached && at < kOvers) top.over[warp][at] = (unsigned short)((__ffs(reached) - 1) * TH + threadIdx.x);
            overs += __popc(some);
        }
        if (overs > kOvers) top.many = 1, overs = 0;
        __syncwarp();
        const int items = overs * each;
        uint4 v[2];
        int at[2];
        auto load_items = [&](int i0) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int i = i0 + k * 32 + lane;
                at[k] = vecs;
                if (i < items) {
                    const int o = i / each, who = top.over[warp][o];
                    at[k] = (who / TH * each + i - o * each) * TH + who % TH;
                }
                if (at[k] < vecs) v[k] = ld_ro16((const uint4 *)base + at[k]);
            }
        };
        load_items(0);
        __syncthreads();   // the groups have been read
        look_at_scalars();
        for (int i0 = 0; i0 < items; i0 += 64) {
            if (i0) load_items(i0);
#pragma unroll
            for (int k = 0; k < 2; ++k)
                if (at[k] < vecs) look(v[k], at[k], 0);
        }
        __syncthreads();
        const int have = top.have;
        if (have <= TH && !top.many) {
            if (threadIdx.x < have) {
                const u64 key = top.cand[threadIdx.x];
                int at = 0;
#pragma unroll 8
                for (int k = 0; k < have; ++k) at += top.cand[k] > key;
                if (at < 32) top.best[at] = key;
            }
        } else if (have <= TopState<W>::kKeys && !top.many) {
            reduce_buffer(top, warp, lane);
        } else {
            // all vectors, in rounds that the buffer holds
            __syncthreads();
            if (threadIdx.x == 0) top.have = 0;
            __syncthreads();
            look_at_scalars();
            __syncthreads();
            reduce_buffer(top, warp, lane);
            u64 least = top.best[p.top - 1];   // the n-th best key so far
            for (int i0 = 0; i0 < vecs; i0 += TH) {
                const int i = i0 + threadIdx.x;
                if (i < vecs) look(ld_ro16((const uint4 *)base + i), i, least);
                __syncthreads();
                if (top.have > 0) {
                    reduce_buffer(top, warp, lane);
                    least = top.best[p.top - 1];
                }
                __syncthreads();   // all have decided before the next keys come
            }
        }
        __syncthreads();
    }

    // join the threads, the warps (by warp 0), the cluster (by every CTA's warp 0)
    auto join_all = [&](Sums a, bool lists) {
        a = warp_join(a);
        if (lane == 0) s_warp[warp] = a;
        __syncthreads();
        if (warp == 0) {
            const Sums none = {-2.f * kFar, 0.f, 0.f, -INFINITY, 0};
            a = warp_join(lane < W ? s_warp[lane] : none);
            if (lane == 0) s_cta = a, s_row = a;
        }
        if (csize > 1) {
            cluster_sync();
            if (warp == 0) {
                Sums b = {-2.f * kFar, 0.f, 0.f, -INFINITY, 0};
                if (lane < csize) {
                    b.r = cluster_load(&s_cta.r, lane), b.s = cluster_load(&s_cta.s, lane), b.t = cluster_load(&s_cta.t, lane);
                    b.most = cluster_load(&s_cta.most, lane), b.before = __float_as_int(cluster_load((const float *)&s_cta.before, lane));
                }
                b = warp_join(b);
                if (lane == 0) s_row = b;
            } else if (TOP && lists && crank == 0 && warp == 1) {
                // meanwhile the CTAs' alternatives
                const float *other = (const float *)&top.best[lane];
                u64 best = top.best[lane];
                float low_half = cluster_load(other, 1), high_half = cluster_load(other + 1, 1);
                for (int k = 1; k < csize; ++k) {
                    const u64 key = (u64)__float_as_uint(low_half) | (u64)__float_as_uint(high_half) << 32;
                    if (k + 1 < csize) low_half = cluster_load(other, k + 1), high_half = cluster_load(other + 1, k + 1);
                    best = warp_merge(best, key, lane);
                }
                top.best[lane] = best;
            }
        }
        __syncthreads();
        return s_row;
    };
    const float2 s1 = unpair(s2), t1 = unpair(t2);
    Sums sums = join_all(Sums{r, s1.x + s1.y, t1.x + t1.y, most, before}, true);
    const bool flat = p.factor < kFlat, far = sums.most < INFINITY && (flat || (sums.most > -INFINITY && fabsf(sums.most * c) >= kFar));
    auto below = [&](float v, float m) { return v * 0.5f - m * 0.5f; };   // half of v - m, which may leave fp32's range
    if (far) {
        // once more, with the maximum (any finite number where all is masked)
        const float m = fmaxf(sums.most, -3.402823466e38f);
        float s = 0.f, t = 0.f;
        auto term = [&](float v) {
            const float d = max_nan(below(v, m) * c * 2.f, -200.f), e = exp2_fast(d);
            s += e, t = fmaf(e, d, t);
        };
        if (crank == 0 && threadIdx.x < head) term(L::value(x[threadIdx.x]));
        if (crank == csize - 1 && threadIdx.x < p.vocab - tail) term(L::value(x[tail + threadIdx.x]));
        for (long long i = threadIdx.x; i < (long long)vecs * VEC; i += TH) term(L::value(base[i]));
        if (csize > 1) cluster_sync();   // the sums have been read
        __syncthreads();
        const int rank = sums.before;
        sums = join_all(Sums{0.f, s, t, m, 0}, false);
        sums.before = rank;
    }
    if (crank == 0 && warp == 0) {
        // a row that holds a NaN has a NaN in s, one with a +inf gets it here
        const float s = sums.most == INFINITY ? NAN : sums.s;
        const float ln_s = logf(s), log2_s = log2f(s);
        auto logprob = [&](float v) {
            if (v == -INFINITY) return -INFINITY + s * 0.f;
            if (far) return fmaf(below(v, sums.most) * p.factor, 2.f, -ln_s);
            if (v * c < -kFar) return fmaf(v, p.factor, -(sums.r + log2_s) * kLn2);   // v c may leave fp32's range
            return (fmaf(v, c, -sums.r) - log2_s) * kLn2;
        };
        if (lane == 0) {
            if (p.lse) p.lse[row] = far ? fmaf(sums.most, p.factor, ln_s) : (sums.r + log2_s) * kLn2;
            if (p.entropy) p.entropy[row] = s == 0.f ? 0.f : (log2_s - sums.t / s) * kLn2;
            if (p.logprob) p.logprob[row] = has ? logprob(mine) : 0.f;
            if (p.rank) p.rank[row] = has ? sums.before : -1;
        }
        if (TOP && lane < p.top) {
            int id;
            float v;
            decode_argmax_key(top.best[lane], &id, &v);
            p.top_ids[(long long)row * p.top + lane] = id;
            if (p.top_logprobs) p.top_logprobs[(long long)row * p.top + lane] = logprob(v);
        }
    }
    if (csize > 1) cluster_arrive(), cluster_wait();   // the first CTA may still be reading the others' lists
}

// grad_i = factor * (g_l (i == given) - p_i (g_l + g_e (ln p_i + h))), ln p_i = (x_i - m) factor - l.
// m and l are 0 and lse, whose roundings make at most 2^-22 |lse| of p, where that stays below
// kExactLse.  Beyond, fp32 has no room for l beside x factor (at -1e9, or with a row of nothing
// but the type's lowest value, all of ln V is gone), so one CTA reads the row once more for its
// maximum m and l = ln sum e^((x - m) factor), and writes all of it.  ln p is held at kNoWeight
// from below, where p is 0, so that masked tokens and 0 * -inf need no branch.  Bound by HBM:
// 1024 rows of 262144 bf16 take 156.4 us, 101 % of a copy's rate; 61 rows of 50021 fp32 3.6 us.
// Read once more they take 350 and 15 us (reading a logit at a time 440 and 17).
constexpr int kGradVecs = 4;   // vectors of a thread
constexpr float kExactLse = 1024.f, kNoWeight = -1024.f;

// The row's largest logit and the logarithm of its sum, for every thread of the CTA.  The row is
// `head` scalars, `vecs` vectors and scalars.
template <bool BF16>
__device__ __forceinline__ float2 largest_and_sum(const typename Logits<BF16>::type *x, int vocab, int head, int vecs, float factor)
{
    typedef Logits<BF16> L;
    __shared__ float s_most[kGradThreads / 32], s_sum[kGradThreads / 32];
    const float c = factor * kLog2e;
    const uint4 *base = (const uint4 *)(x + head);
    constexpr int N = 2;   // vectors at a time: more need more registers, and the common rows want six CTAs per SM
    const uint4 masked = make_uint4(L::masked(), L::masked(), L::masked(), L::masked());
    float most = -INFINITY, sum = 0.f;
    auto raise = [&](float to) {
        if (!(to > most)) return;
        sum *= exp2_fast((most - to) * c);   // 0 for the first
        most = to;
    };
#pragma unroll 1
    for (int i0 = threadIdx.x; i0 < vecs; i0 += N * kGradThreads) {
        uint4 v[N];
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = i0 + j * kGradThreads < vecs ? base[i0 + j * kGradThreads] : masked;
        float high = -INFINITY, part[N] = {};
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
            for (int e = 0; e < L::VEC; ++e) high = fmaxf(high, element<BF16>(v[j], e));
        raise(high);
        const float from = most == -INFINITY ? 0.f : most;
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
            for (int e = 0; e < L::VEC; ++e) part[j] += exp2_fast((element<BF16>(v[j], e) - from) * c);
#pragma unroll
        for (int j = 0; j < N; ++j) sum += part[j];
    }
    auto one = [&](int i) {
        const float v = L::value(x[i]);
        raise(v);
        sum += v == -INFINITY ? 0.f : exp2_fast((v - most) * c);
    };
    if (threadIdx.x < head) one(threadIdx.x);
    if (threadIdx.x < vocab - head - vecs * L::VEC) one(head + vecs * L::VEC + threadIdx.x);
    auto join = [&](float m, float s) {
        const float up = fmaxf(most, m);
        sum = (most == up ? sum : sum * exp2_fast((most - up) * c)) + (m == up ? s : s * exp2_fast((m - up) * c));
        most = up;
    };
    for (int o = 16; o > 0; o >>= 1) join(__shfl_xor_sync(~0u, most, o), __shfl_xor_sync(~0u, sum, o));
    if (threadIdx.x % 32 == 0) s_most[threadIdx.x / 32] = most, s_sum[threadIdx.x / 32] = sum;
    __syncthreads();
    most = s_most[0], sum = s_sum[0];
    for (int w = 1; w < kGradThreads / 32; ++w) join(s_most[w], s_sum[w]);
    return make_float2(most, logf(sum));
}

template <bool BF16> __global__ void __launch_bounds__(kGradThreads, 6) k_token_logprobs_backward(LogprobGradParams p)
{
    typedef Logits<BF16> L;
    typedef typename L::type T;
    constexpr int VEC = L::VEC;
    const int row = blockIdx.x;
    wait_for_previous();
    const T *x = (const T *)p.logits + row * p.ld;
    T *g = (T *)p.grad + row * p.ld_grad;
    const int head = min(p.vocab, (int)((16 - ((uintptr_t)x & 15)) % 16 / sizeof(T)));
    const int vecs = (p.vocab - head) / VEC, tail = head + vecs * VEC;
    const bool together = (((uintptr_t)x ^ (uintptr_t)g) & 15) == 0;   // both on 16-byte boundaries at once
    constexpr int each = kGradVecs * kGradThreads;
    uint4 in[kGradVecs];
    auto load = [&](int v0) {
#pragma unroll
        for (int j = 0; j < kGradVecs; ++j) {
            const int i = v0 + j * kGradThreads + threadIdx.x;
            if (i < vecs) in[j] = __ldcs((const uint4 *)(x + head) + i);
        }
    };
    load(blockIdx.y * each);
    const float lse_in = __ldg(p.lse + row);
    const bool far = fabsf(lse_in) >= kExactLse && lse_in != -INFINITY;
    float most = 0.f, lse = lse_in == -INFINITY ? 0.f : lse_in;   // nothing but masked tokens: all 0
    if (far) {
        if (blockIdx.y > 0) return;
        const float2 exact = largest_and_sum<BF16>(x, p.vocab, head, vecs, p.factor);   // every read is before the first write
        most = exact.x, lse = exact.y;
        load(0);   // again: the first need not stay in registers meanwhile
    }
    const int stride = far ? each : gridDim.y * each;
    const int given = p.tokens ? __ldg(p.tokens + row) : -1;
    const float hot = p.grad_logprob && given >= 0 && given < p.vocab ? __ldg(p.grad_logprob + row) * p.factor : 0.f;
    const float ge = p.grad_entropy ? -__ldg(p.grad_entropy + row) * p.factor : 0.f;
    const float gl = (p.grad_entropy ? ge * __ldg(p.entropy + row) : 0.f) - hot;
    auto pair_of = [&](float a, float b) {   // the gradient of two logits, the given one's 1 apart
        if (far) a -= most, b -= most;
        const float2 l = unpair(fma2(pair(a, b), pair(p.factor, p.factor), pair(-lse, -lse)));
        const u64 d = pair(max_nan(l.x, kNoWeight), max_nan(l.y, kNoWeight));
        const float2 e = unpair(mul2(d, pair(kLog2e, kLog2e)));
        return mul2(pair(exp2_fast(e.x), exp2_fast(e.y)), fma2(d, pair(ge, ge), pair(gl, gl)));
    };
    auto put = [&](T *to, float v) {
        if constexpr (BF16)
            *to = bf16_bits(v);
        else
            *to = v;
    };
    auto one = [&](int i) {
        const float v = L::value(x[i]);
        float r = unpair(pair_of(v, 0.f)).x;
        if (i == given && v != -INFINITY) r += hot;
        put(g + i, r);
    };
    if (blockIdx.y == 0) {
        if (threadIdx.x < head) one(threadIdx.x);
        if (threadIdx.x < p.vocab - tail) one(tail + threadIdx.x);
    }
    for (int v0 = blockIdx.y * each; v0 < vecs; load(v0 += stride)) {
#pragma unroll
        for (int j = 0; j < kGradVecs; ++j) {
            const int i = v0 + j * kGradThreads + threadIdx.x, id = head + i * VEC;
            if (i >= vecs) break;
            float r[VEC];
#pragma unroll
            for (int e = 0; e < VEC; e += 2) {
                const float2 u = unpair(pair_of(element<BF16>(in[j], e), element<BF16>(in[j], e + 1)));
                r[e] = u.x, r[e + 1] = u.y;
            }
            if (given >= id && given < id + VEC) {
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    if (id + e == given && element<BF16>(in[j], e) != -INFINITY) r[e] += hot;
            }
            if (together) {
                uint4 out;
                if (BF16) {
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[e]) : "f"(r[(2 * e + 1) % VEC]), "f"(r[2 * e % VEC]));
                    out = make_uint4(w[0], w[1], w[2], w[3]);
                } else {
                    out = make_uint4(__float_as_uint(r[0]), __float_as_uint(r[1]), __float_as_uint(r[2]), __float_as_uint(r[3]));
                }
                __stcs((uint4 *)(g + id), out);
            } else {
#pragma unroll
                for (int e = 0; e < VEC; ++e) put(g + id + e, r[e]);
            }
        }
    }
}

template <bool BF16, bool TOP, int W> cudaError_t launch_logprobs(const LogprobParams &p, cudaStream_t s)
{
    // CTAs of a row: as many as are resident at once for all rows, of two tiles each at least.
    // Clusters do not fit the last 15 % of the places, and a second wave costs more (rows of
    // 262144 with 20 alternatives; 100 in fp32: 24.3 us with four CTAs, 35.1 with six; 320 in
    // bf16: 42.2 with three, 43.9 with two, 45.0 with four; 64 in fp32: 19.7 with eight, 20.3
    // with four; one masked row: 9.4 with eight, 11.2 with four)
    const long long tile = W * 32 * kVecs * (BF16 ? 8 : 4), slots = 32ll / W * sm_count();
    const int cluster = (int)std::max(1ll, std::min({8ll, slots * 85 / 100 / p.rows, p.vocab / (2 * tile)}));
    return launch_clusters(k_token_logprobs<BF16, TOP, W>, dim3((unsigned)p.rows * cluster), dim3(W * 32), cluster, 0, s, p);
}

// Many rows: CTAs of four warps, whose searches for alternatives hold up less (2000 rows of
// 32003 bf16: 40.8 us, with eight warps 49.4; 320 of 262144: 42.0 and 47.6).  Few: eight (64
// rows of 262144 fp32: 19.7 us, with four warps 21.1; one row: 9.4 and 11.1).
template <bool BF16, bool TOP> cudaError_t launch_logprobs_rows(const LogprobParams &p, cudaStream_t s)
{
    return p.rows > 2 * sm_count() ? launch_logprobs<BF16, TOP, 4>(p, s) : launch_logprobs<BF16, TOP, 8>(p, s);
}

}  // namespace

cudaError_t launch_token_logprobs(const LogprobParams &p, bool bf16, cudaStream_t s)
{
    if (bf16) return p.top ? launch_logprobs_rows<true, true>(p, s) : launch_logprobs_rows<true, false>(p, s);
    return p.top ? launch_logprobs_rows<false, true>(p, s) : launch_logprobs_rows<false, false>(p, s);
}

cudaError_t launch_token_logprobs_backward(const LogprobGradParams &p, bool bf16, cudaStream_t s)
{
    const long long each = (long long)kGradThreads * kGradVecs * (bf16 ? 8 : 4);
    const dim3 grid(p.rows, (unsigned)std::min((p.vocab + each - 1) / each, 65535ll));
    if (bf16)
        return launch_dependent(k_token_logprobs_backward<true>, grid, dim3(kGradThreads), 0, s, p);
    return launch_dependent(k_token_logprobs_backward<false>, grid, dim3(kGradThreads), 0, s, p);
}

}  // namespace mtp
