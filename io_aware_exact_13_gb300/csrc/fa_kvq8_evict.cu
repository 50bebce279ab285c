// fa_kvq8_evict.cu -- the 8-bit cache cut down to a budget of keys by the weight that they have received.
//
// Selection. Of a sequence's n > keep positions each K/V head keeps the last `recent` and, of the earlier ones, the
// keep - recent of the greatest weight (ties: the lower position; NaN counts as the greatest). The weights are mapped to
// integers of the same order, and T, the smallest that is kept, is found by counting how many reach a trial value, which is
// placed by turns where an even spread would have it and in the middle of what is left (about 10 counts for
// weights of a smooth distribution, 32 each way at most). All above T stay and, in order of position, as many equal to T as are missing. So the result
// does not depend on timing.
//
// Moving. The kept tokens go, in their order, to positions 0 .. keep - 1 of the same pages, in place. A page whose tokens
// all stay where they are is left alone. Any other page gets the scale that an append of its tokens to an empty page
// would give it, the smallest power of two that holds them, and their codes rounded to it.
// In place is safe in rounds: token r of the new order comes from a position >= r, so what a round writes, positions
// [r0, r1), no later round reads. A round's own CTAs read all of it before any of them writes (a barrier of the CTA, or of
// the cluster that shares a head's tokens).
//
// Bound: HBM, the kept tokens that move read and written once; for few sequences latency.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <float.h>
#include <stdint.h>

#include "fa_kvq8.cuh"
#include "pdl.cuh"
#include "ptx.cuh"

namespace fa {
namespace {

struct EvictParams {
    uint8_t *codes[2];
    float *scale[2];
    const int *page_table, *kv_lens;
    const float *weight;
    float *weight_out;
    int *lens_out, *kept, *status;
    int n_pages, max_pages, page_shift, Hkv, keep, recent, cluster;
};

__device__ __forceinline__ int evict_len(const EvictParams &p, int b, bool &bad) {
    const int len = __ldg(p.kv_lens + b);
    bad = len < 0 || len > (p.max_pages << p.page_shift);
    return bad ? 0 : len;
}

// Integers of the weights' order; NaN above all, -0 with 0.
__device__ __forceinline__ uint32_t order_of(float w) {
    const uint32_t u = __float_as_uint(w + 0.0f);
    return isnan(w) ? 0xFFFFFFFFu : (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

constexpr int kSelThreads = 1024;
constexpr int kSelEach = 16;  // consecutive positions of a thread
constexpr int kSelChunk = kSelThreads * kSelEach;

// Sum over the CTA; every thread gets it. Two buffers in turn, so one barrier a call.
struct BlockSum {
    int (*buf)[kSelThreads / 32];
    int turn;
    __device__ __forceinline__ int operator()(int x) {
        x = __reduce_add_sync(0xffffffffu, x);
        int *s = buf[turn];
        turn ^= 1;
        if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = x;
        __syncthreads();
        return __reduce_add_sync(0xffffffffu, s[threadIdx.x & 31]);
    }
};

// One CTA for each (sequence, head): the kept positions in order, the weights that go with them, the new length. Up to
// kSelChunk positions stay in registers; longer sequences are read again for every bit.
__global__ void __launch_bounds__(kSelThreads) fa_kvq8_select_kernel(const EvictParams p) {
    __shared__ int sums[2][kSelThreads / 32];
    __shared__ int offs[kSelThreads / 32];
    __shared__ uint32_t ends[2][kSelThreads / 32];
    grid_launch_dependents();
    const int b = blockIdx.x / p.Hkv, head = blockIdx.x - b * p.Hkv;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    bool bad;
    const int n = evict_len(p, b, bad);
    if (threadIdx.x == 0 && head == 0) {
        if (bad) atomicExch(p.status, kStatusSeqlensQ8);
        p.lens_out[b] = min(n, p.keep);
    }
    const size_t cap = (size_t)p.max_pages << p.page_shift;
    const float *w = p.weight + (size_t)blockIdx.x * cap;
    float *w_out = p.weight_out + (size_t)blockIdx.x * cap;
    int *kept = p.kept + (size_t)blockIdx.x * p.keep;
    const int stay = min(n, p.keep);
    for (size_t i = (size_t)stay + threadIdx.x; i < cap; i += kSelThreads) w_out[i] = 0.f;
    for (int i = stay + threadIdx.x; i < p.keep; i += kSelThreads) kept[i] = -1;
    if (n <= p.keep) {
        for (int i = threadIdx.x; i < n; i += kSelThreads) {
            w_out[i] = w[i];
            kept[i] = i;
        }
        return;
    }
    const int old = n - p.recent, need = p.keep - p.recent;  // 0 <= need < old
    for (int i = threadIdx.x; i < p.recent; i += kSelThreads) {
        w_out[need + i] = w[old + i];
        kept[need + i] = old + i;
    }
    if (need == 0) return;

    uint32_t v[kSelEach];
    auto load = [&](int c0) {  // 0, below every weight, for positions past `old`
        const int at = c0 + threadIdx.x * kSelEach;
#pragma unroll
        for (int i = 0; i < kSelEach; i += 4) {
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (at + i < old) x = *reinterpret_cast<const float4 *>(w + at + i);  // cap is a multiple of 16
            v[i] = at + i < old ? order_of(x.x) : 0u;
            v[i + 1] = at + i + 1 < old ? order_of(x.y) : 0u;
            v[i + 2] = at + i + 2 < old ? order_of(x.z) : 0u;
            v[i + 3] = at + i + 3 < old ? order_of(x.w) : 0u;
        }
    };
    const bool once = old <= kSelChunk;
    BlockSum sum{sums, 0};
    // T lies in [lo, hi]: n_lo >= need reach lo, above < need exceed hi
    uint32_t lo = 0xFFFFFFFFu, hi = 0;
    for (int c0 = 0; c0 < old; c0 += kSelChunk) {
        load(c0);
#pragma unroll
        for (int i = 0; i < kSelEach; ++i) {
            hi = max(hi, v[i]);
            if (v[i] != 0u) lo = min(lo, v[i]);
        }
    }
    lo = ~__reduce_max_sync(0xffffffffu, ~lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (lane == 0) {
        ends[0][warp] = lo;
        ends[1][warp] = hi;
    }
    __syncthreads();
    lo = __reduce_min_sync(0xffffffffu, ends[0][lane]);
    hi = __reduce_max_sync(0xffffffffu, ends[1][lane]);
    int n_lo = old, above = 0;
    for (bool halve = false; lo < hi; halve = !halve) {
        // by turns where the count would be reached if it fell evenly, and the middle
        const uint32_t gap = hi - lo;
        uint32_t t = lo + gap / 2 + 1;
        if (!halve) {
            const float share = (float)(n_lo - need) / (float)(n_lo - above);
            t = lo + 1 + min((uint32_t)(share * (float)gap), gap - 1);
        }
        int count = 0;
        for (int c0 = 0; c0 < old; c0 += kSelChunk) {
            if (!once) load(c0);
#pragma unroll
            for (int i = 0; i < kSelEach; ++i) count += v[i] >= t;
        }
        count = sum(count);
        if (count >= need) lo = t, n_lo = count;
        else hi = t - 1, above = count;
        if (count == need) {  // exactly those that reach t
            lo = t - 1;
            above = need;
            break;
        }
    }
    const uint32_t T = lo;
    // in order of position
    int taken = 0, equal_left = need - above;
    for (int c0 = 0; c0 < old; c0 += kSelChunk) {
        if (!once) load(c0);
        const int at = c0 + threadIdx.x * kSelEach;
        int mine = 0;  // above T, and equal to it << 16
#pragma unroll
        for (int i = 0; i < kSelEach; ++i) {
            mine += (v[i] > T) + ((v[i] == T) << 16);
        }
        int incl = mine;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int x = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += x;
        }
        __syncthreads();
        if (lane == 31) offs[warp] = incl;
        __syncthreads();
        int part = offs[lane], scan = part;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int x = __shfl_up_sync(0xffffffffu, scan, d);
            if (lane >= d) scan += x;
        }
        const int total = __shfl_sync(0xffffffffu, scan, 31);
        const int before = __shfl_sync(0xffffffffu, scan - part, warp) + incl - mine;
        int gt = before & 0xFFFF, eq = before >> 16;  // each at most kSelChunk = 2^14
#pragma unroll
        for (int i = 0; i < kSelEach; ++i) {
            if (v[i] > T || (v[i] == T && eq < equal_left)) {
                const int r = taken + gt + min(eq, equal_left);
                kept[r] = at + i;
                w_out[r] = w[at + i];
            }
            gt += v[i] > T;
            eq += v[i] == T;
        }
        taken += (total & 0xFFFF) + min(total >> 16, equal_left);
        equal_left -= min(total >> 16, equal_left);
    }
}

constexpr int kMoveThreads = 256;
constexpr int kMoveTokens = 128;  // tokens of a CTA's round: one page at least
constexpr int kMostCluster = 8;

__device__ __forceinline__ void cluster_barrier() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ float2 half2_at(uint32_t h) { return __half22float2(*reinterpret_cast<const __half2 *>(&h)); }

// One CTA, or a cluster of them, for each (sequence, head, K or V): the kept tokens in rounds of kMoveTokens for each
// CTA. A warp holds 16 tokens in registers, so a page of 16 has its largest value in one warp.
template <int D, int FMT>
__global__ void __launch_bounds__(kMoveThreads) fa_kvq8_move_kernel(const EvictParams p) {
    constexpr int LANES = D / 16;                                   // 16-byte vectors of a token
    constexpr int PER = 32 / LANES;                                 // tokens of a warp's load
    constexpr int VEC = 16 / PER;                                   // loads of a warp
    constexpr int GROUPS = kMoveTokens / 16;                        // of 16 tokens, one for each warp
    static_assert(GROUPS == kMoveThreads / 32, "a group of 16 tokens for each warp");
    __shared__ float top[2][GROUPS];  // largest magnitudes, by turns
    const int rank = blockIdx.x % p.cluster;
    int u = blockIdx.x / p.cluster;
    const int kv = u & 1;
    u >>= 1;
    const int head = u % p.Hkv, b = u / p.Hkv;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    bool bad;
    const int n = evict_len(p, b, bad);
    if (n <= p.keep) return;  // the same in the whole cluster
    grid_dependency_wait();
    const int *kept = p.kept + ((size_t)b * p.Hkv + head) * p.keep;
    const int *table = p.page_table + (size_t)b * p.max_pages;
    const int page = 1 << p.page_shift, per_page = page / 16;  // groups of a page
    const int round = kMoveTokens * p.cluster, rounds = (p.keep + round - 1) / round;
    // The first round with a token that moves (all behind it move too), and the last one.
    int first_round = 0;
    for (int end = rounds; first_round < end;) {
        const int mid = (first_round + end) / 2, last = min((mid + 1) * round, p.keep) - 1;
        if (kept[last] == last) first_round = mid + 1;
        else end = mid;
    }
    // A round's codes and scales are requested while the round before is under way, its positions one round earlier.
    int pos[VEC];
    uint4 x[VEC], ahead[VEC];
    float s[VEC], s_ahead[VEC];
    auto load_pos = [&](int i_round) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const int r = i_round * round + rank * kMoveTokens + warp * 16 + i * PER + lane / LANES;
            pos[i] = r < p.keep && i_round < rounds ? kept[r] : -1;
        }
    };
    auto load_codes = [&]() {
        int phys[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) phys[i] = pos[i] < 0 ? -1 : __ldg(table + (pos[i] >> p.page_shift));
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            ahead[i] = make_uint4(0u, 0u, 0u, 0u);
            s_ahead[i] = 0.f;
            if (phys[i] >= 0 && phys[i] < p.n_pages) {
                const size_t unit = (size_t)phys[i] * p.Hkv + head;
                s_ahead[i] = p.scale[kv][unit];
                ahead[i] = *reinterpret_cast<const uint4 *>(p.codes[kv] + ((unit << p.page_shift) + (pos[i] & (page - 1))) * D + (lane % LANES) * 16);
            } else if (pos[i] >= 0) {
                atomicExch(p.status, kStatusPage);  // such a token becomes zeros
            }
        }
    };
    load_pos(first_round);
    load_codes();
    load_pos(first_round + 1);
    int turn = 0;
    for (int i_round = first_round; i_round < rounds; ++i_round, turn ^= 1) {
        const int g0 = i_round * round + rank * kMoveTokens + warp * 16;  // this warp's tokens of the new order
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            x[i] = ahead[i];
            s[i] = s_ahead[i];
        }
        // (no round writes what a later one reads, so these may run ahead of this round's writes)
        load_codes();
        load_pos(i_round + 2);
        float most = 0.f;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
            __half2 m = __half2half2(__ushort_as_half(0));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                uint32_t lo, hi;
                codes_to_half2<FMT>(w[e], lo, hi);
                m = __hmax2(m, __hmax2(__habs2(*reinterpret_cast<__half2 *>(&lo)), __habs2(*reinterpret_cast<__half2 *>(&hi))));
            }
            const float code = fmaxf(__low2float(m), __high2float(m));
            most = fmaxf(most, code * s[i] > FLT_MAX ? FLT_MAX : product_odd(code, s[i]));
        }
        const float group_most = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(most)));
        if (lane == 0) top[turn][warp] = group_most;
        // every read of the round before its first write
        if (p.cluster > 1) cluster_barrier();
        __syncthreads();
        const int g_page = warp / per_page * per_page;  // the page's first group in this CTA
        float page_most = 0.f;
        for (int i = 0; i < per_page; ++i) page_most = fmaxf(page_most, top[turn][g_page + i]);
        const int first = g0 & ~(page - 1), page_last = min(first + page, p.keep) - 1;
        if (g0 >= p.keep || kept[page_last] == page_last) continue;  // (warp-uniform) no token of the page moves
        const int phys = __ldg(table + (first >> p.page_shift));
        if (phys < 0 || phys >= p.n_pages) {
            if (lane == 0) atomicExch(p.status, kStatusPage);
            continue;
        }
        const size_t unit = (size_t)phys * p.Hkv + head;
        const float now = scale_for<FMT>(page_most);
        const float inv = now > 0.f ? 1.0f / now : 0.f;
        if (warp == g_page && lane == 0) p.scale[kv][unit] = now;
        uint8_t *dst = p.codes[kv] + ((unit << p.page_shift) + (g0 & (page - 1))) * D;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const int t = i * PER + lane / LANES;
            if (g0 + t >= p.keep) continue;
            uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
            if (s[i] != now || now == 0.f) {
                // (a token of zeros may have come under a scale far above the page's)
                const float ratio = fminf(s[i] * inv, 512.0f);
                const bool exact = power_of_two(s[i]);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    uint32_t lo, hi;
                    codes_to_half2<FMT>(w[e], lo, hi);
                    const float2 a = half2_at(lo), c = half2_at(hi);
                    w[e] = exact ? encode4<FMT>(a.x * ratio, a.y * ratio, c.x * ratio, c.y * ratio)
                                 : encode4<FMT>(product_odd(a.x, ratio), product_odd(a.y, ratio), product_odd(c.x, ratio),
                                                product_odd(c.y, ratio));
                }
            }
            *reinterpret_cast<uint4 *>(dst + t * D + (lane % LANES) * 16) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

template <int D, int FMT>
int launch_move(const Kvq8EvictArgs &a, EvictParams p) {
    // A cluster for each head's K or V while there are fewer CTAs than the GPU holds at once, with a round for each CTA.
    const long long units = 2ll * a.nseq * a.c.Hkv;
    p.cluster = 1;
    while (2 * p.cluster <= kMostCluster && 2 * p.cluster * units <= 4ll * a.num_sms && p.cluster * kMoveTokens < a.keep) p.cluster *= 2;
    const long long grid = units * p.cluster;
    if (grid > INT32_MAX) return -3;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kMoveThreads);
    cfg.stream = a.stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = p.cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, fa_kvq8_move_kernel<D, FMT>, p) == cudaSuccess ? 0 : -5;
}

}  // namespace

int launch_kvq8_evict(const Kvq8EvictArgs &a) {
    EvictParams p;
    p.codes[0] = a.c.k_codes;
    p.codes[1] = a.c.v_codes;
    p.scale[0] = a.c.k_scale;
    p.scale[1] = a.c.v_scale;
    p.page_table = a.c.page_table;
    p.kv_lens = a.kv_lens;
    p.weight = a.weight;
    p.weight_out = a.weight_out;
    p.lens_out = a.lens_out;
    p.kept = a.kept;
    p.status = a.status;
    p.n_pages = a.c.n_pages;
    p.max_pages = a.c.max_pages;
    p.page_shift = kvq8_page_shift(a.c.page);
    p.Hkv = a.c.Hkv;
    p.keep = a.keep;
    p.recent = a.recent;
    p.cluster = 1;
    const long long grid = (long long)a.nseq * a.c.Hkv;
    if (grid > INT32_MAX) return -3;
    fa_kvq8_select_kernel<<<(unsigned)grid, kSelThreads, 0, a.stream>>>(p);
    if (cudaGetLastError() != cudaSuccess) return -5;
    const bool i8 = a.c.format == kKvq8Int8;
    if (a.c.d == 128) return i8 ? launch_move<128, kKvq8Int8>(a, p) : launch_move<128, kKvq8E4m3>(a, p);
    return i8 ? launch_move<64, kKvq8Int8>(a, p) : launch_move<64, kKvq8E4m3>(a, p);
}

}  // namespace fa
