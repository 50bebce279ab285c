// fa_kvq8_evict.cu -- the 8-bit cache cut down to a budget of keys by the weight that they have received.
//
// Selection. Of a sequence's n > keep positions each K/V head keeps the last `recent` and, of the earlier ones, the
// keep - recent of the greatest weight (ties: the lower position; NaN counts as the greatest). The weights are mapped to
// integers of the same order, and T, the smallest that is kept, is found by histograms of 2048 bins between the least
// and the greatest, then within the bin that the count is reached in, three at most. All above T stay and, in order of
// position, as many equal to T as are missing. So the result does not depend on timing.
//
// Moving. The kept tokens go, in their order, to positions 0 .. keep - 1 of the same pages, in place. A page whose tokens
// all stay where they are is left alone. Any other page gets the scale that an append of its tokens to an empty page
// would give it, the smallest power of two that holds them, and their codes rounded to it.
// In place is safe in rounds: token r of the new order comes from a position >= r, so what a round writes, positions
// [r0, r1), no later round reads. A round's own CTAs read all of it before any of them writes (a barrier of the CTA, or of
// the cluster that shares a head's tokens).
//
// Bound: HBM, the kept tokens that move read and written once; for few sequences latency. Measured: 24 sequences up to 12000
// tokens of 8 heads of 128 cut to 5000, 88 us (15 of them the selection; the moves run at three quarters of the copy rate), one
// of 1500 tokens of 4 heads of 64 cut to 1100, 14.5 us, some ten dependent passes and barriers. With T found bit by bit and a round's
// codes read when they are needed these were 214 and 63 us, with T by trial values and codes read a round ahead into registers
// 150 and 21.
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
    int nseq, n_pages, max_pages, page_shift, Hkv, keep, recent, cluster;
};

__device__ __forceinline__ int evict_len(const EvictParams &p, int b, bool &bad) {
    const int len = __ldg(p.kv_lens + b);
    bad = len < 0 || len > (p.max_pages << p.page_shift);
    return bad ? 0 : len;
}

// Sequences in the order of the CTAs that work on them: those that are cut down first, then the others, so that every SM gets
// as many of the former. Of many sequences the CTAs are many waves that even out by themselves, and each goes by its own place
// (8 heads of 128, so ordered against as they come; half of them cut: 64 from 2000 tokens to 1500 43.5 / 65.1 us, 128 111.6 /
// 111.0, 256 from 1000 to 700 126.5 / 105.1, 4096 from 100 to 64 5201 / 524). All lanes of a warp call.
constexpr int kOrderMost = 128;
__device__ __forceinline__ int nth_sequence(const EvictParams &p, int nth, bool &cut) {
    const int lane = threadIdx.x & 31;
    if (p.nseq > kOrderMost) {
        bool bad;
        cut = evict_len(p, nth, bad) > p.keep;
        return nth;
    }
    int b = -1, before = 0;
    cut = true;
    for (;;) {
        for (int s0 = 0; s0 < p.nseq && b < 0; s0 += 32) {
            bool bad;
            const bool in = s0 + lane < p.nseq;
            uint32_t mine = __ballot_sync(0xffffffffu, in && (evict_len(p, s0 + lane, bad) > p.keep) == cut);
            const int here = __popc(mine);
            if (nth < before + here) {
                for (int i = before; i < nth; ++i) mine &= mine - 1u;
                b = s0 + __ffs(mine) - 1;
            }
            before += here;
        }
        if (b >= 0 || !cut) return b;
        cut = false;
    }
}

// Integers of the weights' order; NaN above all, -0 with 0.
__device__ __forceinline__ uint32_t order_of(float w) {
    const uint32_t u = __float_as_uint(w + 0.0f);
    return isnan(w) ? 0xFFFFFFFFu : (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
// And back; all NaN are one.
__device__ __forceinline__ float weight_of(uint32_t v) { return __uint_as_float(v & 0x80000000u ? v ^ 0x80000000u : ~v); }

// (With 1024 threads, whose registers spill at two CTAs on an SM, 8 sequences of 8 heads, 8192 tokens to 6144, take 85.1 us for 64.2
// in all, 24 of 6000 to 4000 95.4 for 91.8.)
constexpr int kSelThreads = 512, kSelWarps = kSelThreads / 32;
constexpr int kSelMost = 24576;  // positions whose weights are kept in shared memory (two CTAs on an SM)
constexpr int kBins = 2048, kBinBits = 11;

// One CTA for each (sequence, head): the kept positions in order, the weights that go with them, the new length. Weights
// past the first `held` positions are read again for every count.
__global__ void __launch_bounds__(kSelThreads) fa_kvq8_select_kernel(const EvictParams p, int held) {
    extern __shared__ uint4 order_sm[];  // [held / 4] integers of the weights' order
    __shared__ __align__(16) int bins[kBins];  // from the top down; read four at a time
    __shared__ int sums[kSelWarps];
    __shared__ int2 found[kSelWarps];
    __shared__ int hit[3];
    __shared__ uint32_t ends[2][kSelWarps];
    // (The moving kernel's CTAs are not let in before these have left: beside them they would be spread unevenly.)
    bool cut;
    const int b = nth_sequence(p, blockIdx.x / p.Hkv, cut), head = blockIdx.x % p.Hkv;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    bool bad;
    const int n = evict_len(p, b, bad);
    if (threadIdx.x == 0 && head == 0) {
        if (bad) atomicExch(p.status, kStatusSeqlensQ8);
        p.lens_out[b] = min(n, p.keep);
    }
    const size_t cap = (size_t)p.max_pages << p.page_shift;
    const float *w = p.weight + ((size_t)b * p.Hkv + head) * cap;
    float *w_out = p.weight_out + ((size_t)b * p.Hkv + head) * cap;
    int *kept = p.kept + ((size_t)b * p.Hkv + head) * p.keep;
    const int stay = min(n, p.keep);
    const int old = n - p.recent, need = p.keep - p.recent;  // 0 <= need < old where n > keep
    // the integers' ends: T lies in [lo, hi]
    uint32_t lo = 0xFFFFFFFFu, hi = 0;
    if (n > p.keep && need > 0) {
#pragma unroll 4
        for (int i = threadIdx.x; i < (old + 3) / 4; i += kSelThreads) {
            const float4 x = __ldg(reinterpret_cast<const float4 *>(w) + i);  // cap is a multiple of 16
            uint32_t v[4] = {order_of(x.x), order_of(x.y), order_of(x.z), order_of(x.w)};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (4 * i + e >= old) v[e] = 0u;  // below every weight
                else lo = min(lo, v[e]);
                hi = max(hi, v[e]);
            }
            if (4 * i < held) order_sm[i] = make_uint4(v[0], v[1], v[2], v[3]);
        }
    }
    for (size_t i = (size_t)stay + threadIdx.x; i < cap; i += kSelThreads) w_out[i] = 0.f;
    for (int i = stay + threadIdx.x; i < p.keep; i += kSelThreads) kept[i] = -1;
    if (n <= p.keep) {
        for (int i = threadIdx.x; i < n; i += kSelThreads) {
            w_out[i] = w[i];
            kept[i] = i;
        }
        return;
    }
    for (int i = threadIdx.x; i < p.recent; i += kSelThreads) {
        w_out[need + i] = w[old + i];
        kept[need + i] = old + i;
    }
    if (need == 0) return;
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (lane == 0) {
        ends[0][warp] = lo;
        ends[1][warp] = hi;
    }
    __syncthreads();
    lo = __reduce_min_sync(0xffffffffu, ends[0][lane & (kSelWarps - 1)]);
    hi = __reduce_max_sync(0xffffffffu, ends[1][lane & (kSelWarps - 1)]);

    // Four positions' integers, 0 past `old`.
    auto four = [&](int i4) {
        if (4 * i4 < held) return order_sm[i4];
        const float4 x = __ldg(reinterpret_cast<const float4 *>(w) + i4);
        const int i = 4 * i4;
        return make_uint4(i < old ? order_of(x.x) : 0u, i + 1 < old ? order_of(x.y) : 0u, i + 2 < old ? order_of(x.z) : 0u,
                          i + 3 < old ? order_of(x.w) : 0u);
    };
    const int fours = (old + 3) / 4;
    int above = 0;  // how many exceed hi: fewer than need
    uint32_t T = lo;
    while (lo < hi) {
        const int shift = max(0, 32 - __clz(hi - lo) - kBinBits);
        const int top_bin = (int)((hi - lo) >> shift);
        for (int i = threadIdx.x; i < kBins; i += kSelThreads) bins[i] = 0;
        __syncthreads();
        auto count = [&](uint32_t v) {
            if (v >= lo && v <= hi) atomicAdd(bins + (top_bin - (int)((v - lo) >> shift)), 1);
        };
#pragma unroll 2
        for (int i = threadIdx.x; i < fours; i += kSelThreads) {
            const uint4 v = four(i);
            count(v.x);
            count(v.y);
            count(v.z);
            count(v.w);
        }
        __syncthreads();
        const int4 c = reinterpret_cast<const int4 *>(bins)[threadIdx.x];
        const int mine = c.x + c.y + c.z + c.w;
        int incl = mine;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int x = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += x;
        }
        if (lane == 31) sums[warp] = incl;
        __syncthreads();
        int before = above + incl - mine;
        for (int i = 0; i < warp; ++i) before += sums[i];
        if (before < need && need <= before + mine) {  // one thread: the bin that the count is reached in
            const int each[4] = {c.x, c.y, c.z, c.w};
            int k = 0;
            while (before + each[k] < need) before += each[k++];
            hit[0] = 4 * threadIdx.x + k;
            hit[1] = before;
            hit[2] = each[k];
        }
        __syncthreads();
        lo += (uint32_t)(top_bin - hit[0]) << shift;
        hi = lo + min(hi - lo, (1u << shift) - 1u);  // (the top bin's end may lie past 2^32, where NaN's integer is hi)
        above = hit[1];
        T = lo;
        if (above + hit[2] == need) {  // all that reach lo
            above = need;
            T = lo - 1;
            break;
        }
    }
    // In order of position: a warp takes a run of 128-position groups, first counting its weights above and equal to T.
    const int groups = (fours + 31) / 32, g0 = (int)((long long)warp * groups / kSelWarps);
    const int g1 = (int)((long long)(warp + 1) * groups / kSelWarps);
    auto group = [&](int g) { return 32 * g + lane < fours ? four(32 * g + lane) : make_uint4(0u, 0u, 0u, 0u); };
    int gt = 0, eq = 0;
    for (int g = g0; g < g1; ++g) {
        const uint4 v = group(g);
        gt += (v.x > T) + (v.y > T) + (v.z > T) + (v.w > T);
        eq += (v.x == T) + (v.y == T) + (v.z == T) + (v.w == T);
    }
    gt = __reduce_add_sync(0xffffffffu, gt);
    eq = __reduce_add_sync(0xffffffffu, eq);
    if (lane == 0) found[warp] = make_int2(gt, eq);
    __syncthreads();
    gt = eq = 0;
    for (int i = 0; i < warp; ++i) gt += found[i].x, eq += found[i].y;
    const int equal = need - above;  // how many of those equal to T stay
    const uint32_t below = (1u << lane) - 1u;
    for (int g = g0; g < g1; ++g) {
        const uint4 q = group(g);
        const uint32_t v[4] = {q.x, q.y, q.z, q.w};
        int my_gt = gt, my_eq = eq;  // before this lane's first
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t is_gt = __ballot_sync(0xffffffffu, v[e] > T), is_eq = __ballot_sync(0xffffffffu, v[e] == T);
            my_gt += __popc(is_gt & below);
            my_eq += __popc(is_eq & below);
            gt += __popc(is_gt);
            eq += __popc(is_eq);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (v[e] > T || (v[e] == T && my_eq < equal)) {
                const int r = my_gt + min(my_eq, equal);
                kept[r] = 4 * (32 * g + lane) + e;
                w_out[r] = weight_of(v[e]);
            }
            my_gt += v[e] > T;
            my_eq += v[e] == T;
        }
    }
}

constexpr int kMoveThreads = 256;
constexpr int kMoveTokens = 128;  // tokens of a CTA's round: one page at least
constexpr int kStages = 4;
constexpr int kMostCluster = 8;

__device__ __forceinline__ void cluster_arrive() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// As cp_async16 (ptx.cuh), four bytes.
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src, uint32_t src_bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}

__device__ __forceinline__ __half2 half2_of(uint32_t h) { return *reinterpret_cast<const __half2 *>(&h); }
constexpr float kMostRatio = 0x1p15f;  // the largest power of two in fp16
// Four codes (as fp16) times the power of two r, rounded to codes once, where no product is past the largest code.
// int8: code r + 1536 in one rounding is an integer whose low byte is the code's. e4m3: code r is exact in fp16, or below
// 2^-20, where it becomes 0 either way.
template <int FMT>
__device__ __forceinline__ uint32_t rescaled4(__half2 a, __half2 b, __half2 r) {
    if constexpr (FMT == kKvq8Int8) {
        const __half2 magic = __half2half2(__ushort_as_half(0x6600));
        const __half2 x = __hfma2(a, r, magic), y = __hfma2(b, r, magic);
        return __byte_perm(*reinterpret_cast<const uint32_t *>(&x), *reinterpret_cast<const uint32_t *>(&y), 0x6420);
    } else {
        const uint32_t lo = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(__hmul2(a, r)), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(__hmul2(b, r)), __NV_SATFINITE, __NV_E4M3);
        return lo | (hi << 16);
    }
}

// One CTA, or a cluster of them, for each (sequence, head, K or V): the kept tokens in rounds of kMoveTokens for each
// CTA, whose codes and scales are copied into a ring in shared memory kStages - 1 rounds ahead. (No round writes what a later
// one reads, so the copies may run ahead of the writes.) A warp has 16 tokens of a round, so a page of 16 has its largest
// value in one warp; every thread works on what it copied itself.
template <int D, int FMT>
__global__ void __launch_bounds__(kMoveThreads, 3) fa_kvq8_move_kernel(const __grid_constant__ EvictParams p) {
    constexpr int LANES = D / 16;             // 16-byte vectors of a token
    constexpr int PER = 32 / LANES;           // tokens of a warp's load
    constexpr int VEC = 16 / PER;             // loads of a warp
    constexpr int GROUPS = kMoveTokens / 16;  // of 16 tokens, one for each warp
    static_assert(GROUPS == kMoveThreads / 32, "a group of 16 tokens for each warp");
    extern __shared__ uint4 ring_sm[];  // uint8_t[kStages][kMoveTokens][D]
    __shared__ float ring_scale[kStages][kMoveTokens];
    __shared__ float top[2][GROUPS];  // largest magnitudes, by turns
    const int rank = blockIdx.x % p.cluster;
    int u = blockIdx.x / p.cluster;
    const int kv = u & 1;
    u >>= 1;
    const int head = u % p.Hkv, nth = u / p.Hkv;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    bool cut;
    const int b = nth_sequence(p, nth, cut);
    grid_dependency_wait();  // (before any return: what comes behind this kernel comes behind the selection too)
    if (!cut) return;        // the same in the whole cluster
    const int *kept = p.kept + ((size_t)b * p.Hkv + head) * p.keep;
    const int *table = p.page_table + (size_t)b * p.max_pages;
    const int page = 1 << p.page_shift, per_page = page / 16;  // groups of a page
    const int round = kMoveTokens * p.cluster, rounds = (p.keep + round - 1) / round;
    // The first round with a token that moves (all behind it move too).
    int first_round = 0;
    for (int end = rounds; first_round < end;) {
        const int mid = (first_round + end) / 2, last = min((mid + 1) * round, p.keep) - 1;
        if (kept[last] == last) first_round = mid + 1;
        else end = mid;
    }
    // Every global read is used an iteration after it is requested: positions five rounds ahead, their pages four, codes
    // and scales three; where this warp's tokens go to, and whether they move, one. Lane t < 16 looks after token t.
    int pos = -1, pos_of = -1, phys = -1;  // a position, and the one that the page belongs to
    auto load_pos = [&](int i_round) {
        const int r = i_round * round + rank * kMoveTokens + warp * 16 + lane;
        pos = lane < 16 && i_round < rounds && r < p.keep ? kept[r] : -1;
    };
    auto load_pages = [&]() {
        pos_of = pos;
        phys = pos < 0 ? -1 : __ldg(table + (pos >> p.page_shift));
    };
    const uint8_t *codes = p.codes[kv] + (lane % LANES) * 16;
    const float *scale = p.scale[kv];
    const uint32_t ring_at = smem_u32(ring_sm) + (warp * 16 + lane / LANES) * D + (lane % LANES) * 16;
    auto copy = [&](int stage) {
        const bool there = phys >= 0 && phys < p.n_pages;
        if (!there && pos_of >= 0) atomicExch(p.status, kStatusPage);  // such a token becomes zeros
        const size_t unit = there ? (size_t)phys * p.Hkv + head : 0;
        const size_t row = there ? (unit << p.page_shift) + (pos_of & (page - 1)) : ~(size_t)0;
        if (lane < 16) cp_async4(smem_u32(&ring_scale[stage][warp * 16 + lane]), scale + unit, there ? 4u : 0u);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const size_t from = __shfl_sync(0xffffffffu, row, i * PER + lane / LANES);
            cp_async16(ring_at + stage * (kMoveTokens * D) + i * PER * D, codes + (from == ~(size_t)0 ? 0 : from) * D,
                       from == ~(size_t)0 ? 0u : 16u);
        }
        cp_async_commit();
    };
    int to_phys = -1, to_last = 0;
    auto load_to = [&](int i_round) {  // the page that this warp's tokens go to, the old position of its last token
        const int first = (i_round * round + rank * kMoveTokens + warp * 16) & ~(page - 1);
        to_phys = -1, to_last = 0;
        if (i_round < rounds && first < p.keep) {
            to_phys = __ldg(table + (first >> p.page_shift));
            to_last = kept[min(first + page, p.keep) - 1];
        }
    };
    load_pos(first_round);
    load_pages();
    load_pos(first_round + 1);
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) {
        copy(s);
        load_pages();
        load_pos(first_round + s + 2);
    }
    load_to(first_round);
    cp_async_wait<kStages - 2>();  // the first round's copies
    if (p.cluster > 1) cluster_arrive();
    int turn = 0, stage = 0;
    for (int i_round = first_round; i_round < rounds; ++i_round, turn ^= 1, stage = stage + 1 == kStages ? 0 : stage + 1) {
        const int g0 = i_round * round + rank * kMoveTokens + warp * 16;  // this warp's tokens of the new order
        const int dst_phys = to_phys, dst_last = to_last;
        copy(stage == 0 ? kStages - 1 : stage - 1);
        load_pages();
        load_pos(i_round + kStages + 1);
        load_to(i_round + 1);
        __syncwarp();  // the scales were copied by other lanes
        uint32_t x[VEC][8];  // this thread's codes as pairs of fp16
        float s[VEC], top_code[VEC], most = 0.f;
        bool odd = false;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const int t = warp * 16 + i * PER + lane / LANES;
            const uint4 w = ring_sm[(stage * kMoveTokens + t) * LANES + lane % LANES];
            s[i] = ring_scale[stage][t];
            odd |= !power_of_two(s[i]);
            codes_to_half2<FMT>(w.x, x[i][0], x[i][1]);
            codes_to_half2<FMT>(w.y, x[i][2], x[i][3]);
            codes_to_half2<FMT>(w.z, x[i][4], x[i][5]);
            codes_to_half2<FMT>(w.w, x[i][6], x[i][7]);
            __half2 m = __habs2(half2_of(x[i][0]));
#pragma unroll
            for (int e = 1; e < 8; ++e) m = __hmax2(m, __habs2(half2_of(x[i][e])));
            const float code = fmaxf(__low2float(m), __high2float(m));
            most = fmaxf(most, code * s[i]);
            top_code[i] = code;
        }
        odd = __any_sync(0xffffffffu, odd);
        if (odd) {
            most = 0.f;
#pragma unroll
            for (int i = 0; i < VEC; ++i) most = fmaxf(most, top_code[i] * s[i] > FLT_MAX ? FLT_MAX : product_odd(top_code[i], s[i]));
        }
        const float group_most = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(most)));
        if (lane == 0) top[turn][warp] = group_most;
        // Every read of the round before its first write: the cluster's CTAs said so an iteration ago, and say it now of the
        // next round.
        cp_async_wait<kStages - 2>();
        __syncthreads();
        if (p.cluster > 1) {
            cluster_wait();
            cluster_arrive();
        }
        const int g_page = warp / per_page * per_page;  // the page's first group in this CTA
        float page_most = 0.f;
        for (int i = 0; i < per_page; ++i) page_most = fmaxf(page_most, top[turn][g_page + i]);
        const int first = g0 & ~(page - 1), page_last = min(first + page, p.keep) - 1;
        if (g0 >= p.keep || dst_last == page_last) continue;  // (warp-uniform) no token of the page moves
        if (dst_phys < 0 || dst_phys >= p.n_pages) {
            if (lane == 0) atomicExch(p.status, kStatusPage);
            continue;
        }
        const size_t unit = (size_t)dst_phys * p.Hkv + head;
        const float now = scale_for<FMT>(page_most);
        const float inv = now > 0.f ? 1.0f / now : 0.f;
        if (warp == g_page && lane == 0) p.scale[kv][unit] = now;
        uint8_t *dst = p.codes[kv] + ((unit << p.page_shift) + (g0 & (page - 1))) * D + (lane % LANES) * 16;
        // Scales that no append wrote, or values past the largest scale: codes are rounded from fp32.
        const bool slow = odd || page_most > (FMT == kKvq8Int8 ? 127.0f : 448.0f) * 0x1p120f;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const int t = i * PER + lane / LANES;
            // (at most 127 for a code of int8 that is not 0 and 2^18 for one of e4m3, whose smallest is 2^-9 and most often beside
            // a larger one that has gone; a token of zeros may have come under any scale)
            const float ratio = fminf(s[i] * inv, 0x1p18f);
            uint32_t w[4];
            if (!slow && (FMT == kKvq8Int8 || ratio <= kMostRatio || top_code[i] == 0.f)) {
                const __half2 r = __float2half2_rn(fminf(ratio, kMostRatio));  // a power of two, or so small that every code becomes 0
#pragma unroll
                for (int e = 0; e < 4; ++e) w[e] = rescaled4<FMT>(half2_of(x[i][2 * e]), half2_of(x[i][2 * e + 1]), r);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 a = __half22float2(half2_of(x[i][2 * e])), c = __half22float2(half2_of(x[i][2 * e + 1]));
                    w[e] = encode4<FMT>(product_odd(a.x, ratio), product_odd(a.y, ratio), product_odd(c.x, ratio),
                                        product_odd(c.y, ratio));
                }
            }
            if (g0 + t < p.keep) *reinterpret_cast<uint4 *>(dst + t * D) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
    cp_async_wait<0>();
    if (p.cluster > 1) cluster_wait();
}

template <int D, int FMT>
int launch_move(const Kvq8EvictArgs &a, EvictParams p) {
    // A cluster for each head's K or V while there are fewer CTAs than the GPU holds at once, with a round for each CTA. (At most
    // two, four, six, eight for each SM, 8 heads of 128, 8192 tokens to 6144: 8 sequences 60.1 us, 64.2, 64.5, 66.1; 12 94.0,
    // 74.1, 79.2, 79.5; 16 99.3, 113, 112, 102; 24 127.9, 128.3, 134.7, 135.3.)
    const long long units = 2ll * a.nseq * a.c.Hkv;
    p.cluster = 1;
    while (2 * p.cluster <= kMostCluster && 2 * p.cluster * units <= 4ll * a.num_sms && p.cluster * kMoveTokens < a.keep) p.cluster *= 2;
    const long long grid = units * p.cluster;
    if (grid > INT32_MAX) return -3;
    if (!allow_smem<fa_kvq8_move_kernel<D, FMT>>(kStages * kMoveTokens * D)) return -5;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kMoveThreads);
    cfg.dynamicSmemBytes = kStages * kMoveTokens * D;
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
    p.nseq = a.nseq;
    p.Hkv = a.c.Hkv;
    p.keep = a.keep;
    p.recent = a.recent;
    p.cluster = 1;
    const long long grid = (long long)a.nseq * a.c.Hkv;
    if (grid > INT32_MAX) return -3;
    const long long cap = (long long)a.c.max_pages * a.c.page;
    const int held = (int)(cap < kSelMost ? cap : kSelMost);
    if (!allow_smem<fa_kvq8_select_kernel>(kSelMost * 4)) return -5;  // (beside static shared memory: needed below 48 KB too)
    fa_kvq8_select_kernel<<<(unsigned)grid, kSelThreads, held * 4, a.stream>>>(p, held);
    if (cudaGetLastError() != cudaSuccess) return -5;
    const bool i8 = a.c.format == kKvq8Int8;
    if (a.c.d == 128) return i8 ? launch_move<128, kKvq8Int8>(a, p) : launch_move<128, kKvq8E4m3>(a, p);
    return i8 ? launch_move<64, kKvq8Int8>(a, p) : launch_move<64, kKvq8E4m3>(a, p);
}

}  // namespace fa
