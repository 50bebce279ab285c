// fa_kvq8_prefix_tc.cu -- the keys of a prefix that all sequences of a batch share, attended to by the rows of all of
// them at once, over the 8-bit cache.
//
// The R = B (H / Hkv) Nq query rows of a K/V head are one tall Q: S = Q K^T, O = P V with the running (m, l, a) of the
// forward. A code is read from HBM once for all rows (once for every 256 from L2), turned into fp16 once, and the
// products run on tcgen05.mma. A CTA takes 256 rows (two 128-row tiles) and one run of the prefix's keys and leaves the
// rows' summaries (O / l and the log-sum-exp, fp32).
//
// Scales. A page's values are code * scale. Where all K scales of a run are powers of two (append writes no others) within
// 2^20 of the largest, ks_max, the K tile holds code * 32 ks / ks_max, exact in fp16 (an int8 code and an e4m3 code are
// multiples of 2^0 and 2^-9 of at most 448: 2^-24 is not undercut), so that one factor serves the whole row; V likewise, within
// 2^7: P, which then knows nothing of the V scales, is held 2^7 up, so that what fp16 loses of it (2^-25 at most) is no
// more than 2^-25 of the row's largest contribution p vs, as in fa_kvq8_attn.cuh. (Not raised, and with V within 2^20,
// weights of 2^-26 were lost whose V scale is 2^20 times that of the keys of weight 1.) Any other run (scales further apart
// or no powers of two, K pages of zeros alone, pages that are none) is done with the codes as they are: each 16-key group of
// scores is multiplied by its own page's factor, and P carries 2^(log2 vs) under a running maximum of its own, as there. (64
// sequences of 64 / 8 heads of 128 behind 32768 int8 keys and 2048 of their own: 129 us with V scales up to 2^7 apart, 201
// with 2^8 and more; 16 of 32 / 8 heads behind 8192: 23.6 and 37.)
// Q is fp16, bf16 rows under a power of two that puts the row's largest magnitude into [2^15, 2^16).
//
// Bound: for few rows HBM (2 d bytes a key and head), from about 250 rows on the tensor cores, in effect the softmax's
// issue slots and the order S -> softmax -> P V as in the forward (fa_fwd_bk128.cuh), whose roles, tensor memory and
// barriers this kernel has. What it adds is the way of K and V into shared memory:
//   warps 0-7    softmax and epilogue of the two tiles; each thread first brings its own row of Q
//   warp  8      loader: whole pages by bulk copies into a ring of raw codes, with the pages' scales
//   warp  9      S issuer,  warps 10-11 P V issuers
//   warps 12-19  converters: raw codes -> fp16 in the 128-byte swizzled K and V tiles
// The own keys' kernel behind it is a programmatic dependent that needs nothing of it: it fills the SMs that this one leaves
// free, and ends after it, so that the merge behind may rely on both.
// Measured: 64 sequences of 64 / 8 heads of 128 behind 32768 int8 keys, 88 us (91 where the S issuer waited for K only once the S
// buffer was free); a block of two tiles takes some 3700 cycles, of which the products need
// 2048 and the softmax of a tile about 1500, a block of one tile 1750 to 2300, the first of a CTA 16000. Slower: converters in
// two groups, one for K and one for V (a run of 6 blocks and one tile 28.8 us for 22.8).
#include <float.h>

#include "fa_fwd_bk128.cuh"
#include "fa_kvq8_prefix.cuh"

namespace fa {
namespace {

constexpr int kConv = 256;          // converter threads
constexpr int kPrefixThreads = 384 + kConv;

constexpr int kSpreadK = 20, kSpreadV = 7;  // log2 of the scales' ranges that one factor serves
constexpr float kLift = (float)kSpreadV;    // log2 of what a weight of 1 is in P under such a factor: P is at most 2^(kLift + kTau)
constexpr float kNone = -FLT_MAX;   // a running maximum that has seen no key

template <int D>
struct PrefixCfg {
    using C = Cfg128<__half, D>;
    static constexpr int RK = 2, RV = 2;
    static constexpr int RAW = D == 128 ? 2 : 4;  // tiles of raw codes in flight, and two more where there is no second Q tile
    static constexpr int RAW_TILE = kBK128 * D;
    static constexpr int SMEM_Q = 0;
    static constexpr int SMEM_K = 2 * C::Q_TILE;
    static constexpr int SMEM_V = SMEM_K + RK * C::KV_TILE;
    static constexpr int SMEM_RAW = SMEM_V + RV * C::KV_TILE;
    static constexpr int SMEM_META = SMEM_RAW + RAW * RAW_TILE;  // float[RAW + 2][8]: the scales of a raw tile, -1: no page
    static constexpr int SMEM_SCAN = SMEM_META + (RAW + 2) * 32;  // int[8]
    static constexpr int SMEM_BAR = SMEM_SCAN + 32;
    // raw_full, raw_empty [RAW + 2]; k_full, k_empty [RK]; v_full, v_empty [RV]; q_full[2] s_full[2] s_free p_full[2]
    // pv_done[2][2] drain s_issued[2][2] scan
    static constexpr int B_K = 2 * (RAW + 2), B_V = B_K + 2 * RK, B_Q = B_V + 2 * RV, NUM_BARS = B_Q + 2 + 2 + 1 + 2 + 4 + 1 + 4 + 1;
    static constexpr int SMEM_TMEM_SLOT = SMEM_BAR + NUM_BARS * 8;
    static constexpr int SMEM_ABORT = SMEM_TMEM_SLOT + 8;
    static constexpr int SMEM_USED = SMEM_ABORT + 8;
    static constexpr int SMEM_BYTES = SMEM_USED + 1024;
    static_assert(SMEM_BYTES <= 232448, "shared memory budget");
    static_assert(SMEM_BAR % 8 == 0 && SMEM_META % 16 == 0, "alignment");
};

struct PrefixParams {
    const void *q;
    const uint8_t *k_codes, *v_codes;
    const float *k_scale, *v_scale;
    const int *prefix_table, *prefix_len, *kv_lens;
    float *o_part, *lse_part;
    int *status;
    int B, H, Hkv, Nq, head_rows, rows, row_tiles, splits;  // head_rows = (H / Hkv) Nq of a sequence, rows = B head_rows
    int n_pages, page_shift, max_prefix, max_len, causal;
    float scale_log2;
    uint64_t timeout_ns;
};

// Bounded wait of a whole warp (see wait_bounded in fa_fwd_kernel.cuh).
__device__ __forceinline__ bool wait_all(uint32_t bar, uint32_t parity, volatile int *abort_flag, const PrefixParams &p) {
    bool ok = mbar_try_wait(bar, parity);
    if (!ok) {
        const uint64_t t0 = global_timer_ns();
        for (;;) {
            if (mbar_try_wait_suspend(bar, parity, 100000u)) {
                ok = true;
                break;
            }
            if (*abort_flag) break;
            if (global_timer_ns() - t0 > p.timeout_ns) {
                *abort_flag = 1;
                atomicExch(p.status, kStatusTimeout);
                break;
            }
        }
    }
    return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

__device__ __forceinline__ uint2 ld_shared_v2(uint32_t addr) {
    uint2 w;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w.x), "=r"(w.y) : "r"(addr) : "memory");
    return w;
}
__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t hmul2_bits(uint32_t a, uint32_t b) {
    const __half2 h = __hmul2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&h);
}
// Four codes times the power of two r (both halves of `mul`), exact: for int8 (1152 + code) r - 1152 r.
template <int FMT>
__device__ __forceinline__ void codes_scaled(uint32_t w, uint32_t mul, uint32_t bias, uint32_t &lo, uint32_t &hi) {
    if constexpr (FMT == kKvq8Int8) {
        const uint32_t u = w ^ 0x80808080u;
        const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
        const __half2 m = *reinterpret_cast<const __half2 *>(&mul), c = *reinterpret_cast<const __half2 *>(&bias);
        const __half2 x = __hfma2(*reinterpret_cast<const __half2 *>(&a), m, c);
        const __half2 y = __hfma2(*reinterpret_cast<const __half2 *>(&b), m, c);
        lo = *reinterpret_cast<const uint32_t *>(&x);
        hi = *reinterpret_cast<const uint32_t *>(&y);
    } else {
        e4m3x4_to_half2(w, lo, hi);
        lo = hmul2_bits(lo, mul);
        hi = hmul2_bits(hi, mul);
    }
}

template <typename T, int D, int FMT>
__global__ void __launch_bounds__(kPrefixThreads, 1) fa_kvq8_prefix_kernel(const PrefixParams p) {
    using S = PrefixCfg<D>;
    using C = typename S::C;
    constexpr int RK = S::RK, RV = S::RV;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t pad = (uint32_t)((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *smem = smem_raw + pad;
    const uint32_t bars = smem_u32(smem + S::SMEM_BAR);
    auto raw_full = [&](int s) { return bars + 8 * s; };
    auto raw_empty = [&](int s) { return bars + 8 * (S::RAW + 2 + s); };
    auto k_full = [&](int s) { return bars + 8 * (S::B_K + s); };
    auto k_empty = [&](int s) { return bars + 8 * (S::B_K + RK + s); };
    auto v_full = [&](int s) { return bars + 8 * (S::B_V + s); };
    auto v_empty = [&](int s) { return bars + 8 * (S::B_V + RV + s); };
    auto q_full = [&](int t) { return bars + 8 * (S::B_Q + t); };
    auto s_full = [&](int t) { return bars + 8 * (S::B_Q + 2 + t); };
    const uint32_t s_free = bars + 8 * (S::B_Q + 4);
    auto p_full = [&](int t) { return bars + 8 * (S::B_Q + 5 + t); };
    auto pv_done = [&](int t, int b) { return bars + 8 * (S::B_Q + 7 + 2 * t + b); };
    const uint32_t drain = bars + 8 * (S::B_Q + 11);
    auto s_issued = [&](int t, int b) { return bars + 8 * (S::B_Q + 12 + 2 * t + b); };
    const uint32_t scan_done = bars + 8 * (S::B_Q + 16);
    float *meta = reinterpret_cast<float *>(smem + S::SMEM_META);
    int *scan = reinterpret_cast<int *>(smem + S::SMEM_SCAN);  // most and least exponent of K, of V; irregular
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + S::SMEM_TMEM_SLOT);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + S::SMEM_ABORT);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // work: row tiles of a run beside each other (they share its codes in L2)
    const int rt = blockIdx.x % p.row_tiles;
    const int split = blockIdx.x / p.row_tiles % p.splits;
    const int kvh = blockIdx.x / p.row_tiles / p.splits;
    const int tiles = p.rows - rt * 2 * kBQ > kBQ ? 2 : 1;
    const uint32_t raw_slots = tiles == 1 ? S::RAW + 2 : S::RAW;
    auto raw_tile = [&](int s) {
        return smem_u32(smem) + (s < S::RAW ? S::SMEM_RAW + s * S::RAW_TILE : S::SMEM_Q + C::Q_TILE + (s - S::RAW) * S::RAW_TILE);
    };

    grid_launch_dependents();
    int len = __ldg(p.prefix_len);
    if (len < 0 || len > p.max_prefix) {
        if (blockIdx.x == 0 && threadIdx.x == 0) atomicExch(p.status, kStatusSeqlensQ8);
        len = 0;
    }
    const int blocks = (len + kBK128 - 1) / kBK128;
    const int b0 = (int)((long long)split * blocks / p.splits);
    const int nb = (int)((long long)(split + 1) * blocks / p.splits) - b0;
    const int key_first = b0 * kBK128;
    const int key_end = min(len, (b0 + nb) * kBK128);

    // this thread's query row (softmax warps)
    const int t = warp >> 2, r = threadIdx.x & 127;
    const int row = rt * 2 * kBQ + t * kBQ + r;  // among the K/V head's rows
    const bool live = warp < 8 && row < p.rows;
    const int b = live ? row / p.head_rows : 0, in_head = row - b * p.head_rows;
    const size_t out_row = (size_t)b * p.H * p.Nq + (size_t)kvh * p.head_rows + in_head;
    const size_t part_row = (size_t)split * p.B * p.H * p.Nq + out_row;
    if (nb == 0) {
        if (live) p.lse_part[part_row] = -INFINITY;
        return;
    }

    // What the roles read first is requested before the set-up: the row of Q, the first pages, the scales of the run's pages.
    const int page = 1 << p.page_shift;
    uint32_t qw[D / 2];  // softmax warps
    struct Group {       // loader: page and scales of a 16-key group
        int phys;
        float ks, vs;
    };
    auto entry = [&](int j) {
        const int key = key_first + j * kBK128 + lane * 16;
        return j < nb && lane < 8 && key < key_end ? __ldg(p.prefix_table + (key >> p.page_shift)) : -1;
    };
    auto scales = [&](int phys) {
        Group g = {-1, -1.f, -1.f};
        if (phys >= 0 && phys < p.n_pages) {
            const size_t at = (size_t)phys * p.Hkv + kvh;
            g = {phys, __ldg(p.k_scale + at), __ldg(p.v_scale + at)};
        }
        return g;
    };
    Group next = {-1, -1.f, -1.f};
    int ahead = -1;
    int most_k = 0, least_k = 255, most_v = 0, least_v = 255, odd = 0;  // converters: exponents of the scales
    if (warp < 8) {
        const T *src = static_cast<const T *>(p.q) + out_row * D;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
            const uint4 x = live ? __ldg(reinterpret_cast<const uint4 *>(src) + i) : make_uint4(0u, 0u, 0u, 0u);
            qw[4 * i] = x.x, qw[4 * i + 1] = x.y, qw[4 * i + 2] = x.z, qw[4 * i + 3] = x.w;
        }
    } else if (warp == 8) {
        ahead = entry(1);
        next = scales(entry(0));
    } else if (warp >= 12) {
        const int last = (key_end - 1) >> p.page_shift;
        for (int i = (key_first >> p.page_shift) + (int)threadIdx.x - 12 * 32; i <= last; i += kConv) {
            const int phys = __ldg(p.prefix_table + i);
            if (phys < 0 || phys >= p.n_pages) {
                atomicExch(p.status, kStatusPage);
                odd = 1;
                continue;
            }
            const size_t at = (size_t)phys * p.Hkv + kvh;
            const uint32_t k = __float_as_uint(__ldg(p.k_scale + at)), v = __float_as_uint(__ldg(p.v_scale + at));
            odd |= (k & 0x807FFFFFu) != 0 || (v & 0x807FFFFFu) != 0;
            const int ek = (int)(k >> 23), ev = (int)(v >> 23);
            most_k = max(most_k, ek);
            most_v = max(most_v, ev);
            if (k) least_k = min(least_k, ek);
            if (v) least_v = min(least_v, ev);
        }
    }

    if (threadIdx.x == 0) {
        for (int s = 0; s < S::RAW + 2; ++s) {
            mbar_init(raw_full(s), 1);
            mbar_init(raw_empty(s), kConv);
        }
        for (int s = 0; s < RK; ++s) {
            mbar_init(k_full(s), kConv);
            mbar_init(k_empty(s), 1);
        }
        for (int s = 0; s < RV; ++s) {
            mbar_init(v_full(s), kConv);
            mbar_init(v_empty(s), tiles);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(q_full(i), kBQ);
            mbar_init(s_full(i), 1);
            mbar_init(p_full(i), kBQ);
            for (int j = 0; j < 2; ++j) {
                mbar_init(pv_done(i, j), 1);
                mbar_init(s_issued(i, j), 1);
            }
        }
        mbar_init(s_free, kBQ);
        mbar_init(drain, tiles + 1);
        mbar_init(scan_done, kConv);
        scan[0] = scan[2] = 0;
        scan[1] = scan[3] = 255;
        scan[4] = 0;
        *abort_flag = 0;
        fence_mbar_init();
        fence_proxy_async_smem();
    }
    if (warp == 9) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);

    if (warp >= 8) {
        setmaxnreg_dec<48>();
        if (warp == 8) {
            // ---------------------------------------------------------- loader: K_0, then K_{j+1}, V_j
            // Lane i < 8 looks after the 16-key group i of a block; pages and scales are read a block ahead.
            uint32_t pos = 0;
            bool ok = true;
            auto load = [&](const Group &g, bool v) {
                const int s = pos % raw_slots;
                ok = wait_all(raw_empty(s), ((pos / raw_slots) & 1u) ^ 1u, abort_flag, p);
                if (!ok) return;
                if (lane < 8) meta[s * 8 + lane] = g.phys < 0 ? -1.f : v ? g.vs : g.ks;
                const bool issue = g.phys >= 0 && ((lane * 16) & (page - 1)) == 0;  // a page's first group
                const uint32_t bytes = (uint32_t)page * D;
                __syncwarp();  // the scales are written before lane 0 arrives
                const int n = __popc(__ballot_sync(0xffffffffu, issue));
                if (lane == 0) mbar_arrive_expect_tx(raw_full(s), bytes * n);
                __syncwarp();
                if (issue)
                    bulk_load(raw_tile(s) + lane * 16 * D,
                              (v ? p.v_codes : p.k_codes) + (((size_t)g.phys * p.Hkv + kvh) << p.page_shift) * D, bytes,
                              raw_full(s));
                ++pos;
            };
            Group cur = {-1, 0.f, 0.f};
            for (int j = -1; ok && j < nb; ++j) {
                const Group after = scales(ahead);  // of block j + 2
                ahead = entry(j + 3);
                if (j + 1 < nb) load(next, false);
                if (ok && j >= 0) load(cur, true);
                cur = next;
                next = after;
            }
            if (!ok && lane == 0) {  // let the copies in flight land before the CTA can exit
                const uint64_t t0 = global_timer_ns();
                for (uint32_t i = pos > raw_slots ? pos - raw_slots : 0; i < pos; ++i)
                    while (!mbar_try_wait(raw_full(i % raw_slots), (i / raw_slots) & 1u) && global_timer_ns() - t0 < p.timeout_ns) {
                    }
            }
        } else if (warp == 9) {
            // ---------------------------------------------------------- S issuer
            const uint32_t issue = lane == 0 ? 1u : 0u;
            const uint64_t qd0 = smem_desc_sw128(smem_u32(smem + S::SMEM_Q), 16, 1024);
            const uint64_t kd0 = smem_desc_sw128(smem_u32(smem + S::SMEM_K), 16, 1024);
            uint32_t n_issued = 0;
            bool ok = true;
            for (int i = 0; ok && i < tiles; ++i) ok = wait_all(q_full(i), 0, abort_flag, p);
            if (ok) ok = wait_all(k_full(0), 0, abort_flag, p);
            for (int j = 0; ok && j < nb; ++j) {
                const int slot = j % RK;
                for (int i = 0; ok && i < tiles; ++i) {
                    // the next block's K is waited for while the last product still has the S buffer
                    if (i == tiles - 1 && j + 1 < nb) ok = wait_all(k_full((j + 1) % RK), (uint32_t)((j + 1) / RK) & 1u, abort_flag, p);
                    if (ok && n_issued > 0) ok = wait_all(s_free, (n_issued - 1) & 1u, abort_flag, p);
                    if (!ok) break;
                    ++n_issued;
                    tc_fence_after();
                    const uint64_t a0 = qd0 + (uint64_t)i * (C::Q_TILE >> 4);
                    const uint64_t k0 = kd0 + (uint64_t)slot * (C::KV_TILE >> 4);
#pragma unroll
                    for (int k = 0; k < C::KSTEPS_S; ++k)
                        mma_ss(tmem + C::TM_S, a0 + (uint64_t)(((k / 4) * C::Q_CHUNK + (k % 4) * 32) >> 4),
                               k0 + (uint64_t)(((k / 4) * C::KV_CHUNK + (k % 4) * 32) >> 4), C::IDESC_S, k > 0 ? 1u : 0u, issue);
                    tc_commit(s_full(i), issue);
                    if (lane == 0) mbar_arrive(s_issued(i, j & 1));
                }
                if (ok) tc_commit(k_empty(slot), issue);
            }
            __syncwarp();
            tc_commit(drain, issue);
        } else if (warp < 12) {
            // ---------------------------------------------------------- P V issuer of tile i
            const int i = warp - 10;
            if (i < tiles) {
                const uint32_t issue = lane == 0 ? 1u : 0u;
                const uint64_t vd0 = smem_desc_sw128(smem_u32(smem + S::SMEM_V), C::KV_CHUNK, 1024);
                bool ok = true;
                for (int j = 0; ok && j < nb; ++j) {
                    const int slot = j % RV;
                    ok = wait_all(v_full(slot), (uint32_t)(j / RV) & 1u, abort_flag, p);
                    if (ok) ok = wait_all(p_full(i), (uint32_t)j & 1u, abort_flag, p);
                    // the tile's next S product goes into the queue first (see fa_fwd_bk128.cuh)
                    if (ok && j + 1 < nb) ok = wait_all(s_issued(i, (j + 1) & 1), (uint32_t)((j + 1) >> 1) & 1u, abort_flag, p);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t v0 = vd0 + (uint64_t)slot * (C::KV_TILE >> 4);
#pragma unroll
                    for (int k = 0; k < C::KSTEPS_PV; ++k)
                        mma_ts(tmem + C::TM_O + D * i, tmem + C::TM_P + 64 * i + k * 8,
                               v0 + (uint64_t)((k * C::V_KSTEP_BYTES) >> 4), C::IDESC_PV, (k > 0 || j > 0) ? 1u : 0u, issue);
                    tc_commit(pv_done(i, j & 1), issue);
                    tc_commit(v_empty(slot), issue);
                }
                __syncwarp();
                tc_commit(drain, issue);
            }
        } else {
            // ---------------------------------------------------------- converters
            const int tid = threadIdx.x - 12 * 32;
            {  // the scales of the run's pages
                most_k = __reduce_max_sync(0xffffffffu, most_k);
                most_v = __reduce_max_sync(0xffffffffu, most_v);
                least_k = __reduce_min_sync(0xffffffffu, least_k);
                least_v = __reduce_min_sync(0xffffffffu, least_v);
                odd = __any_sync(0xffffffffu, odd);
                if (lane == 0) {
                    atomicMax(scan + 0, most_k);
                    atomicMin(scan + 1, least_k);
                    atomicMax(scan + 2, most_v);
                    atomicMin(scan + 3, least_v);
                    if (odd) scan[4] = 1;
                }
                named_bar_sync(1, kConv);
                if (tid == 0) {
                    // within 2^-110 .. 2^120, and K not all zeros (V may be)
                    const bool k_ok = scan[0] >= 127 - 110 && scan[0] <= 127 + 120 && scan[0] - scan[1] <= kSpreadK;
                    const bool v_ok = scan[2] == 0 || (scan[2] >= 127 - 110 && scan[2] <= 127 + 120 && scan[2] - scan[3] <= kSpreadV);
                    if (!k_ok || !v_ok || !(p.scale_log2 > 0.f)) scan[4] = 1;
                }
                named_bar_sync(1, kConv);
                mbar_arrive(scan_done);
            }
            const bool regular = scan[4] == 0;
            const float up_k = __uint_as_float((uint32_t)(254 + 5 - scan[0]) << 23);  // 32 / ks_max where regular
            const float up_v = scan[2] == 0 ? 0.f : __uint_as_float((uint32_t)(254 + 5 - scan[2]) << 23);
            constexpr int LANES = D / 16, STEP = kConv / LANES, N = kBK128 / STEP;  // vectors of a key, keys of a pass, passes
            const int c = tid % LANES, swap = D == 128 && c >= 4 ? 1 : 0;
            // the lane's two units in its keys' rows (a pass is a multiple of 8 keys: the swizzle is the same in each)
            const uint32_t unit0 = (uint32_t)((2 * (c % 4) + swap) ^ (tid / LANES & 7)) * 16;
            const uint32_t unit1 = (uint32_t)((2 * (c % 4) + 1 - swap) ^ (tid / LANES & 7)) * 16;
            uint32_t pos = 0;
            bool ok = true;
            auto convert = [&](int j, bool v) {
                const int s = pos % raw_slots, slot = j % 2;
                ok = wait_all(raw_full(s), (pos / raw_slots) & 1u, abort_flag, p);
                if (ok) ok = wait_all(v ? v_empty(slot) : k_empty(slot), ((uint32_t)(j / 2) & 1u) ^ 1u, abort_flag, p);
                if (!ok) return;
                const uint32_t src = raw_tile(s) + tid * 16;
                const uint32_t dst = smem_u32(smem + (v ? S::SMEM_V : S::SMEM_K)) + slot * C::KV_TILE + (c / 4) * C::KV_CHUNK +
                                     (tid / LANES) * 128;
                const uint32_t dst0 = dst + unit0, dst1 = dst + unit1;
                const int in_tile = key_end - (key_first + j * kBK128);  // keys of this block
                const float up = v ? up_v : up_k;
                // A key's 16 dims are two 16-byte units of its 128-byte row. At d = 128 the upper lanes take theirs the
                // other way round, so that eight lanes meet all banks. Every load goes ahead of the first store.
                uint2 w[2][N];
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    w[0][i] = ld_shared_v2(src + i * kConv * 16 + 8 * swap);
                    w[1][i] = ld_shared_v2(src + i * kConv * 16 + 8 - 8 * swap);
                }
                const float scale = meta[s * 8 + (lane & 7)];  // lane e: of the 16-key group e
                const float m = regular ? scale * up : 1.0f;
                const uint32_t mul_of = half2_bits(m, m);
                const bool whole = in_tile >= kBK128 && __all_sync(0xffffffffu, scale >= 0.f);
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const int key = i * STEP + tid / LANES, group = key / 16;  // (of the whole warp)
                    const uint32_t mul = __shfl_sync(0xffffffffu, mul_of, group);
                    const uint32_t bias = FMT == kKvq8Int8 ? hmul2_bits(mul, 0xE480E480u) : 0u;  // -1152
                    uint32_t h[8];
                    codes_scaled<FMT>(w[0][i].x, mul, bias, h[0], h[1]);
                    codes_scaled<FMT>(w[0][i].y, mul, bias, h[2], h[3]);
                    codes_scaled<FMT>(w[1][i].x, mul, bias, h[4], h[5]);
                    codes_scaled<FMT>(w[1][i].y, mul, bias, h[6], h[7]);
                    if (!whole) {  // keys that are none are zeros, whatever the codes were
                        const float there = __shfl_sync(0xffffffffu, scale, group);
                        if (key >= in_tile || there < 0.f) {
#pragma unroll
                            for (int e = 0; e < 8; ++e) h[e] = 0u;
                        }
                    }
                    st_shared_v4(dst0 + i * STEP * 128, h[0], h[1], h[2], h[3]);
                    st_shared_v4(dst1 + i * STEP * 128, h[4], h[5], h[6], h[7]);
                }
                mbar_arrive(raw_empty(s));
                fence_proxy_async_smem();
                mbar_arrive(v ? v_full(slot) : k_full(slot));
                ++pos;
            };
            for (int j = -1; ok && j < nb; ++j) {
                if (j + 1 < nb) convert(j + 1, false);
                if (ok && j >= 0) convert(j, true);
            }
        }
    } else {
        setmaxnreg_inc<168>();
        if (t < tiles) {
            // ---------------------------------------------------------- softmax and epilogue of tile t
            const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
            const uint32_t s_addr = tmem + lane_base + C::TM_S;
            const uint32_t p_addr = tmem + lane_base + C::TM_P + 64 * t;
            const uint32_t o_addr = tmem + lane_base + C::TM_O + D * t;
            const bool warp_live = __any_sync(0xffffffffu, live);
            // Q: this thread's row, in fp16
            float qmul = 1.0f;  // what the row was divided by
            {
                const uint32_t line = smem_u32(smem + S::SMEM_Q) + t * C::Q_TILE + r * 128;
                uint32_t (&w)[D / 2] = qw;
                if constexpr (std::is_same<T, __nv_bfloat16>::value) {
                    uint32_t most = 0;
#pragma unroll
                    for (int i = 0; i < D / 2; ++i) most = max(most, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
                    // (rows below 2^-111 by 2^126, as in fa_kvq8_attn.cuh; a row of zeros stays)
                    const uint32_t ex = max(most >> 7, 16u);
                    const float inv = most == 0 ? 1.0f : __uint_as_float((269u - ex) << 23);
                    qmul = most == 0 ? 1.0f : __uint_as_float(ex << 23) * 0x1p-15f;
#pragma unroll
                    for (int i = 0; i < D / 2; ++i) {
                        const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w[i]));
                        w[i] = half2_bits(f.x * inv, f.y * inv);
                    }
                }
#pragma unroll
                for (int i = 0; i < D / 8; ++i)
                    st_shared_v4(line + (i / 8) * C::Q_CHUNK + (uint32_t)(((i % 8) ^ (r & 7)) * 16), w[4 * i], w[4 * i + 1],
                                 w[4 * i + 2], w[4 * i + 3]);
                fence_proxy_async_smem();
                mbar_arrive(q_full(t));
            }
            // keys of the prefix that the row sees
            int vis = len;
            if (p.causal && live) {
                int own = __ldg(p.kv_lens + b);
                if (own < 0 || own > p.max_len) own = 0;  // reported with the own keys
                vis = min(len, max(0, len + own - p.Nq + in_head % p.Nq + 1));  // (both lengths are below 2^30)
            }
            bool ok = wait_all(scan_done, 0, abort_flag, p);
            const bool regular = scan[4] == 0;
            const float ks_unit = regular ? __uint_as_float((uint32_t)(scan[0] - 5) << 23) : 1.0f;  // ks_max / 32
            const float vs_unit = !regular ? 1.0f : scan[2] == 0 ? 0.0f : __uint_as_float((uint32_t)(scan[2] - 5) << 23);
            const float sl2 = p.scale_log2 * ks_unit * qmul;  // score of the products in log2 units, where regular
            const bool simple = regular && __all_sync(0xffffffffu, sl2 >= FLT_MIN && sl2 <= FLT_MAX);
            float m_ref = simple ? -INFINITY : kNone, mw = kNone, l = 0.0f;
            for (int j = 0; ok && j < nb; ++j) {
                ok = wait_all(s_full(t), (uint32_t)j & 1u, abort_flag, p);
                if (!ok) break;
                tc_fence_after();
                const int kbase = key_first + j * kBK128;
                if (!warp_live) {  // no rows: nothing but the barriers
                    mbar_arrive(s_free);
                    if (j > 0) ok = wait_all(pv_done(t, (j - 1) & 1), (uint32_t)((j - 1) >> 1) & 1u, abort_flag, p);
                    if (ok) mbar_arrive(p_full(t));
                    continue;
                }
                float x[128];
                {
                    uint32_t sr[128];
                    tmem_ld128_wait(s_addr, sr);
#pragma unroll
                    for (int i = 0; i < 128; ++i) x[i] = __uint_as_float(sr[i]);
                }
                tc_fence_before();
                mbar_arrive(s_free);
                const int lim = min(vis, key_end) - kbase;  // columns from here on are not seen
                bool rescale;
                float alpha;
                if (simple) {
                    if (__any_sync(0xffffffffu, lim < kBK128)) {
#pragma unroll
                        for (int i = 0; i < 128; ++i) x[i] = i >= lim ? -INFINITY : x[i];
                    }
                    const float mb = row_max128(x) * sl2;
                    // The exponents are x sl2 - m_ref in one rounding, which takes m_ref for exact: beyond 2^20 its own
                    // rounding would be the exponent, and the scores are rounded first.
                    float mul = sl2;
                    if (__any_sync(0xffffffffu, fabsf(mb) > 0x1p20f && mb != -INFINITY)) {
#pragma unroll
                        for (int i = 0; i < 128; ++i) x[i] *= sl2;
                        mul = 1.0f;
                    }
                    // (the difference, not m_ref + kLift + kTau, which far out may round up and let P past fp16's range)
                    const bool need = mb - m_ref > kLift + kTau;
                    const float m_new = mb - kLift;
                    alpha = need ? ex2_approx(m_ref - m_new) : 1.0f;
                    rescale = __any_sync(0xffffffffu, need) && j > 0;
                    if (need) {
                        l *= alpha;
                        m_ref = m_new;
                    }
                    const float neg = m_ref == -INFINITY ? 0.0f : -m_ref;
                    const float2 sl2v = make_float2(mul, mul), negv = make_float2(neg, neg);
                    float2 ls[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        uint32_t pv[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float2 a = ffma2(make_float2(x[32 * h + 2 * i], x[32 * h + 2 * i + 1]), sl2v, negv);
                            const float2 e = make_float2(ex2_approx(a.x), ex2_approx(a.y));
                            ls[i & 3] = fadd2(ls[i & 3], e);
                            pv[i] = half2_bits(e.x, e.y);
                        }
                        if (h == 0 && j > 0) {  // P_t is free once the tile's previous product has read it
                            ok = wait_all(pv_done(t, (j - 1) & 1), (uint32_t)((j - 1) >> 1) & 1u, abort_flag, p);
                            if (!ok) break;
                            tc_fence_after();
                        }
                        tmem_st16(p_addr + 16 * h, pv);
                    }
                    if (!ok) break;
                    l += ((ls[0].x + ls[0].y) + (ls[1].x + ls[1].y)) + ((ls[2].x + ls[2].y) + (ls[3].x + ls[3].y));
                } else {
                    // each 16-key group under its own page's scales
                    float lv[8];
                    float mx = -INFINITY, mv = -INFINITY;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        float f = sl2;
                        bool good = true;
                        lv[i] = 0.f;
                        if (!regular && kbase + 16 * i < key_end) {
                            const int phys = __ldg(p.prefix_table + ((kbase + 16 * i) >> p.page_shift));
                            good = phys >= 0 && phys < p.n_pages;
                            const size_t at = good ? (size_t)phys * p.Hkv + kvh : 0;
                            f = __ldg(p.k_scale + at) * p.scale_log2 * qmul;
                            lv[i] = lg2_approx(__ldg(p.v_scale + at));  // -inf for a page of zeros
                        }
                        float top = -INFINITY;
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const int col = 16 * i + e;
                            x[col] = col >= lim || !good ? -INFINITY : x[col] * f;
                            top = fmaxf(top, x[col]);
                        }
                        mx = fmaxf(mx, top);
                        mv = fmaxf(mv, top + lv[i]);
                    }
                    if (mx > m_ref + kTau) {
                        l *= ex2_approx(m_ref - mx);
                        m_ref = mx;
                    }
                    const float lift = regular ? kLift : 0.f;  // (lv is 0 where regular)
                    const bool need = mv - mw > lift + kTau;
                    if (need) mv -= lift;
                    alpha = need ? ex2_approx(mw - mv) : 1.0f;
                    rescale = __any_sync(0xffffffffu, need) && j > 0;
                    if (need) mw = mv;
                    if (j > 0) {
                        ok = wait_all(pv_done(t, (j - 1) & 1), (uint32_t)((j - 1) >> 1) & 1u, abort_flag, p);
                        if (!ok) break;
                        tc_fence_after();
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t pv[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const float lvi = lv[4 * h + i / 8];
                            const float f = lvi == -INFINITY ? -INFINITY : fminf(lvi + (m_ref - mw), FLT_MAX);
                            const float a0 = x[64 * h + 2 * i] - m_ref, a1 = x[64 * h + 2 * i + 1] - m_ref;
                            l += ex2_approx(a0) + ex2_approx(a1);
                            pv[i] = half2_bits(ex2_approx(a0 + f), ex2_approx(a1 + f));
                        }
                        tmem_st32(p_addr + 32 * h, pv);
                    }
                }
                if (rescale) {
#pragma unroll
                    for (int c0 = 0; c0 < D; c0 += 32) {
                        uint32_t ov[32];
                        tmem_ld32_wait(o_addr + c0, ov);
#pragma unroll
                        for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
                        tmem_st32(o_addr + c0, ov);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(p_full(t));
            }
            // ---------------------------------------------------------- epilogue
            if (ok && warp_live) ok = wait_all(pv_done(t, (nb - 1) & 1), (uint32_t)((nb - 1) >> 1) & 1u, abort_flag, p);
            if (ok && warp_live) {
                tc_fence_after();
                // (a sum that is NaN, from a NaN query, stays NaN)
                float f = l == 0.0f ? 0.0f : simple ? vs_unit / l : ex2_approx(mw - m_ref) * vs_unit / l;
#pragma unroll
                for (int c0 = 0; c0 < D; c0 += 32) {
                    uint32_t ov[32];
                    tmem_ld32_wait(o_addr + c0, ov);
                    if (live) {
                        float *dst = p.o_part + part_row * D + c0;
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
                            *reinterpret_cast<float4 *>(dst + i) =
                                make_float4(__uint_as_float(ov[i]) * f, __uint_as_float(ov[i + 1]) * f,
                                            __uint_as_float(ov[i + 2]) * f, __uint_as_float(ov[i + 3]) * f);
                    }
                }
                tc_fence_before();
                if (live) p.lse_part[part_row] = l == 0.0f ? -INFINITY : (m_ref + lg2_approx(l)) * 0.6931471805599453f;
            }
        }
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {  // every MMA is complete before the tensor memory is given back
        const uint64_t t0 = global_timer_ns();
        while (!mbar_try_wait(drain, 0) && global_timer_ns() - t0 < p.timeout_ns) {
        }
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <typename T, int D, int FMT>
int launch_tc(const PrefixParams &p, cudaStream_t stream) {
    using S = PrefixCfg<D>;
    if (!allow_smem<fa_kvq8_prefix_kernel<T, D, FMT>>(S::SMEM_BYTES)) return -5;
    const long long grid = (long long)p.Hkv * p.row_tiles * p.splits;
    if (grid > INT32_MAX) return -3;
    fa_kvq8_prefix_kernel<T, D, FMT><<<(unsigned)grid, kPrefixThreads, S::SMEM_BYTES, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? 0 : -5;
}

template <typename T>
int launch_tc_t(const PrefixParams &p, int d, int format, cudaStream_t stream) {
    const bool i8 = format == kKvq8Int8;
    if (d == 128) return i8 ? launch_tc<T, 128, kKvq8Int8>(p, stream) : launch_tc<T, 128, kKvq8E4m3>(p, stream);
    return i8 ? launch_tc<T, 64, kKvq8Int8>(p, stream) : launch_tc<T, 64, kKvq8E4m3>(p, stream);
}

}  // namespace

int launch_kvq8_prefix_tc(const Kvq8AttnArgs &a, bool fp16, float *o_part, float *lse_part) {
    PrefixParams p;
    p.q = a.q;
    p.k_codes = a.c.k_codes;
    p.v_codes = a.c.v_codes;
    p.k_scale = a.c.k_scale;
    p.v_scale = a.c.v_scale;
    p.prefix_table = a.prefix_table;
    p.prefix_len = a.prefix_len;
    p.kv_lens = a.kv_lens;
    p.o_part = o_part;
    p.lse_part = lse_part;
    p.status = a.status;
    p.B = a.B;
    p.H = a.H;
    p.Hkv = a.c.Hkv;
    p.Nq = a.Nq;
    p.head_rows = a.H / a.c.Hkv * a.Nq;
    p.rows = a.B * p.head_rows;
    p.row_tiles = (p.rows + 2 * kBQ - 1) / (2 * kBQ);
    p.splits = a.splits;
    p.n_pages = a.c.n_pages;
    p.page_shift = kvq8_page_shift(a.c.page);
    p.max_prefix = a.max_prefix;
    p.max_len = a.max_len;
    p.causal = a.causal;
    p.scale_log2 = static_cast<float>(static_cast<double>(a.scale) * 1.4426950408889634);
    p.timeout_ns = a.timeout_ns;
    return fp16 ? launch_tc_t<__half>(p, a.c.d, a.c.format, a.stream) : launch_tc_t<__nv_bfloat16>(p, a.c.d, a.c.format, a.stream);
}

}  // namespace fa
