// fa_kvq8_attn.cu -- attention of a few query rows per sequence over the 8-bit key/value cache.
//
// For query row i of head h, with the codes kc, vc and page scales ks, vs of the K/V head it shares,
//     s_j = scale (q_i . kc_j) ks(j),   O_i = sum_j softmax(s)_j vs(j) vc_j,   lse_i = ln sum_j exp(s_j),
// over the visible keys j of the row's sequence. The running maximum, sum and accumulator and the
// merge of key blocks are those of the split-KV forward (fa_splitkv.cu).
//
// Bound: HBM. A step reads every cached byte once and does 2 rows flop per byte for the `rows`
// query rows that share a K/V head, so the design keeps the number of instructions per cached
// byte low enough for the memory rate (24 bytes per clock and SM) and enough bytes in flight:
//   - Both products run on 16x8x16 warp MMAs with the CODES as the 16-row operand A and the query
//     rows as the 8 columns of B: S^T = Kc Q^T, O^T = Vc^T P^T. Eight rows fill a tile (16 with two),
//     and a code is turned into fp16 once for all of them, exactly (int8 and e4m3 are fp16 numbers).
//   - The order of the contraction index, and of the rows of A, is free as long as both sides
//     agree. So a lane loads 16 contiguous codes of a key (K: dims 64 j + 16 c.., four MMA steps'
//     worth; V: dims 16 g.. of four keys), and the fragments are cut from its own registers: no
//     lane ever needs another's codes. Each lane therefore copies into its own slots of shared
//     memory (cp.async, kStages tiles deep) and waits for its own copies only.
//   - The page scales multiply scores, which are few (16 keys x 8 rows per tile and warp): ks goes
//     into the score, log2 vs into the exponent of the weights that multiply Vc. Those weights,
//     w_j = s_j log2 e + log2 vs(j), keep a running maximum of their own: the fp16 rounding of the
//     weights is then relative to the largest contribution, whatever the pages' scales are, and
//     a page of zeros (vs = 0) still counts in the sum. The sum l and all accumulators are fp32.
// Q is rounded to nothing: fp16 as given, and bf16 rows scaled by a power of two into fp16's
// range, which is exact down to 2^-24 of the row's largest magnitude. P (the weights) are rounded
// to fp16, 2^-11 relative.
//
// A CTA takes one chunk of keys of one (sequence, K/V head, row tile); its four warps take every
// fourth 16-key tile and merge at the end. A sequence that needs one chunk is finished by its CTA;
// otherwise the chunks' summaries go to the workspace and fa_kvq8_combine merges them.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "fa_kvq8.cuh"
#include "pdl.cuh"
#include "ptx.cuh"
#include "warp_mma.cuh"

namespace fa {
namespace {

constexpr int kWarps = 4;
constexpr int kTileKeys = 16;
constexpr float kTau = 8.0f;  // log2 units by which a reference maximum may be exceeded before it moves
constexpr float kLn2 = 0.6931471805599453f;

template <int D>
struct Q8Cfg {
    static constexpr int KB = D / 64;                         // 16-byte units of a K row per lane
    static constexpr int VB = D / 8;                          // bytes of a V row per lane
    static constexpr int SLOT = 2 * KB * 16 + 4 * VB;         // bytes per lane and stage
    static constexpr int STAGES = 512 / SLOT;                 // 16 KB per warp: 4 (d = 128) or 8
    static constexpr int STAGE_WARP = SLOT * 32;
    static constexpr int SMEM = kWarps * STAGES * STAGE_WARP;
    static constexpr int PITCH = D + 8;                       // floats per row of the merge buffer
};

struct Q8Params {
    const void *q;
    void *out;
    float *lse;
    const uint8_t *k_codes, *v_codes;
    const float *k_scale, *v_scale;
    const int *page_table, *kv_lens;
    float *o_part, *lse_part;
    int *status;
    int H, Hkv, Nq, rows, row_tiles, rows_total;  // rows = (H / Hkv) Nq; rows_total = B H Nq
    int n_pages, max_pages, page_shift;
    int max_len, split_len, n_splits;
    float scale_log2;
};

// Length of sequence b, 0 when it is out of range (the first CTA to see it reports it).
__device__ __forceinline__ int q8_len(const Q8Params &p, int b, bool &bad) {
    const int len = __ldg(p.kv_lens + b);
    bad = len < 0 || len > p.max_len;
    return bad ? 0 : len;
}

__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
    return v;
}
template <typename T>
__device__ __forceinline__ float to_float(T x) {
    if constexpr (std::is_same<T, __nv_bfloat16>::value) return __bfloat162float(x);
    else return __half2float(x);
}
template <typename T>
__device__ __forceinline__ T from_float(float x) {
    if constexpr (std::is_same<T, __nv_bfloat16>::value) return __float2bfloat16_rn(x);
    else return __float2half_rn(x);
}

template <typename T, int D, int FMT, int NT, bool CAUSAL>
__global__ void __launch_bounds__(kWarps * 32) fa_kvq8_partial(const Q8Params p) {
    using C = Q8Cfg<D>;
    constexpr int KS = D / 16;   // MMA steps over the head dimension
    constexpr int MT = D / 16;   // 16-row tiles of O^T
    constexpr int RT = 8 * NT;   // query rows per CTA
    extern __shared__ __align__(128) uint8_t sm[];
    grid_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, c = lane & 3;
    uint32_t u = blockIdx.x;
    const int split = u % p.n_splits;
    u /= p.n_splits;
    const int rt = u % p.row_tiles;
    u /= p.row_tiles;
    const int kvh = u % p.Hkv, b = u / p.Hkv;
    bool bad;
    const int len = q8_len(p, b, bad);
    if (bad && threadIdx.x == 0) atomicExch(p.status, kStatusSeqlensQ8);
    const int n_chunks = len > 0 ? (len + p.split_len - 1) / p.split_len : 1;
    if (split >= n_chunks) return;
    const int k0 = split * p.split_len, k1 = min(len, k0 + p.split_len);
    const int row0 = rt * RT;  // first of this CTA's rows among the rows of the K/V head
    const size_t row_base = ((size_t)b * p.H + (size_t)kvh * (p.H / p.Hkv)) * p.Nq;

    const int n_tiles = (k1 - k0 + kTileKeys - 1) / kTileKeys;
    const int my_tiles = n_tiles > warp ? (n_tiles - warp + kWarps - 1) / kWarps : 0;
    const int *table = p.page_table + (size_t)b * p.max_pages;
    const int page_mask = (1 << p.page_shift) - 1;

    // Lane i holds the page and the scales of this warp's tile 32 n + i.
    int pg = -1;
    float pg_ks = 0.f, pg_lv = -INFINITY;
    auto load_pages = [&](int it0) {
        const int it = it0 + lane;
        pg = -1;
        pg_ks = 0.f;
        pg_lv = -INFINITY;
        if (it < my_tiles) {
            const int key = k0 + (warp + it * kWarps) * kTileKeys;
            const int phys = __ldg(table + (key >> p.page_shift));
            if (phys >= 0 && phys < p.n_pages) {
                pg = phys;
                const size_t at = (size_t)phys * p.Hkv + kvh;
                pg_ks = __ldg(p.k_scale + at) * p.scale_log2;
                pg_lv = lg2_approx(__ldg(p.v_scale + at));  // -inf for a page of zeros
            } else {
                atomicExch(p.status, kStatusPage);
            }
        }
    };
    const uint32_t my_slots = smem_u32(sm) + warp * C::STAGES * C::STAGE_WARP + lane * 16;
    // Copies of tile it into the stage's slots: unit u of a lane at u * 512 (16-byte units) or,
    // for V rows of 8 bytes, two rows in one unit.
    auto issue = [&](int it, int stage) {
        const int page = __shfl_sync(0xffffffffu, pg, it & 31);
        if (it < my_tiles) {
            const int key0 = k0 + (warp + it * kWarps) * kTileKeys;
            const bool have = page >= 0;
            const size_t off =
                ((((size_t)(have ? page : 0) * p.Hkv + kvh) << p.page_shift) + (size_t)(key0 & page_mask)) * D;
            const uint32_t dst = my_slots + stage * C::STAGE_WARP;
            const uint8_t *ks = p.k_codes + off + c * 16, *vs = p.v_codes + off + g * C::VB;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const uint32_t n = have && key0 + g + 8 * r < k1 ? 16u : 0u;
#pragma unroll
                for (int j = 0; j < C::KB; ++j)
                    cp_async16(dst + (r * C::KB + j) * 512, ks + (g + 8 * r) * D + j * 64, n);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int key = 2 * c + (i & 1) + (i >> 1) * 8;
                const bool in = have && key0 + key < k1;
                if constexpr (D == 128)
                    cp_async16(dst + (2 * C::KB + i) * 512, vs + key * D, in ? 16u : 0u);
                else
                    cp_async8(dst + (2 * C::KB + (i >> 1)) * 512 + (i & 1) * 8, vs + key * D, in ? 8u : 0u);
            }
        }
        cp_async_commit();
    };

    load_pages(0);
    // the copies run ahead: their window of 32 tiles is (pg, pg_ks, pg_lv), the products' the copy below
    bool cur_have = false;
    float cur_ks = 0.f, cur_lv = -INFINITY;
#pragma unroll
    for (int s = 0; s < C::STAGES - 1; ++s) issue(s, s);

    // Q as B fragments: column g of tile t is row row0 + 8 t + g, contraction index in the order of the K codes
    uint32_t qb[NT][KS][2];
    float qmul[NT][2];  // what the rows 2c, 2c + 1 of tile t were divided by
    int lim[NT][2];     // causal: last visible key of those rows
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int row = row0 + 8 * t + g;
        const T *src = static_cast<const T *>(p.q) + (row_base + row) * D;
        float mul = 1.0f;
#pragma unroll
        for (int j = 0; j < C::KB; ++j) {
            uint4 w[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
            if (row < p.rows) {
                w[0] = __ldg(reinterpret_cast<const uint4 *>(src + 64 * j + 16 * c));
                w[1] = __ldg(reinterpret_cast<const uint4 *>(src + 64 * j + 16 * c) + 1);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                qb[t][4 * j + e][0] = e == 0 ? w[0].x : e == 1 ? w[0].z : e == 2 ? w[1].x : w[1].z;
                qb[t][4 * j + e][1] = e == 0 ? w[0].y : e == 1 ? w[0].w : e == 2 ? w[1].y : w[1].w;
            }
        }
        if constexpr (std::is_same<T, __nv_bfloat16>::value) {
            uint32_t most = 0;
#pragma unroll
            for (int s = 0; s < KS; ++s)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    most = max(most, max(qb[t][s][e] & 0x7FFFu, (qb[t][s][e] >> 16) & 0x7FFFu));
            most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
            most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
            const uint32_t ex = min(most >> 7, 253u);  // biased exponent of the row's largest magnitude
            const float inv = __uint_as_float((254u - ex) << 23);
            mul = ex == 0 ? __uint_as_float(1u << 22) : __uint_as_float(ex << 23);  // 2^(ex - 127)
#pragma unroll
            for (int s = 0; s < KS; ++s)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const __nv_bfloat162 h = *reinterpret_cast<const __nv_bfloat162 *>(&qb[t][s][e]);
                    const float2 f = __bfloat1622float2(h);
                    const __half2 o = __floats2half2_rn(f.x * inv, f.y * inv);
                    qb[t][s][e] = *reinterpret_cast<const uint32_t *>(&o);
                }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            qmul[t][e] = __shfl_sync(0xffffffffu, mul, 8 * c + 4 * e);  // lane of column 2c + e
            if constexpr (CAUSAL) lim[t][e] = len - p.Nq + (row0 + 8 * t + 2 * c + e) % p.Nq;
            else lim[t][e] = len - 1;
        }
    }

    float o[NT][MT][4], m[NT][2], mw[NT][2], l[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int i = 0; i < MT; ++i) o[t][i][0] = o[t][i][1] = o[t][i][2] = o[t][i][3] = 0.f;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            m[t][e] = mw[t][e] = -INFINITY;
            l[t][e] = 0.f;
        }
    }

    for (int it = 0; it < my_tiles; ++it) {
        if ((it & 31) == 0) {
            cur_have = pg >= 0;
            cur_ks = pg_ks;
            cur_lv = pg_lv;
        }
        const float ks = __shfl_sync(0xffffffffu, cur_ks, it & 31), lv = __shfl_sync(0xffffffffu, cur_lv, it & 31);
        const bool have = __shfl_sync(0xffffffffu, (int)cur_have, it & 31) != 0;
        cp_async_wait<C::STAGES - 2>();  // this lane's copies of tile it have landed
        const uint32_t slots = my_slots + (it % C::STAGES) * C::STAGE_WARP;

        float s[NT][4];
#pragma unroll
        for (int t = 0; t < NT; ++t) s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
#pragma unroll
        for (int j = 0; j < C::KB; ++j) {
            const uint4 r0 = lds128(slots + j * 512), r1 = lds128(slots + (C::KB + j) * 512);
            const uint32_t w0[4] = {r0.x, r0.y, r0.z, r0.w}, w1[4] = {r1.x, r1.y, r1.z, r1.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                uint32_t a[4];
                codes_to_half2<FMT>(w0[e], a[0], a[2]);
                codes_to_half2<FMT>(w1[e], a[1], a[3]);
#pragma unroll
                for (int t = 0; t < NT; ++t) mma16816<false>(s[t], a, qb[t][4 * j + e][0], qb[t][4 * j + e][1]);
            }
        }
        // scores in log2 units, with the range, page and causal limits
        const int key0 = k0 + (warp + it * kWarps) * kTileKeys;
        const bool mask = !have || key0 + kTileKeys > k1 || (CAUSAL && key0 + kTileKeys - 1 > len - p.Nq);
        bool need = false;
        float x[NT][4];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float v = s[t][e] * (ks * qmul[t][e & 1]);
                if (mask) {
                    const int key = key0 + g + (e >> 1) * 8;
                    if (!have || key >= k1 || key > lim[t][e & 1]) v = -INFINITY;
                }
                x[t][e] = v;
                need |= v > m[t][e & 1] + kTau || v + lv > mw[t][e & 1] + kTau;
            }
        if (__any_sync(0xffffffffu, need)) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float mx = fmaxf(x[t][e], x[t][e + 2]);
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                    if (mx > m[t][e] + kTau) {
                        l[t][e] *= ex2_approx(m[t][e] - mx);  // 0 when m was -inf
                        m[t][e] = mx;
                    }
                    const float mv = mx + lv;
                    if (mv > mw[t][e] + kTau) {
                        const float f = ex2_approx(mw[t][e] - mv);
                        mw[t][e] = mv;
#pragma unroll
                        for (int i = 0; i < MT; ++i) {
                            o[t][i][e] *= f;
                            o[t][i][e + 2] *= f;
                        }
                    }
                }
        }
        uint32_t pb[NT][2];  // weights as B fragments: keys 2c, 2c + 1 (+ 8) of row g
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            float w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float mr = m[t][e & 1] == -INFINITY ? 0.f : m[t][e & 1];
                const float wr = mw[t][e & 1] == -INFINITY ? 0.f : mw[t][e & 1];
                l[t][e & 1] += ex2_approx(x[t][e] - mr);
                w[e] = ex2_approx((x[t][e] + lv) - wr);
            }
            const __half2 h0 = __floats2half2_rn(w[0], w[1]), h1 = __floats2half2_rn(w[2], w[3]);
            pb[t][0] = movmatrix_trans(*reinterpret_cast<const uint32_t *>(&h0));
            pb[t][1] = movmatrix_trans(*reinterpret_cast<const uint32_t *>(&h1));
        }
        // O^T += Vc^T P^T: words of four keys interleaved into pairs of keys
        auto v_words = [&](uint32_t v0, uint32_t v1, uint32_t v2, uint32_t v3, int i) {
            uint32_t a[4];
            codes_to_half2<FMT>(__byte_perm(v0, v1, 0x5140), a[0], a[1]);
            codes_to_half2<FMT>(__byte_perm(v2, v3, 0x5140), a[2], a[3]);
#pragma unroll
            for (int t = 0; t < NT; ++t) mma16816<false>(o[t][i], a, pb[t][0], pb[t][1]);
            codes_to_half2<FMT>(__byte_perm(v0, v1, 0x7362), a[0], a[1]);
            codes_to_half2<FMT>(__byte_perm(v2, v3, 0x7362), a[2], a[3]);
#pragma unroll
            for (int t = 0; t < NT; ++t) mma16816<false>(o[t][i + 1], a, pb[t][0], pb[t][1]);
        };
        const uint32_t vslots = slots + 2 * C::KB * 512;
        if constexpr (D == 128) {
            const uint4 v0 = lds128(vslots), v1 = lds128(vslots + 512), v2 = lds128(vslots + 1024), v3 = lds128(vslots + 1536);
            v_words(v0.x, v1.x, v2.x, v3.x, 0);
            v_words(v0.y, v1.y, v2.y, v3.y, 2);
            v_words(v0.z, v1.z, v2.z, v3.z, 4);
            v_words(v0.w, v1.w, v2.w, v3.w, 6);
        } else {
            const uint4 v01 = lds128(vslots), v23 = lds128(vslots + 512);  // two keys' 8 bytes each
            v_words(v01.x, v01.z, v23.x, v23.z, 0);
            v_words(v01.y, v01.w, v23.y, v23.w, 2);
        }
        // refill: tile it + STAGES - 1 goes into the stage that tile it - 1 left (read before this point)
        const int nx = it + C::STAGES - 1;
        if ((nx & 31) == 0) load_pages(nx);
        issue(nx, nx % C::STAGES);
    }
    cp_async_wait<0>();

    // merge the warps: l over the lanes of a row, O relative to m
    __syncthreads();  // the copies' slots are free
    float *sm_m = reinterpret_cast<float *>(sm), *sm_l = sm_m + kWarps * RT, *sm_o = sm_l + kWarps * RT;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float ls = l[t][e];
            ls += __shfl_xor_sync(0xffffffffu, ls, 4);
            ls += __shfl_xor_sync(0xffffffffu, ls, 8);
            ls += __shfl_xor_sync(0xffffffffu, ls, 16);
            const int r = 8 * t + 2 * c + e;
            if (g == 0) {
                sm_m[warp * RT + r] = m[t][e];
                sm_l[warp * RT + r] = ls;
            }
            const float f = mw[t][e] == -INFINITY ? 0.f : ex2_approx(mw[t][e] - m[t][e]);
            // value (i, e2) of lane g is head column (D / 8) g + 2 i + e2, kept at 16 i + 2 g + e2
            float *dst = sm_o + (warp * RT + r) * C::PITCH + 2 * g;
#pragma unroll
            for (int i = 0; i < MT; ++i)
                *reinterpret_cast<float2 *>(dst + 16 * i) = make_float2(o[t][i][e] * f, o[t][i][e + 2] * f);
        }
    __syncthreads();
    for (int idx = threadIdx.x; idx < RT * D; idx += kWarps * 32) {
        const int r = idx / D, dim = idx % D;
        const int row = row0 + r;
        if (row >= p.rows) continue;
        const int at = ((dim % C::VB) >> 1) * 16 + (dim / C::VB) * 2 + (dim & 1);
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm_m[w * RT + r]);
        float L = 0.f, A = 0.f;
        if (M != -INFINITY) {
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = ex2_approx(sm_m[w * RT + r] - M);  // 0 for a warp that saw nothing
                L += f * sm_l[w * RT + r];
                A += f * sm_o[(w * RT + r) * C::PITCH + at];
            }
        }
        const float val = L > 0.f ? A / L : 0.f;
        const float lse = L > 0.f ? (M + lg2_approx(L)) * kLn2 : -INFINITY;
        const size_t grow = row_base + row;
        if (n_chunks == 1) {
            static_cast<T *>(p.out)[grow * D + dim] = from_float<T>(val);
            if (dim == 0) p.lse[grow] = lse;
        } else {
            const size_t prow = (size_t)split * p.rows_total + grow;
            p.o_part[prow * D + dim] = val;
            if (dim == 0) p.lse_part[prow] = lse;
        }
    }
}

// One CTA of D threads per query row: the chunks' summaries merged onto their common maximum
// (fa_splitkv.cu's rule). Rows whose sequence needed one chunk are already written.
template <typename T, int D>
__global__ void __launch_bounds__(D) fa_kvq8_combine(const Q8Params p) {
    grid_dependency_wait();
    const int row = blockIdx.x;
    bool bad;
    const int len = q8_len(p, row / (p.H * p.Nq), bad);
    const int n = (len + p.split_len - 1) / p.split_len;
    if (n <= 1) return;
    const int e = threadIdx.x;
    float M = -INFINITY;
    for (int s = 0; s < n; ++s) M = fmaxf(M, p.lse_part[(size_t)s * p.rows_total + row]);
    float W = 0.f, A = 0.f;
    if (M != -INFINITY) {
#pragma unroll 4
        for (int s = 0; s < n; ++s) {
            const size_t at = (size_t)s * p.rows_total + row;
            const float w = __expf(p.lse_part[at] - M);  // 0 for an empty chunk
            W += w;
            A = fmaf(w, p.o_part[at * D + e], A);
        }
    }
    static_cast<T *>(p.out)[(size_t)row * D + e] = from_float<T>(W > 0.f ? A / W : 0.f);
    if (e == 0) p.lse[row] = W > 0.f ? M + __logf(W) : -INFINITY;
}

int page_log2(int page) {
    int s = 0;
    while ((1 << s) < page) ++s;
    return s;
}

template <typename T, int D, int FMT, int NT, bool CAUSAL>
int launch_q8(const Kvq8AttnArgs &a) {
    using C = Q8Cfg<D>;
    constexpr int merge = kWarps * 8 * NT * (2 + C::PITCH) * 4;
    constexpr int smem = C::SMEM > merge ? C::SMEM : merge;
    auto kern = fa_kvq8_partial<T, D, FMT, NT, CAUSAL>;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return -5;
    Q8Params p;
    p.q = a.q;
    p.out = a.out;
    p.lse = a.lse;
    p.k_codes = a.c.k_codes;
    p.v_codes = a.c.v_codes;
    p.k_scale = a.c.k_scale;
    p.v_scale = a.c.v_scale;
    p.page_table = a.c.page_table;
    p.kv_lens = a.kv_lens;
    p.o_part = a.o_part;
    p.lse_part = a.lse_part;
    p.status = a.status;
    p.H = a.H;
    p.Hkv = a.c.Hkv;
    p.Nq = a.Nq;
    p.rows = a.H / a.c.Hkv * a.Nq;
    p.row_tiles = (p.rows + 8 * NT - 1) / (8 * NT);
    p.rows_total = a.B * a.H * a.Nq;
    p.n_pages = a.c.n_pages;
    p.max_pages = a.c.max_pages;
    p.page_shift = page_log2(a.c.page);
    p.max_len = a.max_len;
    p.split_len = kvq8_split_len(a.max_len, a.n_splits);
    p.n_splits = (a.max_len + p.split_len - 1) / p.split_len;
    p.scale_log2 = static_cast<float>(static_cast<double>(a.scale) * 1.4426950408889634);
    const long long grid = (long long)p.n_splits * p.row_tiles * a.c.Hkv * a.B;
    if (grid > INT32_MAX) return -3;
    kern<<<static_cast<unsigned>(grid), kWarps * 32, smem, a.stream>>>(p);
    if (cudaGetLastError() != cudaSuccess) return -5;
    if (p.n_splits == 1) return 0;
    return launch_dependent(fa_kvq8_combine<T, D>, dim3(p.rows_total), dim3(D), 0, a.stream, p) == cudaSuccess ? 0 : -5;
}

template <typename T, int D, int FMT>
int launch_q8_rows(const Kvq8AttnArgs &a) {
    const int rows = a.H / a.c.Hkv * a.Nq;
    if (rows <= 8) return a.causal ? launch_q8<T, D, FMT, 1, true>(a) : launch_q8<T, D, FMT, 1, false>(a);
    return a.causal ? launch_q8<T, D, FMT, 2, true>(a) : launch_q8<T, D, FMT, 2, false>(a);
}

template <typename T>
int launch_q8_t(const Kvq8AttnArgs &a) {
    const bool i8 = a.c.format == kKvq8Int8;
    if (a.c.d == 128) return i8 ? launch_q8_rows<T, 128, kKvq8Int8>(a) : launch_q8_rows<T, 128, kKvq8E4m3>(a);
    if (a.c.d == 64) return i8 ? launch_q8_rows<T, 64, kKvq8Int8>(a) : launch_q8_rows<T, 64, kKvq8E4m3>(a);
    return -4;
}

}  // namespace

int kvq8_split_len(int max_len, int n_splits) {
    const int n = (int)(((long long)max_len + n_splits - 1) / n_splits);
    return (int)(((long long)n + 63) / 64 * 64);  // a whole tile for each warp
}

int kvq8_num_splits(int B, int Hkv, int rows, int max_len, int d, int num_sms) {
    const int tiles = rows <= 8 ? 1 : (rows + 15) / 16;
    const long long units = (long long)B * Hkv * tiles;
    const long long slots = 3ll * num_sms;  // resident CTAs: 64 KB of shared memory each
    const long long by_len = ((long long)max_len + 63) / 64;
    long long n = slots / units;
    const long long fine = (max_len + 1023) / 1024;  // at most 1024 keys: ragged batches stay balanced
    if (n < fine) n = fine;
    if (n > by_len) n = by_len;
    return n < 1 ? 1 : (int)n;
}

int launch_kvq8_attention(const Kvq8AttnArgs &a, bool fp16) {
    return fp16 ? launch_q8_t<__half>(a) : launch_q8_t<__nv_bfloat16>(a);
}

}  // namespace fa
