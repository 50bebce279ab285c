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
constexpr float kNone = -1e30f;  // reference maximum of a row that has seen no key
constexpr float kLn2 = 0.6931471805599453f;

template <int D, int NT>
struct Q8Cfg {
    static constexpr int KB = D / 64;                   // 16-byte units of a K row per lane
    static constexpr int VB = D / 8;                    // bytes of a V row per lane
    static constexpr int VW = VB / 4;                   // words of a V row per lane
    static constexpr int PITCH = D + 8;  // floats per row of the merge buffer
    static constexpr int RT = 8 * NT;    // query rows per unit
    static constexpr int CTAS = NT == 1 ? 4 : 3;  // per SM: 128 or 168 registers per thread
};

struct Q8Params {
    const void *q;
    void *out;
    float *lse;
    const uint8_t *k_codes, *v_codes;
    const float *k_scale, *v_scale;
    const int *page_table, *kv_lens;
    float *o_part, *lse_part;  // [parts][2][RT][d], [parts][2][RT]
    int *status;
    int B, H, Hkv, Nq, rows, row_tiles;  // rows = (H / Hkv) Nq query rows share a K/V head, in row_tiles tiles
    int n_pages, max_pages, page_shift;
    int max_len, parts;
    float scale_log2;
};

// The work is a line of 16-key tiles: sequence by sequence, in each the units (K/V head, row tile), in each unit the
// tiles of its keys. Part p takes tiles [p per, (p + 1) per): every part does the same amount of work, whatever the
// lengths are, and they need not be known on the host.
__device__ __forceinline__ int q8_part_tiles(int total, int parts) {
    const int per = (total + parts - 1) / parts;
    return max((per + kWarps - 1) / kWarps * kWarps, kWarps);  // whole rounds of the CTA's warps
}

// 16-key tiles of sequence b; a length out of range counts as 0.
__device__ __forceinline__ int q8_len(const Q8Params &p, int b, bool &bad) {
    const int len = __ldg(p.kv_lens + b);
    bad = len < 0 || len > p.max_len;
    return bad ? 0 : len;
}
__device__ __forceinline__ int q8_tiles(int len) { return (len + kTileKeys - 1) / kTileKeys; }

// Sum over the CTA (THREADS threads, sum[] of THREADS / 32 ints in shared memory); ends with a barrier.
template <int THREADS>
__device__ __forceinline__ int cta_sum(int v, int *sum) {
    v = __reduce_add_sync(0xffffffffu, v);
    if ((threadIdx.x & 31) == 0) sum[threadIdx.x >> 5] = v;
    __syncthreads();
    int s = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) s += sum[w];
    __syncthreads();
    return s;
}

__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// D(16x8, fp32) += A(16x16, row) * B(16x8, col) in fp16 (fragments as in warp_mma.cuh); not volatile, so
// that the compiler may interleave it with the conversions.
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// N words of the cache (16 or 8 bytes), read once.
template <int N>
__device__ __forceinline__ void load_codes(const uint8_t *src, uint32_t (&w)[N]) {
    if constexpr (N == 4) {
        const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(src));
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else {
        const uint2 v = __ldcs(reinterpret_cast<const uint2 *>(src));
        w[0] = v.x, w[1] = v.y;
    }
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
__global__ void __launch_bounds__(kWarps * 32, Q8Cfg<D, NT>::CTAS) fa_kvq8_partial(const Q8Params p) {
    using C = Q8Cfg<D, NT>;
    constexpr int KS = D / 16;   // MMA steps over the head dimension
    constexpr int MT = D / 16;   // 16-row tiles of O^T
    constexpr int RT = C::RT;
    __shared__ float sm_m[kWarps * RT], sm_l[kWarps * RT];
    __shared__ __align__(16) float sm_o[kWarps * RT * C::PITCH];
    __shared__ int sm_scan[kWarps];
    grid_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, c = lane & 3;
    const int page_mask = (1 << p.page_shift) - 1;
    const int units = p.Hkv * p.row_tiles;  // per sequence

    // ---------------------------------------------------------------- this CTA's stretch of the line
    int cur, end, b = 0, base = 0, len = 0;  // base: first tile of sequence b
    {
        int mine = 0, first = 0;  // first: the tiles of this thread's first sequence
        for (int s = threadIdx.x; s < p.B; s += kWarps * 32) {
            bool bad;
            const int n = q8_tiles(q8_len(p, s, bad)) * units;
            if (bad && blockIdx.x == 0) atomicExch(p.status, kStatusSeqlensQ8);
            if (s == threadIdx.x) first = n;
            mine += n;
        }
        const int total = cta_sum<kWarps * 32>(mine, sm_scan);
        const int per = q8_part_tiles(total, p.parts);
        if ((long long)blockIdx.x * per >= total) return;
        cur = blockIdx.x * per;
        end = min(total, cur + per);
        // the sequence that holds tile cur: blocks of 128 sequences, each scanned by the CTA
        for (int s0 = 0;; s0 += kWarps * 32) {
            int n = first;
            if (s0 > 0) {
                bool bad;
                n = s0 + (int)threadIdx.x < p.B ? q8_tiles(q8_len(p, s0 + threadIdx.x, bad)) * units : 0;
            }
            int incl = n;
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const int v = __shfl_up_sync(0xffffffffu, incl, d);
                if (lane >= d) incl += v;
            }
            if (lane == 31) sm_scan[warp] = incl;
            __syncthreads();
            int before = base, all = base;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                before += w < warp ? sm_scan[w] : 0;
                all += sm_scan[w];
            }
            __syncthreads();
            if (cur >= all) {  // the same for every thread; cur < total, so some block holds it
                base = all;
                continue;
            }
            const int from = before + incl - n;
            if (cur >= from && cur < from + n) {  // one thread
                sm_scan[0] = s0 + threadIdx.x;
                sm_scan[1] = from;
            }
            __syncthreads();
            b = sm_scan[0];
            base = sm_scan[1];
            break;
        }
        bool bad;
        len = q8_len(p, b, bad);
    }
    const int start = cur;

    while (cur < end) {
        int seq_tiles = q8_tiles(len);
        while (cur >= base + seq_tiles * units) {  // on to the next sequence that has keys
            base += seq_tiles * units;
            bool bad;
            len = q8_len(p, ++b, bad);
            seq_tiles = q8_tiles(len);
        }
        const int unit = (cur - base) / seq_tiles;
        const int tile0 = cur - base - unit * seq_tiles;
        const int n_tiles = min(seq_tiles - tile0, end - cur);
        const bool whole = n_tiles == seq_tiles;
        const int part_slot = 2 * blockIdx.x + (cur == start ? 0 : 1);
        cur += n_tiles;
        const int kvh = unit / p.row_tiles, rt = unit - kvh * p.row_tiles;
        const int k0 = tile0 * kTileKeys, k1 = min(len, k0 + n_tiles * kTileKeys);
        const int row0 = rt * RT;  // first of the unit's rows among the rows of the K/V head
        const size_t row_base = ((size_t)b * p.H + (size_t)kvh * (p.H / p.Hkv)) * p.Nq;
        const int my_tiles = n_tiles > warp ? (n_tiles - warp + kWarps - 1) / kWarps : 0;

        // Lane i looks after tile 32 n + i of this warp: its page and scales. The page numbers are read a window
        // of 32 tiles ahead.
        const int *table = p.page_table + (size_t)b * p.max_pages;
        const int lane_key = k0 + (warp + lane * kWarps) * kTileKeys;  // + 32 kWarps kTileKeys per window
        int ahead = lane_key < k1 ? __ldg(table + (lane_key >> p.page_shift)) : -1;
        int pg = -1;
        float pg_ks = 0.f, pg_lv = -INFINITY;
        auto load_pages = [&](int it0) {  // the window that starts at tile it0 (a multiple of 32)
            const int key = lane_key + it0 * kWarps * kTileKeys;
            pg = -1;
            if (key < k1) {
                if (ahead >= 0 && ahead < p.n_pages) {
                    pg = ahead;
                    const size_t at = (size_t)pg * p.Hkv + kvh;
                    pg_ks = __ldg(p.k_scale + at) * p.scale_log2;
                    pg_lv = lg2_approx(__ldg(p.v_scale + at));  // -inf for a page of zeros
                } else {
                    atomicExch(p.status, kStatusPage);
                }
            }
            const int next = key + 32 * kWarps * kTileKeys;
            ahead = next < k1 ? __ldg(table + (next >> p.page_shift)) : -1;
        };
        // This lane's codes of one tile: K rows g and g + 8 (dims 64 j + 16 c ..), V rows 2c, 2c + 1, 2c + 8,
        // 2c + 9 (dims VB g ..). Keys past the stretch and pages that are none are read as zeros; only a
        // stretch's last tile looks at single keys.
        uint32_t kw[2][C::KB][4], vw[4][C::VW];
        const uint8_t *k_lane = p.k_codes + g * D + c * 16, *v_lane = p.v_codes + 2 * c * D + g * C::VB;
        size_t off = 0;  // byte offset of the tile whose K was loaded last
        int n_keys = 0;  // how many of its keys there are to read
        auto load_k = [&](int it) {
            const int page = __shfl_sync(0xffffffffu, pg, it & 31);
            const int key0 = k0 + (warp + it * kWarps) * kTileKeys;
            off = ((((size_t)(page >= 0 ? page : 0) * p.Hkv + kvh) << p.page_shift) + (size_t)(key0 & page_mask)) * D;
            n_keys = page >= 0 ? k1 - key0 : 0;
            const uint8_t *src = k_lane + off;
            if (n_keys >= kTileKeys) {
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int j = 0; j < C::KB; ++j) load_codes(src + 8 * r * D + j * 64, kw[r][j]);
            } else {
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int j = 0; j < C::KB; ++j) {
                        kw[r][j][0] = kw[r][j][1] = kw[r][j][2] = kw[r][j][3] = 0u;
                        if (g + 8 * r < n_keys) load_codes(src + 8 * r * D + j * 64, kw[r][j]);
                    }
            }
        };
        auto load_v = [&]() {
            const uint8_t *src = v_lane + off;
            if (n_keys >= kTileKeys) {
#pragma unroll
                for (int i = 0; i < 4; ++i) load_codes(src + ((i & 1) + (i >> 1) * 8) * D, vw[i]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int key = (i & 1) + (i >> 1) * 8;
#pragma unroll
                    for (int e = 0; e < C::VW; ++e) vw[i][e] = 0u;
                    if (2 * c + key < n_keys) load_codes(src + key * D, vw[i]);
                }
            }
        };
        load_pages(0);
        if (my_tiles > 0) {
            load_k(0);
            load_v();
        }

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
                m[t][e] = mw[t][e] = kNone;
                l[t][e] = 0.f;
            }
        }

        for (int it = 0; it < my_tiles; ++it) {
            float x[NT][4];
            const float ks = __shfl_sync(0xffffffffu, pg_ks, it & 31), lv = __shfl_sync(0xffffffffu, pg_lv, it & 31);
            const int key0 = k0 + (warp + it * kWarps) * kTileKeys;
            const int in_tile = n_keys;  // of this tile
            // S^T = Kc Q^T
#pragma unroll
            for (int t = 0; t < NT; ++t) x[t][0] = x[t][1] = x[t][2] = x[t][3] = 0.f;
#pragma unroll
            for (int j = 0; j < C::KB; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    uint32_t a[4];
                    codes_to_half2<FMT>(kw[0][j][e], a[0], a[2]);
                    codes_to_half2<FMT>(kw[1][j][e], a[1], a[3]);
#pragma unroll
                    for (int t = 0; t < NT; ++t) mma_f16(x[t], a, qb[t][4 * j + e][0], qb[t][4 * j + e][1]);
                }
            // the next tile's K, in flight during the rest of this step
            const bool next = it + 1 < my_tiles;
            if (next) {
                if (((it + 1) & 31) == 0) load_pages(it + 1);
                load_k(it + 1);
            }
            // scores in log2 units, with the range, page and causal limits
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[t][e] *= ks * qmul[t][e & 1];
            if (in_tile < kTileKeys || (CAUSAL && key0 + kTileKeys - 1 > len - p.Nq)) {
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int r = g + (e >> 1) * 8;
                        if (r >= in_tile || key0 + r > lim[t][e & 1]) x[t][e] = -INFINITY;
                    }
            }
            bool need = false;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float mx = fmaxf(x[t][e], x[t][e + 2]);
                    need |= mx > m[t][e] + kTau || mx + lv > mw[t][e] + kTau;
                }
            if (__any_sync(0xffffffffu, need)) {
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float mx = fmaxf(x[t][e], x[t][e + 2]);
#pragma unroll
                        for (int s = 4; s <= 16; s *= 2) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
                        if (mx > m[t][e] + kTau) {
                            l[t][e] *= ex2_approx(m[t][e] - mx);  // 0 from kNone
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
            // weights w = p 2^(lv + m - mw) as B fragments: keys 2c, 2c + 1 (+ 8) of row g
            uint32_t pb[NT][2];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                float f[2], w[4];
#pragma unroll
                for (int e = 0; e < 2; ++e)  // (the limit: a row that saw only pages of zeros has m - mw = 1e30, and w = 0 here)
                    f[e] = ex2_approx(fminf(lv + (m[t][e] - mw[t][e]), 120.0f));
#pragma unroll
                for (int e = 0; e < 4; ++e) w[e] = ex2_approx(x[t][e] - m[t][e & 1]);
                l[t][0] += w[0] + w[2];
                l[t][1] += w[1] + w[3];
                const __half2 h0 = __floats2half2_rn(w[0] * f[0], w[1] * f[1]), h1 = __floats2half2_rn(w[2] * f[0], w[3] * f[1]);
                pb[t][0] = movmatrix_trans(*reinterpret_cast<const uint32_t *>(&h0));
                pb[t][1] = movmatrix_trans(*reinterpret_cast<const uint32_t *>(&h1));
            }
            // O^T += Vc^T P^T: words of four keys interleaved into pairs of keys
#pragma unroll
            for (int i = 0; i < C::VW; ++i) {
                uint32_t a[4];
                codes_to_half2<FMT>(__byte_perm(vw[0][i], vw[1][i], 0x5140), a[0], a[1]);
                codes_to_half2<FMT>(__byte_perm(vw[2][i], vw[3][i], 0x5140), a[2], a[3]);
#pragma unroll
                for (int t = 0; t < NT; ++t) mma_f16(o[t][2 * i], a, pb[t][0], pb[t][1]);
                codes_to_half2<FMT>(__byte_perm(vw[0][i], vw[1][i], 0x7362), a[0], a[1]);
                codes_to_half2<FMT>(__byte_perm(vw[2][i], vw[3][i], 0x7362), a[2], a[3]);
#pragma unroll
                for (int t = 0; t < NT; ++t) mma_f16(o[t][2 * i + 1], a, pb[t][0], pb[t][1]);
            }
            if (next) load_v();
        }

        // merge the warps: l over the lanes of a row, O relative to m
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
                const float f = ex2_approx(mw[t][e] - m[t][e]);  // 0 where every weight was (mw = kNone)
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
            float M = kNone;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm_m[w * RT + r]);
            float L = 0.f, A = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = ex2_approx(sm_m[w * RT + r] - M);  // 0 for a warp that saw nothing, unless none did
                L += f * sm_l[w * RT + r];
                A += f * sm_o[(w * RT + r) * C::PITCH + at];
            }
            const float val = L > 0.f ? A / L : 0.f;
            const float lse = L > 0.f ? (M + lg2_approx(L)) * kLn2 : -INFINITY;
            if (whole) {
                static_cast<T *>(p.out)[(row_base + row) * D + dim] = from_float<T>(val);
                if (dim == 0) p.lse[row_base + row] = lse;
            } else {
                const size_t at_part = (size_t)part_slot * RT + r;
                p.o_part[at_part * D + dim] = val;
                if (dim == 0) p.lse_part[at_part] = lse;
            }
        }
        __syncthreads();  // the merge buffer is free
    }
}

// One CTA per query row: the summaries of the parts that share its unit, merged onto their common maximum
// (fa_splitkv.cu's rule), the parts spread over the CTA's groups of D / 4 threads. A unit that one part did alone is
// written already; one without keys gets out = 0, lse = -inf.
constexpr int kCombineThreads = 256;
template <typename T, int D, int RT>
__global__ void __launch_bounds__(kCombineThreads) fa_kvq8_combine(const Q8Params p) {
    constexpr int LANES = D / 4, GROUPS = kCombineThreads / LANES;
    __shared__ int sm_sum[kCombineThreads / 32];
    __shared__ float sm_max[kCombineThreads / 32], sm_w[GROUPS];
    __shared__ float4 sm_a[GROUPS][LANES];
    const int units = p.Hkv * p.row_tiles;
    const int heads_rows = p.rows;  // rows of one K/V head
    const int b = blockIdx.x / (p.Hkv * heads_rows), in_seq = blockIdx.x - b * p.Hkv * heads_rows;
    const int kvh = in_seq / heads_rows, row = in_seq - kvh * heads_rows;
    const int unit = kvh * p.row_tiles + row / RT, r = row % RT;
    int before = 0, after = 0;
    for (int s = threadIdx.x; s < p.B; s += kCombineThreads) {
        bool bad;
        const int n = q8_tiles(q8_len(p, s, bad)) * units;
        if (s < b) before += n;
        else after += n;
    }
    before = cta_sum<kCombineThreads>(before, sm_sum);
    const int total = before + cta_sum<kCombineThreads>(after, sm_sum);
    const int per = q8_part_tiles(total, p.parts);
    bool bad;
    const int tiles = q8_tiles(q8_len(p, b, bad));
    const int first = before + unit * tiles;
    const int p0 = first / per, n = tiles > 0 ? (first + tiles - 1) / per - p0 + 1 : 0;
    grid_dependency_wait();
    if (n == 1) return;
    // part p0 may begin in an earlier unit; every later one begins in this one
    const int slot0 = 2 * p0 + (p0 * per >= first ? 0 : 1);
    auto at = [&](int s) { return (size_t)(s == 0 ? slot0 : 2 * (p0 + s)) * RT + r; };
    float M = -INFINITY;
    for (int s = threadIdx.x; s < n; s += kCombineThreads) M = fmaxf(M, p.lse_part[at(s)]);
#pragma unroll
    for (int d = 16; d > 0; d /= 2) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
    if ((threadIdx.x & 31) == 0) sm_max[threadIdx.x >> 5] = M;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kCombineThreads / 32; ++w) M = fmaxf(M, sm_max[w]);
    const int group = threadIdx.x / LANES, lane = threadIdx.x % LANES;
    float W = 0.f;
    float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
    if (M != -INFINITY) {
#pragma unroll 4
        for (int s = group; s < n; s += GROUPS) {
            const size_t i = at(s);
            const float w = __expf(p.lse_part[i] - M);  // 0 for a part that saw no key
            const float4 v = *reinterpret_cast<const float4 *>(p.o_part + i * D + 4 * lane);
            W += w;
            A.x = fmaf(w, v.x, A.x);
            A.y = fmaf(w, v.y, A.y);
            A.z = fmaf(w, v.z, A.z);
            A.w = fmaf(w, v.w, A.w);
        }
    }
    sm_a[group][lane] = A;
    if (lane == 0) sm_w[group] = W;
    __syncthreads();
    if (threadIdx.x >= D) return;
    float sum = 0.f, den = 0.f;
#pragma unroll
    for (int i = 0; i < GROUPS; ++i) {
        sum += reinterpret_cast<const float *>(sm_a[i])[threadIdx.x];
        den += sm_w[i];
    }
    const size_t out_row = (size_t)blockIdx.x;  // rows are in the order of q
    static_cast<T *>(p.out)[out_row * D + threadIdx.x] = from_float<T>(den > 0.f ? sum / den : 0.f);
    if (threadIdx.x == 0) p.lse[out_row] = den > 0.f ? M + __logf(den) : -INFINITY;
}

int page_log2(int page) {
    int s = 0;
    while ((1 << s) < page) ++s;
    return s;
}

// Row tiles of the kernel: 8 query rows per MMA column tile, one tile or two.
int rows_per_unit(int rows) { return rows <= 8 ? 8 : 16; }

template <typename T, int D, int FMT, int NT, bool CAUSAL>
int launch_q8(const Kvq8AttnArgs &a) {
    using C = Q8Cfg<D, NT>;
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
    p.o_part = a.workspace;
    p.lse_part = a.workspace + (size_t)a.parts * 2 * C::RT * D;
    p.status = a.status;
    p.B = a.B;
    p.H = a.H;
    p.Hkv = a.c.Hkv;
    p.Nq = a.Nq;
    p.rows = a.H / a.c.Hkv * a.Nq;
    p.row_tiles = (p.rows + C::RT - 1) / C::RT;
    p.n_pages = a.c.n_pages;
    p.max_pages = a.c.max_pages;
    p.page_shift = page_log2(a.c.page);
    p.max_len = a.max_len;
    p.parts = a.parts;
    p.scale_log2 = static_cast<float>(static_cast<double>(a.scale) * 1.4426950408889634);
    fa_kvq8_partial<T, D, FMT, NT, CAUSAL><<<a.parts, kWarps * 32, 0, a.stream>>>(p);
    if (cudaGetLastError() != cudaSuccess) return -5;
    return launch_dependent(fa_kvq8_combine<T, D, C::RT>, dim3(a.B * a.H * a.Nq), dim3(kCombineThreads), 0,
                            a.stream, p) == cudaSuccess
               ? 0
               : -5;
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

long long kvq8_tiles(int B, int Hkv, int rows, int max_len) {
    const int rt = rows_per_unit(rows);
    return (long long)B * Hkv * ((rows + rt - 1) / rt) * ((max_len + kTileKeys - 1) / kTileKeys);
}

int kvq8_num_parts(int B, int Hkv, int rows, int max_len, int num_sms) {
    // one part for each CTA that can be resident, and at least one tile for each of a CTA's warps
    const long long slots = (long long)(rows <= 8 ? Q8Cfg<128, 1>::CTAS : Q8Cfg<128, 2>::CTAS) * num_sms;
    const long long by_len = (kvq8_tiles(B, Hkv, rows, max_len) + kWarps - 1) / kWarps;
    return (int)(by_len < slots ? by_len : slots);
}

size_t kvq8_workspace_bytes(int rows, int d, int parts) {
    return (size_t)parts * 2 * rows_per_unit(rows) * (d + 1) * sizeof(float);
}

int launch_kvq8_attention(const Kvq8AttnArgs &a, bool fp16) {
    return fp16 ? launch_q8_t<__half>(a) : launch_q8_t<__nv_bfloat16>(a);
}

}  // namespace fa
