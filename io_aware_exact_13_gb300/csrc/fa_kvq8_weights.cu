// fa_kvq8_weights.cu -- the softmax weight that each key of the 8-bit cache receives.
//
// For K/V head h and key j of a sequence, with the query rows i that share the head and their log-sum-exp as the
// attention left it,
//     weight[h][j] += sum_i exp(s_ij - lse_i),     s_ij = scale (q_i . kc_j) ks(j),
// over the rows that see the key. A row that sees no key (lse = -inf) adds nothing. With lse known a key's sum needs no other
// key's, and nothing is merged.
//
// Bound: HBM, the K codes once and eight bytes of weight for each key and head. As in the attention (fa_kvq8_attn.cuh) the
// codes are the 16-row operand of 16x8x16 MMAs, cut from a lane's own 16-byte loads, and up to 32 query rows are the
// columns; further rows go over the stretch again. bf16 queries enter in fp16 under a power of two for each row.
// Measured: 64 sequences up to 8192 keys, 32 / 8 heads of 128, int8, 64 us (88 % of the copy rate); a CTA for each 256 keys of
// a head 125, the same with all its codes requested at once 115. One sequence of 509 keys, 8 heads of 64: 6.2. 12
// sequences up to 6001 keys, 20 rows for each of 4 heads of 64: 10.4 (12.5 with four tiles of rows instead of three).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "fa_kvq8.cuh"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kWarps = 4;
constexpr int kTileKeys = 16;
__host__ __device__ constexpr int w_ctas(int NT) { return NT >= 3 ? 3 : 4; }  // resident CTAs per SM: 168 or 128 registers

struct WeightParams {
    const void *q;
    const float *lse;
    float *weight;
    const uint8_t *k_codes;
    const float *k_scale;
    const int *page_table, *kv_lens;
    int *status;
    int B, H, Hkv, Nq, rows;
    int n_pages, max_pages, page_shift, max_len;
    float scale_log2;
};

__device__ __forceinline__ int w_len(const WeightParams &p, int b, bool &bad) {
    const int len = __ldg(p.kv_lens + b);
    bad = len < 0 || len > p.max_len;
    return bad ? 0 : len;
}
__host__ __device__ __forceinline__ int w_tiles(int len) { return (len + kTileKeys - 1) / kTileKeys; }

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The 16-key tiles of all sequences and K/V heads are one line, cut into equal stretches for the warps of one wave of CTAs
// (as in fa_kvq8_attn.cuh). A warp keeps the codes of two tiles in flight.
template <typename T, int D, int FMT, int NT, bool CAUSAL>
__global__ void __launch_bounds__(kWarps * 32, w_ctas(NT)) fa_kvq8_weights_kernel(const WeightParams p) {
    constexpr int KB = D / 64, KS = D / 16, DEPTH = 2;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int page_mask = (1 << p.page_shift) - 1;
    // this warp's stretch, and the sequence that it begins in
    int total = 0, s_bad = 0, b = 0, base = 0, len = 0;
    for (int s = lane; s < p.B; s += 32) {
        bool bad;
        total += w_tiles(w_len(p, s, bad)) * p.Hkv;
        s_bad |= bad;
    }
    total = __reduce_add_sync(0xffffffffu, total);
    if (s_bad && blockIdx.x == 0 && warp == 0) atomicExch(p.status, kStatusSeqlensQ8);
    const int warps = gridDim.x * kWarps, per = (total + warps - 1) / warps;
    // (neighbouring stretches in neighbouring CTAs: every SM gets some of a short line)
    const long long first = (long long)(warp * gridDim.x + blockIdx.x) * per;
    if (first >= total) return;
    int cur = (int)first;
    const int end = min(total, cur + per);
    for (int s0 = 0;; s0 += 32) {
        bool bad;
        const int l = s0 + lane < p.B ? w_len(p, s0 + lane, bad) : 0, n = w_tiles(l) * p.Hkv;
        int incl = n;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int v = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += v;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, cur < base + incl);
        if (past != 0) {
            const int at = __ffs(past) - 1;
            b = s0 + at;
            base += __shfl_sync(0xffffffffu, incl - n, at);
            len = __shfl_sync(0xffffffffu, l, at);
            break;
        }
        base += __shfl_sync(0xffffffffu, incl, 31);
    }

    while (cur < end) {
        int seq_tiles = w_tiles(len);
        while (cur >= base + seq_tiles * p.Hkv) {  // on to the next sequence that has keys
            base += seq_tiles * p.Hkv;
            bool bad;
            len = w_len(p, ++b, bad);
            seq_tiles = w_tiles(len);
        }
        const int kvh = (cur - base) / seq_tiles, tile0 = cur - base - kvh * seq_tiles;
        const int n_tiles = min(seq_tiles - tile0, end - cur);
        cur += n_tiles;
        const int k0 = tile0 * kTileKeys;
        const int *table = p.page_table + (size_t)b * p.max_pages;
        float *weight = p.weight + (((size_t)b * p.Hkv + kvh) * p.max_pages << p.page_shift);
        const size_t row_base = ((size_t)b * p.H + (size_t)kvh * (p.H / p.Hkv)) * p.Nq;
        for (int row0 = 0; row0 < p.rows; row0 += 8 * NT) {
            // Lane i looks after tile 32 n + i: its page and scale, the page numbers a window ahead.
            const int lane_key = k0 + lane * kTileKeys, past = k0 + n_tiles * kTileKeys;
            int ahead = lane_key < past ? __ldg(table + (lane_key >> p.page_shift)) : -1, pg = -1;
            float pg_ks = 0.f;
            auto load_pages = [&](int it0) {
                const int key = lane_key + it0 * kTileKeys;
                pg = -1;
                if (key < past) {
                    if (ahead >= 0 && ahead < p.n_pages) {
                        pg = ahead;
                        pg_ks = __ldg(p.k_scale + (size_t)pg * p.Hkv + kvh) * p.scale_log2;
                    } else {
                        atomicExch(p.status, kStatusPage);
                    }
                }
                const int next = key + 32 * kTileKeys;
                ahead = next < past ? __ldg(table + (next >> p.page_shift)) : -1;
            };
            struct Tile {
                uint32_t kw[2][KB][4];  // this lane's codes of keys g and g + 8
                float ks, before;       // scale log2 e times the page's; what key g + 8 c has received so far (c < 2)
                int n_keys;             // of its keys there are
            };
            auto load = [&](Tile &t, int it) {
                const int page = __shfl_sync(0xffffffffu, pg, it & 31);
                t.ks = __shfl_sync(0xffffffffu, pg_ks, it & 31);
                const int key0 = k0 + it * kTileKeys;
                t.n_keys = page < 0 ? 0 : len - key0;
                const uint8_t *src = p.k_codes + (((size_t)(page < 0 ? 0 : page) * p.Hkv + kvh << p.page_shift) + (size_t)(key0 & page_mask)) * D + g * D + c * 16;
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int j = 0; j < KB; ++j) {
                        uint4 v = make_uint4(0u, 0u, 0u, 0u);
                        if (g + 8 * r < t.n_keys) v = __ldcs(reinterpret_cast<const uint4 *>(src + 8 * r * D + j * 64));
                        t.kw[r][j][0] = v.x, t.kw[r][j][1] = v.y, t.kw[r][j][2] = v.z, t.kw[r][j][3] = v.w;
                    }
                t.before = c < 2 && g + 8 * c < t.n_keys ? weight[key0 + g + 8 * c] : 0.f;
            };
            load_pages(0);
            Tile buf[DEPTH];
#pragma unroll
            for (int i = 0; i < DEPTH; ++i)
                if (i < n_tiles) load(buf[i], i);

            // Q as B fragments: column g of tile t is row row0 + 8 t + g, the contraction in the order of the codes
            uint32_t qb[NT][KS][2];
            float qmul[NT][2], lse2[NT][2];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const int row = row0 + 8 * t + g;
                const T *from = static_cast<const T *>(p.q) + (row_base + row) * D;
#pragma unroll
                for (int j = 0; j < KB; ++j) {
                    uint4 w[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
                    if (row < p.rows) {
                        w[0] = __ldg(reinterpret_cast<const uint4 *>(from + 64 * j + 16 * c));
                        w[1] = __ldg(reinterpret_cast<const uint4 *>(from + 64 * j + 16 * c) + 1);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        qb[t][4 * j + e][0] = e == 0 ? w[0].x : e == 1 ? w[0].z : e == 2 ? w[1].x : w[1].z;
                        qb[t][4 * j + e][1] = e == 0 ? w[0].y : e == 1 ? w[0].w : e == 2 ? w[1].y : w[1].w;
                    }
                }
                float mul = 1.0f;
                if constexpr (std::is_same<T, __nv_bfloat16>::value) {
                    // the row's largest magnitude goes to [2^15, 2^16) as in the attention
                    uint32_t most = 0;
#pragma unroll
                    for (int s = 0; s < KS; ++s)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            most = max(most, max(qb[t][s][e] & 0x7FFFu, (qb[t][s][e] >> 16) & 0x7FFFu));
                    most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
                    most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
                    const uint32_t ex = max(most >> 7, 16u);
                    const float inv = __uint_as_float((269u - ex) << 23);
                    mul = __uint_as_float(ex << 23) * 0x1p-15f;
#pragma unroll
                    for (int s = 0; s < KS; ++s)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&qb[t][s][e]));
                            const __half2 o = __floats2half2_rn(f.x * inv, f.y * inv);
                            qb[t][s][e] = *reinterpret_cast<const uint32_t *>(&o);
                        }
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {  // of column 2c + e
                    qmul[t][e] = __shfl_sync(0xffffffffu, mul, 8 * c + 4 * e);
                    const int r = row0 + 8 * t + 2 * c + e;
                    const float l = r < p.rows ? __ldg(p.lse + row_base + r) : -INFINITY;
                    lse2[t][e] = l == -INFINITY ? INFINITY : l * 1.4426950408889634f;  // 2^-inf: such a row adds nothing
                }
            }

            auto step = [&](Tile &tile, int it) {
                float x[NT][4], sum[2] = {0.f, 0.f};
                const float ks = tile.ks, before = tile.before;
                const int key0 = k0 + it * kTileKeys, n_keys = tile.n_keys;
#pragma unroll
                for (int t = 0; t < NT; ++t) x[t][0] = x[t][1] = x[t][2] = x[t][3] = 0.f;
#pragma unroll
                for (int j = 0; j < KB; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t a[4];
                        codes_to_half2<FMT>(tile.kw[0][j][e], a[0], a[2]);
                        codes_to_half2<FMT>(tile.kw[1][j][e], a[1], a[3]);
#pragma unroll
                        for (int t = 0; t < NT; ++t) mma_f16(x[t], a, qb[t][4 * j + e][0], qb[t][4 * j + e][1]);
                    }
                if (it + DEPTH < n_tiles) {  // the tile that takes these registers
                    if (((it + DEPTH) & 31) == 0) load_pages(it + DEPTH);
                    load(tile, it + DEPTH);
                }
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float w = ex2_approx(fmaf(x[t][e], ks * qmul[t][e & 1], -lse2[t][e & 1]));
                        if constexpr (CAUSAL) {
                            const int last = len - p.Nq + (row0 + 8 * t + 2 * c + (e & 1)) % p.Nq;
                            if (key0 + g + (e >> 1) * 8 > last) w = 0.f;
                        }
                        sum[e >> 1] += w;
                    }
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 1);
                    sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 2);
                }
                if (c < 2 && g + 8 * c < n_keys) weight[key0 + g + 8 * c] = before + (c == 0 ? sum[0] : sum[1]);
            };
            for (int it = 0; it < n_tiles; it += DEPTH)
#pragma unroll
                for (int i = 0; i < DEPTH; ++i)
                    if (i == 0 || it + i < n_tiles) step(buf[i], it + i);
        }
    }
}

template <typename T, int D, int FMT, int NT>
int launch_nt(const Kvq8WeightsArgs &a, const WeightParams &p) {
    // one wave, no more CTAs than there can be tiles for their warps
    const long long tiles = (long long)a.B * p.Hkv * w_tiles(a.max_len), most = (long long)w_ctas(NT) * a.num_sms;
    const long long by_len = (tiles + kWarps - 1) / kWarps;
    const unsigned grid = (unsigned)(by_len < most ? by_len : most);
    if (a.causal)
        fa_kvq8_weights_kernel<T, D, FMT, NT, true><<<grid, kWarps * 32, 0, a.stream>>>(p);
    else
        fa_kvq8_weights_kernel<T, D, FMT, NT, false><<<grid, kWarps * 32, 0, a.stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? 0 : -5;
}

template <typename T, int D, int FMT>
int launch_t(const Kvq8WeightsArgs &a) {
    WeightParams p;
    p.q = a.q;
    p.lse = a.lse;
    p.weight = a.weight;
    p.k_codes = a.c.k_codes;
    p.k_scale = a.c.k_scale;
    p.page_table = a.c.page_table;
    p.kv_lens = a.kv_lens;
    p.status = a.status;
    p.B = a.B;
    p.H = a.H;
    p.Hkv = a.c.Hkv;
    p.Nq = a.Nq;
    p.rows = a.H / a.c.Hkv * a.Nq;
    p.n_pages = a.c.n_pages;
    p.max_pages = a.c.max_pages;
    p.page_shift = kvq8_page_shift(a.c.page);
    p.max_len = a.max_len;
    p.scale_log2 = static_cast<float>(static_cast<double>(a.scale) * 1.4426950408889634);
    if (p.rows <= 8) return launch_nt<T, D, FMT, 1>(a, p);
    if (p.rows <= 16) return launch_nt<T, D, FMT, 2>(a, p);
    // Three or four tiles of eight rows for each pass over a stretch: the fewest that hold all, or three where that takes no more
    // passes, or at d 128, where four spill. (64 sequences up to 4000 keys of 4 heads, three / four: d 64, 24 rows 23.4 / 27.0 us,
    // 32 39.2 / 25.9, 48 39.2 / 43.4, 64 51.5 / 41.4, 80 70.0 / 62.0; d 128 29.1 / 40.0, 47.9 / 39.1, 53.7 / 80.0, 72.1 / 74.4,
    // 89.5 / 102.7, 128 rows 148.5 / 152.6. With one tile 16 rows take 28.6 where two take 18.9.)
    const bool three = p.rows <= 24 || (p.rows > 32 && (D == 128 || (p.rows + 23) / 24 == (p.rows + 31) / 32));
    return three ? launch_nt<T, D, FMT, 3>(a, p) : launch_nt<T, D, FMT, 4>(a, p);
}

template <typename T>
int launch_type(const Kvq8WeightsArgs &a) {
    const bool i8 = a.c.format == kKvq8Int8;
    if (a.c.d == 128) return i8 ? launch_t<T, 128, kKvq8Int8>(a) : launch_t<T, 128, kKvq8E4m3>(a);
    return i8 ? launch_t<T, 64, kKvq8Int8>(a) : launch_t<T, 64, kKvq8E4m3>(a);
}

}  // namespace

int launch_kvq8_weights(const Kvq8WeightsArgs &a, bool fp16) {
    return fp16 ? launch_type<__half>(a) : launch_type<__nv_bfloat16>(a);
}

}  // namespace fa
