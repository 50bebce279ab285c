// fa_kvq8_weights.cu -- the softmax weight that each key of the 8-bit cache receives.
//
// For K/V head h and key j of a sequence, with the query rows i that share the head and their log-sum-exp as the
// attention left it,
//     weight[h][j] += sum_i exp(s_ij - lse_i),     s_ij = scale (q_i . kc_j) ks(j),
// over the rows that see the key. A row that sees no key (lse = -inf) adds nothing. With lse known a key's sum needs no other key's,
// so the keys are cut into fixed chunks and nothing is merged.
//
// Bound: HBM, the K codes once and eight bytes of weight for each key and head. As in the attention (fa_kvq8_attn.cu) the
// codes are the 16-row operand of 16x8x16 MMAs, cut from a lane's own 16-byte loads, and up to 32 query rows are the
// columns; further rows use the codes in the registers again. bf16 queries enter in fp16 under a power of two for each row.
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
// 16-key tiles of a warp, all in registers, and keys of a CTA.
__host__ __device__ constexpr int w_tiles(int D, int NT) { return D == 128 || NT == 4 ? 2 : 4; }
__host__ __device__ constexpr int w_chunk(int D, int NT) { return kWarps * w_tiles(D, NT) * kTileKeys; }

struct WeightParams {
    const void *q;
    const float *lse;
    float *weight;
    const uint8_t *k_codes;
    const float *k_scale;
    const int *page_table, *kv_lens;
    int *status;
    int H, Hkv, Nq, rows, chunks;
    int n_pages, max_pages, page_shift, max_len;
    float scale_log2;
};

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// One CTA: a chunk of keys of one (sequence, K/V head); warp w takes tiles w, w + kWarps, ...
template <typename T, int D, int FMT, int NT, bool CAUSAL>
__global__ void __launch_bounds__(kWarps * 32, NT == 4 ? 3 : 4) fa_kvq8_weights_kernel(const WeightParams p) {
    constexpr int KB = D / 64, KS = D / 16, kTiles = w_tiles(D, NT), kChunk = w_chunk(D, NT);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    int u = blockIdx.x;
    const int chunk = u % p.chunks;
    u /= p.chunks;
    const int kvh = u % p.Hkv, b = u / p.Hkv;
    int len = __ldg(p.kv_lens + b);
    if (len < 0 || len > p.max_len) {
        if (threadIdx.x == 0) atomicExch(p.status, kStatusSeqlensQ8);
        len = 0;
    }
    const int k0 = chunk * kChunk + warp * kTileKeys;
    if (k0 >= len) return;
    const int page_mask = (1 << p.page_shift) - 1;

    // this warp's tiles: the page, its scale, and the codes
    int n_keys[kTiles];
    float ks[kTiles];
    const uint8_t *src[kTiles];
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
        const int key = k0 + t * kWarps * kTileKeys;
        n_keys[t] = 0;
        ks[t] = 0.f;
        src[t] = p.k_codes;
        if (key < len) {
            const int pg = __ldg(p.page_table + (size_t)b * p.max_pages + (key >> p.page_shift));
            if (pg >= 0 && pg < p.n_pages) {
                const size_t unit = (size_t)pg * p.Hkv + kvh;
                n_keys[t] = min(len - key, kTileKeys);
                ks[t] = __ldg(p.k_scale + unit) * p.scale_log2;
                src[t] = p.k_codes + ((unit << p.page_shift) + (size_t)(key & page_mask)) * D + g * D + c * 16;
            } else if (lane == 0) {
                atomicExch(p.status, kStatusPage);
            }
        }
    }
    uint32_t kw[kTiles][2][KB][4];  // rows g and g + 8 of each tile
    float sum[kTiles][2], before[kTiles];
    float *weight = p.weight + (((size_t)b * p.Hkv + kvh) * p.max_pages << p.page_shift) + k0 + g + 8 * c;
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int j = 0; j < KB; ++j) {
                uint4 v = make_uint4(0u, 0u, 0u, 0u);
                if (g + 8 * r < n_keys[t]) v = __ldcs(reinterpret_cast<const uint4 *>(src[t] + 8 * r * D + j * 64));
                kw[t][r][j][0] = v.x, kw[t][r][j][1] = v.y, kw[t][r][j][2] = v.z, kw[t][r][j][3] = v.w;
            }
        sum[t][0] = sum[t][1] = 0.f;
    }
#pragma unroll
    for (int t = 0; t < kTiles; ++t)  // lanes c = 0, 1 look after keys g and g + 8
        before[t] = c < 2 && g + 8 * c < n_keys[t] ? weight[t * kWarps * kTileKeys] : 0.f;

    const size_t row_base = ((size_t)b * p.H + (size_t)kvh * (p.H / p.Hkv)) * p.Nq;
    for (int row0 = 0; row0 < p.rows; row0 += 8 * NT) {
        // Q as B fragments: column g of tile t is row row0 + 8 t + g, the contraction in the order of the codes
        uint32_t qb[NT][KS][2];
        float qmul[NT][2], lse2[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int row = row0 + 8 * t + g;
            const T *from = static_cast<const T *>(p.q) + (row_base + row) * D;
            uint32_t most = 0;
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
#pragma unroll
        for (int i = 0; i < kTiles; ++i) {
            float x[NT][4];
#pragma unroll
            for (int t = 0; t < NT; ++t) x[t][0] = x[t][1] = x[t][2] = x[t][3] = 0.f;
#pragma unroll
            for (int j = 0; j < KB; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    uint32_t a[4];
                    codes_to_half2<FMT>(kw[i][0][j][e], a[0], a[2]);
                    codes_to_half2<FMT>(kw[i][1][j][e], a[1], a[3]);
#pragma unroll
                    for (int t = 0; t < NT; ++t) mma_f16(x[t], a, qb[t][4 * j + e][0], qb[t][4 * j + e][1]);
                }
            const int key0 = k0 + i * kWarps * kTileKeys;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float w = ex2_approx(fmaf(x[t][e], ks[i] * qmul[t][e & 1], -lse2[t][e & 1]));
                    if constexpr (CAUSAL) {
                        const int last = len - p.Nq + (row0 + 8 * t + 2 * c + (e & 1)) % p.Nq;
                        if (key0 + g + (e >> 1) * 8 > last) w = 0.f;
                    }
                    sum[i][e >> 1] += w;
                }
        }
    }
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
        if (n_keys[i] == 0) continue;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            sum[i][r] += __shfl_xor_sync(0xffffffffu, sum[i][r], 1);
            sum[i][r] += __shfl_xor_sync(0xffffffffu, sum[i][r], 2);
        }
        if (c < 2 && g + 8 * c < n_keys[i]) weight[i * kWarps * kTileKeys] = before[i] + (c == 0 ? sum[i][0] : sum[i][1]);
    }
}

template <typename T, int D, int FMT, int NT>
int launch_nt(const Kvq8WeightsArgs &a, WeightParams &p) {
    p.chunks = (a.max_len + w_chunk(D, NT) - 1) / w_chunk(D, NT);
    const long long grid = (long long)p.chunks * p.Hkv * a.B;
    if (grid > INT32_MAX) return -3;
    if (a.causal)
        fa_kvq8_weights_kernel<T, D, FMT, NT, true><<<(unsigned)grid, kWarps * 32, 0, a.stream>>>(p);
    else
        fa_kvq8_weights_kernel<T, D, FMT, NT, false><<<(unsigned)grid, kWarps * 32, 0, a.stream>>>(p);
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
    return launch_nt<T, D, FMT, 4>(a, p);
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
