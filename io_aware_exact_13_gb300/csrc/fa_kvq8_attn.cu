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
//     lane ever needs another's codes and nothing passes through shared memory. (A ring of
//     asynchronous copies in shared memory was slower, 272 us against 214 on the large case below:
//     its loads and copies crowd the pipe that the shuffles use.) The next tile's K is loaded into
//     the registers as soon as the scores have read them, its V at the end of the step; bringing
//     tiles further ahead to L2 first was slower too (219 to 271 us).
//   - The page scales multiply scores, which are few (16 keys x 8 rows per tile and warp): ks goes
//     into the score, log2 vs into the exponent of the weights that multiply Vc. Those weights,
//     w_j = s_j log2 e + log2 vs(j), keep a running maximum of their own: the fp16 rounding of the
//     weights is then relative to the largest contribution, whatever the pages' scales are, and
//     a page of zeros (vs = 0) still counts in the sum. The sum l and all accumulators are fp32.
// Q goes into the products in fp16, as given or (bf16) scaled by a power of two that puts the row's largest magnitude
// into [2^15, 2^16): exact for elements down to 2^-32 of it, and off by at most 2^-40 of it below. The weights are
// rounded to fp16, 2^-11 relative (2^-25 of the largest below fp16's normal range).
//
// Ragged batches: all sequences' tiles are one line (sequence by sequence, head by head) that the warps of one
// wave of CTAs cut into equal stretches, whatever the lengths are; each warp finds its place by adding the
// lengths up. (A CTA per fixed chunk of keys left most of a second wave idle: 51 us against 38 on the ragged
// case below.) A unit that one warp does alone is written at once; the warps of a CTA merge theirs in shared
// memory; what several CTAs share goes through the workspace to fa_kvq8_combine.
//
// Short contexts, and longer ones of few sequences, take a CTA or a cluster of CTAs per unit instead, in one launch: the
// CTAs of a cluster merge through each other's shared memory (see kvq8_num_parts).
//
// Measured on one GB300 (copy rate 6.80 TB/s): B 64, H 64 / 8, d 128, e4m3, ragged up to 16384 keys 210 us (92 % of the
// copy rate); B 16, H 32 / 8, d 128, int8, ragged up to 8192 keys 40 us (63 %); time is about bytes / rate + 14 us, of
// which launch and lengths are 2.3 and the merge kernel 4.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <float.h>
#include <stdint.h>

#include <type_traits>

#include "fa_kvq8.cuh"
#include "pdl.cuh"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kWarps = 4;
constexpr int kMostCluster = 8;  // CTAs of a unit, all of a portable cluster
constexpr int kTileKeys = 16;
constexpr float kTau = 8.0f;  // log2 units by which a reference maximum may be exceeded before it moves
// Reference maximum of a row that has seen no key: below every finite score, and finite itself, so that the differences
// with it that empty rows and stretches form are numbers.
constexpr float kNone = -FLT_MAX;
constexpr float kLn2 = 0.6931471805599453f;

// Resident CTAs per SM that the kernel is compiled for: 128, 168 or 255 registers per thread. At d = 128 with one tile the
// four CTAs' 128 registers leave 20 to 52 bytes spilled; three CTAs, without spills, are slower (B 64, H 64 / 8, up to 16384
// keys 230 us against 210, B 16, H 32 / 8, up to 8192 keys 43.4 against 40.3).
__host__ __device__ constexpr int q8_ctas(int D, int NT) { return NT == 1 ? 4 : NT == 2 && D == 64 ? 3 : 2; }

template <int D, int NT>
struct Q8Cfg {
    static constexpr int KB = D / 64;                   // 16-byte units of a K row per lane
    static constexpr int VB = D / 8;                    // bytes of a V row per lane
    static constexpr int VW = VB / 4;                   // words of a V row per lane
    static constexpr int KS = D / 16;    // MMA steps over the head dimension
    static constexpr int MT = D / 16;    // 16-row tiles of O^T
    static constexpr int RT = 8 * NT;    // query rows per unit
    static constexpr int DEPTH = D == 64 || NT == 2 ? 2 : 1;  // tiles in flight per warp: 4 KB (8 KB where CTAs are few)
    static constexpr int PITCH = D + 4;  // floats per row of a shared stretch's summary
    static constexpr int CTAS = q8_ctas(D, NT);
    static constexpr int SM_O = 0;                                           // [2 kWarps][RT][PITCH] floats
    static constexpr int SM_ML = SM_O + 2 * kWarps * RT * PITCH * 4;         // m, l: [2 kWarps][RT] floats each
    static constexpr int SM_SEG = SM_ML + 2 * 2 * kWarps * RT * 4;           // Q8Stretch[2 kWarps]
    static constexpr int SMEM = SM_SEG + 2 * kWarps * 32;
};

// What a warp left in shared memory of a unit that it did not do alone: tiles [beg, end) of the unit's [first, last).
struct Q8Stretch {
    int unit;  // b * units + unit, or -1
    int first, last, beg, end;
    int pad[3];
};

struct Q8Params {
    const void *q;
    void *out;
    float *lse;
    const uint8_t *k_codes, *v_codes;
    const float *k_scale, *v_scale;
    const int *page_table, *kv_lens;
    float *o_part, *lse_part;  // [parts][2][RT][d], [parts][2][RT]
    int4 *shared;              // [parts]: the unit that holds the part's first tile, if it began in an earlier part
    int *status;
    int B, H, Hkv, Nq, rows, row_tiles;  // rows = (H / Hkv) Nq query rows share a K/V head, in row_tiles tiles
    int n_pages, max_pages, page_shift;
    int max_len, parts, cluster;  // cluster: CTAs of a unit when parts is 0
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
__host__ __device__ __forceinline__ int q8_tiles(int len) { return (len + kTileKeys - 1) / kTileKeys; }

// All threads of the cluster's CTAs: what any wrote to its shared memory before is seen by every one after.
__device__ __forceinline__ void cluster_sync() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Shared memory of another CTA of the cluster, at the address that `here` has in this one.
__device__ __forceinline__ uint32_t cluster_addr(const void *here, int rank) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(here)), "r"(rank));
    return a;
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t a) {
    float x;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(a) : "memory");
    return x;
}
__device__ __forceinline__ float4 ld_cluster_v4f(uint32_t a) {
    float4 x;
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w) : "r"(a) : "memory");
    return x;
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
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
    if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}
template <typename T>
__device__ __forceinline__ T from_float(float x) {
    if constexpr (std::is_same<T, __nv_bfloat16>::value) return __float2bfloat16_rn(x);
    else return __float2half_rn(x);
}

template <typename T, int D, int FMT, int NT, bool CAUSAL>
__global__ void __launch_bounds__(kWarps * 32, Q8Cfg<D, NT>::CTAS) fa_kvq8_partial(const Q8Params p) {
    using C = Q8Cfg<D, NT>;
    constexpr int KS = C::KS, MT = C::MT, RT = C::RT;
    extern __shared__ __align__(128) uint8_t sm[];
    float *sm_o = reinterpret_cast<float *>(sm + C::SM_O), *sm_m = reinterpret_cast<float *>(sm + C::SM_ML);
    float *sm_l = sm_m + 2 * kWarps * RT;
    Q8Stretch *seg = reinterpret_cast<Q8Stretch *>(sm + C::SM_SEG);
    grid_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, c = lane & 3;
    const int page_mask = (1 << p.page_shift) - 1;
    const int units = p.Hkv * p.row_tiles;  // per sequence

    // ---------------------------------------------------------------- this warp's stretch of the line
    // Each warp adds the lengths up for itself: no barrier between the lengths' arrival and the first page's read.
    int cur, end, b = 0, base = 0, len = 0, per;  // base: first tile of sequence b
    int start;  // the CTA's first tile
    const int rank = p.parts == 0 ? (int)blockIdx.x % p.cluster : 0;  // of this CTA in its cluster
    if (p.parts == 0) {  // a cluster for each unit, its tiles shared out evenly over all warps; the line begins with the sequence
        b = blockIdx.x / p.cluster / units;
        const int unit = blockIdx.x / p.cluster - b * units;
        bool bad;
        len = q8_len(p, b, bad);
        if (bad && threadIdx.x == 0) atomicExch(p.status, kStatusSeqlensQ8);
        const int n = q8_tiles(len), each = (n + kWarps * p.cluster - 1) / (kWarps * p.cluster), w = rank * kWarps + warp;
        if (n == 0) {
            const int kvh = unit / p.row_tiles, row0 = (unit - kvh * p.row_tiles) * RT, rows = min(RT, p.rows - row0);
            const size_t at = ((size_t)b * p.H + (size_t)kvh * (p.H / p.Hkv)) * p.Nq + row0;
            uint4 *o = reinterpret_cast<uint4 *>(static_cast<T *>(p.out) + at * D);
            for (int i = w * 32 + lane; i < rows * (D / 8); i += p.cluster * kWarps * 32) o[i] = make_uint4(0u, 0u, 0u, 0u);
            for (int i = w * 32 + lane; i < rows; i += p.cluster * kWarps * 32) p.lse[at + i] = -INFINITY;
            return;
        }
        per = n;
        start = unit * n;
        cur = start + min(n, w * each);
        end = start + min(n, (w + 1) * each);
        if (lane < 2) seg[2 * warp + lane].unit = -1;
        for (int r = lane; r < RT; r += 32) {  // what a warp without tiles leaves
            sm_m[2 * warp * RT + r] = kNone;
            sm_l[2 * warp * RT + r] = 0.f;
        }
        __syncwarp();
    } else {
        int total = 0, first_len = 0, s_bad = 0;  // first_len: the length of this lane's first sequence
#pragma unroll 4
        for (int s = lane; s < p.B; s += 32) {
            bool bad;
            const int n = q8_len(p, s, bad);
            s_bad |= bad;
            if (s == lane) first_len = n;
            total += q8_tiles(n) * units;
        }
        total = __reduce_add_sync(0xffffffffu, total);
        per = q8_part_tiles(total, p.parts);
        if (s_bad && blockIdx.x == 0 && warp == 0) atomicExch(p.status, kStatusSeqlensQ8);
        // sequences without keys: zeros, by the CTAs in turn
        for (int s = blockIdx.x; s < p.B; s += gridDim.x) {
            bool bad;
            if (q8_len(p, s, bad) != 0) continue;
            const size_t rows = (size_t)p.H * p.Nq;
            uint4 *o = reinterpret_cast<uint4 *>(static_cast<T *>(p.out) + s * rows * D);
            for (size_t i = threadIdx.x; i < rows * (D / 8); i += kWarps * 32) o[i] = make_uint4(0u, 0u, 0u, 0u);
            for (size_t i = threadIdx.x; i < rows; i += kWarps * 32) p.lse[s * rows + i] = -INFINITY;
        }
        if (threadIdx.x == 0) p.shared[blockIdx.x] = make_int4(-1, 0, 0, 0);
        if ((long long)blockIdx.x * per >= total) return;
        cur = blockIdx.x * per + warp * (per / kWarps);
        end = min(total, cur + per / kWarps);
        if (lane < 2) seg[2 * warp + lane].unit = -1;
        // the sequence that holds tile cur, 32 at a time
        for (int s0 = 0; cur < total; s0 += 32) {
            bool bad;
            const int l = s0 == 0 ? first_len : s0 + lane < p.B ? q8_len(p, s0 + lane, bad) : 0;
            const int n = q8_tiles(l) * units;
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
        __syncwarp();
        start = blockIdx.x * per;
    }
    const int warp_start = cur;

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
        const int slot = 2 * warp + (cur == warp_start ? 0 : 1);  // a stretch that is not whole is the first or the last
        if (!whole && lane == 0) {
            seg[slot].unit = b * units + unit;
            seg[slot].first = base + unit * seq_tiles;
            seg[slot].last = base + (unit + 1) * seq_tiles;
            seg[slot].beg = cur;
            seg[slot].end = cur + n_tiles;
        }
        cur += n_tiles;
        const int kvh = unit / p.row_tiles, rt = unit - kvh * p.row_tiles;
        const int k0 = tile0 * kTileKeys, k1 = min(len, k0 + n_tiles * kTileKeys);
        const int row0 = rt * RT;  // first of the unit's rows among the rows of the K/V head
        const size_t row_base = ((size_t)b * p.H + (size_t)kvh * (p.H / p.Hkv)) * p.Nq;

        // Lane i looks after tile 32 n + i of the stretch: its page and scales. The page numbers are read a window
        // of 32 tiles ahead.
        const int *table = p.page_table + (size_t)b * p.max_pages;
        const int lane_key = k0 + lane * kTileKeys;  // + 32 kTileKeys per window
        int ahead = lane_key < k1 ? __ldg(table + (lane_key >> p.page_shift)) : -1;
        int pg = -1;
        float pg_ks = 0.f, pg_lv = -INFINITY;
        auto load_pages = [&](int it0) {  // the window that starts at tile it0 (a multiple of 32)
            const int key = lane_key + it0 * kTileKeys;
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
            const int next = key + 32 * kTileKeys;
            ahead = next < k1 ? __ldg(table + (next >> p.page_shift)) : -1;
        };
        // This lane's codes of one tile: K rows g and g + 8 (dims 64 j + 16 c ..), V rows 2c, 2c + 1, 2c + 8,
        // 2c + 9 (dims VB g ..). Keys past the stretch and pages that are none are read as zeros; only a
        // stretch's last tile looks at single keys. DEPTH tiles are in flight.
        struct Tile {
            uint32_t kw[2][C::KB][4], vw[4][C::VW];
            size_t off;    // byte offset of its codes
            int n_keys;    // how many of its keys there are to read
            float ks, lv;  // scale log2 e times the page's K scale, log2 of its V scale
        };
        Tile buf[C::DEPTH];
        const uint8_t *k_lane = p.k_codes + g * D + c * 16, *v_lane = p.v_codes + 2 * c * D + g * C::VB;
        auto load_k = [&](Tile &b, int it) {
            const int page = __shfl_sync(0xffffffffu, pg, it & 31);
            b.ks = __shfl_sync(0xffffffffu, pg_ks, it & 31);
            b.lv = __shfl_sync(0xffffffffu, pg_lv, it & 31);
            const int key0 = k0 + it * kTileKeys;
            b.off = ((((size_t)(page >= 0 ? page : 0) * p.Hkv + kvh) << p.page_shift) + (size_t)(key0 & page_mask)) * D;
            b.n_keys = page >= 0 ? k1 - key0 : 0;
            const uint8_t *src = k_lane + b.off;
            if (b.n_keys >= kTileKeys) {
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int j = 0; j < C::KB; ++j) load_codes(src + 8 * r * D + j * 64, b.kw[r][j]);
            } else {
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int j = 0; j < C::KB; ++j) {
                        b.kw[r][j][0] = b.kw[r][j][1] = b.kw[r][j][2] = b.kw[r][j][3] = 0u;
                        if (g + 8 * r < b.n_keys) load_codes(src + 8 * r * D + j * 64, b.kw[r][j]);
                    }
            }
        };
        auto load_v = [&](Tile &b) {
            const uint8_t *src = v_lane + b.off;
            if (b.n_keys >= kTileKeys) {
#pragma unroll
                for (int i = 0; i < 4; ++i) load_codes(src + ((i & 1) + (i >> 1) * 8) * D, b.vw[i]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int key = (i & 1) + (i >> 1) * 8;
#pragma unroll
                    for (int e = 0; e < C::VW; ++e) b.vw[i][e] = 0u;
                    if (2 * c + key < b.n_keys) load_codes(src + key * D, b.vw[i]);
                }
            }
        };
        // Q as B fragments: column g of tile t is row row0 + 8 t + g, contraction index in the order of the K codes
        uint32_t qb[NT][KS][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int row = row0 + 8 * t + g;
            const T *src = static_cast<const T *>(p.q) + (row_base + row) * D;
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
        }
        load_pages(0);
#pragma unroll
        for (int i = 0; i < C::DEPTH; ++i)
            if (i < n_tiles) {
                load_k(buf[i], i);
                load_v(buf[i]);
            }

        float qmul[NT][2];  // what the rows 2c, 2c + 1 of a tile were divided by
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            uint32_t (&qt)[KS][2] = qb[t];
            float mul = 1.0f;
            if constexpr (std::is_same<T, __nv_bfloat16>::value) {
                uint32_t most = 0;
#pragma unroll
                for (int s = 0; s < KS; ++s)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        most = max(most, max(qt[s][e] & 0x7FFFu, (qt[s][e] >> 16) & 0x7FFFu));
                most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
                most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
                // The row's largest magnitude, of biased exponent ex, goes to [2^15, 2^16) (rows below 2^-111 are scaled
                // by 2^126, whose inverse is a normal number too: bf16's smallest number is then 2^-7).
                const uint32_t ex = max(most >> 7, 16u);
                const float inv = __uint_as_float((269u - ex) << 23);
                mul = __uint_as_float(ex << 23) * 0x1p-15f;  // 1 / inv (as an integer subtraction the kernel
                                                             // was 0.6 us slower on B 16, H 32 / 8, 8192 keys)
#pragma unroll
                for (int s = 0; s < KS; ++s)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const __nv_bfloat162 h = *reinterpret_cast<const __nv_bfloat162 *>(&qt[s][e]);
                        const float2 f = __bfloat1622float2(h);
                        const __half2 o = __floats2half2_rn(f.x * inv, f.y * inv);
                        qt[s][e] = *reinterpret_cast<const uint32_t *>(&o);
                    }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) qmul[t][e] = __shfl_sync(0xffffffffu, mul, 8 * c + 4 * e);  // of column 2c + e
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

        auto step = [&](Tile &b, int it) {
            float x[NT][4];
            const float ks = b.ks, lv = b.lv;
            const int key0 = k0 + it * kTileKeys, in_tile = b.n_keys;
            // S^T = Kc Q^T
#pragma unroll
            for (int t = 0; t < NT; ++t) x[t][0] = x[t][1] = x[t][2] = x[t][3] = 0.f;
#pragma unroll
            for (int j = 0; j < C::KB; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    uint32_t a[4];
                    codes_to_half2<FMT>(b.kw[0][j][e], a[0], a[2]);
                    codes_to_half2<FMT>(b.kw[1][j][e], a[1], a[3]);
#pragma unroll
                    for (int t = 0; t < NT; ++t) mma_f16(x[t], a, qb[t][4 * j + e][0], qb[t][4 * j + e][1]);
                }
            // K of the tile that takes this one's registers, in flight from here on; its V at the end
            const bool more = it + C::DEPTH < n_tiles;
            if (more) {
                if (((it + C::DEPTH) & 31) == 0) load_pages(it + C::DEPTH);
                load_k(b, it + C::DEPTH);
            }
            // scores in log2 units, with the range, page and causal limits
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const float2 mul = make_float2(ks * qmul[t][0], ks * qmul[t][1]);
                x[t][0] *= mul.x;
                x[t][1] *= mul.y;
                x[t][2] *= mul.x;
                x[t][3] *= mul.y;
            }
            if (in_tile < kTileKeys || (CAUSAL && key0 + kTileKeys - 1 > len - p.Nq)) {
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int r = g + (e >> 1) * 8;
                        const int last = CAUSAL ? len - p.Nq + (row0 + 8 * t + 2 * c + (e & 1)) % p.Nq : len;
                        if (r >= in_tile || key0 + r > last) x[t][e] = -INFINITY;
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
            // weights w = 2^(x + lv - mw) as B fragments: keys 2c, 2c + 1 (+ 8) of row g. One exponential for the whole
            // exponent: 2^(x - m) and 2^(lv + m - mw) may each leave fp32's range where their product does not.
            uint32_t pb[NT][2];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                float f[2], s[4], w[4];
#pragma unroll
                for (int e = 0; e < 2; ++e)  // (a row that saw only pages of zeros has mw = kNone; m - mw may be infinite)
                    f[e] = lv == -INFINITY ? -INFINITY : fminf(lv + (m[t][e] - mw[t][e]), FLT_MAX);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float a = x[t][e] - m[t][e & 1];
                    s[e] = ex2_approx(a);
                    w[e] = ex2_approx(a + f[e & 1]);
                }
                l[t][0] += s[0] + s[2];
                l[t][1] += s[1] + s[3];
                const __half2 h0 = __floats2half2_rn(w[0], w[1]), h1 = __floats2half2_rn(w[2], w[3]);
                pb[t][0] = movmatrix_trans(*reinterpret_cast<const uint32_t *>(&h0));
                pb[t][1] = movmatrix_trans(*reinterpret_cast<const uint32_t *>(&h1));
            }
            // O^T += Vc^T P^T: words of four keys interleaved into pairs of keys
#pragma unroll
            for (int i = 0; i < C::VW; ++i) {
                uint32_t a[4];
                codes_to_half2<FMT>(__byte_perm(b.vw[0][i], b.vw[1][i], 0x5140), a[0], a[1]);
                codes_to_half2<FMT>(__byte_perm(b.vw[2][i], b.vw[3][i], 0x5140), a[2], a[3]);
#pragma unroll
                for (int t = 0; t < NT; ++t) mma_f16(o[t][2 * i], a, pb[t][0], pb[t][1]);
                codes_to_half2<FMT>(__byte_perm(b.vw[0][i], b.vw[1][i], 0x7362), a[0], a[1]);
                codes_to_half2<FMT>(__byte_perm(b.vw[2][i], b.vw[3][i], 0x7362), a[2], a[3]);
#pragma unroll
                for (int t = 0; t < NT; ++t) mma_f16(o[t][2 * i + 1], a, pb[t][0], pb[t][1]);
            }
            if (more) load_v(b);
        };
        for (int it = 0; it < n_tiles; it += C::DEPTH)
#pragma unroll
            for (int i = 0; i < C::DEPTH; ++i)
                if (i == 0 || it + i < n_tiles) step(buf[i], it + i);


        // Lane (g, c) holds head columns VB g .. VB g + VB - 1 of rows 2c, 2c + 1 of every tile: value (i, e2) is
        // column VB g + 2 i + e2. A whole unit is written out, any other stretch left for the CTA's merge.
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float ls = l[t][e];
                ls += __shfl_xor_sync(0xffffffffu, ls, 4);
                ls += __shfl_xor_sync(0xffffffffu, ls, 8);
                ls += __shfl_xor_sync(0xffffffffu, ls, 16);
                const int r = 8 * t + 2 * c + e;
                float f = ex2_approx(mw[t][e] - m[t][e]);  // 0 where every weight was (mw = kNone)
                if (whole) {
                    f = ls == 0.f ? 0.f : f / ls;  // (a sum that is NaN, from a NaN query, stays NaN)
                    if (row0 + r < p.rows) {
                        uint32_t w[MT];
#pragma unroll
                        for (int i = 0; i < MT; ++i) w[i] = pack16<T>(o[t][i][e] * f, o[t][i][e + 2] * f);
                        T *dst = static_cast<T *>(p.out) + (row_base + row0 + r) * D + C::VB * g;
#pragma unroll
                        for (int i = 0; i < MT; i += 4) st_global_v4(dst + 2 * i, w[i], w[i + 1], w[i + 2], w[i + 3]);
                        if (g == 0) p.lse[row_base + row0 + r] = ls == 0.f ? -INFINITY : (m[t][e] + lg2_approx(ls)) * kLn2;
                    }
                } else {
                    float4 *dst = reinterpret_cast<float4 *>(sm_o + (slot * RT + r) * C::PITCH + C::VB * g);
#pragma unroll
                    for (int i = 0; i < MT; i += 2)
                        dst[i / 2] = make_float4(o[t][i][e] * f, o[t][i][e + 2] * f, o[t][i + 1][e] * f, o[t][i + 1][e + 2] * f);
                    if (g == 0) {
                        sm_m[slot * RT + r] = m[t][e];
                        sm_l[slot * RT + r] = ls;
                    }
                }
            }
    }

    // ---------------------------------------------------------------- a unit shared by the CTAs of a cluster
    // Each CTA merges its warps' summaries (into slot 1, which no warp has used); then the CTAs share out the unit's
    // rows and columns and merge each other's. One tile is one warp's, which has written the rows.
    if (p.parts == 0 && p.cluster > 1) {
        if (per == 1) return;
        const int unit = blockIdx.x / p.cluster - b * units;
        const int kvh = unit / p.row_tiles, row0 = (unit - kvh * p.row_tiles) * RT, rows = min(RT, p.rows - row0);
        const size_t row_base = ((size_t)b * p.H + (size_t)kvh * (p.H / p.Hkv)) * p.Nq + row0;
        __syncthreads();
        for (int idx = threadIdx.x; idx < rows * (D / 4); idx += kWarps * 32) {
            const int r = idx / (D / 4), e4 = idx % (D / 4);
            float M = kNone, L = 0.f;
            float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm_m[2 * w * RT + r]);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                if (seg[2 * w].unit < 0) continue;  // a warp without tiles
                const float f = ex2_approx(sm_m[2 * w * RT + r] - M);
                const float4 v = *reinterpret_cast<const float4 *>(sm_o + (2 * w * RT + r) * C::PITCH + 4 * e4);
                L += f * sm_l[2 * w * RT + r];
                A.x = fmaf(f, v.x, A.x);
                A.y = fmaf(f, v.y, A.y);
                A.z = fmaf(f, v.z, A.z);
                A.w = fmaf(f, v.w, A.w);
            }
            *reinterpret_cast<float4 *>(sm_o + (RT + r) * C::PITCH + 4 * e4) = A;
            if (e4 == 0) {
                sm_m[RT + r] = M;
                sm_l[RT + r] = L;
            }
        }
        cluster_sync();
        for (int idx = rank * kWarps * 32 + threadIdx.x; idx < rows * (D / 4); idx += p.cluster * kWarps * 32) {
            const int r = idx / (D / 4), e4 = idx % (D / 4);
            float m[kMostCluster], l[kMostCluster];
            float4 v[kMostCluster];
#pragma unroll
            for (int q = 0; q < kMostCluster; ++q) {
                m[q] = kNone, l[q] = 0.f, v[q] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (q < p.cluster) {
                    m[q] = ld_cluster_f32(cluster_addr(sm_m + RT + r, q));
                    l[q] = ld_cluster_f32(cluster_addr(sm_l + RT + r, q));
                    v[q] = ld_cluster_v4f(cluster_addr(sm_o + (RT + r) * C::PITCH + 4 * e4, q));
                }
            }
            float M = m[0], L = 0.f;
            float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int q = 1; q < kMostCluster; ++q) M = fmaxf(M, m[q]);
#pragma unroll
            for (int q = 0; q < kMostCluster; ++q) {
                const float f = ex2_approx(m[q] - M);
                L += f * l[q];
                A.x = fmaf(f, v[q].x, A.x);
                A.y = fmaf(f, v[q].y, A.y);
                A.z = fmaf(f, v[q].z, A.z);
                A.w = fmaf(f, v[q].w, A.w);
            }
            const float inv = L == 0.f ? 0.f : 1.0f / L;
            uint2 w;
            w.x = pack16<T>(A.x * inv, A.y * inv);
            w.y = pack16<T>(A.z * inv, A.w * inv);
            *reinterpret_cast<uint2 *>(static_cast<T *>(p.out) + (row_base + r) * D + 4 * e4) = w;
            if (e4 == 0) p.lse[row_base + r] = L == 0.f ? -INFINITY : (M + lg2_approx(L)) * kLn2;
        }
        cluster_sync();  // a CTA's shared memory stays until its neighbours have read it
        return;
    }

    // ---------------------------------------------------------------- units shared by warps or CTAs
    // Neighbouring stretches of one unit are merged. Where they are all of it the rows are written, otherwise the
    // CTA's summary: slot 0 of the part for the unit that holds the CTA's first tile, slot 1 for its last one.
    __syncthreads();
    for (int a = 0; a < 2 * kWarps;) {
        const int uid = seg[a].unit;
        if (uid < 0) {
            ++a;
            continue;
        }
        int z = a, next = a + 1;  // stretches a .. z (some slots between may be empty)
        for (; next < 2 * kWarps && (seg[next].unit < 0 || seg[next].unit == uid); ++next)
            if (seg[next].unit == uid) z = next;
        const bool all = seg[a].beg == seg[a].first && seg[z].end == seg[z].last;
        const size_t part = 2 * (size_t)blockIdx.x + (seg[a].first <= start ? 0 : 1);
        if (threadIdx.x == 0 && !all && seg[a].first < start) p.shared[blockIdx.x] = make_int4(uid, seg[a].first, seg[a].last, per);
        const int ub = uid / units, unit = uid - ub * units;
        const int kvh = unit / p.row_tiles, row0 = (unit - kvh * p.row_tiles) * RT;
        const size_t row_base = ((size_t)ub * p.H + (size_t)kvh * (p.H / p.Hkv)) * p.Nq + row0;
        for (int idx = threadIdx.x; idx < RT * D / 4; idx += kWarps * 32) {
            const int r = idx / (D / 4), e4 = idx % (D / 4);
            if (row0 + r >= p.rows) break;
            float M = kNone, L = 0.f;
            float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int s = a; s <= z; ++s)
                if (seg[s].unit >= 0) M = fmaxf(M, sm_m[s * RT + r]);
            for (int s = a; s <= z; ++s) {
                if (seg[s].unit < 0) continue;
                const float f = ex2_approx(sm_m[s * RT + r] - M);  // 0 for a stretch that saw nothing, unless none did
                const float4 v = *reinterpret_cast<const float4 *>(sm_o + (s * RT + r) * C::PITCH + 4 * e4);
                L += f * sm_l[s * RT + r];
                A.x = fmaf(f, v.x, A.x);
                A.y = fmaf(f, v.y, A.y);
                A.z = fmaf(f, v.z, A.z);
                A.w = fmaf(f, v.w, A.w);
            }
            const float inv = L == 0.f ? 0.f : 1.0f / L;
            const float lse = L == 0.f ? -INFINITY : (M + lg2_approx(L)) * kLn2;
            if (all) {
                uint2 w;
                w.x = pack16<T>(A.x * inv, A.y * inv);
                w.y = pack16<T>(A.z * inv, A.w * inv);
                *reinterpret_cast<uint2 *>(static_cast<T *>(p.out) + (row_base + r) * D + 4 * e4) = w;
                if (e4 == 0) p.lse[row_base + r] = lse;
            } else {
                *reinterpret_cast<float4 *>(p.o_part + (part * RT + r) * D + 4 * e4) =
                    make_float4(A.x * inv, A.y * inv, A.z * inv, A.w * inv);
                if (e4 == 0) p.lse_part[part * RT + r] = lse;
            }
        }
        a = next;
    }
}

// The units that several parts share: their summaries merged onto their common maximum (fa_splitkv.cu's rule). A unit
// that n parts share is merged by the CTAs of its parts but the first, each doing every (n - 1)-th row; where a CTA has
// few rows, several groups of threads share a row's summaries out.
constexpr int kCombineThreads = 128;
template <typename T, int D, int RT>
__global__ void __launch_bounds__(kCombineThreads) fa_kvq8_combine(const Q8Params p) {
    constexpr int LANES = D / 4, SLOTS = kCombineThreads / LANES;  // four columns of a row per thread
    constexpr int AHEAD = 8;                                      // summaries loaded before the first is used
    __shared__ float4 sm_a[SLOTS][LANES];
    __shared__ float sm_m[SLOTS], sm_w[SLOTS];
    grid_dependency_wait();
    const int4 d = p.shared[blockIdx.x];
    if (d.x < 0) return;
    const int first = d.y, per = d.w, p0 = first / per, n = (d.z - 1) / per - p0 + 1;
    const int units = p.Hkv * p.row_tiles;
    const int b = d.x / units, unit = d.x - b * units, kvh = unit / p.row_tiles, rt = unit - kvh * p.row_tiles;
    const size_t row_base = ((size_t)b * p.H + (size_t)kvh * (p.H / p.Hkv)) * p.Nq + rt * RT;
    const int mine = (int)blockIdx.x - p0 - 1, n_rows = min(RT, p.rows - rt * RT);
    if (mine >= n_rows) return;
    const int rows = (n_rows - mine + n - 2) / (n - 1);  // rows mine, mine + (n - 1), ...
    int groups = 1;
    while (2 * groups * rows <= SLOTS && groups < n) groups *= 2;
    // part p0 may begin in an earlier unit; every later one begins in this one
    const int slot0 = 2 * p0 + (p0 * per >= first ? 0 : 1);
    const int slot = threadIdx.x / LANES, lane = threadIdx.x % LANES, group = slot % groups;
    for (int r0 = slot / groups; r0 - slot / groups < rows; r0 += SLOTS / groups) {  // as often for every thread
        const bool in = r0 < rows;
        const int r = mine + (in ? r0 : 0) * (n - 1);
        float M = -INFINITY, W = 0.f;
        float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int s0 = in ? group : n; s0 < n; s0 += AHEAD * groups) {
            float l[AHEAD];
            float4 v[AHEAD];
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {
                const int s = s0 + k * groups;
                const size_t at = (size_t)(s == 0 ? slot0 : 2 * (p0 + s)) * RT + r;
                l[k] = -INFINITY;
                v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (s < n) {
                    l[k] = p.lse_part[at];
                    v[k] = *reinterpret_cast<const float4 *>(p.o_part + at * D + 4 * lane);
                }
            }
            float m = M;
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) m = fmaxf(m, isnan(l[k]) ? 0.f : l[k]);  // NaN goes through the weights
            if (m == -INFINITY) continue;  // parts that saw no key
            const float f = __expf(M - m);
            W *= f;
            A.x *= f, A.y *= f, A.z *= f, A.w *= f;
            M = m;
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {
                const float w = __expf(l[k] - m);
                W += w;
                A.x = fmaf(w, v[k].x, A.x);
                A.y = fmaf(w, v[k].y, A.y);
                A.z = fmaf(w, v[k].z, A.z);
                A.w = fmaf(w, v[k].w, A.w);
            }
        }
        if (groups > 1) {
            sm_a[slot][lane] = A;
            if (lane == 0) {
                sm_m[slot] = M;
                sm_w[slot] = W;
            }
            __syncthreads();
            if (group == 0) {
                for (int i = 1; i < groups; ++i) M = fmaxf(M, sm_m[slot + i]);
                W = 0.f;
                A = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int i = 0; i < groups && M != -INFINITY; ++i) {
                    const float f = __expf(sm_m[slot + i] - M);
                    const float4 v = sm_a[slot + i][lane];
                    W += f * sm_w[slot + i];
                    A.x = fmaf(f, v.x, A.x);
                    A.y = fmaf(f, v.y, A.y);
                    A.z = fmaf(f, v.z, A.z);
                    A.w = fmaf(f, v.w, A.w);
                }
            }
            __syncthreads();
        }
        if (group == 0 && in) {
            const float inv = W == 0.f ? 0.f : 1.0f / W;
            uint2 o;
            o.x = pack16<T>(A.x * inv, A.y * inv);
            o.y = pack16<T>(A.z * inv, A.w * inv);
            *reinterpret_cast<uint2 *>(static_cast<T *>(p.out) + (row_base + r) * D + 4 * lane) = o;
            if (lane == 0) p.lse[row_base + r] = W == 0.f ? -INFINITY : M + __logf(W);
        }
    }
}

int page_log2(int page) {
    int s = 0;
    while ((1 << s) < page) ++s;
    return s;
}

// Query rows that share a K/V head, in 8-row MMA tiles: as few units as the accumulators' registers allow (two
// tiles at d = 128, four at d = 64), the tiles spread evenly over them.
int tiles_per_unit(int rows, int d) {
    const int most = d == 64 ? 4 : 2, n = (rows + 7) / 8;
    const int units = (n + most - 1) / most;
    return (n + units - 1) / units;
}
int units_per_head(int rows, int d) { return (rows + 8 * tiles_per_unit(rows, d) - 1) / (8 * tiles_per_unit(rows, d)); }

// CTAs for each unit when parts is 0: as many as fit in one wave and have a tile for every warp, up to 8. (B 1, H 8, d 64:
// 500 keys 7.8, 5.9, 4.9, 4.6 us with 1, 2, 4, 8; with two waves instead of one, B 16, H 32 / 8, d 128, 8.8 becomes 14.0.)
int cluster_size(long long units, int tiles, long long slots) {
    int c = 1;
    while (2 * c <= kMostCluster && 2 * c * units <= slots && tiles > kWarps * c) c *= 2;
    return c;
}

template <typename T, int D, int FMT, int NT, bool CAUSAL>
int launch_q8(const Kvq8AttnArgs &a) {
    using C = Q8Cfg<D, NT>;
    auto kern = fa_kvq8_partial<T, D, FMT, NT, CAUSAL>;
    if (C::SMEM > 48 * 1024 &&
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) != cudaSuccess)
        return -5;
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
    p.shared = reinterpret_cast<int4 *>(a.workspace + (size_t)a.parts * 2 * C::RT * (D + 1));
    p.status = a.status;
    p.B = a.B;
    p.H = a.H;
    p.Hkv = a.c.Hkv;
    p.Nq = a.Nq;
    p.rows = a.H / a.c.Hkv * a.Nq;
    p.row_tiles = units_per_head(p.rows, D);
    p.n_pages = a.c.n_pages;
    p.max_pages = a.c.max_pages;
    p.page_shift = page_log2(a.c.page);
    p.max_len = a.max_len;
    p.parts = a.parts;
    p.scale_log2 = static_cast<float>(static_cast<double>(a.scale) * 1.4426950408889634);
    // (not as a programmatic dependent: its CTAs would take their places beside those of the kernel ahead, and
    // the one wave that the parts are sized for would become two)
    p.cluster = a.parts > 0 ? 1 : cluster_size((long long)a.B * a.c.Hkv * p.row_tiles, q8_tiles(a.max_len),
                                               (long long)C::CTAS * a.num_sms);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.parts > 0 ? a.parts : a.B * a.c.Hkv * p.row_tiles * p.cluster);
    cfg.blockDim = dim3(kWarps * 32);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = a.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = p.cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.cluster > 1 ? 1 : 0;
    if (cudaLaunchKernelEx(&cfg, kern, p) != cudaSuccess) return -5;
    if (cudaGetLastError() != cudaSuccess) return -5;
    if (a.parts <= 1) return 0;
    return launch_dependent(fa_kvq8_combine<T, D, C::RT>, dim3(a.parts), dim3(kCombineThreads), 0,
                            a.stream, p) == cudaSuccess
               ? 0
               : -5;
}

template <typename T, int D, int FMT, int NT>
int launch_q8_causal(const Kvq8AttnArgs &a) {
    return a.causal ? launch_q8<T, D, FMT, NT, true>(a) : launch_q8<T, D, FMT, NT, false>(a);
}
template <typename T, int D, int FMT>
int launch_q8_rows(const Kvq8AttnArgs &a) {
    const int nt = tiles_per_unit(a.H / a.c.Hkv * a.Nq, D);
    if (nt == 1) return launch_q8_causal<T, D, FMT, 1>(a);
    if (nt == 2) return launch_q8_causal<T, D, FMT, 2>(a);
    if constexpr (D == 64) return nt == 3 ? launch_q8_causal<T, D, FMT, 3>(a) : launch_q8_causal<T, D, FMT, 4>(a);
    return -4;
}

template <typename T>
int launch_q8_t(const Kvq8AttnArgs &a) {
    const bool i8 = a.c.format == kKvq8Int8;
    if (a.c.d == 128) return i8 ? launch_q8_rows<T, 128, kKvq8Int8>(a) : launch_q8_rows<T, 128, kKvq8E4m3>(a);
    if (a.c.d == 64) return i8 ? launch_q8_rows<T, 64, kKvq8Int8>(a) : launch_q8_rows<T, 64, kKvq8E4m3>(a);
    return -4;
}

}  // namespace

long long kvq8_tiles(int B, int Hkv, int rows, int max_len, int d) {
    return (long long)B * Hkv * units_per_head(rows, d) * ((max_len + kTileKeys - 1) / kTileKeys);
}

// Parts 0, a cluster of CTAs for each unit and no merge kernel, while no warp has many tiles: 8, or more where the clusters
// fill most of a wave, since the line then has little to spread (16; 12 with one CTA for a unit). Measured, cluster against
// line, each case alone in its process (the first is 4.85 us among other work): B 1, H 8, d 64: 500 keys 4.6 against 7.6 us,
// 4000 8.0 / 8.8, 8000 11.8 / 9.6. B 4, H 32 / 8, d 128: 1000 keys 7.5 / 10.1, 4000 15.6 / 16.5, 8000 24.7 / 21.5. B 16,
// H 32 / 8, d 128: 500 keys 8.8 / 12.2, 2000 18.6 / 22.8, 4000 30.7 / 33.9, ragged 27.1 / 27.4. B 32: 2000 30.8 / 33.9,
// ragged 27.0 / 26.4. B 64, one CTA: 600 21.0 / 25.1, 1000 ragged 26.4 / 26.6.
// Otherwise one part for each CTA that can be resident, and at least one tile for each of a CTA's warps.
int kvq8_num_parts(int B, int Hkv, int rows, int max_len, int d, int num_sms) {
    const int nt = tiles_per_unit(rows, d), tiles = q8_tiles(max_len);
    const long long slots = (long long)q8_ctas(d, nt) * num_sms, units = (long long)B * Hkv * units_per_head(rows, d);
    const int c = cluster_size(units, tiles, slots), each = (tiles + kWarps * c - 1) / (kWarps * c);
    const bool full = 2 * c * units > slots && c * units <= slots;
    if (each <= (!full ? 8 : c > 1 ? 16 : 12)) return 0;
    const long long by_len = (kvq8_tiles(B, Hkv, rows, max_len, d) + kWarps - 1) / kWarps;
    return (int)(by_len < slots ? by_len : slots);
}

size_t kvq8_workspace_bytes(int rows, int d, int parts) {
    return (size_t)parts * (2 * 8 * tiles_per_unit(rows, d) * (d + 1) * sizeof(float) + sizeof(int4));
}

int launch_kvq8_attention(const Kvq8AttnArgs &a, bool fp16) {
    return fp16 ? launch_q8_t<__half>(a) : launch_q8_t<__nv_bfloat16>(a);
}

}  // namespace fa
