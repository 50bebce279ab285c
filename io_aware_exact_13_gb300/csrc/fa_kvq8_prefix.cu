// fa_kvq8_prefix.cu -- attention over the 8-bit cache for a batch whose sequences share a prefix: the choice between
// reading the prefix with each sequence's own keys (fa_kvq8_attn.cuh) and once for the rows of all (fa_kvq8_prefix_tc.cu),
// and the merge of the latter's summaries with those of the own keys.
#include "fa_kvq8_attn.cuh"
#include "fa_kvq8_prefix.cuh"

namespace fa {
namespace {

constexpr int kMergeThreads = 128;

// out = sum_s w_s o_s / sum_s w_s with w_s = exp(lse_s - max lse), over the own keys' summary and those of the prefix's
// runs (fa_splitkv.cu's rule). Four columns of a row for each thread; the lanes of a row share the weights out.
template <typename T, int D>
__global__ void __launch_bounds__(kMergeThreads)
    fa_kvq8_prefix_merge(const float *own_o, const float *own_lse, const float *o_part, const float *lse_part, T *out,
                         float *lse, int rows, int splits) {
    constexpr int LANES = D / 4, AHEAD = 16;
    grid_dependency_wait();
    const long long id = (long long)blockIdx.x * kMergeThreads + threadIdx.x;
    const long long row = id / LANES;
    const int lane = (int)(id % LANES);
    const uint32_t mask = LANES == 32 ? 0xffffffffu : 0xffffu << (threadIdx.x & 16);
    if (row >= rows) return;
    float M = -INFINITY;  // NaN goes through the weights
    for (int s = lane; s <= splits; s += LANES) M = fmaxf(M, s == 0 ? own_lse[row] : lse_part[(long long)(s - 1) * rows + row]);
#pragma unroll
    for (int d = LANES / 2; d > 0; d /= 2) M = fmaxf(M, __shfl_xor_sync(mask, M, d, LANES));
    const float ref = M == -INFINITY ? 0.f : M;
    float W = 0.f;
    float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = 0; s0 <= splits; s0 += LANES) {
        float w = 0.f;
        if (s0 + lane <= splits) w = __expf((s0 + lane == 0 ? own_lse[row] : lse_part[(long long)(s0 + lane - 1) * rows + row]) - ref);
        const int n = min(LANES, splits + 1 - s0);
        for (int i0 = 0; i0 < n; i0 += AHEAD) {
            float f[AHEAD];
            float4 v[AHEAD];
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {
                f[k] = __shfl_sync(mask, w, (i0 + k) % LANES, LANES);
                if (i0 + k >= n) f[k] = 0.f;
                const int s = s0 + i0 + k;
                v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (f[k] != 0.f)  // a summary without keys holds nothing
                    v[k] = *reinterpret_cast<const float4 *>((s == 0 ? own_o : o_part + (long long)(s - 1) * rows * D) + row * D + 4 * lane);
            }
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {
                W += f[k];
                A.x = fmaf(f[k], v[k].x, A.x);
                A.y = fmaf(f[k], v[k].y, A.y);
                A.z = fmaf(f[k], v[k].z, A.z);
                A.w = fmaf(f[k], v[k].w, A.w);
            }
        }
    }
    store4(out + row * D + 4 * lane, A, W == 0.f ? 0.f : 1.0f / W);
    if (lane == 0) lse[row] = W == 0.f ? -INFINITY : M + __logf(W);
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

template <typename T, int D>
int launch_merge(const Kvq8AttnArgs &a, const float *own_o, const float *own_lse, const float *o_part, const float *lse_part) {
    const int rows = a.B * a.H * a.Nq;
    const long long grid = ((long long)rows * (D / 4) + kMergeThreads - 1) / kMergeThreads;
    if (grid > INT32_MAX) return -3;
    return launch_dependent(fa_kvq8_prefix_merge<T, D>, dim3((unsigned)grid), dim3(kMergeThreads), 0, a.stream, own_o, own_lse,
                            o_part, lse_part, static_cast<T *>(a.out), a.lse, rows, a.splits) == cudaSuccess
               ? 0
               : -5;
}

// How the prefix is done, by estimates of each way's time in us. They go by max_prefix and max_len, and were fitted to
// measured times (below); what they decide is never more than speed.
//   with every sequence's own keys: a start, the merge of parts, and all keys at the rate of L2, or at that of the products where
//   many rows share a head; or as many waves as there are clusters (no parts);
//   once for all, in s runs for each 256 rows: waves of a start and the run's blocks, and the merge of summaries; the own keys
//   beside it on the SMs that are left, or after it on all.
// Measured (us; with every sequence's own keys against once for all), int8, 8 K/V heads. 4 heads share one, d 128: prefix 2048, B 1 to
// 32: 12.4 / 16.6, 12.9 / 16.6, 14.0 / 16.5, 16.6 / 16.6, 20.7 / 18.6, 30.4 / 20.6; prefix 8192: 16.7 / 22.4, 18.6 / 21.5,
// 22.8 / 22.3, 30.9 / 22.6, 46.2 / 22.7, 80.0 / 28.1. 8 share one, 32768: 25.0 / 39.1, 33.6 / 39.1, 49.3 / 40.6, 85.9 / 41.9, 152 /
// 45.3, 289 / 57.5. d 64, not shared, prefix 1000: 8.4 / 14.5 up to 4, 10.4 / 14.5, 10.7 / 14.5, 14.5 / 14.5. With own keys, beside
// and after: B 16, 8192 + up to 1024: 13 runs after 33.0, 11 beside 24.9; B 64, 8 share one, 32768 + up to 2048: 9 runs after
// 118.8, 7 beside 107, 6 104; B 256, 4 rows each, 2048 + up to 1000: in the line 290, one run beside 494, after 171; B 4096, not
// shared, 1000 + up to 100: in the line 1183, after 378; B 200, 16 heads, 1500 + up to 1500: 9 runs after 175, one beside 159.
// Against the best of all run and part counts at 32 sizes (2 to 4096 sequences, 1 to 16 rows, prefixes of 200 to 32768) what is chosen
// takes 1.4 % longer on the average, 16 % at most.
struct Batch {
    int B, Hkv, rows, max_prefix, max_len, d;
};

double tile_cost(int nt) { return nt == 1 ? 1.0 : nt == 2 ? 1.6 : nt == 3 ? 3.5 : 4.5; }  // of a key, by tiles of rows

// The attention over `keys` keys of each sequence without parts: how often its clusters fill the SMs, and the time of each.
struct Waves {
    double count, time;
};
Waves line_waves(const Batch &b, double keys, int max_keys, int sms) {
    const int nt = tiles_per_unit(b.rows, b.d);
    const long long slots = (long long)q8_ctas(b.d, nt) * sms, units = (long long)b.B * b.Hkv * units_per_head(b.rows, b.d);
    const int c = cluster_size(units, q8_tiles(max_keys), slots);
    const double count = (double)(units * c) / (double)slots;
    return {count > 1.0 ? count : 1.0, 5.0 + 0.0001 * b.d * (1.0 + tile_cost(nt)) * keys / c};
}
double own_time(const Batch &b, int sms) {
    const double cost = units_per_head(b.rows, b.d) * tile_cost(tiles_per_unit(b.rows, b.d));
    const double bytes = 0.65 * b.B * b.max_len * 2.0 * b.d * b.Hkv * cost;
    if (kvq8_num_parts(b.B, b.Hkv, b.rows, b.max_len, b.d, sms) > 0) {
        const double rate = 60e3 * b.max_len / (b.max_len + 1000.0) * sms;
        return 10.0 + bytes / (rate < 6.2e6 ? rate : 6.2e6);
    }
    const Waves w = line_waves(b, 0.65 * b.max_len, b.max_len, sms);
    const double rate = 60e3 * sms, all = 6.0 + bytes / (rate < 6.2e6 ? rate : 6.2e6), waves = w.count * w.time;
    return all > waves ? all : waves;
}

// The prefix's kernel in s runs.
double prefix_time(const Batch &b, int s, int num_sms) {
    const long long all = (long long)b.B * b.rows, units = b.Hkv * ((all + 255) / 256), blocks = (b.max_prefix + 127) / 128;
    const double block = all <= 128 ? (b.d == 64 ? 1.5 : 1.35) : b.d == 64 ? 1.75 : 2.0;
    return (double)((units * s + num_sms - 1) / num_sms) * ((b.d == 64 ? 9.0 : 11.0) + block * (double)((blocks + s - 1) / s));
}

// Both kernels, and the SMs that the own keys' is sized for: those that the prefix's leaves free, where they are an eighth and
// that is faster, or all.
struct Both {
    double time;
    int own_sms;
};
Both both(const Batch &b, int s, double prefix, double own_all, int num_sms) {
    const long long left = num_sms - b.Hkv * (((long long)b.B * b.rows + 255) / 256) * s;
    const double after = prefix + own_all + 4.0;
    if (left < num_sms / 8) return {after, num_sms};
    const double own = own_time(b, (int)left), beside = prefix > own ? prefix : own;
    return beside < after ? Both{beside, (int)left} : Both{after, num_sms};
}
int own_sms(const Batch &b, int s, int num_sms) {
    return both(b, s, prefix_time(b, s, num_sms), own_time(b, num_sms), num_sms).own_sms;
}

}  // namespace

void kvq8_prefix_plan(int B, int Hkv, int rows, int max_prefix, int max_len, int d, int num_sms, int *splits, int *parts) {
    const Batch b = {B, Hkv, rows, max_prefix, max_len, d};
    const long long all = (long long)B * rows, units = Hkv * ((all + 255) / 256), blocks = (max_prefix + 127) / 128;
    const int line_len = q8_tiles(max_prefix) * kTileKeys + max_len, nt = tiles_per_unit(rows, d);
    const double keys = max_prefix + 0.65 * max_len;
    *splits = 0;
    *parts = kvq8_num_parts(B, Hkv, rows, line_len, d, num_sms);
    double best = 10.0 + (*parts > 0 ? 4.0 : 0.0) + max_prefix / 6000.0 +
                  units_per_head(rows, d) * tile_cost(nt) * B * keys * 2.0 * d * Hkv / 8.3e6;
    if (*parts == 0) {
        const Waves w = line_waves(b, keys, line_len, num_sms);
        if (w.count * w.time > best) best = w.count * w.time;
    }
    const double own_all = own_time(b, num_sms);
    const long long most = units <= num_sms ? num_sms / units : 1;
    int sms = num_sms;
    for (int s = 1; s <= most && s <= blocks; ++s) {
        const double merge = 3.5 + 0.2 * s + (double)all * Hkv * (s + 1) * d * 4 / 6e6, prefix = prefix_time(b, s, num_sms);
        if (prefix + merge >= best) continue;
        const Both x = both(b, s, prefix, own_all, num_sms);
        if (x.time + merge < best) {
            best = x.time + merge;
            *splits = s;
            sms = x.own_sms;
        }
    }
    if (*splits == 0) return;
    *parts = kvq8_num_parts(B, Hkv, rows, max_len, d, sms);
    // Beside a longer prefix the own keys need no parts, and so no merge of their own. (One sequence of 16 rows, 4 heads share
    // one, 32768 + 1000: 50.2 us with parts, 44.2 without.)
    const Waves w = line_waves(b, 0.65 * max_len, max_len, sms);
    if (sms < num_sms && (int)(w.count + 0.999) * w.time < prefix_time(b, *splits, num_sms)) *parts = 0;
}

// Own summary, the runs' summaries, and what the own keys' parts take.
size_t kvq8_prefix_workspace_bytes(int B, int Hkv, int rows, int d, int splits, int parts) {
    const size_t own = kvq8_workspace_bytes(rows, d, parts);
    if (splits == 0) return own;
    const size_t n = (size_t)B * Hkv * rows;
    return align256(n * d * 4) + align256(n * 4) + align256(splits * n * d * 4) + align256(splits * n * 4) + own;
}

int launch_kvq8_prefix(const Kvq8AttnArgs &a, bool fp16) {
    if (a.splits == 0) return fp16 ? launch_q8_t<__half, kQ8Prefix>(a) : launch_q8_t<__nv_bfloat16, kQ8Prefix>(a);
    const size_t n = (size_t)a.B * a.H * a.Nq, d = a.c.d;
    char *at = reinterpret_cast<char *>(a.workspace);
    auto take = [&](size_t bytes) {
        float *x = reinterpret_cast<float *>(at);
        at += align256(bytes);
        return x;
    };
    float *own_o = take(n * d * 4), *own_lse = take(n * 4), *o_part = take(a.splits * n * d * 4), *lse_part = take(a.splits * n * 4);
    Kvq8AttnArgs own = a;
    own.out = own_o;
    own.lse = own_lse;
    own.workspace = reinterpret_cast<float *>(at);
    own.max_prefix = 0;
    if (a.parts == 0) own.num_sms = own_sms({a.B, a.c.Hkv, a.H / a.c.Hkv * a.Nq, a.max_prefix, a.max_len, (int)d}, a.splits, a.num_sms);
    int rc = launch_kvq8_prefix_tc(a, fp16, o_part, lse_part);
    if (rc == 0) rc = launch_kvq8_prefix_own(own, fp16);
    if (rc != 0) return rc;
    if (a.c.d == 128)
        return fp16 ? launch_merge<__half, 128>(a, own_o, own_lse, o_part, lse_part)
                    : launch_merge<__nv_bfloat16, 128>(a, own_o, own_lse, o_part, lse_part);
    return fp16 ? launch_merge<__half, 64>(a, own_o, own_lse, o_part, lse_part)
                : launch_merge<__nv_bfloat16, 64>(a, own_o, own_lse, o_part, lse_part);
}

}  // namespace fa
