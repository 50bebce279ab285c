// fa_kvq8.cuh -- the 8-bit key/value cache: its layout, host-side arguments, and the
// device helpers its kernels (append, read, attention, weights, eviction) share.
//
// A cache is n_pages pages of `page` tokens (16, 32, 64 or 128). Codes are
// [n_pages][Hkv][page][d] bytes, scales [n_pages][Hkv] floats, K and V apart; a value is
// code * scale. Sequence s keeps position t in page page_table[s][t / page], slot t % page.
#pragma once
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

namespace fa {

constexpr int kKvq8Int8 = 0, kKvq8E4m3 = 1;  // FA_KVQ8_INT8, FA_KVQ8_E4M3
constexpr int kStatusSeqlensQ8 = -8;         // FA_ERR_SEQLENS
constexpr int kStatusPage = -10;             // FA_ERR_PAGE
constexpr int kStatusValue = -11;            // FA_ERR_VALUE
constexpr int kKvq8MaxNq = 16;

struct Kvq8Cache {
    uint8_t *k_codes, *v_codes;
    float *k_scale, *v_scale;
    const int *page_table;  // [nseq][max_pages]
    int n_pages, max_pages, page, Hkv, d, format;
};

struct Kvq8AppendArgs {
    Kvq8Cache c;
    const void *k, *v;  // [total][Hkv][d] with element strides between tokens and heads
    long long k_token, k_head, v_token, v_head;
    const int *cu_seqlens, *cache_lens;
    int nseq, total, max_new;
    int *status;
    cudaStream_t stream;
};

struct Kvq8ReadArgs {
    Kvq8Cache c;
    void *k, *v;  // [total][Hkv][d]
    const int *cu_seqlens, *first;  // first: position of each sequence's first token read, or NULL (0)
    int nseq, total, max_len;
    int *status;
    cudaStream_t stream;
};

struct Kvq8AttnArgs {
    Kvq8Cache c;
    const void *q;
    void *out;
    float *lse;
    const int *kv_lens;
    int B, H, Nq, max_len;
    float scale;
    int causal, parts, num_sms;
    float *workspace;
    int *status;
    cudaStream_t stream;
    const int *prefix_table = nullptr, *prefix_len = nullptr;  // of the prefix that all sequences share
    int max_prefix = 0, splits = 0;
    unsigned long long timeout_ns = 0;
};

struct Kvq8WeightsArgs {
    Kvq8Cache c;
    const void *q;
    const float *lse;
    float *weight;  // [B][Hkv][max_pages * page]
    const int *kv_lens;
    int B, H, Nq, max_len;
    float scale;
    int causal, num_sms;
    int *status;
    cudaStream_t stream;
};

struct Kvq8EvictArgs {
    Kvq8Cache c;
    const int *kv_lens;
    const float *weight;  // [nseq][Hkv][max_pages * page]
    float *weight_out;    // the same shape
    int *lens_out, *kept;  // [nseq], [nseq][Hkv][keep]
    int nseq, keep, recent, num_sms;
    int *status;
    cudaStream_t stream;
};

int launch_kvq8_append(const Kvq8AppendArgs &a, bool fp16);
int launch_kvq8_read(const Kvq8ReadArgs &a, bool fp16);
int launch_kvq8_attention(const Kvq8AttnArgs &a, bool fp16);
int launch_kvq8_prefix(const Kvq8AttnArgs &a, bool fp16);
// Runs of keys that a shared prefix is cut into (0: it is read with each sequence's own keys), the parts of the own keys,
// and the workspace.
void kvq8_prefix_plan(int B, int Hkv, int rows, int max_prefix, int max_len, int d, int num_sms, int *splits, int *parts);
size_t kvq8_prefix_workspace_bytes(int B, int Hkv, int rows, int d, int splits, int parts);
int launch_kvq8_weights(const Kvq8WeightsArgs &a, bool fp16);
int launch_kvq8_evict(const Kvq8EvictArgs &a);
// 16-key tiles of B sequences of max_len keys, over K/V heads and tiles of the `rows` = (H / Hkv) * Nq query rows
// that share one; a part count for them, and the workspace that it takes.
long long kvq8_tiles(int B, int Hkv, int rows, int max_len, int d);
int kvq8_num_parts(int B, int Hkv, int rows, int max_len, int d, int num_sms);
size_t kvq8_workspace_bytes(int rows, int d, int parts);

// A kernel's dynamic shared memory allowed beyond 48 KB, once for each device (the driver's call costs half a microsecond).
template <auto KERNEL>
bool allow_smem(int bytes) {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    const uint64_t bit = 1ull << (dev & 63);
    if (done.load(std::memory_order_relaxed) & bit) return true;
    if (cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
    done.fetch_or(bit, std::memory_order_relaxed);
    return true;
}

inline int kvq8_page_shift(int page) {
    int s = 0;
    while ((1 << s) < page) ++s;
    return s;
}

// Scales that are no powers of two (append writes none, but a cache may come from elsewhere): a product or quotient with
// one is rounded to fp32 before it is rounded to a code or to 16 bits, and twice is not once: what fp32 rounds to the
// middle between two results need not lie there. So fp32's rounding is made one to odd: an inexact result takes the
// neighbour whose last bit is 1, and the second rounding is then that of the exact value.
__device__ __forceinline__ bool power_of_two(float s) { return (__float_as_uint(s) & 0x7FFFFFu) == 0u; }  // or 0
// q = fl(exact), not 0 or far from the second rounding's middles; rest has the sign of exact - q.
__device__ __forceinline__ float to_odd(float q, float rest) {
    const int b = __float_as_int(q);
    if (rest == 0.0f || (b & 1) || q == 0.0f) return q;
    return __int_as_float((b ^ __float_as_int(rest)) >= 0 ? b + 1 : b - 1);
}
__device__ __forceinline__ float product_odd(float a, float b) {
    const float q = a * b;
    return to_odd(q, fmaf(a, b, -q));
}
__device__ __forceinline__ float quotient_odd(float a, float s) {  // s > 0
    const float q = __fdiv_rn(a, s);
    return to_odd(q, fmaf(-q, s, a));
}

// Four int8 codes -> two pairs of fp16, exact: code + 128 under the exponent of 1024 is the
// fp16 number 1152 + code.
__device__ __forceinline__ void int8x4_to_half2(uint32_t w, uint32_t &lo, uint32_t &hi) {
    const uint32_t u = w ^ 0x80808080u;
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 bias = __half2half2(__ushort_as_half(0x6480));  // 1152
    const __half2 x = __hsub2(*reinterpret_cast<const __half2 *>(&a), bias);
    const __half2 y = __hsub2(*reinterpret_cast<const __half2 *>(&b), bias);
    lo = *reinterpret_cast<const uint32_t *>(&x);
    hi = *reinterpret_cast<const uint32_t *>(&y);
}
// Four e4m3 codes -> two pairs of fp16 (every e4m3 number is an fp16 number).
__device__ __forceinline__ void e4m3x4_to_half2(uint32_t w, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}
template <int FMT>
__device__ __forceinline__ void codes_to_half2(uint32_t w, uint32_t &lo, uint32_t &hi) {
    if constexpr (FMT == kKvq8Int8) int8x4_to_half2(w, lo, hi);
    else e4m3x4_to_half2(w, lo, hi);
}

// Four values already divided by the scale -> four codes, rounded to nearest even and saturated.
template <int FMT>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
    if constexpr (FMT == kKvq8Int8) {
        // adding 1.5 * 2^23 leaves the rounded integer in the low bits
        auto code = [](float x) { return __float_as_uint(fminf(fmaxf(x, -127.0f), 127.0f) + 12582912.0f); };
        return __byte_perm(__byte_perm(code(a), code(b), 0x0040), __byte_perm(code(c), code(d), 0x0040), 0x5410);
    } else {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
        return lo | (hi << 16);
    }
}

// Smallest power of two s with a <= QMAX s, from the bits of a > 0 (QMAX = 1.984375 * 2^6 or
// 1.75 * 2^8: one more when a's mantissa is above QMAX's); 0 for a = 0.
template <int FMT>
__device__ __forceinline__ float scale_for(float a) {
    if (a == 0.0f) return 0.0f;
    const uint32_t bits = __float_as_uint(a);
    const uint32_t over = (bits & 0x7FFFFFu) > (FMT == kKvq8Int8 ? 0x7E0000u : 0x600000u) ? 1u : 0u;
    int e = (int)(bits >> 23) - 127 + (int)over - (FMT == kKvq8Int8 ? 6 : 8);
    e = min(max(e, -110), 120);
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

}  // namespace fa
