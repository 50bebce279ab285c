// fa_kvq8.cuh -- the 8-bit key/value cache: its layout, host-side arguments, and the
// device helpers its three kernels (append, read, attention) share.
//
// A cache is n_pages pages of `page` tokens (16, 32, 64 or 128). Codes are
// [n_pages][Hkv][page][d] bytes, scales [n_pages][Hkv] floats, K and V apart; a value is
// code * scale. Sequence s keeps position t in page page_table[s][t / page], slot t % page.
#pragma once
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

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
};

int launch_kvq8_append(const Kvq8AppendArgs &a, bool fp16);
int launch_kvq8_read(const Kvq8ReadArgs &a, bool fp16);
int launch_kvq8_attention(const Kvq8AttnArgs &a, bool fp16);
// 16-key tiles of B sequences of max_len keys, over K/V heads and tiles of the `rows` = (H / Hkv) * Nq query rows
// that share one; a part count for them, and the workspace that it takes.
long long kvq8_tiles(int B, int Hkv, int rows, int max_len, int d);
int kvq8_num_parts(int B, int Hkv, int rows, int max_len, int d, int num_sms);
size_t kvq8_workspace_bytes(int rows, int d, int parts);

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

}  // namespace fa
