// fa_kvq8_cache.cu -- writing new tokens into the 8-bit key/value cache, and reading tokens back.
//
// Writing. One scale serves the `page` tokens of a page and head. With a the largest magnitude
// of the tokens in the page, the scale is the smallest power of two s with a <= QMAX s
// (QMAX = 127 for int8, 448 for e4m3), kept within 2^-110 .. 2^120 and 0 while every value is 0;
// a code is x / s rounded to nearest even. A page that held tokens before the call keeps its
// scale or, when the new tokens need a larger one, takes that and has its codes rounded to it:
//     s = max(s_old, s_new),   c' = rne(c s_old / s),   c = rne(x / s).
// (A page whose scale came from elsewhere keeps it while it is large enough; its codes are rounded once as well, and once
// more when it first grows, by a factor that need not be two.)
// Why powers of two: x / s and c s_old / s are then exact, so a code depends on the values alone
// and not on how a division rounds; and a scale that grows at least doubles, so a code's
// roundings in all of its page's growths add up to less than one step (1/2 + 1/4 + ...). With
// amax / 127 a page that fills token by token could round every code at every token. For e4m3
// nothing is lost; for int8 the step is at most twice that of amax / 127.
//
// Reading is code * scale, rounded once to the 16-bit type.
//
// Both are bound by HBM: 2 bytes + 1 byte per value.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "fa_kvq8.cuh"

namespace fa {
namespace {

template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t v) {
    if constexpr (std::is_same<T, __nv_bfloat16>::value) return __bfloat1622float2(*reinterpret_cast<__nv_bfloat162 *>(&v));
    else return __half22float2(*reinterpret_cast<__half2 *>(&v));
}
template <typename T>
__device__ __forceinline__ uint32_t pack2h(float lo, float hi) {
    if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<uint32_t *>(&h);
    } else {
        __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<uint32_t *>(&h);
    }
}
template <typename T>
constexpr uint32_t exponent_mask() { return std::is_same<T, __nv_bfloat16>::value ? 0x7F80u : 0x7C00u; }

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

struct AppendParams {
    const void *src[2];
    long long token[2], head[2];
    uint8_t *codes[2];
    float *scale[2];
    const int *page_table, *cu_seqlens, *cache_lens;
    int *status;
    int n_pages, max_pages, page_shift, Hkv, d_shift;
    int nseq, total, max_new, pages_per_seq;
};

// One CTA writes the new tokens of one (sequence, page, head), K or V, or both (KVS = 2, small pages): every value is
// read once into registers (VEC 16-byte vectors per thread hold the whole page), the page's largest magnitude is
// reduced over the CTA, and the codes are written as 8-byte vectors.
template <typename T, int FMT, int NT, int VEC, int KVS>
__global__ void __launch_bounds__(NT, KVS == 1 ? 1024 / NT : 28) fa_kvq8_append_kernel(const AppendParams p) {
    __shared__ uint32_t warp_max[NT / 32];
    uint32_t u = blockIdx.x;
    const int kv0 = KVS == 2 ? 0 : u & 1u;
    if (KVS == 1) u >>= 1;
    const int head = u % p.Hkv;
    u /= p.Hkv;
    const int ord = u % p.pages_per_seq, seq = u / p.pages_per_seq;
    const int held = __ldg(p.cache_lens + seq);
    const int c0 = __ldg(p.cu_seqlens + seq), c1 = __ldg(p.cu_seqlens + seq + 1);
    const int page = 1 << p.page_shift;
    if (c0 < 0 || c1 < c0 || c1 > p.total || c1 - c0 > p.max_new || held < 0 ||
        (long long)held + (c1 - c0) > (long long)p.max_pages * page) {
        if (threadIdx.x == 0) atomicExch(p.status, kStatusSeqlensQ8);
        return;
    }
    const int n = c1 - c0;
    const int pg = (held >> p.page_shift) + ord;
    if (n == 0 || pg > ((held + n - 1) >> p.page_shift)) return;
    const int phys = __ldg(p.page_table + (long long)seq * p.max_pages + pg);  // looked at once the values are on their way
    const int t0 = pg << p.page_shift;  // position of the page's first slot
    const int lo = max(held, t0) - t0;  // slots [lo, hi) take new tokens, [0, lo) hold earlier ones
    const int hi = min(held + n - t0, page);

    const int vec_shift = p.d_shift - 3;  // 8-value vectors per row
    uint4 xs[KVS][VEC];
#pragma unroll
    for (int j = 0; j < KVS; ++j) {
        const T *src = static_cast<const T *>(p.src[kv0 + j]) + (long long)head * p.head[kv0 + j];
        const long long token = p.token[kv0 + j];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const int vec = threadIdx.x + i * NT;
            const int slot = vec >> vec_shift, chunk = vec & ((1 << vec_shift) - 1);
            xs[j][i] = make_uint4(0u, 0u, 0u, 0u);
            if (slot >= lo && slot < hi)
                xs[j][i] = __ldg(reinterpret_cast<const uint4 *>(src + (long long)(c0 + (t0 + slot - held)) * token + chunk * 8));
        }
    }
    if (phys < 0 || phys >= p.n_pages) {
        if (threadIdx.x == 0) atomicExch(p.status, kStatusPage);
        return;
    }
    const long long unit = (long long)phys * p.Hkv + head;
#pragma unroll
    for (int j = 0; j < KVS; ++j) {
        if (j > 0) __syncthreads();  // warp_max is used again
        float *scale = p.scale[kv0 + j] + unit;
        const float s_old = lo > 0 ? *scale : 0.0f;
        uint4 (&x)[VEC] = xs[j];
        uint32_t most = 0;  // the largest magnitude's 15 bits, in either half
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const uint32_t a = __vmaxs2(x[i].x & 0x7FFF7FFFu, x[i].y & 0x7FFF7FFFu);
            const uint32_t b = __vmaxs2(x[i].z & 0x7FFF7FFFu, x[i].w & 0x7FFF7FFFu);
            most = __vmaxs2(most, __vmaxs2(a, b));
        }
        auto block_max = [&](uint32_t m) {
            m = __reduce_max_sync(0xffffffffu, max(m & 0xFFFFu, m >> 16));
            if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = m;
            __syncthreads();
            m = warp_max[0];
#pragma unroll
            for (int w = 1; w < NT / 32; ++w) m = max(m, warp_max[w]);
            return m;
        };
        uint32_t top = block_max(most);
        if (top >= exponent_mask<T>()) {  // infinities or NaN: no code stands for them; they are written as 0 and reported
            if (threadIdx.x == 0) atomicExch(p.status, kStatusValue);
            most = 0;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                uint32_t *w = reinterpret_cast<uint32_t *>(&x[i]);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if ((w[e] & 0x7FFFu) >= exponent_mask<T>()) w[e] &= 0xFFFF0000u;
                    if (((w[e] >> 16) & 0x7FFFu) >= exponent_mask<T>()) w[e] &= 0x0000FFFFu;
                    most = __vmaxs2(most, w[e] & 0x7FFF7FFFu);
                }
            }
            __syncthreads();  // every thread has read the first maxima
            top = block_max(most);
        }
        const float s = fmaxf(scale_for<FMT>(unpack2<T>(top).x), s_old);
        const float inv = s > 0.0f ? 1.0f / s : 0.0f;
        if (threadIdx.x == 0) *scale = s;  // every thread read the old one before block_max's barrier
        uint8_t *dst = p.codes[kv0 + j] + (unit << (p.page_shift + p.d_shift));
        const bool grew = lo > 0 && s != s_old;
        const float ratio = s_old * inv;
        if (!power_of_two(s) || (grew && !power_of_two(s_old))) {  // a scale from elsewhere: a rare, slower way
            const T *src = static_cast<const T *>(p.src[kv0 + j]) + (long long)head * p.head[kv0 + j];
            const float up = s < 0x1p-60f ? 0x1p60f : 1.0f;  // (keeps the quotient's remainder in range; exact)
#pragma unroll 1
            for (int vec = threadIdx.x; vec < NT * VEC; vec += NT) {
                const int slot = vec >> vec_shift, chunk = vec & ((1 << vec_shift) - 1);
                float f[8];
                if (slot >= lo && slot < hi) {
                    const uint4 y = __ldg(reinterpret_cast<const uint4 *>(
                        src + (long long)(c0 + (t0 + slot - held)) * p.token[kv0 + j] + chunk * 8));
                    const uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 a = unpack2<T>(w[e]);
                        f[2 * e] = isfinite(a.x) ? quotient_odd(a.x * up, s * up) : 0.0f;
                        f[2 * e + 1] = isfinite(a.y) ? quotient_odd(a.y * up, s * up) : 0.0f;
                    }
                } else if (grew && slot < lo) {
                    const uint2 was = *reinterpret_cast<const uint2 *>(dst + (long long)vec * 8);
                    const uint32_t w[2] = {was.x, was.y};
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        uint32_t h[2];
                        codes_to_half2<FMT>(w[e], h[0], h[1]);
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float2 a = unpack2<__half>(h[i]);
                            f[4 * e + 2 * i] = product_odd(a.x, ratio);
                            f[4 * e + 2 * i + 1] = product_odd(a.y, ratio);
                        }
                    }
                } else {
                    continue;
                }
                *reinterpret_cast<uint2 *>(dst + (long long)vec * 8) =
                    make_uint2(encode4<FMT>(f[0], f[1], f[2], f[3]), encode4<FMT>(f[4], f[5], f[6], f[7]));
            }
            continue;
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const int vec = threadIdx.x + i * NT;
            const int slot = vec >> vec_shift;
            if (slot >= lo && slot < hi) {
                const float2 a = unpack2<T>(x[i].x), b = unpack2<T>(x[i].y), c = unpack2<T>(x[i].z), d = unpack2<T>(x[i].w);
                uint2 o;
                o.x = encode4<FMT>(a.x * inv, a.y * inv, b.x * inv, b.y * inv);
                o.y = encode4<FMT>(c.x * inv, c.y * inv, d.x * inv, d.y * inv);
                *reinterpret_cast<uint2 *>(dst + (long long)vec * 8) = o;
            } else if (grew && slot < lo) {
                const uint2 was = *reinterpret_cast<const uint2 *>(dst + (long long)vec * 8);
                uint2 o;
                const uint32_t w[2] = {was.x, was.y};
                uint32_t r[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    uint32_t h0, h1;
                    codes_to_half2<FMT>(w[e], h0, h1);
                    const float2 a = unpack2<__half>(h0), b = unpack2<__half>(h1);
                    r[e] = encode4<FMT>(a.x * ratio, a.y * ratio, b.x * ratio, b.y * ratio);
                }
                o.x = r[0];
                o.y = r[1];
                *reinterpret_cast<uint2 *>(dst + (long long)vec * 8) = o;
            }
        }
    }
}

struct ReadParams {
    const uint8_t *codes[2];
    const float *scale[2];
    void *dst[2];
    const int *page_table, *cu_seqlens, *first;
    int *status;
    int n_pages, max_pages, page_shift, Hkv, d_shift;
    int nseq, total, max_len, groups_per_seq;
};

// Small CTAs again: 64 threads and 16 tokens 80.0 us, 128 and 32 82.9, 256 and 64 86.0 (87000 tokens, 8 heads, d 128).
// (The first is 76.3 since scales that are no powers of two have a branch of their own; one sequence of 700 tokens is 2.03
// instead of 1.93.)
constexpr int kReadThreads = 64;
constexpr int kReadTokens = 16;  // tokens per CTA: K and V of one head

// One CTA reads kReadTokens tokens of one (sequence, head), K and V: a thread's loads (16 codes
// each) are all issued before the first is used.
template <typename T, int FMT, int D>
__global__ void __launch_bounds__(kReadThreads) fa_kvq8_read_kernel(const ReadParams p) {
    constexpr int VPR = D / 16;                                      // 16-code vectors per row
    constexpr int VEC = kReadTokens * VPR / kReadThreads;            // vectors per thread and tensor
    static_assert(VEC >= 1 && kReadTokens * VPR % kReadThreads == 0, "whole vectors per thread");
    uint32_t u = blockIdx.x;
    const int head = u % p.Hkv;
    u /= p.Hkv;
    const int group = u % p.groups_per_seq, seq = u / p.groups_per_seq;
    const int c0 = __ldg(p.cu_seqlens + seq), c1 = __ldg(p.cu_seqlens + seq + 1);
    const int from = p.first ? __ldg(p.first + seq) : 0;
    const int page = 1 << p.page_shift;
    if (c0 < 0 || c1 < c0 || c1 > p.total || c1 - c0 > p.max_len || from < 0 ||
        (long long)from + (c1 - c0) > (long long)p.max_pages * page) {
        if (threadIdx.x == 0) atomicExch(p.status, kStatusSeqlensQ8);
        return;
    }
    const int n = c1 - c0;
    if (group * kReadTokens >= n) return;
    uint4 x[2][VEC];
    float s[2][VEC];
    bool ok[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        const int vec = threadIdx.x + i * kReadThreads;
        const int t = group * kReadTokens + vec / VPR, chunk = vec % VPR;
        ok[i] = t < n;
        if (ok[i]) {
            const int pos = from + t;
            const int phys = __ldg(p.page_table + (long long)seq * p.max_pages + (pos >> p.page_shift));
            if (phys < 0 || phys >= p.n_pages) {
                atomicExch(p.status, kStatusPage);
                ok[i] = false;
            } else {
                const long long unit = (long long)phys * p.Hkv + head;
                const long long off = ((unit << p.page_shift) + (pos & (page - 1))) * D + chunk * 16;
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    x[kv][i] = __ldg(reinterpret_cast<const uint4 *>(p.codes[kv] + off));
                    s[kv][i] = __ldg(p.scale[kv] + unit);
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        if (!ok[i]) continue;
        const int vec = threadIdx.x + i * kReadThreads;
        const int t = group * kReadTokens + vec / VPR, chunk = vec % VPR;
        const long long row = ((long long)(c0 + t) * p.Hkv + head) * D + chunk * 16;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            const uint32_t w[4] = {x[kv][i].x, x[kv][i].y, x[kv][i].z, x[kv][i].w};
            uint32_t o[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                uint32_t h0, h1;
                codes_to_half2<FMT>(w[e], h0, h1);
                const float2 a = unpack2<__half>(h0), b = unpack2<__half>(h1);
                if (power_of_two(s[kv][i])) {
                    o[2 * e] = pack2h<T>(a.x * s[kv][i], a.y * s[kv][i]);
                    o[2 * e + 1] = pack2h<T>(b.x * s[kv][i], b.y * s[kv][i]);
                } else {
                    o[2 * e] = pack2h<T>(product_odd(a.x, s[kv][i]), product_odd(a.y, s[kv][i]));
                    o[2 * e + 1] = pack2h<T>(product_odd(b.x, s[kv][i]), product_odd(b.y, s[kv][i]));
                }
            }
            uint4 *dst = reinterpret_cast<uint4 *>(static_cast<T *>(p.dst[kv]) + row);
            dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
            dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
        }
    }
}

int log2i(int x) {
    int s = 0;
    while ((1 << s) < x) ++s;
    return s;
}

template <typename T, int FMT>
int launch_append_t(const Kvq8AppendArgs &a) {
    AppendParams p;
    p.src[0] = a.k;
    p.src[1] = a.v;
    p.token[0] = a.k_token;
    p.token[1] = a.v_token;
    p.head[0] = a.k_head;
    p.head[1] = a.v_head;
    p.codes[0] = a.c.k_codes;
    p.codes[1] = a.c.v_codes;
    p.scale[0] = a.c.k_scale;
    p.scale[1] = a.c.v_scale;
    p.page_table = a.c.page_table;
    p.cu_seqlens = a.cu_seqlens;
    p.cache_lens = a.cache_lens;
    p.status = a.status;
    p.n_pages = a.c.n_pages;
    p.max_pages = a.c.max_pages;
    p.page_shift = log2i(a.c.page);
    p.Hkv = a.c.Hkv;
    p.d_shift = log2i(a.c.d);
    p.nseq = a.nseq;
    p.total = a.total;
    p.max_new = a.max_new;
    // max_new tokens that start in a page's last slot touch this many pages
    long long pages = ((long long)a.max_new + a.c.page - 2) / a.c.page + 1;
    if (pages > a.c.max_pages) pages = a.c.max_pages;
    p.pages_per_seq = static_cast<int>(pages);
    const int vecs = a.c.page * a.c.d / 8;
    const long long grid = (vecs > 128 ? 2ll : 1ll) * a.c.Hkv * pages * a.nseq;
    if (grid > INT32_MAX) return -3;
    const unsigned g = static_cast<unsigned>(grid);
    // Eight vectors per thread (a warp at least): small CTAs keep more of them, and of their dependent first reads (lengths,
    // page), on an SM. With 128 or 256 threads for every page size, pages of 16 tokens took 86 us instead of 72, of 64
    // tokens 77 instead of 65 (74000 tokens, 8 heads, d 128). At 16 tokens of d 64 a warp takes K and V: 36 us instead of 53
    // (e4m3; 35.0 with 28 CTAs an SM asked for, 38.3 at the 77 registers that the branch for other scales would take).
    switch (vecs) {
        case 128: fa_kvq8_append_kernel<T, FMT, 32, 4, 2><<<g, 32, 0, a.stream>>>(p); break;
        case 256: fa_kvq8_append_kernel<T, FMT, 32, 8, 1><<<g, 32, 0, a.stream>>>(p); break;
        case 512: fa_kvq8_append_kernel<T, FMT, 64, 8, 1><<<g, 64, 0, a.stream>>>(p); break;
        case 1024: fa_kvq8_append_kernel<T, FMT, 128, 8, 1><<<g, 128, 0, a.stream>>>(p); break;
        case 2048: fa_kvq8_append_kernel<T, FMT, 256, 8, 1><<<g, 256, 0, a.stream>>>(p); break;
        default: return -4;
    }
    return cudaGetLastError() == cudaSuccess ? 0 : -5;
}

template <typename T, int FMT>
int launch_read_t(const Kvq8ReadArgs &a) {
    ReadParams p;
    p.codes[0] = a.c.k_codes;
    p.codes[1] = a.c.v_codes;
    p.scale[0] = a.c.k_scale;
    p.scale[1] = a.c.v_scale;
    p.dst[0] = a.k;
    p.dst[1] = a.v;
    p.page_table = a.c.page_table;
    p.cu_seqlens = a.cu_seqlens;
    p.first = a.first;
    p.status = a.status;
    p.n_pages = a.c.n_pages;
    p.max_pages = a.c.max_pages;
    p.page_shift = log2i(a.c.page);
    p.Hkv = a.c.Hkv;
    p.d_shift = log2i(a.c.d);
    p.nseq = a.nseq;
    p.total = a.total;
    p.max_len = a.max_len;
    p.groups_per_seq = (a.max_len + kReadTokens - 1) / kReadTokens;
    const long long grid = (long long)a.c.Hkv * p.groups_per_seq * a.nseq;
    if (grid > INT32_MAX) return -3;
    if (a.c.d == 128)
        fa_kvq8_read_kernel<T, FMT, 128><<<static_cast<unsigned>(grid), kReadThreads, 0, a.stream>>>(p);
    else
        fa_kvq8_read_kernel<T, FMT, 64><<<static_cast<unsigned>(grid), kReadThreads, 0, a.stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? 0 : -5;
}

}  // namespace

int launch_kvq8_append(const Kvq8AppendArgs &a, bool fp16) {
    if (a.c.format == kKvq8Int8)
        return fp16 ? launch_append_t<__half, kKvq8Int8>(a) : launch_append_t<__nv_bfloat16, kKvq8Int8>(a);
    return fp16 ? launch_append_t<__half, kKvq8E4m3>(a) : launch_append_t<__nv_bfloat16, kKvq8E4m3>(a);
}

int launch_kvq8_read(const Kvq8ReadArgs &a, bool fp16) {
    if (a.c.format == kKvq8Int8)
        return fp16 ? launch_read_t<__half, kKvq8Int8>(a) : launch_read_t<__nv_bfloat16, kKvq8Int8>(a);
    return fp16 ? launch_read_t<__half, kKvq8E4m3>(a) : launch_read_t<__nv_bfloat16, kKvq8E4m3>(a);
}

}  // namespace fa
