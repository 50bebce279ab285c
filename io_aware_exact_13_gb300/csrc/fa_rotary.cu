// fa_rotary.cu -- rotary positions with several axes (text, images, video): queries and keys turned by angles that go
// by each token's position along its axes, and turned back for the gradient.
//
// Pair i of a row is dims i and r + i (r pairs, the dims from 2 r on pass through). With p = positions[axis(i)] of the
// token and f_i its frequency,
//     y_i = x_i cos(p f_i) - x_{r+i} sin(p f_i),     y_{r+i} = x_i sin(p f_i) + x_{r+i} cos(p f_i).
// The gradient of a rotation is the rotation back: dx is dy turned by -p f_i.
//
// Angles: p f_i in 32 bits is off by 2^-24 of itself, 6e-3 at position 100000, more than bf16's rounding. So a frequency
// is held as the fraction of a turn that one position makes, t_i = f_i / 2 pi mod 1 in 64 bits of fixed point. The integer
// product p t_i mod 2^64 is then the angle's place on the circle with all whole turns taken out exactly, for any 32-bit
// position of either sign (off by |p| (f_i 2^-54 + 2^-64) turns at most, from the 53 bits of f_i / 2 pi and their cut to 64 of
// fixed point). It goes to sincospi in fp32.
// Products and sums are fp32, and each result is rounded once.
//
// Bound: HBM, each value read and written once. A thread turns the same 16 dims of up to ten heads by one set of eight
// angles, all its loads requested before the angles are formed, and nothing stays in the caches. Measured: 30011 tokens of
// 32 + 8 heads of 128, 96.5 us (94 % of the copy rate); 16 tokens 6.3 us with the launch.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "fa_rotary.cuh"

namespace fa {
namespace {

constexpr int kThreads = 128;

struct RotaryParams {
    RotaryTensor x[2];
    const int *positions;
    uint64_t turns[kRotaryMaxPairs];
    uint8_t axis[kRotaryMaxPairs];
    int pairs, N, lane_shift, slots, inverse;
    long long tokens, threads;
};

template <typename T>
__device__ __forceinline__ float2 to_float2(uint32_t v) {
    if constexpr (std::is_same<T, __nv_bfloat16>::value) return __bfloat1622float2(*reinterpret_cast<__nv_bfloat162 *>(&v));
    else return __half22float2(*reinterpret_cast<__half2 *>(&v));
}
template <typename T>
__device__ __forceinline__ uint32_t from_float2(float a, float b) {
    if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<uint32_t *>(&h);
    } else {
        __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<uint32_t *>(&h);
    }
}

// A row (token, head) is d / 16 units of two 16-byte vectors: dims 8 u and r + 8 u for the first r / 8, then pairs of
// vectors that pass through. Threads are numbered unit, head slot, token, and a thread does HEADS heads, `slots` apart.
template <typename T, int HEADS, int MINB>
__global__ void __launch_bounds__(kThreads, MINB) fa_rotary_kernel(const __grid_constant__ RotaryParams p) {
    const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
    if (id >= p.threads) return;
    const int u = (int)(id & ((1 << p.lane_shift) - 1));
    const long long row = id >> p.lane_shift, token = row / p.slots;
    const int slot = (int)(row - token * p.slots);
    const long long b = token / p.N, n = token - b * p.N;
    const int rotated = p.pairs / 8;  // units that are turned
    const bool turn = u < rotated;
    const int lo = turn ? 8 * u : 2 * p.pairs + 16 * (u - rotated), hi = turn ? lo + p.pairs : lo + 8;

    uint4 a[HEADS], c[HEADS];
    T *dst[HEADS];
#pragma unroll
    for (int j = 0; j < HEADS; ++j) {
        int head = slot + j * p.slots;
        dst[j] = nullptr;
        const bool second = head >= p.x[0].heads;
        if (second) head -= p.x[0].heads;
        const RotaryTensor &t = p.x[second];
        if (head < t.heads) {
            const T *src = static_cast<const T *>(t.in) + b * t.in_b + n * t.in_n + head * t.in_h;
            dst[j] = static_cast<T *>(t.out) + b * t.out_b + n * t.out_n + head * t.out_h;
            a[j] = __ldcs(reinterpret_cast<const uint4 *>(src + lo));
            c[j] = __ldcs(reinterpret_cast<const uint4 *>(src + hi));
        }
    }
    float sn[8], cs[8];
    if (turn) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int pos = __ldg(p.positions + (long long)p.axis[lo + i] * p.tokens + token);
            const long long at = (long long)((uint64_t)(long long)pos * p.turns[lo + i]);  // 2^-64 turns, mod one turn
            sincospif(__ll2float_rn(at) * 0x1p-63f, &sn[i], &cs[i]);
            if (p.inverse) sn[i] = -sn[i];
        }
    }
#pragma unroll
    for (int j = 0; j < HEADS; ++j) {
        if (dst[j] == nullptr) continue;
        if (turn) {
            uint32_t (&av)[4] = *reinterpret_cast<uint32_t (*)[4]>(&a[j]);
            uint32_t (&cv)[4] = *reinterpret_cast<uint32_t (*)[4]>(&c[j]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 x = to_float2<T>(av[e]), y = to_float2<T>(cv[e]);
                av[e] = from_float2<T>(fmaf(x.x, cs[2 * e], -(y.x * sn[2 * e])), fmaf(x.y, cs[2 * e + 1], -(y.y * sn[2 * e + 1])));
                cv[e] = from_float2<T>(fmaf(x.x, sn[2 * e], y.x * cs[2 * e]), fmaf(x.y, sn[2 * e + 1], y.y * cs[2 * e + 1]));
            }
        }
        __stcs(reinterpret_cast<uint4 *>(dst[j] + lo), a[j]);
        __stcs(reinterpret_cast<uint4 *>(dst[j] + hi), c[j]);
    }
}

template <typename T, int HEADS, int MINB>
int launch_heads(RotaryParams &p, long long tokens, int heads, cudaStream_t stream) {
    p.slots = (heads + HEADS - 1) / HEADS;
    p.threads = (tokens * p.slots) << p.lane_shift;
    const long long grid = (p.threads + kThreads - 1) / kThreads;
    if (grid > INT32_MAX) return -3;
    fa_rotary_kernel<T, HEADS, MINB><<<static_cast<unsigned>(grid), kThreads, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? 0 : -5;
}

template <typename T>
int launch_t(const RotaryArgs &a) {
    RotaryParams p;
    p.x[0] = a.x[0];
    p.x[1] = a.x[1];
    p.positions = a.positions;
    for (int i = 0; i < kRotaryMaxPairs; ++i) {
        p.turns[i] = i < a.pairs ? a.turns[i] : 0;
        p.axis[i] = i < a.pairs ? a.axis[i] : 0;
    }
    p.pairs = a.pairs;
    p.N = a.N;
    p.lane_shift = a.d == 128 ? 3 : 2;
    p.inverse = a.inverse;
    p.tokens = (long long)a.B * a.N;
    const int heads = a.x[0].heads + a.x[1].heads;
    // Heads of a thread: eight, or ten or four where those leave fewer threads with less to do. (32 + 8 heads of 128, 65536
    // tokens: four 212 us, five 198, eight 197, ten 197; 8 + 1 heads: 63.8, 55.4, 63.6, 51.5; up to 64 tokens all 6.3.)
    auto idle = [&](int h) { return (heads + h - 1) / h * h - heads; };
    if (idle(8) <= idle(10) && idle(8) <= idle(4)) return launch_heads<T, 8, 4>(p, p.tokens, heads, a.stream);
    if (idle(10) <= idle(4)) return launch_heads<T, 10, 4>(p, p.tokens, heads, a.stream);
    return launch_heads<T, 4, 8>(p, p.tokens, heads, a.stream);
}

}  // namespace

int launch_rotary(const RotaryArgs &a, bool fp16) { return fp16 ? launch_t<__half>(a) : launch_t<__nv_bfloat16>(a); }

}  // namespace fa
