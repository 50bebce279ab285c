// fa_rotary.cuh -- host-side arguments of the rotary positions (fa_rotary.cu).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

namespace fa {

constexpr int kRotaryMaxPairs = 64, kRotaryMaxAxes = 8;

struct RotaryTensor {  // [B][heads][N][d] by element strides, head dimension contiguous
    const void *in;
    void *out;
    long long in_b, in_n, in_h, out_b, out_n, out_h;
    int heads;
};

struct RotaryArgs {
    RotaryTensor x[2];     // q, k (heads 0: none)
    const int *positions;  // [n_axes][B * N]
    uint64_t turns[kRotaryMaxPairs];  // what one position turns a pair by, in 2^-64 of a full turn
    uint8_t axis[kRotaryMaxPairs];
    int pairs, B, N, d, inverse;
    cudaStream_t stream;
};

int launch_rotary(const RotaryArgs &a, bool fp16);

}  // namespace fa
