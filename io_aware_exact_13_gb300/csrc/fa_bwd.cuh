// fa_bwd.cuh -- host-side arguments of the attention backward (recomputation).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

namespace fa {

constexpr int kBwdRows = 128;  // query rows per recomputed tile and keys per CTA

struct BwdArgs {
    const void *q, *k, *v, *out, *dout;  // [B][H][N][d]
    const float *lse;                    // [B][H][N], natural log
    void *dq, *dk, *dv;                  // [B][H][N][d]
    int B, H, N, d;
    float scale;
    int causal;
    float *dq_acc;   // workspace: fp32 [B*H][N][d]
    float *lse2;     // workspace: fp32 [B*H][Npad], lse * log2(e), +inf past N
    float *dsum;     // workspace: fp32 [B*H][Npad], rowsum(dO o O), 0 past N
    cudaStream_t stream;
    int *status;
    uint64_t timeout_ns;
    // keys of another sequence (launch_bwd_cross): k, v, dk, dv [B][Hkv][Nk][d], N query rows
    int Hkv = 0, Nk = 0, num_sms = 0;
    const int *kv_lens = nullptr;  // [B] keys in use, or nullptr (Nk)
    int parts = 1;                 // CTAs that share the query blocks of a key block
    float *kv_part = nullptr;      // workspace for parts > 1: fp32 [parts][2][B*Hkv][Nk][d] (dK, dV)
};

// CTAs per key block for the backward over keys of another length: where there are fewer key blocks than half the
// SMs, as many as fill the GPU, each with at least one (head, query block).
inline int bwd_cross_parts(int64_t BHkv, int group, int Nq, int Nk, int num_sms) {
    const int64_t blocks = BHkv * ((static_cast<int64_t>(Nk) + kBwdRows - 1) / kBwdRows);
    const int64_t n_it = group * ((static_cast<int64_t>(Nq) + kBwdRows - 1) / kBwdRows);
    int64_t n = num_sms / blocks;
    if (n > n_it) n = n_it;
    return n < 1 ? 1 : static_cast<int>(n);
}
inline size_t bwd_cross_part_bytes(int64_t BHkv, int Nk, int d, int parts) {
    return parts > 1 ? static_cast<size_t>(parts) * 2 * static_cast<size_t>(BHkv) * Nk * d * sizeof(float) : 0;
}

inline int64_t bwd_padded_rows(int N) { return ((static_cast<int64_t>(N) + kBwdRows - 1) / kBwdRows) * kBwdRows; }

// Workspace bytes for B*H heads of N rows and head dimension d, each part
// 256-byte aligned: dQ accumulator, then lse2, then dsum.
inline size_t bwd_workspace_bytes(int64_t BH, int N, int d) {
    const size_t acc = static_cast<size_t>(BH) * static_cast<size_t>(N) * static_cast<size_t>(d) * sizeof(float);
    const size_t row = static_cast<size_t>(BH) * static_cast<size_t>(bwd_padded_rows(N)) * sizeof(float);
    return ((acc + 255) / 256) * 256 + 2 * (((row + 255) / 256) * 256);
}

int launch_bwd(const BwdArgs &a, bool fp16);
int launch_bwd_cross(const BwdArgs &a, bool fp16);

}  // namespace fa
