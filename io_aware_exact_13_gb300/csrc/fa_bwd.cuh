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
    float *kv_part = nullptr;      // workspace: the cut blocks, then fp32 [bwd_cross_slots][2][128][d] (dK, dV)
};

// How the key blocks that hold keys are shared out over the CTAs of the backward over keys of another length. With a CTA
// per block the last wave of blocks may leave most SMs idle (768 blocks on 152 SMs: 6 waves for 5.05). So the blocks of
// that wave, [full, valid) of `valid` in line, are cut into `parts` runs of neighbouring iterations (head, query block),
// each an item of its own with fp32 dK and dV that are added up in order at the end. Items [0, full) are whole blocks,
// item full + t * parts + i is run i of block full + t. A run costs its iterations and about two more (its start and end,
// and the adding up); parts fill one or two waves, whichever is shorter, or are 1 when neither gains. Measured: B 4,
// H 32 / 8, d 128, 2500 queries, up to 4096 keys ragged (those 768 blocks) 1650 -> 1475 us, B 8, H 16, d 64, 448
// queries, up to 1500 keys ragged 99 -> 95 us, B 3, H 16 / 2, d 128, 1153 queries, 57 keys (6 blocks) 276 -> 45 us.
struct BwdCrossPlan {
    int valid, full, parts, items;
};
__host__ __device__ inline BwdCrossPlan bwd_cross_plan(int valid, int n_it, int num_sms) {
    BwdCrossPlan r;
    const int tail = valid % num_sms;
    r.valid = valid;
    r.full = valid - tail;
    r.parts = 1;
    int best = n_it + 1;
    for (int m = 1; m <= 2 && tail > 0; ++m) {
        int k = m * num_sms / tail;
        if (k > n_it) k = n_it;
        const int cost = (tail * k + num_sms - 1) / num_sms * ((n_it + k - 1) / k + 2);
        if (k > 1 && cost < best) {
            best = cost;
            r.parts = k;
        }
    }
    r.items = r.full + tail * r.parts;
    return r;
}
// At most so many items are cut blocks' runs, whatever the key counts are.
inline int64_t bwd_cross_slots(int64_t blocks, int64_t n_it, int num_sms) {
    const int64_t tail = blocks < num_sms ? blocks : num_sms;
    return n_it < 2 ? 0 : (tail * n_it < 2 * num_sms ? tail * n_it : 2 * num_sms);
}
inline int64_t bwd_cross_iters(int group, int Nq) {
    return group * ((static_cast<int64_t>(Nq) + kBwdRows - 1) / kBwdRows);
}
inline int64_t bwd_cross_blocks(int64_t BHkv, int Nk) {
    return BHkv * ((static_cast<int64_t>(Nk) + kBwdRows - 1) / kBwdRows);
}
inline size_t bwd_cross_cut_bytes(int num_sms) { return (static_cast<size_t>(num_sms + 1) * 16 + 255) / 256 * 256; }
inline size_t bwd_cross_part_bytes(int64_t slots, int d, int num_sms) {
    return bwd_cross_cut_bytes(num_sms) + static_cast<size_t>(slots) * 2 * kBwdRows * static_cast<size_t>(d) * sizeof(float);
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
