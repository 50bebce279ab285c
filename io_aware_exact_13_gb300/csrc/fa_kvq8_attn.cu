// fa_kvq8_attn.cu -- sizes and launches of the attention over the 8-bit cache (fa_kvq8_attn.cuh).
#include "fa_kvq8_attn.cuh"

namespace fa {

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
    return fp16 ? launch_q8_t<__half, kQ8Plain>(a) : launch_q8_t<__nv_bfloat16, kQ8Plain>(a);
}

}  // namespace fa
