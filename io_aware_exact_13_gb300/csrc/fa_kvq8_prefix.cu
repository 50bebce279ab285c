// fa_kvq8_prefix.cu -- attention over the 8-bit cache for a batch whose sequences share a prefix.
#include "fa_kvq8_attn.cuh"

namespace fa {

int kvq8_prefix_splits(int, int, int, int, int, int, int) { return 0; }

size_t kvq8_prefix_workspace_bytes(int, int, int rows, int d, int, int parts) { return kvq8_workspace_bytes(rows, d, parts); }

int launch_kvq8_prefix(const Kvq8AttnArgs &a, bool fp16) {
    return fp16 ? launch_q8_t<__half, true>(a) : launch_q8_t<__nv_bfloat16, true>(a);
}

}  // namespace fa
