// fa_kvq8_prefix_own.cu -- behind a shared prefix that is done apart: each sequence's own keys as a summary in fp32.
#include "fa_kvq8_attn.cuh"
#include "fa_kvq8_prefix.cuh"

namespace fa {

int launch_kvq8_prefix_own(const Kvq8AttnArgs &a, bool fp16) {
    return fp16 ? launch_q8_t<__half, kQ8Summary>(a) : launch_q8_t<__nv_bfloat16, kQ8Summary>(a);
}

}  // namespace fa
