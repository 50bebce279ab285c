// fp16 instantiations of the forward over keys of another length (the 128-key-block
// kernel).
#include "fa_launch.cuh"

namespace fa {
int launch_fwd_cross_fp16(const LaunchArgs &a) { return launch_cross_fwd<__half>(a); }
}  // namespace fa
