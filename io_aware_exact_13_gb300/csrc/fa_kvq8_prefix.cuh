// fa_kvq8_prefix.cuh -- host-side interface of the shared prefix's kernels: the prefix for all rows at once
// (fa_kvq8_prefix_tc.cu) and each sequence's own keys as a summary (fa_kvq8_prefix_own.cu).
#pragma once
#include "fa_kvq8.cuh"

namespace fa {

// Summaries of `splits` runs of the prefix's keys: o_part [splits][B * H * Nq][d] fp32, normalised, and lse_part
// [splits][B * H * Nq], natural log; a row that sees no key of a run has lse -inf and any o.
int launch_kvq8_prefix_tc(const Kvq8AttnArgs &a, bool fp16, float *o_part, float *lse_part);
// The own keys' summary, fp32, into a.out and a.lse (0 and -inf for rows without keys).
int launch_kvq8_prefix_own(const Kvq8AttnArgs &a, bool fp16);

}  // namespace fa
