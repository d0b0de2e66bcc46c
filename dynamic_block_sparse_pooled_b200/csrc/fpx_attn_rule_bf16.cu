// fpx_attn_rule_bf16.cu -- the tensor-core attention under a score rule, bf16 inputs: one kernel for
// each set of parts that a rule can have (fpx_attn_sm100.cuh).
#include "fpx_attn_sm100.cuh"

namespace fpx {
namespace sm100 {

AttnKernel rule_kernel_bf16(int rules) {
  switch (rules) {
    case 1: return attn_tc_kernel<false, false, 1>;
    case 3: return attn_tc_kernel<false, false, 3>;
    case 5: return attn_tc_kernel<false, false, 5>;
    default: return attn_tc_kernel<false, false, 7>;
  }
}

}  // namespace sm100
}  // namespace fpx
