// fpx_attn_rule_e4m3.cu -- the tensor-core attention under a score rule, e4m3 inputs: one kernel for
// each set of parts that a rule can have (fpx_attn_sm100.cuh).
#include "fpx_attn_sm100.cuh"

namespace fpx {
namespace sm100 {

AttnKernel rule_kernel_e4m3(int rules) {
  switch (rules) {
    case 1: return attn_tc_kernel<true, false, 1>;
    case 3: return attn_tc_kernel<true, false, 3>;
    case 5: return attn_tc_kernel<true, false, 5>;
    default: return attn_tc_kernel<true, false, 7>;
  }
}

}  // namespace sm100
}  // namespace fpx
