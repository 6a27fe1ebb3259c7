// rssm_inst_norm_bf16.hip -- block-norm kernel instances with bf16 inputs.
#include "norm_inst.h"

namespace rssm {

const void* norm_bf16_for(int residual_dtype, int channels) { return norm_pick<kBF16>(residual_dtype, channels); }

}  // namespace rssm
