// rssm_inst_norm_f16.hip -- block-norm kernel instances with f16 inputs.
#include "norm_inst.h"

namespace rssm {

const void* norm_f16_for(int residual_dtype, int channels) { return norm_pick<kF16>(residual_dtype, channels); }

}  // namespace rssm
