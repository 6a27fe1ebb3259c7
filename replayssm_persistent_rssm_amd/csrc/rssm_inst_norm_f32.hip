// rssm_inst_norm_f32.hip -- block-norm kernel instances with f32 inputs.
#include "norm_inst.h"

namespace rssm {

const void* norm_f32_for(int residual_dtype, int channels) { return norm_pick<kF32>(residual_dtype, channels); }

}  // namespace rssm
