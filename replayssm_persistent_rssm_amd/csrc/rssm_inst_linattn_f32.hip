// rssm_inst_linattn_f32.hip -- linear-attention kernel instances with f32 inputs.
#include "linattn_inst.h"

namespace rssm {

const void* linattn_f32_for(int which, int state_dtype, int dstate) { return linattn_pick<kF32>(which, state_dtype, dstate); }

}  // namespace rssm
