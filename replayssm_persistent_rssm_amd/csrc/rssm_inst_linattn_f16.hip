// rssm_inst_linattn_f16.hip -- linear-attention kernel instances with f16 inputs.
#include "linattn_inst.h"

namespace rssm {

const void* linattn_f16_for(int which, int state_dtype, int dstate) { return linattn_pick<kF16>(which, state_dtype, dstate); }

}  // namespace rssm
