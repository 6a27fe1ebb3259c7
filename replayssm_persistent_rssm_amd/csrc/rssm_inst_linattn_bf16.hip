// rssm_inst_linattn_bf16.hip -- linear-attention kernel instances with bf16 inputs.
#include "linattn_inst.h"

namespace rssm {

const void* linattn_bf16_for(int which, int state_dtype, int dstate) { return linattn_pick<kBF16>(which, state_dtype, dstate); }

}  // namespace rssm
