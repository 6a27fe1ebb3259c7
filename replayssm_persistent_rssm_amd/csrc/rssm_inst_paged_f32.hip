// rssm_inst_paged_f32.hip -- paged-attention kernel instances for f32.
#include "paged_inst.h"

namespace rssm {

const void* paged_f32_for(int which, int head_dim) { return paged_pick<kF32>(which, head_dim); }

}  // namespace rssm
