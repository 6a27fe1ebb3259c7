// rssm_inst_paged_f16.hip -- paged-attention kernel instances for f16.
#include "paged_inst.h"

namespace rssm {

const void* paged_f16_for(int which, int head_dim) { return paged_pick<kF16>(which, head_dim); }

}  // namespace rssm
