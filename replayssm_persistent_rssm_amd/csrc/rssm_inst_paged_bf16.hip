// rssm_inst_paged_bf16.hip -- paged-attention kernel instances for bf16.
#include "paged_inst.h"

namespace rssm {

const void* paged_bf16_for(int which, int head_dim) { return paged_pick<kBF16>(which, head_dim); }

}  // namespace rssm
