// rssm_inst_scan_bf16.hip -- selective-scan kernel instances with bf16 inputs.
#include "scan_inst.h"

namespace rssm {

const void* scan_bf16_for(int which, int state_dtype, int dstate) { return scan_pick<kBF16>(which, state_dtype, dstate); }

}  // namespace rssm
