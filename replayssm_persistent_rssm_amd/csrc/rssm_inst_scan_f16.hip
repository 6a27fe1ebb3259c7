// rssm_inst_scan_f16.hip -- selective-scan kernel instances with fp16 inputs.
#include "scan_inst.h"

namespace rssm {

const void* scan_f16_for(int which, int state_dtype, int dstate) { return scan_pick<kF16>(which, state_dtype, dstate); }

}  // namespace rssm
