// rssm_inst_scan_f32.hip -- selective-scan kernel instances with fp32 inputs.
#include "scan_inst.h"

namespace rssm {

const void* scan_f32_for(int which, int state_dtype, int dstate) { return scan_pick<kF32>(which, state_dtype, dstate); }

}  // namespace rssm
