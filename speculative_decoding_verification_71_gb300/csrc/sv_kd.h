// What the distillation kernels (sv_kd.cu, sv_toploss.cu) share with the C ABI.
#pragma once

namespace sv {

// The limit of their waits for staged logits, a call's at the time of the call
// (sv_api.cu: spec_kd_set_wait_limit_ns).
long long kd_wait_limit_ns();

}  // namespace sv
