// Host-only stand-ins for the kernel launchers that token_api.cpp calls.
#include "delta.h"
#include "internal.h"
#include "norm.h"

namespace s4 {
s4dplr_status hip_failure(hipError_t) { return S4DPLR_ERR_HIP; }
hipError_t launch_norm_fwd(const NormArgs&, int, hipStream_t) { return hipSuccess; }
hipError_t launch_norm_bwd(const NormArgs&, int, hipStream_t) { return hipSuccess; }
hipError_t launch_delta_steps(const s4dplr_delta_plan*, const DeltaArgs&, hipStream_t) {
  return hipSuccess;
}
hipError_t launch_delta_prep(const s4dplr_delta_plan*, const DeltaArgs&, bool, hipStream_t) {
  return hipSuccess;
}
hipError_t launch_delta_scan(const s4dplr_delta_plan*, const DeltaArgs&, hipStream_t) {
  return hipSuccess;
}
hipError_t launch_delta_scan_bwd(const s4dplr_delta_plan*, const DeltaArgs&, hipStream_t) {
  return hipSuccess;
}
hipError_t launch_delta_grads(const s4dplr_delta_plan*, const DeltaArgs&, hipStream_t) {
  return hipSuccess;
}
}  // namespace s4
