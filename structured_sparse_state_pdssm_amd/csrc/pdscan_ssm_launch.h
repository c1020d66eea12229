// Declarations of the launchers of the selective scan, the convolution and the norm.
#pragma once

#include <hip/hip_runtime_api.h>

#include "pdscan_ssm_plan.h"

namespace pdscan {

hipError_t launch_selscan_fwd(const SsArgs& a, int bf16, hipStream_t st);
hipError_t launch_selscan_state(const SsArgs& a, int bf16, hipStream_t st);   // with a.adj backwards too
hipError_t launch_selscan_carry(const SsCarryArgs& a, hipStream_t st);
hipError_t launch_selscan_bwd(const SsArgs& a, int bf16, hipStream_t st);
hipError_t launch_selscan_fold(const SsFoldArgs& a, int bf16, hipStream_t st);
hipError_t launch_ssm_sum(const SsSumArgs& a, hipStream_t st);
hipError_t launch_selscan_step(const SsStepArgs& a, int bf16, hipStream_t st);

hipError_t launch_conv_fwd(const CvArgs& a, int bf16, hipStream_t st);
hipError_t launch_conv_bwd(const CvArgs& a, int bf16, hipStream_t st);
hipError_t launch_conv_step(const CvStepArgs& a, int bf16, hipStream_t st);

hipError_t launch_norm_fwd(const NmArgs& a, int bf16, hipStream_t st);
hipError_t launch_norm_bwd(const NmArgs& a, int bf16, hipStream_t st);

}  // namespace pdscan
