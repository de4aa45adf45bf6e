// spec_head_norm.cu -- static kernels of the projections with the norm of each head and rotary positions
// (compiled apart from the others to keep builds parallel).
#include "programs.cuh"

namespace ge {

const KernelSpec kSpecsHeadNorm[] = {
    make_spec<ProgNormRotary>("head_norm_rotary"),
    make_spec<ProgBiasNormRotary>("bias_head_norm_rotary"),
    make_spec<ProgRmsNormRotary>("row_scale_head_norm_rotary"),
};
const int kNumSpecsHeadNorm = sizeof(kSpecsHeadNorm) / sizeof(kSpecsHeadNorm[0]);

}  // namespace ge
