// spec_rotary.cu -- static kernels of the projections with rotary positions
// (compiled apart from the others to keep builds parallel).
#include "programs.cuh"

namespace ge {

const KernelSpec kSpecsRotary[] = {
    make_spec<ProgRotary>("rotary"),
    make_spec<ProgBiasRotary>("bias_rotary"),
    make_spec<ProgRmsRotary>("row_scale_rotary"),
};
const int kNumSpecsRotary = sizeof(kSpecsRotary) / sizeof(kSpecsRotary[0]);

}  // namespace ge
