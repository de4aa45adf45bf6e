// spec_dropout.cu -- static kernels of the programs with dropout (compiled apart
// from the others to keep builds parallel).
#include "programs.cuh"

namespace ge {

const KernelSpec kSpecsDropout[] = {
    make_spec<ProgDropResidual>("dropout_residual"),
    make_spec<ProgBiasDropResidual>("bias_dropout_residual"),
    make_spec<ProgBiasGeluDrop>("bias_gelu_dropout"),
    make_spec<ProgDropGeluGradColSum>("dropout_gelu_grad_col_sum"),
    make_spec<ProgSwiGLUDrop>("swiglu_dropout"),
    make_spec<ProgDropDSwiGLU>("dropout_dswiglu"),
};
const int kNumSpecsDropout = sizeof(kSpecsDropout) / sizeof(kSpecsDropout[0]);

}  // namespace ge
