// spec_heads.cu -- the interpreting kernels of the programs with HEAD_RMS or
// ROTARY (the norm and rotary positions of a projection's heads), compiled
// apart from the others to keep builds parallel.
#include "programs.cuh"

namespace ge {

const void* const kDynamicHeads[2][3] = {
    {reinterpret_cast<const void*>(&fused_gemm_epilogue_kernel<1, DynamicHeadProgram>),
     reinterpret_cast<const void*>(&fused_gemm_epilogue_kernel<2, DynamicHeadProgram>),
     split_kernel_for<DynamicHeadProgram, 0>()},
    {reinterpret_cast<const void*>(&fused_gemm_epilogue_kernel<1, DynamicHeadProgram, 1>),
     reinterpret_cast<const void*>(&fused_gemm_epilogue_kernel<2, DynamicHeadProgram, 1>),
     split_kernel_for<DynamicHeadProgram, 1>()}};

}  // namespace ge
