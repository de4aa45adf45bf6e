// spec_dropout_any.cu -- the interpreting kernels of the programs with dropout
// (compiled apart from the others to keep builds parallel).
#include "programs.cuh"

namespace ge {

const void* const kDynamicDrop[2][2] = {
    {reinterpret_cast<const void*>(&fused_gemm_epilogue_kernel<1, DynamicDropProgram>),
     reinterpret_cast<const void*>(&fused_gemm_epilogue_kernel<2, DynamicDropProgram>)},
    {reinterpret_cast<const void*>(&fused_gemm_epilogue_kernel<1, DynamicDropProgram, 1>),
     reinterpret_cast<const void*>(&fused_gemm_epilogue_kernel<2, DynamicDropProgram, 1>)}};

}  // namespace ge
