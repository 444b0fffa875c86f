// What every kernel of the int8 product does with a sum: one rounding to FP32 a step
// and none of them joined, so that all kernels give the same bits.
#pragma once

#include "common.cuh"

namespace nvm {

NVM_DEV float int8_scaled(int sum, float xs, float ws) { return __fmul_rn(__fmul_rn((float)sum, xs), ws); }
NVM_DEV float int8_biased(float v, float bias) { return __fadd_rn(v, bias); }

}  // namespace nvm
