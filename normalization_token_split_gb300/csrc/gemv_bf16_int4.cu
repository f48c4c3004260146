// gemv_bf16_int4.cu -- products of bf16 rows with int4 weights.
#include "gemv_kernel.cuh"

namespace nts {

template GemvKernel pick_gemv<false, true>(int group, int nt);

}  // namespace nts
