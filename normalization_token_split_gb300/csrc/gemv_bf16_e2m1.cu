// gemv_bf16_e2m1.cu -- products of bf16 rows with e2m1 weights.
#include "gemv_kernel.cuh"

namespace nts {

template GemvKernel pick_gemv<false, false>(int group, int nt);

}  // namespace nts
