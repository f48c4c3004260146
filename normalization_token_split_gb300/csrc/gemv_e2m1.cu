// gemv_e2m1.cu -- products with e2m1 weights.
#include "gemv_kernel.cuh"

namespace nts {

template GemvKernel pick_gemv<false>(int group, int nt);

}  // namespace nts
