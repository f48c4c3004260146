// gemv_int4.cu -- products with int4 weights.
#include "gemv_kernel.cuh"

namespace nts {

template GemvKernel pick_gemv<true>(int group, int nt);

}  // namespace nts
