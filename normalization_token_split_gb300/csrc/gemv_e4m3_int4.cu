// gemv_e4m3_int4.cu -- products of e4m3 rows with int4 weights.
#include "gemv_kernel.cuh"

namespace nts {

template GemvKernel pick_gemv<true, true>(int group, int nt);

}  // namespace nts
