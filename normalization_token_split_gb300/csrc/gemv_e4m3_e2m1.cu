// gemv_e4m3_e2m1.cu -- products of e4m3 rows with e2m1 weights.
#include "gemv_kernel.cuh"

namespace nts {

template GemvKernel pick_gemv<true, false>(int group, int nt);

}  // namespace nts
