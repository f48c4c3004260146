// gemv_e2m1.cu -- products with e2m1 weights.
#include "gemv_kernel.cuh"
#include "gemv_tile.cuh"

namespace nts {

template GemvKernel pick_gemv<false>(int group, int nt);
template GemvTileKernel pick_gemv_tile<false>(int group, bool e4m3, size_t* smem);
template int read_and_clear_gemv_unit<false>(unsigned* out);

}  // namespace nts
