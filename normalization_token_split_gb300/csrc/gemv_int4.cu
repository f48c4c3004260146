// gemv_int4.cu -- products with int4 weights.
#include "gemv_kernel.cuh"
#include "gemv_tile.cuh"

namespace nts {

template GemvKernel pick_gemv<true>(int group, int nt);
template GemvTileKernel pick_gemv_tile<true>(int group, bool e4m3, size_t* smem);
template int read_and_clear_gemv_unit<true>(unsigned* out);

}  // namespace nts
