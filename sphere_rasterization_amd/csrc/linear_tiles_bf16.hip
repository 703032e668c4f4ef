// Products of any size in bf16: a file for each type, so that they compile side by side.
#include "linear_tiles_kernels.h"

int launch_product_bf16(const ProductArgs &a, bool qt, bool pt, int out, hipStream_t stream) {
  return product<bf16_t>(a, qt, pt, out, stream);
}
