// Products of any size in fp32: a file for each type, so that they compile side by side.
#include "linear_tiles_kernels.h"

int launch_product_f32(const ProductArgs &a, bool qt, bool pt, int out, hipStream_t stream) {
  return product<float>(a, qt, pt, out, stream);
}
