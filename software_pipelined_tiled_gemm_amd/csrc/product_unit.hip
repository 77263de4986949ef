// Instantiations of the tiled kernel for one element type, product and copy mode:
// build.py compiles this file once per combination, with -DSPG_ET, -DSPG_PRODUCT and
// -DSPG_REG.
#define SPG_DEFINE_PRODUCT
#include "product_launch.hpp"

template void spg::launch_product<SPG_ET, SPG_PRODUCT, (SPG_REG != 0)>(int, const spg::ProductArgs&, dim3, hipStream_t);
