// Instantiations of the tiled kernel for one element type, product and copy mode:
// build.py compiles this file once per combination, with -DSPG_ET, -DSPG_PRODUCT and
// -DSPG_REG (products 2 and 3, the input gradients, also as one launch with the weights').
#define SPG_DEFINE_PRODUCT
#include "product_launch.hpp"

template void spg::launch_product<SPG_ET, SPG_PRODUCT, (SPG_REG != 0)>(int, const spg::ProductArgs&, dim3, hipStream_t);
#if SPG_PRODUCT == 2 || SPG_PRODUCT == 3
template void spg::launch_gradients<SPG_ET, SPG_PRODUCT, (SPG_REG != 0)>(int, const spg::ProductArgs&,
                                                                       const spg::ProductArgs&, int, dim3, hipStream_t);
#endif
