// Instantiations of the tiled products by group for one element type, product and copy mode:
// build.py compiles this file once per combination, with -DSPG_ET, -DSPG_PRODUCT and -DSPG_REG.
#define SPG_DEFINE_GROUPED
#include "grouped_launch.hpp"

template void spg::launch_grouped<SPG_ET, SPG_PRODUCT, (SPG_REG != 0)>(int, const spg::ProductArgs&, const spg::GroupArgs&, int,
                                                                     dim3, hipStream_t);
