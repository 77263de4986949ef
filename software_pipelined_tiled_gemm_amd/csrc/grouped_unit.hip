// Instantiations of the tiled products by group for one element type, product and copy mode:
// with rows of X
// in order or by their source: build.py compiles this file once per combination, with -DSPG_ET, -DSPG_PRODUCT,
// -DSPG_REG and -DSPG_GATHER.
#define SPG_DEFINE_GROUPED
#include "grouped_launch.hpp"

template void spg::launch_grouped<SPG_ET, SPG_PRODUCT, (SPG_REG != 0), (SPG_GATHER != 0)>(int, const spg::ProductArgs&,
                                                                                        const spg::GroupArgs&, int, dim3, hipStream_t);
#if SPG_PRODUCT >= 2 && SPG_PRODUCT <= 5 && !SPG_GATHER
template void spg::launch_group_gradients<SPG_ET, SPG_PRODUCT, (SPG_REG != 0)>(int, const spg::ProductArgs&, const spg::ProductArgs&,
                                                                             const spg::GroupArgs&, int, int, dim3, hipStream_t);
#endif
