// linear_w8a8.hip -- the MFMA GEMMs of qw_w8a8_linear.
#include "linear_mfma.h"

namespace qw {

hipError_t launch_mfma_linear_a8(int tile, const LinearArgs &a, hipStream_t stream)
{
    return launch_linear_tiles<true, false>(tile, a, Experts{}, stream);
}

hipError_t launch_mfma_split_a8(int splits, const LinearArgs &a, void *workspace, hipStream_t stream)
{
    return launch_split<true>(splits, a, workspace, stream);
}

} // namespace qw
