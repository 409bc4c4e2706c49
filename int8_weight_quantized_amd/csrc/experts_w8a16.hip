// experts_w8a16.hip -- the MFMA GEMMs of qw_w8a16_experts.
#include "linear_mfma.h"

namespace qw {

hipError_t launch_mfma_experts(int tile, const LinearArgs &a, const Experts &ex, hipStream_t stream)
{
    return launch_linear_tiles<false, true>(tile, a, ex, stream);
}

} // namespace qw
