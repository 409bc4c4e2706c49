// linear_w8a16.hip -- the MFMA GEMMs of qw_w8a16_linear.
#include "linear_mfma.h"

namespace qw {

// A gated product's weight tile spans both halves of the weight, in 32-bit
// offsets from its first row.
bool mfma_linear_supported(int64_t n, int64_t k, bool gated)
{
    return k <= kMfmaMaxK && (!gated || n * k < int64_t(1) << 32);
}

hipError_t launch_mfma_linear(int tile, const LinearArgs &a, hipStream_t stream)
{
    return launch_linear_tiles<false, false>(tile, a, Experts{}, stream);
}

} // namespace qw
