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

int64_t mfma_split_bytes(int64_t m, int64_t n, int splits)
{
    // (a gated product's tiles hold as many rows of the weight)
    const int64_t tiles = ((m + pp::kBM - 1) / pp::kBM) * ((n + pp::kBN - 1) / pp::kBN);
    return tiles * splits * pp::kBM * pp::kBN * 4;
}

hipError_t launch_mfma_split(int splits, const LinearArgs &a, void *workspace, hipStream_t stream)
{
    return launch_split<false>(splits, a, workspace, stream);
}

} // namespace qw
