// experts_w8a16.hip -- the MFMA GEMMs of qw_w8a16_experts, with outputs in fp16 or
// fp32.  The latter for a sum over a token's entries that rounds once: entries
// rounded to fp16 first were its largest error, and infinite beyond 65504.  Us,
// product / product and sum, fp16 and fp32, 64 experts: 32 tokens x 8, 2048 by 1024
// 28 / 34 and 28 / 34; 1024 x 8 67 / 79 and 75 / 88; 4096 x 8, 4096 by 1536 476 /
// 532 and 569 / 679 (twice the bytes between the two).
#include "linear_mfma.h"

namespace qw {

hipError_t launch_mfma_experts(int tile, const LinearArgs &a, const Experts &ex, bool f32, hipStream_t stream)
{
    return f32 ? launch_linear_tiles<false, true, true>(tile, a, ex, stream) : launch_linear_tiles<false, true>(tile, a, ex, stream);
}

} // namespace qw
