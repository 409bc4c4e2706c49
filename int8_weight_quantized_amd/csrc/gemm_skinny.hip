// gemm_skinny.hip -- launch configuration of the skinny GEMM
// (gemm_skinny_kernel.h) for the plain products.
#include "gemm_skinny_kernel.h"

namespace qw {
namespace {

template <int RT, int MT, int KSPLIT, bool A8>
hipError_t launch_cfg(const void *x, const uint16_t *sx, const int8_t *q, const uint16_t *scales,
                      const int8_t *zeros, OutlierList ol, uint16_t *y, int64_t m, int64_t n, int64_t k,
                      hipStream_t stream)
{
    const dim3 grid((unsigned)((n + 16 * RT - 1) / (16 * RT)), (unsigned)((m + 16 * MT - 1) / (16 * MT)));
    if constexpr (!A8) {
        if (zeros != nullptr) {
            hipLaunchKernelGGL((skinny_gemm_kernel<RT, MT, KSPLIT, false, true>), grid, dim3(KSPLIT * kWave), 0,
                               stream, x, sx, q, scales, zeros, ol, y, (int)m, (int)n, (int)k, Epilogue{}, Experts{}, nullptr, 1);
            return hipGetLastError();
        }
    }
    hipLaunchKernelGGL((skinny_gemm_kernel<RT, MT, KSPLIT, A8>), grid, dim3(KSPLIT * kWave), 0, stream,
                       x, sx, q, scales, zeros, ol, y, (int)m, (int)n, (int)k, Epilogue{}, Experts{}, nullptr, 1);
    return hipGetLastError();
}

// Largest k split per kernel variant: a workgroup of 16 waves leaves each
// lane 128 registers, which the int8 kernel and the two-tile fp16 kernel
// exceed (they spilled); they stop at 8 waves.  Four weight tiles with two
// activation tiles stop at 4: at 8 they spilled, and their staging slices
// would fill most of the LDS.
template <int RT, int MT, bool A8>
constexpr int max_split()
{
    return RT == 4 ? 4 : (A8 || MT > 1) ? 8 : 16;
}

template <int RT, int MT, bool A8>
hipError_t launch_mt(const void *x, const uint16_t *sx, const int8_t *q, const uint16_t *scales,
                     const int8_t *zeros, OutlierList ol, uint16_t *y, int64_t m, int64_t n, int64_t k,
                     hipStream_t stream)
{
    // split k until the grid holds about kSkinnyTargetWaves waves, keeping
    // at least one 64-wide step per wave
    const int64_t tiles = ((n + 16 * RT - 1) / (16 * RT)) * ((m + 16 * MT - 1) / (16 * MT));
    const int64_t steps = (k + 63) / 64;
    constexpr int kMaxSplit = max_split<RT, MT, A8>();
    int ksplit = 1;
    while (ksplit < kMaxSplit && tiles * ksplit < kSkinnyTargetWaves && steps >= 2 * ksplit)
        ksplit *= 2;
    if (ksplit == 1)
        return launch_cfg<RT, MT, 1, A8>(x, sx, q, scales, zeros, ol, y, m, n, k, stream);
    if (ksplit == 2)
        return launch_cfg<RT, MT, 2, A8>(x, sx, q, scales, zeros, ol, y, m, n, k, stream);
    if (ksplit == 4)
        return launch_cfg<RT, MT, 4, A8>(x, sx, q, scales, zeros, ol, y, m, n, k, stream);
    if constexpr (kMaxSplit >= 8)
        if (ksplit == 8)
            return launch_cfg<RT, MT, 8, A8>(x, sx, q, scales, zeros, ol, y, m, n, k, stream);
    if constexpr (kMaxSplit >= 16)
        if (ksplit == 16)
            return launch_cfg<RT, MT, 16, A8>(x, sx, q, scales, zeros, ol, y, m, n, k, stream);
    return hipErrorInvalidValue; // not reached: ksplit <= kMaxSplit
}

// Activation tiles per wave from m and k.  For 17..32 rows with k >= 2048,
// two tiles per wave take one pass over the weights instead of two
// (measured 10% faster at k = 4096, n = 4608 and 27392).  Otherwise one
// tile per wave and one pass per 16 rows: the passes run side by side and
// their repeated weight reads hit in cache, so more, shorter waves win
// (four tiles per wave measured 7-10% slower than four passes at 48 and 64
// rows; two tiles 2-5% slower at k = 1024, where the k split then has too
// few steps to fill the chip).
template <int RT, bool A8>
hipError_t launch_rt(const void *x, const uint16_t *sx, const int8_t *q, const uint16_t *scales,
                     const int8_t *zeros, OutlierList ol, uint16_t *y, int64_t m, int64_t n, int64_t k,
                     hipStream_t stream)
{
    if (skinny_rows_per_pass(m, k) == 32)
        return launch_mt<RT, 2, A8>(x, sx, q, scales, zeros, ol, y, m, n, k, stream);
    return launch_mt<RT, 1, A8>(x, sx, q, scales, zeros, ol, y, m, n, k, stream);
}

} // namespace

int skinny_rows_per_pass(int64_t m, int64_t k)
{
    return (m > 16 && m <= 32 && k >= 2048) ? 32 : 16;
}

namespace {

// Weight tiles per workgroup.  Two 16-row tiles share each activation
// operand load, but each workgroup holds all the k-split waves of its tiles,
// so the grid has one workgroup per RT x 16 weight rows (per pass).  Where
// one tile per workgroup still fits the grid on the chip in one round, the
// doubled workgroup count keeps twice the CUs streaming: at n = 4096, m = 8
// it measured 24% faster at k = 1024 and 12% at k = 4096 (128 two-tile
// workgroups leave half the CUs idle).  At n = 4608 (288 one-tile
// workgroups, a second round) two tiles stay faster.
template <bool A8>
hipError_t launch_auto_rt(const void *x, const uint16_t *sx, const int8_t *q, const uint16_t *scales,
                          const int8_t *zeros, OutlierList ol, uint16_t *y, int64_t m, int64_t n, int64_t k,
                          hipStream_t stream)
{
    const int64_t rows = skinny_rows_per_pass(m, k);
    const int64_t one_tile_grid = ((n + 15) / 16) * ((m + rows - 1) / rows);
    if (one_tile_grid <= device_cu_count())
        return launch_rt<1, A8>(x, sx, q, scales, zeros, ol, y, m, n, k, stream);
    // Two activation tiles read 32 activation rows per k step, once per
    // workgroup: four weight tiles halve those reads where the grid stays
    // large (n >= 12288 at one pass).  Measured at k = 4096: 49.4 -> 37.0 us
    // at m = 32 and n = 27392, 31.8 -> 26.7 us at m = 32 and n = 13824,
    // W8A8 m = 32, n = 27392 33.9 -> 28.1 us.  With one activation tile
    // four tiles measured slower on some of these grids.
    if (rows == 32 && one_tile_grid >= 3 * (int64_t)device_cu_count())
        return launch_mt<4, 2, A8>(x, sx, q, scales, zeros, ol, y, m, n, k, stream);
    return launch_rt<2, A8>(x, sx, q, scales, zeros, ol, y, m, n, k, stream);
}

} // namespace

hipError_t launch_skinny_gemm(const uint16_t *x, const int8_t *q, const uint16_t *scales,
                              const int8_t *zeros, OutlierList ol, uint16_t *y, int64_t m, int64_t n, int64_t k, hipStream_t stream)
{
    // one, two or four 16-row weight tiles per wave (more tiles reuse the
    // activation operand; four only with two activation tiles on a large
    // grid, elsewhere they measured slower: fewer waves, longer dependent
    // MFMA chains)
    return launch_auto_rt<false>(x, nullptr, q, scales, zeros, ol, y, m, n, k, stream);
}

hipError_t launch_w8a8_skinny(const int8_t *qx, const uint16_t *sx, const int8_t *q, const uint16_t *scales,
                              uint16_t *y, int64_t m, int64_t n, int64_t k, hipStream_t stream)
{
    return launch_auto_rt<true>(qx, sx, q, scales, nullptr, OutlierList{nullptr, nullptr, 0}, y, m, n, k, stream);
}

} // namespace qw
