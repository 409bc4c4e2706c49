// linear_skinny.hip -- the skinny GEMM with an epilogue: qw_w8a16_linear and
// qw_w8a8_linear for a few activation rows, qw_w8a16_experts for a few a expert.
#include "gemm_skinny_kernel.h"

namespace qw {
namespace {

template <int RT, int MT, int KSPLIT, bool A8, int EPI, bool GRP, int RW = 1>
hipError_t launch_cfg(const LinearArgs &a, const Experts &ex, hipStream_t stream)
{
    constexpr int kCols = RW * (EPI == kGated ? 8 * RT : 16 * RT);
    const int64_t columns = EPI == kGated ? a.n / 2 : a.n;
    const int64_t tiles_n = (columns + kCols - 1) / kCols;
    const int64_t tiles_m = GRP ? a.m / (16 * MT) + ex.count + 1 : (a.m + 16 * MT - 1) / (16 * MT);
    if (tiles_m > 65535)
        return hipErrorInvalidConfiguration;
    const dim3 grid((unsigned)tiles_n, (unsigned)tiles_m);
    hipLaunchKernelGGL((skinny_gemm_kernel<RT, MT, KSPLIT, A8, false, EPI, GRP, RW>), grid, dim3(RW * KSPLIT * kWave), 0,
                       stream, a.x, a.sx, a.q, a.scales, (const int8_t *)nullptr, OutlierList{nullptr, nullptr, 0}, a.y, (int)a.m,
                       (int)a.n, (int)a.k, a.ep, ex);
    return hipGetLastError();
}

// As for the plain products: k is split until the grid holds about
// kSkinnyTargetWaves waves, within the largest split of each variant.
template <int RT, int MT, bool A8, int EPI, bool GRP>
hipError_t launch_split(const LinearArgs &a, const Experts &ex, int64_t row_tiles, hipStream_t stream)
{
    constexpr int kMaxSplit = RT == 4 ? 4 : (A8 || MT > 1 || GRP) ? 8 : 16;
    const int64_t tiles = (a.n + 16 * RT - 1) / (16 * RT) * row_tiles;
    const int64_t steps = (a.k + 63) / 64;
    int ksplit = 1;
    while (ksplit < kMaxSplit && tiles * ksplit < kSkinnyTargetWaves && steps >= 2 * ksplit)
        ksplit *= 2;
    switch (ksplit) {
    case 1:
        return launch_cfg<RT, MT, 1, A8, EPI, GRP>(a, ex, stream);
    case 2:
        return launch_cfg<RT, MT, 2, A8, EPI, GRP>(a, ex, stream);
    case 4:
        return launch_cfg<RT, MT, 4, A8, EPI, GRP>(a, ex, stream);
    case 8:
        if constexpr (kMaxSplit >= 8)
            return launch_cfg<RT, MT, 8, A8, EPI, GRP>(a, ex, stream);
        break;
    default:
        if constexpr (kMaxSplit >= 16)
            return launch_cfg<RT, MT, 16, A8, EPI, GRP>(a, ex, stream);
        break;
    }
    return hipErrorInvalidValue; // not reached: ksplit <= kMaxSplit
}

// One pass by workgroups of eight waves, four row blocks wide, that share the
// activations, where their grid gives three quarters of the CUs one; returns
// whether it launched.  With fewer the workgroups of one row block and more parts
// of k have more loads in flight (16 rows: 4608 x 4096 11 us and 13 here, gated
// 16384 x 4096 18 and 22), and four rows are as fast there.
//
// 64 weight rows a workgroup (one tile a wave) where two of them fit a CU's LDS,
// so with one tile of activations, or where 128 would be too few: 32 rows, n =
// 16384 / 27392 / 65024 18 / 33 / 67 us, with 128 weight rows 26 / 29 / 61; 16 rows
// 15 / 25 / 46 and 22 / 25 / 53.  The gate and its partner are two tiles.  A grid
// of 128 rows and several rounds gains where the activations are many bytes: gated
// 57344 x 8192, 8 / 16 / 32 rows 92 / 93 / 103, one row block 86 / 97 / 116; W8A8
// 88 / 89 / 93 and 86 / 87 / 93.
template <int MT, bool A8, int EPI>
bool launch_shared(const LinearArgs &a, hipStream_t stream, hipError_t &result)
{
    if (a.m <= 4 || a.m > 16 * MT || a.k > (1 << 30)) // (its loads ahead count past k in 32 bits)
        return false;
    const Experts none = {};
    const int64_t cus = device_cu_count(), least = 3 * cus / 4;
    const int64_t wide = (a.n + 127) / 128, narrow = (a.n + 63) / 64;
    if constexpr (EPI != kGated) {
        if (narrow >= least && (MT == 1 || wide < least)) {
            result = launch_cfg<1, MT, 2, A8, EPI, false, 4>(a, none, stream);
            return true;
        }
    }
    if constexpr (EPI == kGated || MT > 1) {
        if (wide >= least && (wide <= cus || (!A8 && a.m > 8))) {
            result = launch_cfg<2, MT, 2, A8, EPI, false, 4>(a, none, stream);
            return true;
        }
    }
    return false;
}

// Weight tiles a workgroup as for the plain products, but at least the pair
// that a gated product takes.
template <bool A8, int EPI>
hipError_t launch_rows(const LinearArgs &a, hipStream_t stream)
{
    const int64_t rows = skinny_rows_per_pass(a.m, a.k);
    const int64_t passes = (a.m + rows - 1) / rows;
    const int64_t one_tile_grid = ((a.n + 15) / 16) * passes;
    const Experts none = {};
    hipError_t result = hipSuccess;
    if (rows == 32 ? launch_shared<2, A8, EPI>(a, stream, result) : launch_shared<1, A8, EPI>(a, stream, result))
        return result;
    if (rows == 32 && one_tile_grid >= 3 * (int64_t)device_cu_count())
        return launch_split<4, 2, A8, EPI, false>(a, none, passes, stream);
    if constexpr (EPI != kGated)
        if (one_tile_grid <= device_cu_count())
            return rows == 32 ? launch_split<1, 2, A8, EPI, false>(a, none, passes, stream)
                              : launch_split<1, 1, A8, EPI, false>(a, none, passes, stream);
    return rows == 32 ? launch_split<2, 2, A8, EPI, false>(a, none, passes, stream)
                      : launch_split<2, 1, A8, EPI, false>(a, none, passes, stream);
}

} // namespace

hipError_t launch_skinny_linear(const LinearArgs &a, hipStream_t stream)
{
    if (a.sx)
        return a.gated ? launch_rows<true, kGated>(a, stream) : launch_rows<true, kLinear>(a, stream);
    return a.gated ? launch_rows<false, kGated>(a, stream) : launch_rows<false, kLinear>(a, stream);
}

hipError_t launch_skinny_experts(const LinearArgs &a, const Experts &ex, hipStream_t stream)
{
    const int64_t row_tiles = a.m < ex.count ? a.m : ex.count; // (about as many have rows)
    return a.gated ? launch_split<2, 1, false, kGated, true>(a, ex, row_tiles, stream)
                   : launch_split<2, 1, false, kLinear, true>(a, ex, row_tiles, stream);
}

} // namespace qw
