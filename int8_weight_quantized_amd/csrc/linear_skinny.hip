// linear_skinny.hip -- the skinny GEMM with an epilogue: qw_w8a16_linear and
// qw_w8a8_linear for a few activation rows, qw_w8a16_experts for a few a expert.
#include "gemm_skinny_kernel.h"

namespace qw {
namespace {

template <int RT, int MT, int KSPLIT, bool A8, int EPI, bool GRP, int RW = 1, int PART = kWhole, bool F32 = false>
hipError_t launch_cfg(const LinearArgs &a, const Experts &ex, hipStream_t stream, void *sums = nullptr, int parts = 1)
{
    constexpr int kCols = RW * (EPI == kGated ? 8 * RT : 16 * RT);
    const int64_t columns = EPI == kGated ? a.n / 2 : a.n;
    const int64_t tiles_n = (columns + kCols - 1) / kCols;
    const int64_t tiles_m = GRP ? a.m / (16 * MT) + ex.count + 1 : (a.m + 16 * MT - 1) / (16 * MT);
    if (tiles_m > 65535)
        return hipErrorInvalidConfiguration;
    const dim3 grid((unsigned)tiles_n, (unsigned)tiles_m, PART == kParts ? (unsigned)parts : 1u);
    hipLaunchKernelGGL((skinny_gemm_kernel<RT, MT, KSPLIT, A8, false, EPI, GRP, RW, PART, F32>), grid, dim3(RW * KSPLIT * kWave), 0,
                       stream, a.x, a.sx, a.q, a.scales, (const int8_t *)nullptr, OutlierList{nullptr, nullptr, 0}, a.y, (int)a.m,
                       (int)a.n, (int)a.k, a.ep, ex, sums, parts);
    return hipGetLastError();
}

// As for the plain products: k is split until the grid holds about
// kSkinnyTargetWaves waves, within the largest split of each variant.
template <int RT, int MT, bool A8, int EPI, bool GRP, bool F32 = false>
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
        return launch_cfg<RT, MT, 1, A8, EPI, GRP, 1, kWhole, F32>(a, ex, stream);
    case 2:
        return launch_cfg<RT, MT, 2, A8, EPI, GRP, 1, kWhole, F32>(a, ex, stream);
    case 4:
        return launch_cfg<RT, MT, 4, A8, EPI, GRP, 1, kWhole, F32>(a, ex, stream);
    case 8:
        if constexpr (kMaxSplit >= 8)
            return launch_cfg<RT, MT, 8, A8, EPI, GRP, 1, kWhole, F32>(a, ex, stream);
        break;
    default:
        if constexpr (kMaxSplit >= 16)
            return launch_cfg<RT, MT, 16, A8, EPI, GRP, 1, kWhole, F32>(a, ex, stream);
        break;
    }
    return hipErrorInvalidValue; // not reached: ksplit <= kMaxSplit
}

// One pass by workgroups of eight waves, four row blocks wide, that share the
// activations; returns whether it launched.  Four rows are as fast without.
//
// 64 weight rows a workgroup (one tile a wave) where they give more than half of
// the CUs one (4096 deep, 16 / 32 rows: n = 8704 13 / 16 us, one row block 18 / 29;
// 8192 13 / 16 and 13 / 17, and 8 rows 13 and 11), as long as two fit a CU's LDS, so
// with one tile of activations, or 128 would be too few: 32 rows, n = 16384 / 27392
// / 65024 18 / 33 / 67, with 128 weight rows 26 / 29 / 61; 16 rows 15 / 25 / 46 and
// 22 / 25 / 53.
//
// 128 weight rows (the gate and its partner are two tiles) where they give three
// quarters of the CUs one, or with many bytes of activations more than half:
// gated, 4096 deep, n = 17408, 8 / 16 / 32 rows 21 / 21 / 25, one row block 20 / 24 /
// 33, W8A8 18 / 18 / 20 and 17 / 19 / 25.  In several rounds with many bytes too:
// gated 57344 x 8192 92 / 93 / 103 and 86 / 97 / 116, W8A8 88 / 89 / 93 and 86 / 87 / 93.
template <int MT, bool A8, int EPI>
bool launch_shared(const LinearArgs &a, hipStream_t stream, hipError_t &result)
{
    // (its loads ahead count past k in 32 bits, and its grid of up to 8 n threads
    // has to stay below 2^32)
    if (a.m <= 4 || a.m > 16 * MT || a.k > (1 << 30) || a.n > (1 << 28))
        return false;
    const Experts none = {};
    const int64_t cus = device_cu_count(), wide = (a.n + 127) / 128, narrow = (a.n + 63) / 64;
    if constexpr (EPI != kGated) {
        if (2 * narrow > cus && (MT == 1 || 4 * wide < 3 * cus)) {
            result = launch_cfg<1, MT, 2, A8, EPI, false, 4>(a, none, stream);
            return true;
        }
    }
    if constexpr (EPI == kGated || MT > 1) {
        const bool many = !A8 && a.m > 8;
        if ((EPI == kGated && (many || MT > 1) ? 2 * wide > cus : 4 * wide >= 3 * cus) && (wide <= cus || many)) {
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

// Two launches: the parts' sums, and these joined with the epilogue.
template <int RT, int MT, bool A8, int EPI>
hipError_t launch_parts(const LinearArgs &a, int parts, void *sums, hipStream_t stream)
{
    const Experts none = {};
    const hipError_t e = launch_cfg<RT, MT, 2, A8, EPI, false, 4, kParts>(a, none, stream, sums, parts);
    return e != hipSuccess ? e : launch_cfg<RT, MT, 1, A8, EPI, false, 4, kJoin>(a, none, stream, sums, parts);
}

template <bool A8>
hipError_t launch_parts_rows(const LinearArgs &a, int parts, void *sums, hipStream_t stream)
{
    const bool two = skinny_rows_per_pass(a.m, a.k) == 32;
    if (a.gated)
        return two ? launch_parts<2, 2, A8, kGated>(a, parts, sums, stream) : launch_parts<2, 1, A8, kGated>(a, parts, sums, stream);
    return two ? launch_parts<1, 2, A8, kLinear>(a, parts, sums, stream) : launch_parts<1, 1, A8, kLinear>(a, parts, sums, stream);
}

} // namespace

int64_t skinny_parts_bytes(int64_t m, int64_t n, int64_t k, bool gated, int parts)
{
    const int64_t wide = gated ? 128 : 64, rows = skinny_rows_per_pass(m, k);
    return parts * ((n + wide - 1) / wide * wide) * ((m + rows - 1) / rows * rows) * 4;
}

hipError_t launch_skinny_parts(int parts, const LinearArgs &a, void *workspace, hipStream_t stream)
{
    return a.sx ? launch_parts_rows<true>(a, parts, workspace, stream) : launch_parts_rows<false>(a, parts, workspace, stream);
}

hipError_t launch_skinny_linear(const LinearArgs &a, hipStream_t stream)
{
    if (a.sx)
        return a.gated ? launch_rows<true, kGated>(a, stream) : launch_rows<true, kLinear>(a, stream);
    return a.gated ? launch_rows<false, kGated>(a, stream) : launch_rows<false, kLinear>(a, stream);
}

hipError_t launch_skinny_experts(const LinearArgs &a, const Experts &ex, bool f32, hipStream_t stream)
{
    const int64_t row_tiles = a.m < ex.count ? a.m : ex.count; // (about as many have rows)
    if (f32)
        return a.gated ? launch_split<2, 1, false, kGated, true, true>(a, ex, row_tiles, stream)
                       : launch_split<2, 1, false, kLinear, true, true>(a, ex, row_tiles, stream);
    return a.gated ? launch_split<2, 1, false, kGated, true>(a, ex, row_tiles, stream)
                   : launch_split<2, 1, false, kLinear, true>(a, ex, row_tiles, stream);
}

} // namespace qw
