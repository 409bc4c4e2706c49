// gemm_mfma.hip -- launch and tile choice of the LDS-tiled MFMA GEMMs
// (gemm_mfma_kernels.h) for the plain products.
#include "gemm_mfma_kernels.h"

#include <algorithm>
#include <atomic>
#include <cmath>

namespace qw {
namespace {

template <int BN, int BM, bool A8>
int64_t slots_per_cu();

// Weight-tile columns per group of the tile order.  An XCD holds about r =
// min(its share of the grid, its resident workgroups) tiles at once; as an
// a x (r / a) block of weight x activation tiles they fetch a * BN weight
// rows and (r / a) * BM activation rows per k step, least at
// a = sqrt(r * BM * e / BN) with e the bytes of one activation element.
// With few activation tiles (prefill: 4) the block needs at least
// r / tiles_m columns; a group that wide also makes consecutive workgroups
// share an activation tile, which measured 3-7% faster there than narrower
// groups.  Measured on MI355X against one column per group: 5-14% faster
// for the W8A8 tiles and 1-7% for the fp16 tiles with 256 weight rows; the
// fp16 tiles with 128 weight rows ran 1-5% slower grouped, at either width,
// and keep one.
template <int BN, int BM, bool A8>
int group_width(int64_t blocks, int64_t tiles_m, int64_t tiles_n)
{
    if constexpr (!A8 && BN == 128)
        return 1;
    const int64_t share = (blocks + 7) / 8;
    const int64_t resident = slots_per_cu<BN, BM, A8>() * (int64_t)device_cu_count() / 8;
    const double r = (double)std::max<int64_t>(1, std::min(share, resident));
    int64_t a = std::llround(std::sqrt(r * BM * (A8 ? 1 : 2) / BN));
    a = std::max<int64_t>(a, ((int64_t)r + tiles_m - 1) / tiles_m);
    return (int)std::max<int64_t>(1, std::min(a, tiles_n));
}

template <int NW, int BN, int BM, bool A8>
hipError_t launch_dma(const void *x, const uint16_t *sx, const int8_t *q, const uint16_t *scales,
                      const int8_t *zeros, OutlierList ol, uint16_t *y, int64_t m, int64_t n, int64_t k,
                      hipStream_t stream)
{
    const int64_t tiles_m = (m + BM - 1) / BM;
    const int64_t tiles_n = (n + BN - 1) / BN;
    const int64_t blocks = tiles_m * tiles_n;
    if (blocks > 0x7fffffff)
        return hipErrorInvalidConfiguration;
    const int group = group_width<BN, BM, A8>(blocks, tiles_m, tiles_n);
    if constexpr (!A8) {
        if (ol.idx != nullptr) {
            if (ol.cap > kMfmaOutlierSlots)
                return hipErrorInvalidValue;
            hipLaunchKernelGGL((mfma_gemm_dma_kernel<NW, BN, BM, false, true>), dim3((unsigned)blocks),
                               dim3(NW * kWave), 0, stream, x, sx, q, scales, zeros, ol, y, (int)m, (int)n,
                               (int)k, (int)tiles_m, (int)tiles_n, group, Epilogue{}, Experts{});
            return hipGetLastError();
        }
    }
    if (ol.idx != nullptr)
        return hipErrorInvalidValue;
    if constexpr (!A8) {
        if (zeros != nullptr) {
            hipLaunchKernelGGL((mfma_gemm_dma_kernel<NW, BN, BM, false, false, true>), dim3((unsigned)blocks),
                               dim3(NW * kWave), 0, stream, x, sx, q, scales, zeros, ol, y, (int)m, (int)n,
                               (int)k, (int)tiles_m, (int)tiles_n, group, Epilogue{}, Experts{});
            return hipGetLastError();
        }
    }
    hipLaunchKernelGGL((mfma_gemm_dma_kernel<NW, BN, BM, A8>), dim3((unsigned)blocks), dim3(NW * kWave),
                       0, stream, x, sx, q, scales, zeros, ol, y, (int)m, (int)n, (int)k, (int)tiles_m,
                       (int)tiles_n, group, Epilogue{}, Experts{});
    return hipGetLastError();
}

// Workgroups of this tile shape one CU holds at once (registers and LDS),
// queried once per device.  Host threads may race on the first query; they
// store the same value.
template <int BN, int BM, bool A8>
int64_t slots_per_cu()
{
    static std::atomic<int> cached[64];
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64)
        return 1;
    int blocks = cached[dev].load(std::memory_order_relaxed);
    if (blocks == 0) {
        if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&blocks, mfma_gemm_dma_kernel<4, BN, BM, A8>,
                                                        4 * kWave, 0) != hipSuccess || blocks < 1)
            blocks = 1;
        cached[dev].store(blocks, std::memory_order_relaxed);
    }
    return blocks;
}

template <int BN, int BM, bool A8>
bool fills(int64_t m, int64_t n)
{
    const int64_t tiles = ((n + BN - 1) / BN) * ((m + BM - 1) / BM);
    // The fp16 128 x 128 tile is counted at two workgroups per CU even where
    // its registers allow three: per-shape tuning measured it fastest at 256
    // rows (N = 27392), where counting the third slot would pass it over
    // for 128 x 64.
    int64_t per_cu = slots_per_cu<BN, BM, A8>();
    if (!A8 && BN == 128 && BM == 128 && per_cu > 2)
        per_cu = 2;
    const int64_t slots = per_cu * (int64_t)device_cu_count();
    return 4 * tiles >= 3 * slots;
}

// The ping-pong tile (fp16 activations) where its grid covers at least half
// the CUs (one workgroup per CU) and rounding m up to 256 rows costs at most
// 10% more rows than rounding it to 64 (the smallest 4-wave tile).
// Measured on MI355X against the 4-wave tiles: 10-13% faster at 512 x 4096
// x 27392, 8% at 2048 x 4096 x 4608 (144 tiles), even at 4096 x 1024 x
// 4096; 20% slower at 256 x 4096 x 27392 (107 tiles).
bool pp_fills(int64_t m, int64_t n, int64_t k)
{
    if (k > kPingPongMaxK)
        return false;
    const int64_t tiles = ((m + pp::kBM - 1) / pp::kBM) * ((n + pp::kBN - 1) / pp::kBN);
    const int64_t rows256 = (m + 255) / 256 * 256, rows64 = (m + 63) / 64 * 64;
    return 2 * tiles >= (int64_t)device_cu_count() && 10 * rows256 <= 11 * rows64;
}

// PP: the ping-pong tile may be chosen.  Calls with outlier side lists keep
// the 4-wave tiles: the ping-pong kernel's epilogue gather of the side
// lists' activation columns, one workgroup per CU with nothing to overlap
// it, measured 54% above the plain GEMM on 4096 x 1024 x 4096 (one slot)
// against 43% for the 256 x 128 tile.
template <bool A8>
int tile_choice(int64_t m, int64_t n, int64_t k, bool pp = true)
{
    if (pp && pp_fills(m, n, k))
        return 256256;
    // largest tile first (more reuse per byte staged); 256 x 64 before
    // 128 x 128 (same area, half the activation bytes per tile)
    if (fills<256, 128, A8>(m, n))
        return 256128;
    if (fills<256, 64, A8>(m, n))
        return 256064;
    // W8A8: the 128 x 128 tile holds four workgroups per CU (int8 activation
    // tiles are half the LDS), so it fills the chip only where 256 x 64
    // already does and is never the choice
    if (!A8 && fills<128, 128, A8>(m, n))
        return 128128;
    return 128064;
}

template <bool A8>
int pp_group_width(int64_t blocks, int64_t tiles_m, int64_t tiles_n)
{
    const int64_t share = (blocks + 7) / 8;
    const int64_t resident = std::max<int64_t>(1, (int64_t)device_cu_count() / 8);
    const double r = (double)std::max<int64_t>(1, std::min(share, resident));
    int64_t a = std::llround(std::sqrt(r * pp::kBM * (A8 ? 1 : 2) / pp::kBN));
    a = std::max<int64_t>(a, ((int64_t)r + tiles_m - 1) / tiles_m);
    return (int)std::max<int64_t>(1, std::min(a, tiles_n));
}

// Ping-pong launch: one 512-thread workgroup per 256 x 256 tile, one per CU
// (144 KiB of LDS).  Grouped tile order as for the 4-wave tiles, with one
// resident workgroup per CU.
template <bool A8>
hipError_t launch_pp(const void *x, const uint16_t *sx, const int8_t *q, const uint16_t *scales,
                     const int8_t *zeros, OutlierList ol, uint16_t *y, int64_t m, int64_t n, int64_t k,
                     hipStream_t stream)
{
    const int64_t tiles_m = (m + pp::kBM - 1) / pp::kBM;
    const int64_t tiles_n = (n + pp::kBN - 1) / pp::kBN;
    const int64_t blocks = tiles_m * tiles_n;
    if (blocks > 0x7fffffff || k < 1 || k > kPingPongMaxK || (ol.idx != nullptr && ol.cap > kMfmaOutlierSlots))
        return hipErrorInvalidValue;
    const int group = pp_group_width<A8>(blocks, tiles_m, tiles_n);
#define QW_PP_LAUNCH(A, O, Z)                                                                                   \
    hipLaunchKernelGGL((mfma_pp_kernel<A, O, Z>), dim3((unsigned)blocks), dim3(pp::kThreads), 0, stream, x, sx, q,  \
                       scales, zeros, ol, y, (int)m, (int)n, (int)k, (int)tiles_m, (int)tiles_n, group, Epilogue{}, Experts{}, 1, nullptr)
    if constexpr (A8) {
        if (ol.idx != nullptr || zeros != nullptr)
            return hipErrorInvalidValue;
        QW_PP_LAUNCH(true, false, false);
    } else {
        // side lists come with symmetric codes only (as in the 4-wave kernels)
        if (ol.idx != nullptr)
            QW_PP_LAUNCH(false, true, false);
        else if (zeros != nullptr)
            QW_PP_LAUNCH(false, false, true);
        else
            QW_PP_LAUNCH(false, false, false);
    }
#undef QW_PP_LAUNCH
    return hipGetLastError();
}

template <bool A8>
hipError_t launch_tiles(const void *x, const uint16_t *sx, const int8_t *q, const uint16_t *scales,
                        const int8_t *zeros, OutlierList ol, uint16_t *y, int64_t m, int64_t n, int64_t k,
                        hipStream_t stream, int forced_tile = 0)
{
    if (k > kMfmaMaxK) // the entry points route such rows elsewhere
        return hipErrorInvalidValue;
    const int tile = forced_tile != 0 ? forced_tile : tile_choice<A8>(m, n, k, ol.idx == nullptr);
    switch (tile) {
    case 256256:
        return launch_pp<A8>(x, sx, q, scales, zeros, ol, y, m, n, k, stream);
    case 256128:
        return launch_dma<4, 256, 128, A8>(x, sx, q, scales, zeros, ol, y, m, n, k, stream);
    case 256064:
        return launch_dma<4, 256, 64, A8>(x, sx, q, scales, zeros, ol, y, m, n, k, stream);
    case 128128:
        if constexpr (!A8)
            return launch_dma<4, 128, 128, A8>(x, sx, q, scales, zeros, ol, y, m, n, k, stream);
        [[fallthrough]];
    default:
        return launch_dma<4, 128, 64, A8>(x, sx, q, scales, zeros, ol, y, m, n, k, stream);
    }
}

} // namespace

int mfma_tile_group(int tile, bool a8, int64_t tiles_m, int64_t tiles_n)
{
    const int64_t blocks = tiles_m * tiles_n;
    switch (tile) {
    case 256256:
        return a8 ? pp_group_width<true>(blocks, tiles_m, tiles_n) : pp_group_width<false>(blocks, tiles_m, tiles_n);
    case 256128:
        return a8 ? group_width<256, 128, true>(blocks, tiles_m, tiles_n) : group_width<256, 128, false>(blocks, tiles_m, tiles_n);
    case 256064:
        return a8 ? group_width<256, 64, true>(blocks, tiles_m, tiles_n) : group_width<256, 64, false>(blocks, tiles_m, tiles_n);
    case 128128:
        return group_width<128, 128, false>(blocks, tiles_m, tiles_n);
    default:
        return a8 ? group_width<128, 64, true>(blocks, tiles_m, tiles_n) : group_width<128, 64, false>(blocks, tiles_m, tiles_n);
    }
}

int mfma_tile_choice(int64_t m, int64_t n, int64_t k)
{
    return tile_choice<false>(m, n, k);
}

int w8a8_tile_choice(int64_t m, int64_t n, int64_t k)
{
    return tile_choice<true>(m, n, k);
}

hipError_t launch_mfma_gemm(const uint16_t *x, const int8_t *q, const uint16_t *scales,
                            const int8_t *zeros, OutlierList ol, uint16_t *y, int64_t m, int64_t n,
                            int64_t k, hipStream_t stream)
{
    return launch_tiles<false>(x, nullptr, q, scales, zeros, ol, y, m, n, k, stream);
}

hipError_t launch_mfma_gemm_tile(int tile, const uint16_t *x, const int8_t *q, const uint16_t *scales,
                                 const int8_t *zeros, OutlierList ol, uint16_t *y, int64_t m, int64_t n,
                                 int64_t k, hipStream_t stream)
{
    if (tile != 256256 && tile != 256128 && tile != 256064 && tile != 128128 && tile != 128064)
        return hipErrorInvalidValue;
    if (tile == 256256 && k > kPingPongMaxK)
        return hipErrorInvalidValue;
    return launch_tiles<false>(x, nullptr, q, scales, zeros, ol, y, m, n, k, stream, tile);
}

hipError_t launch_w8a8_gemm_tile(int tile, const int8_t *qx, const uint16_t *sx, const int8_t *q,
                                 const uint16_t *scales, uint16_t *y, int64_t m, int64_t n, int64_t k,
                                 hipStream_t stream)
{
    if (tile != 256256 && tile != 256128 && tile != 256064 && tile != 128064)
        return hipErrorInvalidValue;
    return launch_tiles<true>(qx, sx, q, scales, nullptr, OutlierList{nullptr, nullptr, 0}, y, m, n, k, stream,
                              tile);
}

hipError_t launch_w8a8_gemm(const int8_t *qx, const uint16_t *sx, const int8_t *q,
                            const uint16_t *scales, uint16_t *y, int64_t m, int64_t n, int64_t k,
                            hipStream_t stream)
{
    return launch_tiles<true>(qx, sx, q, scales, nullptr, OutlierList{nullptr, nullptr, 0}, y, m, n, k, stream);
}

} // namespace qw
