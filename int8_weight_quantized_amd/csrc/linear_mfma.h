// linear_mfma.h -- launch of the MFMA GEMMs with an epilogue, one translation
// unit per activation type.
#pragma once

#include "gemm_mfma_kernels.h"

namespace qw {
namespace {

template <int NW, int BN, int BM, bool A8, bool GRP, bool F32>
hipError_t launch_linear_tile(int tile, const LinearArgs &a, const Experts &ex, hipStream_t stream)
{
    constexpr bool kPp = BN == 256 && BM == 256;
    const int64_t columns = a.gated ? a.n / 2 : a.n, bn = a.gated ? BN / 2 : BN;
    const int64_t tiles_n = (columns + bn - 1) / bn;
    // GRP: every number that group_tile() gives out.  A tile row's columns lie
    // next to each other there, so that an expert's weight and rows stay in an
    // XCD's cache while it is worked on.
    const int64_t tiles_m = GRP ? a.m / BM + ex.count + 1 : (a.m + BM - 1) / BM;
    const int64_t blocks = tiles_m * tiles_n;
    if (blocks > 0x7fffffff)
        return hipErrorInvalidConfiguration;
    const int group = GRP ? (int)tiles_n : mfma_tile_group(tile, A8, tiles_m, tiles_n);
    const OutlierList none = {nullptr, nullptr, 0};
    auto launch = [&](auto kernel, int threads, auto... more) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(threads), 0, stream, a.x, a.sx, a.q, a.scales,
                           (const int8_t *)nullptr, none, a.y, (int)a.m, (int)a.n, (int)a.k, (int)tiles_m, (int)tiles_n,
                           group, a.ep, ex, more...);
        return hipGetLastError();
    };
    if constexpr (kPp)
        return a.gated ? launch(mfma_pp_kernel<A8, false, false, kGated, GRP, F32>, pp::kThreads, 1, (u32x4_t *)nullptr)
                       : launch(mfma_pp_kernel<A8, false, false, kLinear, GRP, F32>, pp::kThreads, 1, (u32x4_t *)nullptr);
    else
        return a.gated ? launch(mfma_gemm_dma_kernel<NW, BN, BM, A8, false, false, kGated, GRP, F32>, NW * kWave)
                       : launch(mfma_gemm_dma_kernel<NW, BN, BM, A8, false, false, kLinear, GRP, F32>, NW * kWave);
}

template <bool A8, bool GRP, bool F32 = false>
hipError_t launch_linear_tiles(int tile, const LinearArgs &a, const Experts &ex, hipStream_t stream)
{
    switch (tile) {
    case 256256:
        return launch_linear_tile<8, 256, 256, A8, GRP, F32>(tile, a, ex, stream);
    case 256128:
        return launch_linear_tile<4, 256, 128, A8, GRP, F32>(tile, a, ex, stream);
    case 256064:
        return launch_linear_tile<4, 256, 64, A8, GRP, F32>(tile, a, ex, stream);
    case 128128:
        if constexpr (!A8 && !GRP)
            return launch_linear_tile<4, 128, 128, A8, GRP, F32>(tile, a, ex, stream);
        return hipErrorInvalidValue;
    case 128064:
        return launch_linear_tile<4, 128, 64, A8, GRP, F32>(tile, a, ex, stream);
    default:
        return hipErrorInvalidValue;
    }
}

// Two launches: the parts of the products, and their sum with the epilogue.
template <bool A8>
hipError_t launch_split(int splits, const LinearArgs &a, void *workspace, hipStream_t stream)
{
    const int64_t columns = a.gated ? a.n / 2 : a.n, bn = a.gated ? pp::kBN / 2 : pp::kBN;
    const int64_t tiles_n = (columns + bn - 1) / bn, tiles_m = (a.m + pp::kBM - 1) / pp::kBM, tiles = tiles_m * tiles_n;
    if (tiles * splits > 0x7fffffff || tiles > 0x0fffffff)
        return hipErrorInvalidConfiguration;
    const int group = mfma_tile_group(256256, A8, tiles_m, tiles_n);
    u32x4_t *partial = static_cast<u32x4_t *>(workspace);
    const OutlierList none = {nullptr, nullptr, 0};
    auto product = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)(tiles * splits)), dim3(pp::kThreads), 0, stream, a.x, a.sx, a.q, a.scales,
                           (const int8_t *)nullptr, none, a.y, (int)a.m, (int)a.n, (int)a.k, (int)tiles_m, (int)tiles_n, group,
                           a.ep, Experts{}, splits, partial);
        return hipGetLastError();
    };
    const hipError_t e = a.gated ? product(mfma_pp_kernel<A8, false, false, kPartialGated>)
                                 : product(mfma_pp_kernel<A8, false, false, kPartial>);
    if (e != hipSuccess)
        return e;
    auto join = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)(2 * pp::kSJ * tiles)), dim3(pp::kThreads / 2), 0, stream, (const u32x4_t *)partial,
                           splits, a.sx, a.scales, a.y, (int)a.m, (int)a.n, (int)tiles_m, (int)tiles_n, group, a.ep);
        return hipGetLastError();
    };
    return a.gated ? join(mfma_join_kernel<A8, kGated>) : join(mfma_join_kernel<A8, kLinear>);
}

} // namespace
} // namespace qw
