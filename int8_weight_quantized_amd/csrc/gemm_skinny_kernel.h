// gemm_skinny_kernel.h -- W8A16 skinny GEMM (a few activation rows) on the
// matrix cores (gfx950): the kernel.
//
// Between decode (one token) and prefill (max_length tokens) the matmul has
// a handful of activation rows: the weight stream from HBM still sets the
// time ("探索ChatGLM2在算能BM1684X上INT8量化部署", section 4: small left
// matrix => bound by loading the right matrix), but the per-row VALU dot
// products of the GEMV path grow with m.  Here the contraction runs on
// v_mfma_f32_16x16x32_f16 instead: the int8 weights are cast to fp16 exactly
// in registers and used as the MFMA "A" operand; the activations are the "B"
// operand (16 columns, rows beyond m are zero).
//
// Work split: a workgroup of KSPLIT waves owns RT x 16 weight rows x MT x 16
// activation rows; wave w walks the k steps [w*S/KSPLIT, (w+1)*S/KSPLIT)
// of the S = ceil(k/64) steps of 64, four steps (256 codes of each row) per
// iteration.  The MFMA layout wants lane l (row r = l % 16, group
// g = l / 16) to hold bytes [64 s + 16 g, +16) of row r, which as a load
// would touch sixteen 64-byte row segments per instruction; instead each
// load instruction reads four rows x 256 contiguous bytes (16-byte
// nontemporal loads), the wave writes them into its own slice of LDS and
// reads them back in the MFMA layout (measured 12-25% faster).  Of the 16
// codes a lane holds per step, the first 8 feed one MFMA (k slots
// 8 g .. 8 g + 7 of a 32-wide k block), the last 8 a second one; the
// activation operand is loaded once with the same k assignment and reused
// by all RT row tiles, and each cast weight operand feeds the MFMAs of all
// MT activation tiles (so up to 16 MT activation rows take one pass over the
// weights).  KSPLIT is chosen so the grid has enough waves to
// keep HBM busy.  The KSPLIT partial tiles are summed in LDS in wave order
// (deterministic), then scaled (the scales are loaded at the start, so their
// latency hides under the main loop), rounded to fp16 and transposed
// through LDS, so that Y is written in whole 16-byte pieces of its rows.
#pragma once

#include "epilogue_device.h"
#include "qw_device.h"
#include "qw_internal.h"

#include <type_traits>

namespace qw {
namespace {

typedef float float4v __attribute__((ext_vector_type(4)));
typedef int int4v __attribute__((ext_vector_type(4)));

constexpr int kSkinnyUnroll = 4;
constexpr int kSkinnyTargetWaves = 2048; // enough in-flight loads to fill HBM

// A8 (W8A8): the activations are int8 codes with one fp16 scale per row
// (sx); the 16 codes a lane holds per step are exactly the A operand of one
// v_mfma_i32_16x16x64_i8 (k slots 16 g .. 16 g + 15 of the 64-wide step),
// the activation codes the B operand with the same assignment, the
// accumulators are exact int32, and the epilogue scales by S[n] * Sx[m].
// Zero points and side lists are W8A16 only (null with A8).
//
// EPI: the products with an epilogue (qw_w8a16_linear and its kind), without
// zero points or side lists.  A gated product (kGated) pairs weight tile 2 t of
// the gate's channels with tile 2 t + 1 of the same channels of the other half,
// so that a lane holds both factors of its outputs.  The finished tile is fp32
// in LDS, and the residual is added where it is stored: one rounding.
// GRP: a grouped product (qw_w8a16_experts); blockIdx.y is a row tile of
// 16 MT entries of one expert, and m the expert's end.
//
// RW > 1: RW waves of neighbouring weight rows for each part of k, RW * KSPLIT in
// all.  They share the activations of an iteration through LDS, each wave loading
// its part of them: with a row block a wave, every wave reads all of the
// activations again, which for 16 rows in fp16 and 32 weight rows are as many
// bytes as its weights.  All waves keep step (a barrier an iteration, two tiles of
// activations in turn), and the loads of two iterations are in flight.  Us, 4096
// deep, 16 rows, n = 27392 (gated) / 16384 / 65024: 24.2 / 15.5 / 46.3, without
// 30.1 / 18.1 / 55.3; 32 rows 28.1 / 18.4 / 60.5 and 34.9 / 26.4 / 72.2.  Three
// iterations ahead were 4 to 20 % slower.
//
// PART (with RW > 1): the reduction split over `parts` workgroups too (blockIdx.z).
// kParts leaves each one's sums in `partial`, and kJoin, a launch of its own with
// the same RT, MT and RW, adds them in the parts' order for the epilogue.
//
// F32: a grouped product's outputs stay in fp32.
enum { kWhole = 0, kParts = 1, kJoin = 2 };
template <int RT, int MT, int KSPLIT, bool A8 = false, bool ZP = false, int EPI = kPlain, bool GRP = false, int RW = 1,
          int PART = kWhole, bool F32 = false>
__global__ __launch_bounds__(RW * KSPLIT * 64) void skinny_gemm_kernel(
    const void *__restrict__ xv, const uint16_t *__restrict__ sx, const int8_t *__restrict__ q,
    const uint16_t *__restrict__ scales, const int8_t *__restrict__ zeros, OutlierList ol,
    uint16_t *__restrict__ y, int m, int n, int k, Epilogue ep, Experts ex, void *__restrict__ partial_sums, int parts)
{
    static_assert(EPI == kPlain || !ZP, "symmetric codes");
    static_assert(EPI != kGated || RT % 2 == 0, "gate and up in pairs of tiles");
    static_assert(!GRP || (EPI != kPlain && !A8), "grouped products are W8A16 with an epilogue");
    static_assert(GRP || !F32, "fp32 outputs: grouped products");
    static_assert(RW == 1 || (EPI != kPlain && !GRP), "shared activations: products with an epilogue");
    static_assert(PART == kWhole || (RW > 1 && (PART == kParts || KSPLIT == 1)), "parts of wide workgroups");
    const uint16_t *__restrict__ x = static_cast<const uint16_t *>(xv);
    using acc_t = std::conditional_t<A8, int4v, float4v>;
    // Per wave, a staging slice for the weight codes of one iteration:
    // [tile][row][256 bytes + 16 pad].  After the main loop the same memory
    // holds the partial tiles of the parts 1 .. KSPLIT-1.
    constexpr int kStageRow = 64 * kSkinnyUnroll + 16; // 256 codes + pad
    constexpr int kStageBytes = RW * KSPLIT * RT * 16 * kStageRow;
    constexpr int kPartialBytes = RW * (KSPLIT > 1 ? KSPLIT - 1 : 1) * RT * MT * kWave * (int)sizeof(acc_t);
    __shared__ __attribute__((aligned(16))) uint8_t smem[kStageBytes > kPartialBytes ? kStageBytes : kPartialBytes];
    // the finished tile (fp16, or fp32 with EPI), [activation row][channel], padded rows
    constexpr int kCols = EPI == kGated ? 8 * RT : 16 * RT; // columns of Y a workgroup
    using tile_t = std::conditional_t<EPI == kPlain, uint16_t, float>;
    __shared__ __attribute__((aligned(16))) tile_t ytiles[RW * 16 * MT][kCols + (EPI == kPlain ? 8 : 4)];
    static_assert(kSkinnyUnroll == 4, "one iteration covers 256 codes of a row");

    const int lane = __lane_id();
    const int wave_id = threadIdx.x / kWave;
    const int wave = RW > 1 ? wave_id / RW : wave_id; // part of k
    const int rw = RW > 1 ? wave_id % RW : 0;         // row block of the workgroup
    auto *ytile = ytiles + rw * 16 * MT;
    const int r = lane % 16;
    const int g = lane / 16;
    const int n_out = EPI == kGated ? n / 2 : n;
    const int n0 = (blockIdx.x * RW + rw) * kCols; // first column of Y
    // weight row r16 of tile t, and whether it is one
    auto row_of = [&](int t, int r16) { return EPI == kGated ? (t & 1) * n_out + n0 + 16 * (t / 2) + r16 : n0 + 16 * t + r16; };
    auto row_in = [&](int t, int r16) { return EPI == kGated ? n0 + 16 * (t / 2) + r16 < n_out : n0 + 16 * t + r16 < n; };
    int m0 = blockIdx.y * 16 * MT;
    if constexpr (GRP) {
        const GroupTile tile = group_tile<16 * MT>(ex, blockIdx.y);
        if (tile.end <= tile.begin)
            return;
        m0 = tile.begin;
        m = tile.end;
        if (tile.expert == ex.count) { // entries of no expert: rows of zeros
            for (int e = threadIdx.x; e < 16 * MT * kCols; e += KSPLIT * kWave)
                if (m0 + e / kCols < m && n0 + e % kCols < n_out)
                    reinterpret_cast<std::conditional_t<F32, float, uint16_t> *>(y)[(int64_t)(m0 + e / kCols) * n_out + n0 +
                                                                                    e % kCols] = 0;
            return;
        }
        q += (int64_t)tile.expert * n * k;
        scales += (int64_t)tile.expert * n;
        if (ep.bias)
            ep.bias += (int64_t)tile.expert * n;
    }

    const int steps_total = (k + 63) / 64;
    const int s_first = PART == kParts ? (int)((int64_t)blockIdx.z * steps_total / parts) : 0;
    const int steps = PART == kParts ? (int)((int64_t)(blockIdx.z + 1) * steps_total / parts) - s_first : steps_total;
    const int s_begin = s_first + (int)(((int64_t)wave * steps) / KSPLIT);
    const int s_end = s_first + (int)(((int64_t)(wave + 1) * steps) / KSPLIT);

    const int8_t *qrow[RT];
    bool row_ok[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        const int row = row_of(t, r);
        row_ok[t] = row_in(t, r);
        qrow[t] = q + (int64_t)(row_ok[t] ? row : 0) * k;
    }
    // activation row m0 + 16 mt + r is what this lane feeds into the B
    // operand of activation tile mt
    const uint16_t *xrow[MT];
    const int8_t *qxrow[MT];
    bool col_ok[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        int col = m0 + 16 * mt + r;
        col_ok[mt] = col < m;
        if constexpr (GRP) {
            col = col_ok[mt] ? entry_row(ex, col) : -1;
            col_ok[mt] = col >= 0;
        }
        xrow[mt] = x + (int64_t)(col_ok[mt] ? col : 0) * k;
        qxrow[mt] = static_cast<const int8_t *>(xv) + (int64_t)(col_ok[mt] ? col : 0) * k;
    }

    // the scales of the outputs this lane ends up holding (channels
    // n0 + 16 t + 4 g + i), loaded now so that they arrive during the main
    // loop instead of stalling the epilogue
    uint16_t sc[RT][4], bias[RT][4];
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int yn = row_of(t, 4 * g + i);
            const bool in = row_in(t, 4 * g + i);
            sc[t][i] = in ? scales[yn] : (uint16_t)0;
            if constexpr (EPI != kPlain)
                bias[t][i] = in && ep.bias ? ep.bias[yn] : (uint16_t)0;
        }

    // asymmetric weights: the cast subtracts the zero point of weight row
    // n0 + 16 t + r (zeros == nullptr: symmetric)
    // (a template parameter: the symmetric kernels keep the constant bias
    // and its registers free)
    half2_t zbias[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t)
        zbias[t] = zero_point_bias(ZP && row_ok[t] ? (int)zeros[n0 + 16 * t + r] : 0);

    acc_t acc[RT][MT];
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
            acc[t][mt] = (acc_t){};

    // this lane's sums of tile (t, mt) of part p
    auto sums_of = [&](int p, int t, int mt) {
        const int64_t block = ((int64_t)p * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x;
        return static_cast<acc_t *>(partial_sums) + (block * (RW * RT * MT) + (rw * RT + t) * MT + mt) * kWave + lane;
    };
    if constexpr (PART == kJoin) {
        for (int p = 0; p < parts; ++p)
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
                    acc[t][mt] += *sums_of(p, t, mt);
    } else if constexpr (RW > 1) {
        constexpr int kElem = A8 ? 1 : 2;
        constexpr int kXRow = 64 * kSkinnyUnroll * kElem + 16; // an iteration's activations of a row + pad
        constexpr int kXTile = 16 * MT * kXRow;
        constexpr int kXLanes = 4 * kSkinnyUnroll * kElem;     // lanes a row, 16 bytes each
        constexpr int kXLoads = 16 * MT * kXLanes / (RW * kWave);
        static_assert(kXLoads * RW * kWave == 16 * MT * kXLanes, "a whole number of loads");
        __shared__ __attribute__((aligned(16))) uint8_t xtiles[KSPLIT * 2 * kXTile];
        uint8_t *slice = smem + wave_id * RT * 16 * kStageRow;
        uint8_t *xtile = xtiles + wave * 2 * kXTile;
        u32x4_t raw[2][4][RT], xraw[2][kXLoads];
        const uint8_t *xp[kXLoads];
        bool xin[kXLoads];
        const int xpiece = lane % kXLanes; // of the row
#pragma unroll
        for (int i = 0; i < kXLoads; ++i) {
            const int col = m0 + (i * RW * kWave + rw * kWave + lane) / kXLanes;
            xin[i] = col < m;
            xp[i] = static_cast<const uint8_t *>(xv) + (int64_t)(xin[i] ? col : 0) * k * kElem + 16 * xpiece;
        }
        // Both loads leave what is behind the part's end, k, m or n zero.
        auto load = [&](int d, int s) {
#pragma unroll
            for (int i = 0; i < kXLoads; ++i) {
                const int kk = s * 64 + 16 / kElem * xpiece;
                xraw[d][i] = (u32x4_t){0u, 0u, 0u, 0u};
                if (xin[i] && kk < 64 * s_end && kk < k)
                    xraw[d][i] = *reinterpret_cast<const u32x4_t *>(xp[i] + (int64_t)s * 64 * kElem);
            }
            const int kl = s * 64 + 16 * (lane % 16);
            const bool okl = kl < 64 * s_end && kl < k;
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = row_of(t, 4 * i + lane / 16);
                    raw[d][i][t] = (u32x4_t){0u, 0u, 0u, 0u};
                    if (okl && row_in(t, 4 * i + lane / 16))
                        raw[d][i][t] = __builtin_nontemporal_load(
                            reinterpret_cast<const u32x4_t *>(q + (int64_t)row * k + kl));
                }
        };
        // (as many for every wave: the longest part's)
        const int rounds = ((steps + KSPLIT - 1) / KSPLIT + kSkinnyUnroll - 1) / kSkinnyUnroll;
        load(0, s_begin);
        load(1, s_begin + kSkinnyUnroll);
        for (int i0 = 0; i0 < rounds; i0 += 2) {
#pragma unroll
            for (int d = 0; d < 2; ++d) {
                if (i0 + d >= rounds)
                    break;
                uint8_t *xs = xtile + d * kXTile;
#pragma unroll
                for (int i = 0; i < kXLoads; ++i)
                    *reinterpret_cast<u32x4_t *>(xs + (i * RW * kWave + rw * kWave + lane) / kXLanes * kXRow + 16 * xpiece) =
                        xraw[d][i];
#pragma unroll
                for (int t = 0; t < RT; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        *reinterpret_cast<u32x4_t *>(slice + (t * 16 + 4 * i + lane / 16) * kStageRow + 16 * (lane % 16)) =
                            raw[d][i][t];
                __builtin_amdgcn_sched_barrier(0); // (the loads into these registers not before)
                load(d, s_begin + (i0 + d + 2) * kSkinnyUnroll);
                // This tile of activations was read two iterations ago, before
                // the barrier of the last one.  The asm waits for LDS alone: the
                // loads stay in flight.
                asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
                for (int u = 0; u < kSkinnyUnroll; ++u) {
                    u32x4_t xa[MT], xb[MT];
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        const uint8_t *p = xs + (16 * mt + r) * kXRow + (64 * u + 16 * g) * kElem;
                        xa[mt] = *reinterpret_cast<const u32x4_t *>(p);
                        if constexpr (!A8)
                            xb[mt] = *reinterpret_cast<const u32x4_t *>(p + 16);
                    }
#pragma unroll
                    for (int t = 0; t < RT; ++t) {
                        const u32x4_t w = *reinterpret_cast<const u32x4_t *>(slice + (t * 16 + r) * kStageRow + 64 * u + 16 * g);
                        if constexpr (A8) {
#pragma unroll
                            for (int mt = 0; mt < MT; ++mt)
                                acc[t][mt] = __builtin_amdgcn_mfma_i32_16x16x64_i8(
                                    __builtin_bit_cast(int4v, w), __builtin_bit_cast(int4v, xa[mt]), acc[t][mt], 0, 0, 0);
                        } else {
                            const half8_t a0 = i8x8_to_half8(w.x, w.y, zbias[t]);
                            const half8_t a1 = i8x8_to_half8(w.z, w.w, zbias[t]);
#pragma unroll
                            for (int mt = 0; mt < MT; ++mt) {
                                acc[t][mt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a0, __builtin_bit_cast(half8_t, xa[mt]),
                                                                                   acc[t][mt], 0, 0, 0);
                                acc[t][mt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a1, __builtin_bit_cast(half8_t, xb[mt]),
                                                                                   acc[t][mt], 0, 0, 0);
                            }
                        }
                    }
                }
                // (the next codes go into the slice behind these reads, as below)
                __builtin_amdgcn_wave_barrier();
            }
        }
    }

    for (int s = s_begin; RW == 1 && s < s_end; s += kSkinnyUnroll) {
        u32x4_t wv[kSkinnyUnroll][RT];
        u32x4_t xa[kSkinnyUnroll][MT], xb[kSkinnyUnroll][MT];
        // Activation operands.  For the fp16 kernel with one activation
        // tile they are requested before the weight codes, so the two
        // loads' latencies overlap (measured 2-4% faster); otherwise after
        // the weight staging (two tiles measured 5% slower the other way,
        // and the int8 kernel kept its operand arrays in scratch memory).
        constexpr bool kXFirst = MT == 1 && !A8;
        if constexpr (kXFirst) {
#pragma unroll
            for (int u = 0; u < kSkinnyUnroll; ++u) {
                const int kk = (s + u) * 64 + g * 16;
                const bool ok = (s + u) < s_end && kk < k;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    xa[u][mt] = (u32x4_t){0u, 0u, 0u, 0u};
                    xb[u][mt] = (u32x4_t){0u, 0u, 0u, 0u};
                    if (ok && col_ok[mt]) {
                        if constexpr (A8) {
                            xa[u][mt] = *reinterpret_cast<const u32x4_t *>(qxrow[mt] + kk);
                        } else {
                            xa[u][mt] = *reinterpret_cast<const u32x4_t *>(xrow[mt] + kk);
                            xb[u][mt] = *reinterpret_cast<const u32x4_t *>(xrow[mt] + kk + 8);
                        }
                    }
                }
            }
        }
        {
            // Weight codes, loaded contiguously: instruction i of tile t
            // covers rows 4 i .. 4 i + 3, 256 bytes each (lane l: row
            // 4 i + l / 16, bytes 16 (l % 16) of the 256), so every load
            // instruction touches four 256-byte row segments instead of
            // sixteen 64-byte ones.  They go through this wave's slice of
            // LDS and come back in the MFMA layout (lane (r, g): row r,
            // bytes 64 u + 16 g for step u).
            uint8_t *slice = smem + wave * RT * 16 * kStageRow;
            const int ul = (lane % 16) / 4; // step this lane's 16 bytes belong to
            const int kl = s * 64 + 16 * (lane % 16);
            const bool okl = (s + ul) < s_end && kl < k;
            u32x4_t raw[4][RT];
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = row_of(t, 4 * i + lane / 16);
                    raw[i][t] = (u32x4_t){0u, 0u, 0u, 0u};
                    if (okl && row_in(t, 4 * i + lane / 16))
                        raw[i][t] = __builtin_nontemporal_load(
                            reinterpret_cast<const u32x4_t *>(q + (int64_t)row * k + kl));
                }
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    *reinterpret_cast<u32x4_t *>(slice + (t * 16 + 4 * i + lane / 16) * kStageRow +
                                                 16 * (lane % 16)) = raw[i][t];
            // Each lane reads back bytes that other lanes of the wave wrote.
            // LDS executes a wave's accesses in order, but per lane the read
            // and write addresses never coincide, so without these barriers
            // the compiler may move reads above the writes they depend on
            // (or the next iteration's writes above these reads).
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int u = 0; u < kSkinnyUnroll; ++u)
#pragma unroll
                for (int t = 0; t < RT; ++t)
                    wv[u][t] = *reinterpret_cast<const u32x4_t *>(slice + (t * 16 + r) * kStageRow + 64 * u + 16 * g);
            __builtin_amdgcn_wave_barrier();
        }
        if constexpr (!kXFirst) {
#pragma unroll
            for (int u = 0; u < kSkinnyUnroll; ++u) {
                const int kk = (s + u) * 64 + g * 16;
                const bool ok = (s + u) < s_end && kk < k;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    xa[u][mt] = (u32x4_t){0u, 0u, 0u, 0u};
                    xb[u][mt] = (u32x4_t){0u, 0u, 0u, 0u};
                    if (ok && col_ok[mt]) {
                        if constexpr (A8) {
                            xa[u][mt] = *reinterpret_cast<const u32x4_t *>(qxrow[mt] + kk);
                        } else {
                            xa[u][mt] = *reinterpret_cast<const u32x4_t *>(xrow[mt] + kk);
                            xb[u][mt] = *reinterpret_cast<const u32x4_t *>(xrow[mt] + kk + 8);
                        }
                    }
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kSkinnyUnroll; ++u) {
            if constexpr (A8) {
#pragma unroll
                for (int t = 0; t < RT; ++t)
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
                        acc[t][mt] = __builtin_amdgcn_mfma_i32_16x16x64_i8(
                            __builtin_bit_cast(int4v, wv[u][t]), __builtin_bit_cast(int4v, xa[u][mt]), acc[t][mt],
                            0, 0, 0);
            } else {
#pragma unroll
                for (int t = 0; t < RT; ++t) {
                    const half8_t a0 = i8x8_to_half8(wv[u][t].x, wv[u][t].y, zbias[t]);
                    const half8_t a1 = i8x8_to_half8(wv[u][t].z, wv[u][t].w, zbias[t]);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        const half8_t b0 = __builtin_bit_cast(half8_t, xa[u][mt]);
                        const half8_t b1 = __builtin_bit_cast(half8_t, xb[u][mt]);
                        acc[t][mt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a0, b0, acc[t][mt], 0, 0, 0);
                        acc[t][mt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a1, b1, acc[t][mt], 0, 0, 0);
                    }
                }
            }
        }
    }

    if (KSPLIT > 1) {
        acc_t *partial = reinterpret_cast<acc_t *>(smem); // [KSPLIT-1][RW][RT][MT][kWave]
        __syncthreads(); // every wave is done with its staging slice
        if (wave > 0) {
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
                    partial[((((wave - 1) * RW + rw) * RT + t) * MT + mt) * kWave + lane] = acc[t][mt];
        }
        __syncthreads();
        if (wave != 0)
            return;
#pragma unroll
        for (int w = 0; w < KSPLIT - 1; ++w)
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
                    acc[t][mt] += partial[(((w * RW + rw) * RT + t) * MT + mt) * kWave + lane];
    }
    if constexpr (PART == kParts) {
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
                *sums_of(blockIdx.z, t, mt) = acc[t][mt];
        return;
    }
    if constexpr (EPI == kPlain) {
        // lane holds channels n0 + 16 t + 4 g + i (i = 0..3) of activation row
        // m0 + 16 mt + r: scale, round, and transpose through LDS so that the
        // stores are whole 16-byte pieces of Y rows
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const float xscale = A8 && col_ok[mt] ? f16_bits_to_f32(sx[m0 + 16 * mt + r]) : 0.0f;
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float out;
                    if constexpr (A8) // exact int32 sum, then S[n] * Sx[m] (exact in fp32)
                        out = (float)acc[t][mt][i] * (f16_bits_to_f32(sc[t][i]) * xscale);
                    else
                        out = acc[t][mt][i] * f16_bits_to_f32(sc[t][i]);
                    // exact outliers of channel n0 + 16 t + 4 g + i, with X read
                    // from global memory (a few activation rows: L2-resident)
                    const int yn = n0 + 16 * t + 4 * g + i;
                    if (!A8 && ol.idx != nullptr && yn < n && col_ok[mt]) {
                        for (int e = 0; e < ol.cap; ++e) {
                            const int kk = ol.idx[(int64_t)yn * ol.cap + e];
                            if (kk < 0 || kk >= k)
                                break; // used slots come first
                            out += f16_bits_to_f32(xrow[mt][kk]) * ol.val[(int64_t)yn * ol.cap + e];
                        }
                    }
                    ytile[16 * mt + r][16 * t + 4 * g + i] = f32_to_f16_bits(out);
                }
        }
    } else {
        // the same channels with bias, activation and the gate's partner
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const float xscale = A8 && col_ok[mt] ? f16_bits_to_f32(sx[m0 + 16 * mt + r]) : 0.0f;
            auto value = [&](int t, int i) -> float {
                const float s = f16_bits_to_f32(sc[t][i]);
                const float v = A8 ? (float)acc[t][mt][i] * (s * xscale) : acc[t][mt][i] * s;
                return v + from16(bias[t][i], ep.bf16);
            };
            constexpr int kStep = EPI == kGated ? 2 : 1;
#pragma unroll
            for (int t = 0; t < RT; t += kStep)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float v = activate(ep.activation, value(t, i));
                    if constexpr (EPI == kGated)
                        v *= value(t + 1, i);
                    ytile[16 * mt + r][16 * (t / kStep) + 4 * g + i] = v;
                }
        }
    }
    // the tile is written and read back by the same wave: LDS keeps a
    // wave's accesses in order; the barrier only stops the compiler from
    // moving the reads above the writes
    __builtin_amdgcn_wave_barrier();
    constexpr int kPieces = kCols / 8;  // 8-column pieces per tile row
    const bool vec_ok = (n_out % 8) == 0 && n0 + kCols <= n_out;
    for (int e = lane; e < 16 * MT * kPieces; e += kWave) {
        const int row = e / kPieces;
        const int pc = e % kPieces;
        const int ym = m0 + row;
        if (ym >= m)
            continue;
        uint16_t *dst = y + (int64_t)ym * n_out + n0 + 8 * pc;
        if constexpr (EPI == kPlain) {
            if (vec_ok) {
                *reinterpret_cast<u32x4_t *>(dst) = *reinterpret_cast<const u32x4_t *>(&ytile[row][8 * pc]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (n0 + 8 * pc + j < n)
                        dst[j] = ytile[row][8 * pc + j];
            }
        } else if constexpr (F32) {
            float *to = reinterpret_cast<float *>(y) + (int64_t)ym * n_out + n0 + 8 * pc;
            const float *from = &ytile[row][8 * pc];
            if (vec_ok) {
                *reinterpret_cast<float4v *>(to) = *reinterpret_cast<const float4v *>(from);
                *reinterpret_cast<float4v *>(to + 4) = *reinterpret_cast<const float4v *>(from + 4);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (n0 + 8 * pc + j < n_out)
                        to[j] = from[j];
            }
        } else {
            const uint16_t *res = ep.residual ? ep.residual + (int64_t)ym * n_out + n0 + 8 * pc : nullptr;
            uint32_t w[4];
            if (vec_ok) {
                u32x4_t rv = {0u, 0u, 0u, 0u};
                if (res)
                    rv = *reinterpret_cast<const u32x4_t *>(res);
                const uint32_t rw[4] = {rv.x, rv.y, rv.z, rv.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float a = ytile[row][8 * pc + 2 * j], b = ytile[row][8 * pc + 2 * j + 1];
                    if (res) {
                        a += from16((uint16_t)rw[j], ep.bf16);
                        b += from16((uint16_t)(rw[j] >> 16), ep.bf16);
                    }
                    w[j] = to16(a, ep.bf16) | ((uint32_t)to16(b, ep.bf16) << 16);
                }
                *reinterpret_cast<u32x4_t *>(dst) = (u32x4_t){w[0], w[1], w[2], w[3]};
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (n0 + 8 * pc + j < n_out) {
                        float a = ytile[row][8 * pc + j];
                        if (res)
                            a += from16(res[j], ep.bf16);
                        dst[j] = to16(a, ep.bf16);
                    }
            }
        }
    }
}

} // namespace
} // namespace qw
