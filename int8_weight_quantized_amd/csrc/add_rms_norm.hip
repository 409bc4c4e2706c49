// add_rms_norm.hip -- the residual's addition and the RMS norm of the rows of
// a residual stream, with an output in 16 bits or in int8 codes.
//
//   h = round(x + r)                       (no residual: h = x)
//   y = h w / sqrt(mean(h^2) + eps)
//   codes: S = fp16(max|y| / 127), q = clamp(round_half_even(y / S))
//
// in fp32 from the rounded h, so that y is a function of the h that is stored.
// The row's sum of squares and its largest |h w| come from one pass over the
// loads: the largest |y| is the latter over the root of the former, so the
// codes need no second reduction.
//
// Bound by HBM: 7 bytes an element with a residual and codes.  A row is held in
// registers, 8 elements (16 bytes) a lane and vector, as the 16-bit h.
//
// Waves before vectors: a row's latency is that of its loads and of the one
// barrier, and a lane with one vector has the fewest of them in a row.  Us, fp16
// with a residual / and codes, as launched and with four waves of four vectors:
// 1 x 4096 2.5 / 2.7 and 3.1 / 3.4, 256 x 8192 4.2 / 4.6 and 5.0 / 5.4, 8192 x
// 4096 38.9 / 35.0 and 40.2 / 38.8, 8192 x 8192 91 / 83 (5.9 and 5.6 TB/s) and
// 95 / 89.  4096 x 16384 with two vectors 97 / 87, with eight 104 / 109.  Beyond,
// eight for all: 4096 x 20480 128 / 129, 2048 x 32768 107 / 106, 2048 x 65536
// 207 / 203 (5.0 to 5.3 and 4.4 to 4.6 TB/s).  Short rows leave waves without work
// (four a row up to 2048 elements): 16384 x 256 11 / 17, 512 13 / 18, 1024 21 / 22.
#include "ff_internal.h"
#include "kv_device.h"

namespace qw {

namespace {

// W waves a row, at most V vectors a lane.
template <int DT, bool CODES, int W, int V>
__global__ __launch_bounds__(W * kWave) void add_rms_norm_kernel(AddNormArgs a)
{
    __shared__ float part[2 * W];
    const int lane = __lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int64_t row = blockIdx.x;
    const int first = (int)threadIdx.x; // vector of the row
    const int vectors = (int)(a.k / 8);
    const uint16_t *x = a.x + row * a.x_stride, *r = a.residual + row * a.residual_stride;
    uint16_t *hrow = a.h + row * a.h_stride;
    u32x4_t h[V], w[V], more[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int v = first + i * W * kWave;
        if (v < vectors) {
            h[i] = *reinterpret_cast<const u32x4_t *>(x + v * 8);
            if (a.residual)
                more[i] = *reinterpret_cast<const u32x4_t *>(r + v * 8);
            w[i] = *reinterpret_cast<const u32x4_t *>(a.weight + v * 8);
        }
    }
    float squares = 0.0f, most = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int v = first + i * W * kWave;
        if (v < vectors) {
            float f[8], g[8];
            unpack8<DT>(h[i], f);
            if (a.residual) {
                unpack8<DT>(more[i], g);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    f[e] += g[e];
                h[i] = pack8<DT>(f);
                *reinterpret_cast<u32x4_t *>(hrow + v * 8) = h[i];
                unpack8<DT>(h[i], f);
            }
            unpack8<DT>(w[i], g);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                squares += f[e] * f[e];
                if (CODES)
                    most = fmaxf(most, fabsf(f[e] * g[e]));
            }
        }
    }
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        squares += shfl_xor_f32(squares, d);
        if (CODES)
            most = fmaxf(most, shfl_xor_f32(most, d));
    }
    if (lane == 0) {
        part[wave] = squares;
        part[W + wave] = most;
    }
    __syncthreads();
    squares = 0.0f;
#pragma unroll
    for (int i = 0; i < W; ++i) {
        squares += part[i];
        most = fmaxf(most, part[W + i]);
    }
    const float inv = 1.0f / sqrtf(squares / (float)a.k + a.eps);
    float step = 0.0f; // codes a unit of h w
    if (CODES) {
        const uint16_t bits = f32_to_f16_bits(most * inv / 127.0f);
        const float scale = f16_bits_to_f32(bits);
        step = scale > 0.0f ? inv / scale : 0.0f;
        if (first == 0)
            a.scales[row] = bits;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int v = first + i * W * kWave;
        if (v < vectors) {
            float f[8], g[8];
            unpack8<DT>(h[i], f);
            unpack8<DT>(w[i], g);
            if (CODES) {
                uint32_t c[2] = {0, 0};
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float t = fminf(fmaxf(rintf(f[e] * g[e] * step), -127.0f), 127.0f);
                    c[e / 4] |= ((uint32_t)(int)t & 255u) << (8 * (e % 4));
                }
                *reinterpret_cast<u32x2_t *>(a.q + row * a.k + v * 8) = (u32x2_t){c[0], c[1]};
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    f[e] = f[e] * inv * g[e];
                *reinterpret_cast<u32x4_t *>(a.y + row * a.k + v * 8) = pack8<DT>(f);
            }
        }
    }
}

template <int DT, bool CODES, int W, int V>
hipError_t launch(const AddNormArgs &a, hipStream_t stream)
{
    // (a grid holds fewer than 2^32 threads: more rows go in several launches)
    constexpr int64_t kMost = (int64_t(1) << 31) / (W * kWave);
    for (int64_t first = 0; first < a.tokens; first += kMost) {
        AddNormArgs part = a;
        part.x += first * a.x_stride;
        if (a.residual) {
            part.residual += first * a.residual_stride;
            part.h += first * a.h_stride;
        }
        if (CODES) {
            part.q += first * a.k;
            part.scales += first;
        } else {
            part.y += first * a.k;
        }
        const int64_t rows = a.tokens - first < kMost ? a.tokens - first : kMost;
        add_rms_norm_kernel<DT, CODES, W, V><<<dim3((unsigned)rows), dim3(W * kWave), 0, stream>>>(part);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

template <int DT, bool CODES>
hipError_t launch_sizes(const AddNormArgs &a, hipStream_t stream)
{
    const int64_t vectors = a.k / 8;
    if (vectors <= 256)
        return launch<DT, CODES, 4, 1>(a, stream);
    if (vectors <= 512)
        return launch<DT, CODES, 8, 1>(a, stream);
    if (vectors <= 1024)
        return launch<DT, CODES, 16, 1>(a, stream);
    if (vectors <= 2048)
        return launch<DT, CODES, 16, 2>(a, stream);
    return launch<DT, CODES, 16, 8>(a, stream);
}

} // namespace

hipError_t launch_add_rms_norm(const AddNormArgs &a, int dtype, hipStream_t stream)
{
    if (dtype == QW_F16)
        return a.q ? launch_sizes<QW_F16, true>(a, stream) : launch_sizes<QW_F16, false>(a, stream);
    return a.q ? launch_sizes<QW_BF16, true>(a, stream) : launch_sizes<QW_BF16, false>(a, stream);
}

} // namespace qw
