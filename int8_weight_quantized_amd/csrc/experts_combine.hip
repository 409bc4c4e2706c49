// experts_combine.hip -- the sum over a token's experts.
//
//   out[t] = residual[t] + sum_j weights[t][j] y[places[t][j]]
//
// in fp32, in the order of j, rounded once.  Bound by memory: top_k rows in, one
// out (and the residual in).  A lane takes 8 columns (16 bytes) of a token and
// asks for kBatch rows at a time, so that their latencies overlap.  4096 tokens of
// 2048, 8 experts: 23 us (6.4 TB/s), with a residual 26; 16 tokens 3.4 us; 4096 of
// 2047, by elements, 82.  Rows of fp16 or fp32.
#include "ff_internal.h"
#include "kv_device.h"

namespace qw {

namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 8;

// WHOLE: n is a multiple of 8, so that every row is aligned.
template <bool WHOLE>
__device__ __forceinline__ u32x4_t load8(const uint16_t *p, int left)
{
    if (WHOLE)
        return *reinterpret_cast<const u32x4_t *>(p);
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < left)
            w[e / 2] |= (uint32_t)p[e] << (16 * (e % 2));
    return (u32x4_t){w[0], w[1], w[2], w[3]};
}

// Eight entries' values of a row: as they are loaded, and in fp32.
template <bool WHOLE, bool F32>
struct Entries;
template <bool WHOLE>
struct Entries<WHOLE, false> {
    u32x4_t v;
    __device__ __forceinline__ void load(const void *y, int64_t at, int left)
    {
        v = load8<WHOLE>(static_cast<const uint16_t *>(y) + at, left);
    }
    __device__ __forceinline__ void values(float (&f)[8]) const { unpack8<QW_F16>(v, f); }
};
template <bool WHOLE>
struct Entries<WHOLE, true> {
    float v[8];
    __device__ __forceinline__ void load(const void *y, int64_t at, int left)
    {
        const float *p = static_cast<const float *>(y) + at;
        if (WHOLE) {
            const float4_t a = *reinterpret_cast<const float4_t *>(p), b = *reinterpret_cast<const float4_t *>(p + 4);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                v[e] = a[e], v[4 + e] = b[e];
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = e < left ? p[e] : 0.0f;
        }
    }
    __device__ __forceinline__ void values(float (&f)[8]) const
    {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            f[e] = v[e];
    }
};

template <bool WHOLE, bool F32>
__global__ __launch_bounds__(kThreads) void experts_combine_kernel(CombineArgs a, int pieces, int64_t first)
{
    const int64_t id = (first + blockIdx.x) * kThreads + threadIdx.x;
    const int64_t token = id / pieces;
    if (token >= a.tokens)
        return;
    const int64_t c = (id - token * pieces) * 8;
    const int left = (int)(a.n - c < 8 ? a.n - c : 8);
    float sum[8] = {};
    if (a.residual)
        unpack8<QW_F16>(load8<WHOLE>(a.residual + token * a.n + c, left), sum);
    const int32_t *places = a.places + token * a.top_k;
    const float *weights = a.weights + token * a.top_k;
    for (int j0 = 0; j0 < a.top_k; j0 += kBatch) {
        Entries<WHOLE, F32> v[kBatch];
        float w[kBatch];
        bool in[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int32_t p = j0 + b < a.top_k ? places[j0 + b] : -1;
            in[b] = p >= 0 && p < a.entries;
            if (in[b]) {
                v[b].load(a.y, p * a.n + c, left);
                w[b] = weights[j0 + b];
            }
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
            if (in[b]) {
                float f[8];
                v[b].values(f);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    sum[e] = fmaf(w[b], f[e], sum[e]);
            }
    }
    uint16_t *dst = a.out + token * a.n + c;
    if (WHOLE) {
        *reinterpret_cast<u32x4_t *>(dst) = pack8<QW_F16>(sum);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < left)
                dst[e] = f32_to_f16_bits(sum[e]);
    }
}

} // namespace

hipError_t launch_experts_combine(const CombineArgs &a, hipStream_t stream)
{
    const int64_t pieces = (a.n + 7) / 8;
    const int64_t blocks = (a.tokens * pieces + kThreads - 1) / kThreads;
    // (a grid holds fewer than 2^32 threads: more go in several launches)
    constexpr int64_t kMost = (int64_t(1) << 31) / kThreads;
    auto launch = [&](auto kernel) {
        for (int64_t first = 0; first < blocks; first += kMost) {
            const int64_t count = blocks - first < kMost ? blocks - first : kMost;
            hipLaunchKernelGGL(kernel, dim3((unsigned)count), dim3(kThreads), 0, stream, a, (int)pieces, first);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess)
                return e;
        }
        return hipSuccess;
    };
    if (a.f32)
        return a.n % 8 == 0 ? launch(experts_combine_kernel<true, true>) : launch(experts_combine_kernel<false, true>);
    return a.n % 8 == 0 ? launch(experts_combine_kernel<true, false>) : launch(experts_combine_kernel<false, false>);
}

} // namespace qw
