// route_experts.hip -- which experts a token goes to, with what weights, and
// the entries (a token and one of its experts) listed expert by expert.
//
//   s = softmax(l) or 1 / (1 + exp(-l))
//   choice c = s + bias, or without a bias the order of l itself
//   groups: the top_groups with the largest group scores (the sum of a group's
//           two largest c with a bias, else its largest) keep their experts
//   the top_k experts of the largest c, ties to the lowest index
//   w = s of those [/ their sum] * scale
//
// The choice is made in fp64: with a bias two experts' c often lie closer than
// fp32's rounding of the scores, and the choice would go by that rounding.
//
// A wave takes a token; a lane holds P neighbouring experts, so that the lowest
// lane of those with the largest value also holds the lowest index.
//
// The list is a counting sort that keeps the entries' order and adds nothing in
// an order that varies: each workgroup counts the entries of its tokens by
// expert (integers, in LDS), and a second kernel sums the counts of the
// workgroups before its own and numbers its entries wave by wave, lanes with
// the same expert by their bits in a ballot.
//
// Neither kernel moves enough bytes to matter but for prompts; what counts is
// the length of the chain of selections.
#include "epilogue_device.h"
#include "ff_internal.h"
#include "kv_device.h"

namespace qw {

namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / kWave;
constexpr int kMaxBlocks = 256;

__device__ __forceinline__ double shfl_xor_f64(double v, int mask)
{
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = shfl_xor_u32((uint32_t)b, mask), hi = shfl_xor_u32((uint32_t)(b >> 32), mask);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

__device__ __forceinline__ double wave_max_f64(double v)
{
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) {
        const double o = shfl_xor_f64(v, d);
        v = o > v ? o : v;
    }
    return v;
}

__device__ __forceinline__ double wave_sum_f64(double v)
{
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1)
        v += shfl_xor_f64(v, d);
    return v;
}

template <int DT>
__device__ __forceinline__ float logit(const void *logits, int64_t at)
{
    if constexpr (DT == QW_F32)
        return static_cast<const float *>(logits)[at];
    else
        return from16(static_cast<const uint16_t *>(logits)[at], DT == QW_BF16);
}

// The experts of one token: lane j < top_k gets the j-th (-1: there is none)
// and its weight.  `scratch`: this wave's [experts] of LDS.
template <int DT, int P>
__device__ __forceinline__ void choose(const RouteArgs &a, int64_t token, double *scratch, int &id, float &weight)
{
    const double kNone = -__builtin_inf();
    const int lane = __lane_id();
    float l[P];
    double c[P];
    float most = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int e = lane * P + i;
        float v = e < a.experts ? logit<DT>(a.logits, token * a.experts + e) : -__builtin_inff();
        if (!(v > -__builtin_inff())) // (a NaN too)
            v = -__builtin_inff();
        l[i] = fminf(v, 3.402823466e38f); // infinity counts as the largest number
        most = fmaxf(most, l[i]);
        c[i] = (double)l[i];
    }
    most = wave_max_f32(most);
    double total = 1.0; // softmax: the sum of exp(l - most)
    if (!a.sigmoid && (a.bias || !a.renormalize)) {
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < P; ++i)
            if (l[i] > -__builtin_inff())
                sum += exp((double)l[i] - (double)most);
        total = wave_sum_f64(sum);
    }
    if (a.bias) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int e = lane * P + i;
            if (e < a.experts && l[i] > -__builtin_inff()) {
                const double s = a.sigmoid ? 1.0 / (1.0 + exp(-(double)l[i])) : exp((double)l[i] - (double)most) / total;
                const double v = s + (double)a.bias[e];
                c[i] = v > kNone ? v : kNone; // (a NaN is not chosen)
            }
        }
    }
    if (a.groups > 1) {
        const int size = a.experts / a.groups;
#pragma unroll
        for (int i = 0; i < P; ++i)
            if (lane * P + i < a.experts)
                scratch[lane * P + i] = c[i];
        __builtin_amdgcn_wave_barrier();
        double score = kNone;
        if (lane < a.groups) {
            double first = kNone, second = kNone;
            for (int i = 0; i < size; ++i) {
                const double v = scratch[lane * size + i];
                second = v > first ? first : (v > second ? v : second);
                first = v > first ? v : first;
            }
            score = a.bias && second > kNone ? first + second : first;
        }
        __builtin_amdgcn_wave_barrier();
        uint64_t kept = 0;
        for (int g = 0; g < a.top_groups; ++g) {
            const double top = wave_max_f64(score);
            if (!(top > kNone))
                break;
            const int at = __builtin_ctzll(__ballot(score == top));
            kept |= 1ull << at;
            score = lane == at ? kNone : score;
        }
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int e = lane * P + i;
            if (e < a.experts && !(kept >> (e / size) & 1))
                c[i] = kNone;
        }
    }
    id = -1;
    float mine = 0.0f; // the chosen expert's logit
    for (int j = 0; j < a.top_k; ++j) {
        double best = c[0];
        int at = 0;
#pragma unroll
        for (int i = 1; i < P; ++i)
            if (c[i] > best) {
                best = c[i];
                at = i;
            }
        const double top = wave_max_f64(best);
        if (!(top > kNone))
            break;
        const int from = __builtin_ctzll(__ballot(best == top));
        const int which = __builtin_amdgcn_readlane(at, from);
        float v = l[0];
#pragma unroll
        for (int i = 1; i < P; ++i)
            v = at == i ? l[i] : v;
        const int bits = __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), from);
        if (lane == j) {
            id = from * P + which;
            mine = __builtin_bit_cast(float, bits);
        }
        if (lane == from) {
#pragma unroll
            for (int i = 0; i < P; ++i)
                c[i] = at == i ? kNone : c[i];
        }
    }
    double s = 0.0;
    if (id >= 0)
        s = a.sigmoid ? 1.0 / (1.0 + exp(-(double)mine)) : exp((double)mine - (double)most) / total;
    if (a.renormalize) {
        const double sum = wave_sum_f64(s);
        s = sum > 0.0 ? s / sum : 0.0;
    }
    weight = (float)(s * (double)a.scale);
}

template <int DT, int P>
__global__ __launch_bounds__(kThreads) void route_kernel(RouteArgs a)
{
    extern __shared__ double lds[];
    // counts [experts] ints, then (with groups) a wave's scratch each
    int *counts = reinterpret_cast<int *>(lds);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = __lane_id();
    double *scratch = lds + (a.experts + 1) / 2 + wave * a.experts;
    for (int e = threadIdx.x; e < a.experts; e += kThreads)
        counts[e] = 0;
    __syncthreads();
    const int64_t begin = (int64_t)blockIdx.x * a.tokens_a_block;
    const int64_t end = begin + a.tokens_a_block < a.tokens ? begin + a.tokens_a_block : a.tokens;
    for (int64_t token = begin + wave; token < end; token += kWaves) {
        int id;
        float weight;
        choose<DT, P>(a, token, scratch, id, weight);
        if (lane < a.top_k) {
            a.ids[token * a.top_k + lane] = id;
            a.weights[token * a.top_k + lane] = weight;
            if (id >= 0)
                atomicAdd(&counts[id], 1);
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.experts; e += kThreads)
        a.counts[(int64_t)blockIdx.x * a.experts + e] = counts[e];
}

// Inclusive sum over the workgroup (every thread takes part).
__device__ __forceinline__ int block_scan(int v, int *sums)
{
    const int lane = __lane_id(), wave = threadIdx.x / kWave;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        const int o = __builtin_amdgcn_ds_bpermute((lane - d) << 2, v);
        v += lane >= d ? o : 0;
    }
    if (lane == kWave - 1)
        sums[wave] = v;
    __syncthreads();
    for (int w = 0; w < wave; ++w)
        v += sums[w];
    return v;
}

// Lists the entries of this workgroup's tokens.  experts <= kThreads.
__global__ __launch_bounds__(kThreads) void list_kernel(RouteArgs a)
{
    extern __shared__ int at[]; // [kWaves][experts]: first a wave's entries of an expert, then where its next one goes
    __shared__ int sums[kWaves];
    __shared__ int used;
    const int tid = threadIdx.x, lane = __lane_id(), wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int64_t begin = (int64_t)blockIdx.x * a.tokens_a_block;
    const int64_t end = begin + a.tokens_a_block < a.tokens ? begin + a.tokens_a_block : a.tokens;
    const int64_t entries = (end - begin) * a.top_k, first = begin * a.top_k;
    // a wave's entries: whole chunks of 64 in a row
    const int64_t chunks = (entries + kWave - 1) / kWave, per = (chunks + kWaves - 1) / kWaves;
    const int64_t lo = wave * per * kWave, hi = lo + per * kWave < entries ? lo + per * kWave : entries;
    for (int i = tid; i < kWaves * a.experts; i += kThreads)
        at[i] = 0;
    // this workgroup's first place of each expert
    int before = 0, total = 0;
    if (tid < a.experts)
        for (int b = 0; b < a.blocks; ++b) {
            const int n = a.counts[(int64_t)b * a.experts + tid];
            before += b < (int)blockIdx.x ? n : 0;
            total += n;
        }
    const int upto = block_scan(total, sums); // (with a barrier: `at` is clear)
    for (int64_t i = lo + lane; i < hi; i += kWave) {
        const int id = a.ids[first + i];
        if (id >= 0)
            atomicAdd(&at[wave * a.experts + id], 1);
    }
    if (tid == kThreads - 1)
        used = upto;
    __syncthreads();
    if (tid < a.experts) {
        int next = upto - total + before;
        for (int w = 0; w < kWaves; ++w) {
            const int n = at[w * a.experts + tid];
            at[w * a.experts + tid] = next;
            next += n;
        }
        if (blockIdx.x == 0) {
            a.offsets[tid] = upto - total;
            if (tid == a.experts - 1)
                a.offsets[a.experts] = upto;
        }
    }
    __syncthreads();
    for (int64_t i0 = lo; i0 < hi; i0 += kWave) {
        const int64_t i = i0 + lane;
        const int id = i < hi ? a.ids[first + i] : -1;
        uint64_t same = __ballot(id >= 0); // the lanes with this lane's expert
        for (int bit = 1; bit < a.experts; bit <<= 1) {
            const uint64_t set = __ballot((id & bit) != 0);
            same &= id & bit ? set : ~set;
        }
        int place = -1;
        if (id >= 0) {
            const uint64_t lower = same & ((1ull << lane) - 1);
            place = at[wave * a.experts + id] + __popcll(lower);
            a.rows[place] = (int32_t)(first + i);
        }
        __builtin_amdgcn_wave_barrier(); // (a wave's LDS accesses are in order)
        if (id >= 0 && (same >> lane) == 1)
            at[wave * a.experts + id] = place + 1;
        __builtin_amdgcn_wave_barrier();
        if (i < hi)
            a.places[first + i] = place;
    }
    // places behind the last expert's: this workgroup's share of them
    for (int64_t p = first + tid; p < first + entries; p += kThreads)
        if (p >= used)
            a.rows[p] = -1;
}

template <int DT, int P>
hipError_t launch(const RouteArgs &a, hipStream_t stream)
{
    const size_t counts = (size_t)((a.experts + 1) / 2) * sizeof(double);
    const size_t scratch = a.groups > 1 ? (size_t)kWaves * a.experts * sizeof(double) : 0;
    if (a.blocks > 0) {
        route_kernel<DT, P><<<dim3((unsigned)a.blocks), dim3(kThreads), counts + scratch, stream>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    // (without tokens: the offsets)
    list_kernel<<<dim3(a.blocks > 0 ? (unsigned)a.blocks : 1u), dim3(kThreads), (size_t)kWaves * a.experts * sizeof(int), stream>>>(a);
    return hipGetLastError();
}

template <int DT>
hipError_t launch_type(const RouteArgs &a, hipStream_t stream)
{
    if (a.experts <= 64)
        return launch<DT, 1>(a, stream);
    if (a.experts <= 128)
        return launch<DT, 2>(a, stream);
    if (a.experts <= 256)
        return launch<DT, 4>(a, stream);
    return launch<DT, 8>(a, stream);
}

} // namespace

// A multiple of the waves of a workgroup, so that there are at most kMaxBlocks.
int64_t route_tokens_a_block(int64_t tokens)
{
    const int64_t per = tokens > 0 ? (tokens + kMaxBlocks - 1) / kMaxBlocks : 1;
    return (per + kWaves - 1) / kWaves * kWaves;
}

hipError_t launch_route_experts(const RouteArgs &a, int dtype, hipStream_t stream)
{
    if (dtype == QW_F32)
        return launch_type<QW_F32>(a, stream);
    return dtype == QW_F16 ? launch_type<QW_F16>(a, stream) : launch_type<QW_BF16>(a, stream);
}

} // namespace qw
