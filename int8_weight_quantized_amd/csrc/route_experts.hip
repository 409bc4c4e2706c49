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
// With a bias two experts' c often lie closer than fp32's rounding of the
// scores, so what decides is computed in fp64.  But not for every expert:
//
//   - L lanes take a token (16, 32 or 64: at least its groups and its top_k), P
//     experts a lane, so that a wave works on up to four tokens in the same
//     instructions; every fourth load is four neighbours of the next four lanes'
//     (a lane with 16 neighbours of its own read 64 lines an instruction, which
//     took half the time);
//   - each expert gets a choice in fp32, and all a bound on its error (0 without
//     a bias: the logit itself);
//   - the top_k-th largest of the lanes' own maxima, less twice the error, bounds
//     the top_k-th choice from below, and only the few experts whose choice may
//     reach it go on, to a list in LDS;
//   - those are computed in fp64, and each counts the ones that come before it,
//     which is its place.
//
// Groups are chosen by the fp32 choices too.  Where two are closer than their
// errors, or a list overflows (ties, or more than kListed places), the wave does
// its tokens one expert after the other, all in fp64.  Us, 16384 tokens of 256
// experts, eight of them, with bias and groups / with neither: a token a wave with
// every expert in fp64 40 / 21, this 31 / 14.  Softmax with a bias goes that way
// for every token, as a choice needs the sum over all experts first: with the
// lists 58 with groups and 52 without, where the sigmoid takes 39 and 26; 64
// tokens of 256 50 and 44 for 23 and 18.
//
// The list is a counting sort that keeps the entries' order and adds nothing in
// an order that varies: each workgroup counts the entries of its tokens by
// expert (integers, in LDS), and a second kernel sums the counts of the
// workgroups before its own and numbers its entries wave by wave, lanes with
// the same expert by their bits in a ballot.  Where one workgroup takes all
// tokens it lists them too, without a second launch.
//
// Neither kernel moves enough bytes to matter; what counts is the number of
// instructions in the chain of selections, and for a decode batch the launches.
#include "epilogue_device.h"
#include "ff_internal.h"
#include "kv_device.h"

#include <type_traits>

namespace qw {

namespace {

typedef int int4v __attribute__((ext_vector_type(4)));

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / kWave;
constexpr int kMaxBlocks = 256;
constexpr int kListed = 32; // experts of a token that a list in LDS holds (16 at least)

// v of another lane of the row of 16, by a DPP control: a VALU move.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, false);
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kHalfMirror = 0x141, kMirror = 0x140;

__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return a > b ? a : b; }

// The largest of L neighbouring lanes, in each of them (VALU only: a trip
// through LDS for each step cost ten times as much).
template <int L>
__device__ __forceinline__ uint32_t most_of(uint32_t v)
{
    v = larger(v, dpp<kXor1>(v));
    v = larger(v, dpp<kXor2>(v));
    v = larger(v, dpp<kHalfMirror>(v));
    v = larger(v, dpp<kMirror>(v));
    if constexpr (L >= 32) {
        const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        v = larger(a[0], a[1]);
    }
    if constexpr (L >= 64) {
        const auto a = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        v = larger(a[0], a[1]);
    }
    return v;
}

// v of the lanes up to this one, of L, summed: shifts within the rows of 16
// (zeros come in), then the rows' totals.
template <int L>
__device__ __forceinline__ int sum_upto(int v)
{
    v += (int)dpp<0x111>((uint32_t)v);
    v += (int)dpp<0x112>((uint32_t)v);
    v += (int)dpp<0x114>((uint32_t)v);
    v += (int)dpp<0x118>((uint32_t)v);
#pragma unroll
    for (int d = 16; d < L; d <<= 1) {
        const int before = __builtin_amdgcn_ds_bpermute(((__lane_id() & ~(d - 1)) - 1) << 2, v);
        v += __lane_id() & d ? before : 0;
    }
    return v;
}

// The lanes of this lane's L that are set in `lanes`, from bit 0 on.
template <int L>
__device__ __forceinline__ uint64_t own_lanes(uint64_t lanes)
{
    if constexpr (L == 64)
        return lanes;
    const uint32_t half = __lane_id() & 32 ? (uint32_t)(lanes >> 32) : (uint32_t)lanes;
    return L == 32 ? half : half >> (__lane_id() & 16) & 0xffffu;
}

template <int B, int E, class F>
__device__ __forceinline__ void static_for(F &&f)
{
    if constexpr (B < E) {
        f(std::integral_constant<int, B>{});
        static_for<B + 1, E>(f);
    }
}

// What is chosen by: a number that orders like the value, 0 for what is not
// eligible.  Two words for an fp64 value, the second 0 for an fp32 one.
struct Key {
    uint32_t hi, lo;
};
__device__ __forceinline__ Key key_of(float v) // of a number, or -infinity
{
    const uint32_t b = __builtin_bit_cast(uint32_t, v);
    return {v == -__builtin_inff() ? 0u : b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u), 0u};
}
__device__ __forceinline__ Key key_of(double v)
{
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint64_t k = v == -__builtin_inf() ? 0u : b ^ ((uint64_t)((int64_t)b >> 63) | 0x8000000000000000u);
    return {(uint32_t)(k >> 32), (uint32_t)k};
}

// The lowest of the L lanes with the largest key, from 0; -1 where none is
// eligible.  TWO: keys of two words; the second is looked at where a token of
// the wave needs it.
template <int L, bool TWO>
__device__ __forceinline__ int best_lane(const Key &k)
{
    const uint32_t hi = most_of<L>(k.hi);
    bool top = k.hi == hi && hi != 0;
    uint64_t own = own_lanes<L>(__ballot(top));
    if (TWO && __any((own & (own - 1)) != 0)) {
        // (by all lanes, so not behind `top &&`: moves between lanes read nothing
        // from lanes that are switched off)
        const uint32_t mine = top ? k.lo : 0u, lo = most_of<L>(mine);
        top = top && mine == lo;
        own = own_lanes<L>(__ballot(top));
    }
    return L == 64 ? __ffsll((unsigned long long)own) - 1 : __ffs((uint32_t)own) - 1;
}

__device__ __forceinline__ double shfl_xor_f64(double v, int mask)
{
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = shfl_xor_u32((uint32_t)b, mask), hi = shfl_xor_u32((uint32_t)(b >> 32), mask);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

template <int CTRL>
__device__ __forceinline__ double dpp_f64(double v)
{
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = dpp<CTRL>((uint32_t)b), hi = dpp<CTRL>((uint32_t)(b >> 32));
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

template <int L>
__device__ __forceinline__ double sum_of(double v)
{
    v += dpp_f64<kXor1>(v);
    v += dpp_f64<kXor2>(v);
    v += dpp_f64<kHalfMirror>(v);
    v += dpp_f64<kMirror>(v);
    if constexpr (L >= 32)
        v += shfl_xor_f64(v, 16);
    if constexpr (L >= 64)
        v += shfl_xor_f64(v, 32);
    return v;
}

// exp(x) for x from kLeast to 0, subnormal results included.  x = n ln 2
// + r with ln 2 in two parts (Cody and Waite's reduction), and exp(r) by its
// series up to r^13 (|r| < 0.347: what is left out is below 2^-57).  The library's
// function and its division took more than twice as long.
constexpr double kLeast = -747.0; // (exp(-745.2) rounds to 0; larger |x| would leave n's range)
__device__ __forceinline__ double exp_f64(double x)
{
    constexpr double kSeries[14] = {1.0, 1.0, 1.0 / 2, 1.0 / 6, 1.0 / 24, 1.0 / 120, 1.0 / 720, 1.0 / 5040, 1.0 / 40320,
                                    1.0 / 362880, 1.0 / 3628800, 1.0 / 39916800, 1.0 / 479001600, 1.0 / 6227020800};
    const double n = rint(x * 1.4426950408889634);
    const double r = fma(n, -1.9082149292705877e-10, fma(n, -0.6931471803691238, x));
    double p = kSeries[13];
#pragma unroll
    for (int i = 12; i >= 0; --i)
        p = fma(p, r, kSeries[i]);
    return __builtin_amdgcn_ldexp(p, (int)n);
}

// 1 / (1 + exp(-x)), for negative x as exp(x) / (1 + exp(x)), which keeps its bits
// where exp(-x) leaves the range: the reciprocal by two steps of Newton's
// iteration from the hardware's estimate.
__device__ __forceinline__ double sigmoid_f64(double x)
{
    const double e = exp_f64(fmax(-fabs(x), kLeast)), d = 1.0 + e;
    double r = __builtin_amdgcn_rcp(d);
    r = fma(fma(-d, r, 1.0), r, r);
    r = fma(fma(-d, r, 1.0), r, r);
    return x < 0.0 ? e * r : r;
}

template <int DT>
__device__ __forceinline__ float logit(const void *logits, int64_t at)
{
    if constexpr (DT == QW_F32)
        return static_cast<const float *>(logits)[at];
    else
        return from16(static_cast<const uint16_t *>(logits)[at], DT == QW_BF16);
}

__device__ __forceinline__ float eligible(float l)
{
    // a NaN is not; infinity counts as the largest number, and -0 as 0 (keys tell
    // them apart)
    return l > -__builtin_inff() ? fminf(l, 3.402823466e38f) + 0.0f : -__builtin_inff();
}

// Lanes that share a group of experts: neighbours, a power of two.
template <int L>
__device__ __forceinline__ int lanes_a_group(const RouteArgs &a)
{
    return 1 << (31 - __builtin_clz(L / a.groups));
}

// The largest and the second largest of a group's values; the lanes of the
// group each look at a share of them.
template <class T>
__device__ __forceinline__ void two_largest(const T *values, int size, int share, T &first, T &second)
{
    first = second = -__builtin_inf();
#pragma unroll 4
    for (int i = __lane_id() & (share - 1); i < size; i += share) {
        const T v = values[i];
        second = v > first ? first : (v > second ? v : second);
        first = v > first ? v : first;
    }
}
__device__ __forceinline__ float from_lane_xor(float v, int d) { return shfl_xor_f32(v, d); }
__device__ __forceinline__ double from_lane_xor(double v, int d) { return shfl_xor_f64(v, d); }
template <class T>
__device__ __forceinline__ void merge_largest(int share, T &first, T &second)
{
    for (int d = 1; d < share; d <<= 1) {
        const T f = from_lane_xor(first, d), s = from_lane_xor(second, d);
        const T low = f > first ? first : f;
        second = s > second ? s : second;
        second = low > second ? low : second;
        first = f > first ? f : first;
    }
}

// What the choice of a wave's tokens leaves in LDS: ids and logits of each
// token's experts, [top_k] each.
struct Chosen {
    int32_t *id;
    float *logit;
};

// The experts of the wave's tokens, one after the other, in fp64.  `choices`:
// this token's [experts] of LDS.
template <int DT, int L, int P>
__device__ __forceinline__ void choose_one_by_one(const RouteArgs &a, int64_t row, bool live, double most, double *choices,
                                                  const Chosen &chosen)
{
    const double kNone = -__builtin_inf();
    int lane = __lane_id() & (L - 1);
    __asm__ volatile("" : "+v"(lane)); // (as in choose)
    const int first = lane * P, end = min(first + P, a.experts);
    double total = 1.0;
    if (a.bias && !a.sigmoid) {
        double sum = 0.0;
#pragma unroll 1
        for (int e = first; e < end; ++e)
            sum += exp_f64(fmax((double)eligible(logit<DT>(a.logits, row + e)) - most, kLeast));
        total = sum_of<L>(sum);
    }
#pragma unroll 1
    for (int e = first; e < end; ++e) {
        const double l = (double)eligible(logit<DT>(a.logits, row + e));
        double c = l;
        if (a.bias) {
            const double v = (a.sigmoid ? sigmoid_f64(l) : exp_f64(fmax(l - most, kLeast)) / total) + (double)a.bias[e];
            c = l > kNone && v > kNone ? v : kNone; // (a NaN is not chosen)
        }
        choices[e] = live ? c : kNone;
    }
    __builtin_amdgcn_wave_barrier(); // (a wave's LDS accesses are in order)
    if (a.groups > 1) {
        const int size = a.experts / a.groups, share = lanes_a_group<L>(a), group = lane / share;
        double one, two;
        two_largest(choices + group * size, group < a.groups ? size : 0, share, one, two);
        merge_largest(share, one, two);
        Key score = key_of(a.bias && two > kNone ? one + two : one);
        if (lane % share || group >= a.groups)
            score = {0, 0};
        uint64_t kept = 0;
#pragma unroll 1
        for (int g = 0; g < a.top_groups; ++g) {
            const int at = best_lane<L, true>(score);
            kept |= at < 0 ? 0ull : 1ull << (at / share);
            score = lane == at ? (Key){0, 0} : score;
        }
        __builtin_amdgcn_wave_barrier();
#pragma unroll 1
        for (int e = first; e < end; ++e)
            if (!(kept >> (e / size) & 1))
                choices[e] = kNone;
        __builtin_amdgcn_wave_barrier();
    }
#pragma unroll 1
    for (int j = 0; j < a.top_k; ++j) {
        double best = kNone;
        int at = first;
#pragma unroll 1
        for (int e = first; e < end; ++e) {
            const double c = choices[e];
            at = c > best ? e : at;
            best = c > best ? c : best;
        }
        const int from = best_lane<L, true>(key_of(best));
        if (lane == from) {
            chosen.id[j] = at;
            chosen.logit[j] = eligible(logit<DT>(a.logits, row + at));
            choices[at] = kNone;
        } else if (from < 0 && lane == 0) {
            chosen.id[j] = -1;
        }
        __builtin_amdgcn_wave_barrier();
    }
}

// Four neighbouring logits or biases of a row of `count` (16-byte aligned rows
// where `whole`); beyond its end, any of it.
template <int DT>
__device__ __forceinline__ void load4(const void *values, int64_t row, int e, int count, bool whole, float (&v)[4])
{
    if (whole) {
        const int at = min(e, count - 4);
        if constexpr (DT == QW_F32) {
            const float4_t x = *reinterpret_cast<const float4_t *>(static_cast<const float *>(values) + row + at);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = x[i];
        } else {
            const u32x2_t x = *reinterpret_cast<const u32x2_t *>(static_cast<const uint16_t *>(values) + row + at);
            const uint32_t w[2] = {x.x, x.y};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = from16((uint16_t)(w[i / 2] >> (16 * (i % 2))), DT == QW_BF16);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = logit<DT>(values, row + min(e + i, count - 1));
    }
}

// The experts of the wave's tokens; L lanes each, P experts a lane: those of
// element i are (i / 4) 4 L + 4 lane + i % 4.  `scratch`: this token's
// scratch_of() numbers of LDS.
template <int DT, int L, int P>
__device__ __forceinline__ void choose(const RouteArgs &a, int64_t token, bool live, double *scratch, const Chosen &chosen)
{
    static_assert(P % 4 == 0, "fours");
    const float kNone = -__builtin_inff();
    int lane = __lane_id() & (L - 1);
    // (opaque: else all that depends on the lane alone moves out of the loop over
    // tokens into registers that are spilled, which took most of the time)
    __asm__ volatile("" : "+v"(lane));
    const int64_t row = (live ? token : 0) * a.experts;
    const bool whole = a.experts % 4 == 0;
    auto expert = [&](int i) { return i / 4 * 4 * L + 4 * lane + i % 4; };
    float l[P], b[P], c[P];
    // (all loads at once, without a branch around each)
#pragma unroll
    for (int i = 0; i < P; i += 4) {
        float v[4];
        load4<DT>(a.logits, row, expert(i), a.experts, whole, v);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            l[i + e] = v[e];
    }
#pragma unroll
    for (int i = 0; i < P; i += 4) {
        float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (a.bias)
            load4<QW_F32>(a.bias, 0, expert(i), a.experts, whole, v);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            b[i + e] = v[e];
    }
    float top = kNone, size_b = 0.0f;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        l[i] = live && expert(i) < a.experts ? eligible(l[i]) : kNone;
        top = fmaxf(top, l[i]);
        c[i] = l[i];
        if (a.bias) {
            const float v = times_sigmoid(1.0f, l[i]) + b[i];
            const bool in = l[i] > kNone && v > kNone;
            c[i] = in ? v : kNone;
            size_b = in ? fmaxf(size_b, fabsf(b[i])) : size_b;
        }
    }
    double most = 0.0; // softmax: the largest logit
    if (!a.sigmoid) {
        const uint32_t m = most_of<L>(key_of(top).hi);
        most = m ? (double)__builtin_bit_cast(float, m & 0x80000000u ? m ^ 0x80000000u : ~m) : 0.0;
    }
    bool slow = a.bias && !a.sigmoid; // (a choice needs the softmax's sum over all)
    // How far an fp32 choice may be off.  The sigmoid's error is below 2^-20: the
    // exponential's is at most 2^-23 (1 + 1.45 |x|) relative, on a term that
    // counts s (1 - s); the sum with the bias adds 2^-24 of it.
    float error = 0.0f;
    if (a.bias) {
        const uint32_t bits = most_of<L>(__builtin_bit_cast(uint32_t, size_b)); // (not negative: ordered as it is)
        error = 0x1p-18f * (1.0f + __builtin_bit_cast(float, bits));
        slow = slow || !(error < 0x1p60f); // (an infinite bias, or one whose sums may be, has no bounds)
    }
    if (a.groups > 1 && !slow) {
        const int size = a.experts / a.groups, share = lanes_a_group<L>(a), group = lane / share;
        // (exact: e + 1/2 is at least 1/2 from a multiple of size, and below 2^10)
        const float part = 1.0f / (float)size;
        auto group_of = [&](int e) { return (int)(((float)e + 0.5f) * part); };
        // (groups one number further apart than their size: in distinct banks)
        float *values = reinterpret_cast<float *>(scratch);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int e = expert(i);
            if (e < a.experts)
                values[e + group_of(e)] = c[i];
        }
        __builtin_amdgcn_wave_barrier(); // (a wave's LDS accesses are in order)
        float one, two;
        two_largest(values + group * (size + 1), group < a.groups ? size : 0, share, one, two);
        merge_largest(share, one, two);
        __builtin_amdgcn_wave_barrier();
        const bool counts = lane % share == 0 && group < a.groups;
        const float sum = a.bias && two > kNone ? one + two : one;
        Key score = counts ? key_of(sum) : (Key){0, 0};
        uint64_t kept = 0;
        uint32_t last = 0; // the lowest that was kept
#pragma unroll 1
        for (int g = 0; g < a.top_groups; ++g) {
            last = most_of<L>(score.hi);
            const int at = best_lane<L, false>(score);
            kept |= at < 0 ? 0ull : 1ull << (at / share);
            score = lane == at ? (Key){0, 0} : score;
        }
        if (a.bias) {
            // a group that was not kept may be as good as one that was: each sum
            // is off by twice the error and its own rounding
            const float lowest = __builtin_bit_cast(float, last & 0x80000000u ? last ^ 0x80000000u : ~last);
            const float off = 4.0f * error + 0x1p-22f * (fabsf(sum) + fabsf(lowest));
            slow = counts && !(kept >> group & 1) && last != 0 && sum > kNone && sum >= lowest - off;
        }
#pragma unroll
        for (int i = 0; i < P; ++i)
            c[i] = kept >> group_of(min(expert(i), a.experts - 1)) & 1 ? c[i] : kNone;
    }
    slow = __any(slow);
    if (!slow) {
        float own_top = kNone;
#pragma unroll
        for (int i = 0; i < P; ++i)
            own_top = fmaxf(own_top, c[i]);
        uint32_t m = key_of(own_top).hi, t = 0;
#pragma unroll 1
        for (int j = 0; j < a.top_k; ++j) {
            t = most_of<L>(m);
            const uint64_t own = own_lanes<L>(__ballot(m == t));
            m = (own & ((1ull << lane) - 1)) == 0 && m == t ? 0u : m; // the lowest lane's
        }
        // what may be a choice: all that are eligible, or those that reach the bound
        float least = -3.402823466e38f;
        if (t != 0) {
            const float kth = __builtin_bit_cast(float, t & 0x80000000u ? t ^ 0x80000000u : ~t);
            least = a.bias ? kth - 2.0f * error - 0x1p-22f * fabsf(kth) : kth;
        }
        uint32_t mask = 0; // of this lane's experts
#pragma unroll
        for (int i = 0; i < P; ++i)
            mask |= c[i] >= least ? 1u << i : 0u;
        const int mine = __popc(mask);
        const int upto = sum_upto<L>(mine); // experts of the list up to this lane's
        const int n = (int)most_of<L>((uint32_t)upto);
        slow = __any(n > kListed);
        if (!slow) {
            u32x4_t *list = reinterpret_cast<u32x4_t *>(scratch), *keys = list + kListed;
            const int first = upto - mine;
#pragma unroll
            for (int i = 0; i < P; ++i)
                if (mask >> i & 1)
                    list[first + __popc(mask & ((1u << i) - 1))] =
                        (u32x4_t){__builtin_bit_cast(uint32_t, (float)l[i]), __builtin_bit_cast(uint32_t, (float)b[i]),
                                  (uint32_t)expert(i), 0u};
            __builtin_amdgcn_wave_barrier();
            const int longest = __builtin_amdgcn_readfirstlane((int)most_of<64>((uint32_t)n));
#pragma unroll 1
            for (int at = lane; at < (longest < 16 ? 16 : longest); at += L) {
                const u32x4_t x = list[at];
                const uint32_t lb = x.x, bb = x.y;
                const float lf = __builtin_bit_cast(float, lb);
                const Key k = a.bias ? key_of(sigmoid_f64((double)lf) + (double)__builtin_bit_cast(float, bb)) : key_of(lf);
                keys[at] = at < n ? (u32x4_t){k.hi, k.lo, x.z, lb} : (u32x4_t){0u, 0u, 0u, 0u}; // (comes before nothing)
            }
            __builtin_amdgcn_wave_barrier();
            auto put = [&](const u32x4_t own, int place) {
                const uint32_t bits = own.w;
                if (place < a.top_k) {
                    chosen.id[place] = (int)own.z;
                    chosen.logit[place] = __builtin_bit_cast(float, bits);
                }
            };
            if (longest <= 16) {
                // one a lane: the others' come round by DPP (read from LDS by
                // every lane they took six times as long)
                const u32x4_t own = keys[lane & 15]; // (the same in every row of the token)
                int place = 0;
                static_for<1, 16>([&](auto turn) {
                    constexpr int kTurn = 0x120 + decltype(turn)::value; // row_ror
                    const uint32_t hi = dpp<kTurn>(own.x), lo = dpp<kTurn>(own.y), z = dpp<kTurn>(own.z);
                    place += hi > own.x || (hi == own.x && (lo > own.y || (lo == own.y && z < own.z))) ? 1 : 0;
                });
                if (lane < n)
                    put(own, place);
            } else {
#pragma unroll 1
                for (int at = lane; at - lane < longest; at += L) {
                    const u32x4_t own = keys[at < n ? at : 0];
                    int place = 0;
#pragma unroll 1
                    for (int o = 0; o < longest; ++o) {
                        const u32x4_t x = keys[o];
                        const bool more = x.x > own.x || (x.x == own.x && (x.y > own.y || (x.y == own.y && x.z < own.z)));
                        place += o < n && more ? 1 : 0;
                    }
                    if (at < n)
                        put(own, place);
                }
            }
            for (int j = n + lane; j < a.top_k; j += L)
                chosen.id[j] = -1;
        }
    }
    __builtin_amdgcn_wave_barrier();
    if (slow)
        choose_one_by_one<DT, L, P>(a, row, live, most, scratch, chosen);
    // the weights
    double total = 1.0; // softmax: the sum of exp(l - most)
    if (!a.sigmoid && !a.renormalize) {
        double sum = 0.0;
#pragma unroll 1
        for (int e = lane * P; e < min(lane * P + P, a.experts); ++e)
            sum += exp_f64(fmax((double)eligible(logit<DT>(a.logits, row + e)) - most, kLeast)); // (0 where there is none)
        total = sum_of<L>(sum);
    }
    __builtin_amdgcn_wave_barrier();
    const int id = live && lane < a.top_k ? chosen.id[lane] : -1; // (top_k <= L)
    const double v = id >= 0 ? (double)chosen.logit[lane] : 0.0;
    const double e = a.sigmoid ? sigmoid_f64(v) : exp_f64(fmax(v - most, kLeast));
    double w = id >= 0 ? e : 0.0;
    if (a.renormalize)
        total = sum_of<L>(w);
    w = total > 0.0 ? w / total * a.scale : 0.0;
    if (live && lane < a.top_k) {
        a.weights[token * a.top_k + lane] = (float)w;
        a.ids[token * a.top_k + lane] = id;
    }
}

// Inclusive sum over the workgroup (every thread takes part).
__device__ __forceinline__ int block_scan(int v, int *sums) // sums: a wave's each
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

// Lists the entries of this workgroup's tokens: `total` entries of expert tid
// (experts <= kThreads), `before` of them of earlier workgroups.  `at`:
// [kWaves][experts] of LDS.
__device__ __forceinline__ void list_entries(const RouteArgs &a, int before, int total, int *at)
{
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
    const int upto = block_scan(total, sums); // (with a barrier: `at` is clear)
    const int waves = (int)((chunks + per - 1) / (per > 0 ? per : 1)); // that have entries
    int id = lo + lane < hi ? a.ids[first + lo + lane] : -1;
    if (id >= 0)
        atomicAdd(&at[wave * a.experts + id], 1);
    for (int64_t i = lo + kWave + lane; i < hi; i += kWave) {
        const int e = a.ids[first + i];
        if (e >= 0)
            atomicAdd(&at[wave * a.experts + e], 1);
    }
    if (tid == kThreads - 1)
        used = upto;
    __syncthreads();
    if (tid < a.experts) {
        int next = upto - total + before;
#pragma unroll 4
        for (int w = 0; w < waves; ++w) {
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
        if (i0 != lo)
            id = i < hi ? a.ids[first + i] : -1;
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

// The list of a workgroup's tokens, from the counts of all.
__global__ __launch_bounds__(kThreads) void list_kernel(RouteArgs a)
{
    // [2 slices][stride]: sums of counts; then list_entries' [kWaves][experts]
    extern __shared__ int at[];
    const int tid = threadIdx.x;
    // The counts of the workgroups before this one and of all: four experts a
    // thread, the workgroups shared out to as many threads as there are.
    int before = 0, total = 0;
    const int stride = a.counts_stride, quads = stride / 4;
    const int slices = kThreads / quads < 32 ? kThreads / quads : 32; // (their sums fit in `at`)
    const int slice = tid / quads, quad = tid % quads;
    if (slice < slices) {
        int4v all = {0, 0, 0, 0}, mine = {0, 0, 0, 0};
        const int4v *rows = reinterpret_cast<const int4v *>(a.counts) + quad;
#pragma unroll 16
        for (int b = slice; b < a.blocks; b += slices) {
            const int4v n = rows[(int64_t)b * quads];
            all += n;
            mine += b < (int)blockIdx.x ? n : (int4v){0, 0, 0, 0};
        }
        *reinterpret_cast<int4v *>(at + (2 * slice) * stride + 4 * quad) = all;
        *reinterpret_cast<int4v *>(at + (2 * slice + 1) * stride + 4 * quad) = mine;
    }
    __syncthreads();
    if (tid < a.experts)
        for (int i = 0; i < slices; ++i) {
            total += at[2 * i * stride + tid];
            before += at[(2 * i + 1) * stride + tid];
        }
    __syncthreads();
    list_entries(a, before, total, at);
}

// Numbers of LDS that a token takes (an even count: 16 bytes): its experts'
// choices, or two lists.  (Room for the groups' values with their gaps, half as
// large and at most as many again, is among these.)
__host__ __device__ __forceinline__ int scratch_of(const RouteArgs &a)
{
    const int lists = 2 * kListed * 16 / (int)sizeof(double), choices = (a.experts + 1) / 2 * 2;
    return lists > choices ? lists : choices;
}

template <int DT, int L, int P>
__global__ __launch_bounds__(kThreads) void route_kernel(RouteArgs a)
{
    extern __shared__ double lds[];
    // the tokens' scratch; [tokens at once][top_k]: their experts, and as much:
    // the logits of these; counts [experts].  With one workgroup for all tokens,
    // then list_entries' places.
    constexpr int kTokens = kThreads / L; // at once
    const int each = scratch_of(a), tid = threadIdx.x, slot = tid / L, lane = tid & (L - 1);
    int *ids = reinterpret_cast<int *>(lds + kTokens * each), *counts = ids + kTokens * 2 * a.top_k;
    const Chosen chosen = {ids + slot * a.top_k, reinterpret_cast<float *>(ids + (kTokens + slot) * a.top_k)};
    for (int e = tid; e < a.experts; e += kThreads)
        counts[e] = 0;
    __syncthreads();
    const int64_t begin = (int64_t)blockIdx.x * a.tokens_a_block;
    const int64_t end = begin + a.tokens_a_block < a.tokens ? begin + a.tokens_a_block : a.tokens;
    for (int64_t t0 = begin; t0 < end; t0 += kTokens) {
        const int64_t token = t0 + slot;
        if (t0 + slot / (kWave / L) * (kWave / L) >= end)
            break; // (a wave without a token)
        choose<DT, L, P>(a, token, token < end, lds + slot * each, chosen);
        if (token < end && lane < a.top_k && chosen.id[lane] >= 0)
            atomicAdd(&counts[chosen.id[lane]], 1);
        __builtin_amdgcn_wave_barrier();
    }
    __syncthreads();
    if (a.blocks == 1) {
        const int total = tid < a.experts ? counts[tid] : 0;
        __syncthreads();
        list_entries(a, 0, total, reinterpret_cast<int *>(lds));
        return;
    }
    for (int e = tid; e < a.experts; e += kThreads)
        a.counts[(int64_t)blockIdx.x * a.counts_stride + e] = counts[e];
}

template <int DT, int L, int P>
hipError_t launch(const RouteArgs &a, hipStream_t stream)
{
    const size_t tokens = kThreads / L, places = (size_t)(kThreads / kWave) * a.experts * sizeof(int);
    if (a.blocks > 0) {
        size_t lds = tokens * scratch_of(a) * sizeof(double) + (tokens * 2 * a.top_k + a.experts) * sizeof(int);
        if (a.blocks == 1 && lds < places)
            lds = places;
        route_kernel<DT, L, P><<<dim3((unsigned)a.blocks), dim3(kThreads), lds, stream>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess || a.blocks == 1)
            return e;
    }
    // (2 slices of 4 quads each: at most 8 a thread; without tokens: the offsets)
    const size_t sums = 8 * (size_t)kThreads * sizeof(int);
    list_kernel<<<dim3(a.blocks > 0 ? (unsigned)a.blocks : 1u), dim3(kThreads), sums > places ? sums : places, stream>>>(a);
    return hipGetLastError();
}

// At least as many lanes a token as it has groups and places, and at most 8
// experts a lane.  Us, 16384 tokens of 256 experts with bias and groups: 16 lanes
// of 16 experts 120 (264 registers spilled) or, in workgroups of 512, 49; 32 of
// 8 30; 64 of 4 39.
template <int DT>
hipError_t launch_type(const RouteArgs &a, hipStream_t stream)
{
    const int least = a.groups > a.top_k ? a.groups : a.top_k;
    if (least <= 16 && a.experts <= 64)
        return launch<DT, 16, 4>(a, stream);
    if (least <= 16 && a.experts <= 128)
        return launch<DT, 16, 8>(a, stream);
    if (least <= 32 && a.experts <= 256)
        return launch<DT, 32, 8>(a, stream);
    return launch<DT, 64, 8>(a, stream);
}

} // namespace

// A multiple of 64, so that there are at most kMaxBlocks; up to 64 tokens are
// one workgroup's, which lists them too.
int64_t route_tokens_a_block(int64_t tokens)
{
    const int64_t per = (tokens + kMaxBlocks - 1) / kMaxBlocks;
    return tokens <= 64 ? 64 : (per + 63) / 64 * 64;
}

hipError_t launch_route_experts(const RouteArgs &a, int dtype, hipStream_t stream)
{
    if (dtype == QW_F32)
        return launch_type<QW_F32>(a, stream);
    return dtype == QW_F16 ? launch_type<QW_F16>(a, stream) : launch_type<QW_BF16>(a, stream);
}

} // namespace qw
