// kv_cache.hip -- the quantizing write into the paged int8 KV cache, and
// the read back.
//
// Write.  The new tokens of one call that fall into one block form a run
// (consecutive slots).  With o the run's first offset in the block, per head
//
//   S' = fp32(max |x| / 127) over the run (0 below 2^-100)
//   S  = o > 0 ? max(S_old, S') : S'
//   q  = clamp(round_half_even(fp32(x / S)), -127, 127)      (S = 0: 0)
//   q_kept = round_half_even(fp32(q_kept * fp32(S_old / S))) where S > S_old
//
// so a block's scale is the largest value that tokens brought since its offset
// 0 was written (also tokens that others have replaced since, as after rejected
// drafts), a token at offset 0 starts the block afresh, and nothing before the
// run is read unless the scale grows.
//
// Bound by HBM for prompts (2 bytes in, 1 byte out an element: 4 prompts of
// 4000 tokens, 8 heads of 128, in 26 us, 3.8 TB/s) and by latency for single
// tokens (64 of them: 4.5 us, of which a launch is about 4).  A run is read
// once, into the registers of a wave or of a workgroup, which hold it from
// the maximum to the codes (read twice, from L2 the second time, with windows
// of 16 tokens and general divisions: 62 us for those prompts).  Values are
// stored transposed: a lane packs 16 tokens of two channels into two 16-byte
// stores.
//
// This unit is compiled without floating-point contraction: codes and
// scales are bit-exact by the formulas above.
#include "kv_device.h"
#include "kv_internal.h"

namespace qw {

namespace {

constexpr int kThreads = 256;

template <int N>
struct Int {
    static constexpr int value = N;
};

// x / s correctly rounded, from the correctly rounded inverse of s: the
// residual of x * inverse is exact, and one step along it lands on the
// nearest float (tests/test_kv_quotient.py: scales from the floor up, each with
// every 11-bit significand of x and quotients of 2^-2 to 2^8; below, the code is
// 0 whatever the last bit).
// A third of a general division's instructions.
struct Scale {
    float s, inverse; // both 0 for a run of zeros
};

__device__ __forceinline__ uint32_t code_of(float x, Scale k)
{
    const float y = x * k.inverse;
    const float r = fminf(fmaxf(rintf(fmaf(fmaf(-y, k.s, x), k.inverse, y)), -127.0f), 127.0f);
    return (uint32_t)(int)r & 0xffu;
}

__device__ __forceinline__ uint32_t rescaled(uint32_t byte, float ratio)
{
    return (uint32_t)(int)rintf((float)(int8_t)byte * ratio) & 0xffu;
}

__device__ __forceinline__ uint32_t rescaled4(uint32_t w, float ratio)
{
    return rescaled(w & 0xffu, ratio) | rescaled(w >> 8 & 0xffu, ratio) << 8 | rescaled(w >> 16 & 0xffu, ratio) << 16 |
           rescaled(w >> 24, ratio) << 24;
}

// The low n bytes.
__device__ __forceinline__ uint32_t low_bytes(int n) { return n >= 4 ? ~0u : n > 0 ? (1u << (8 * n)) - 1 : 0u; }

// One run of `len` tokens from token t on, at offset `off` of block `blk`,
// for one head and for keys (VALUES false) or values, by NW waves (this one
// is `wave` of them).  MOST bounds the run: the block size, or 16 for a run
// within one segment of 16 places.  Its elements stay in registers from the
// maximum to the codes; loads beyond the run repeat its last token, so that
// they need no branch.
template <int DT, int D, int NW, int MOST, bool VALUES>
__device__ __forceinline__ void write_run(const KvCacheArgs &a, int64_t t, int64_t blk, int off, int len, int head, int wave, float *lds)
{
    const int lane = __lane_id();
    const int64_t block = int64_t(1) << a.block_shift;
    const int64_t stride = VALUES ? a.v_stride : a.k_stride;
    const uint16_t *x = (VALUES ? a.v : a.k) + t * stride + (int64_t)head * D;
    const int64_t bh = blk * a.kv_heads + head;
    int8_t *codes = (VALUES ? a.v_cache : a.k_cache) + bh * block * D;
    float *scale = (VALUES ? a.v_scales : a.k_scales) + bh;

    // keys: 16 bytes of a token a lane; values: two channels of 16 tokens a lane
    constexpr int LPT = D / 8, TPW = 64 / LPT; // lanes a token, tokens a wave
    constexpr int LPS = D / 2, SPW = 64 / LPS; // lanes a segment of 16 tokens, segments a wave
    constexpr int N = VALUES ? (MOST / 16 + NW * SPW - 1) / (NW * SPW) : MOST / (NW * TPW);
    constexpr int DWORDS = VALUES ? 16 : 4;
    const int unit = VALUES ? wave * SPW + lane / LPS : wave * TPW + lane / LPT;
    const int d = VALUES ? 2 * (lane & (LPS - 1)) : 8 * (lane & (LPT - 1));
    const int first = MOST == 16 ? off & ~15 : 0; // place of the first segment
    uint32_t raw[N][DWORDS];
#pragma unroll
    for (int n = 0; n < N; ++n) {
        if (VALUES) {
            const int lo = first + (n * NW * SPW + unit) * 16 - off;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const int i = lo + j < 0 ? 0 : lo + j < len ? lo + j : len - 1;
                raw[n][j] = *reinterpret_cast<const uint32_t *>(x + i * stride + d);
            }
        } else {
            const int at = n * NW * TPW + unit, i = at < len ? at : len - 1;
            const u32x4_t piece = *reinterpret_cast<const u32x4_t *>(x + i * stride + d);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                raw[n][j] = piece[j];
        }
    }
    const float was = off > 0 ? *scale : 0.0f;
    float top = 0.0f;
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int j = 0; j < DWORDS; ++j)
            top = fmaxf(top, fmaxf(fabsf(Act<DT>::lo(raw[n][j])), fabsf(Act<DT>::hi(raw[n][j]))));
    top = wave_max_f32(top);
    if (NW > 1) {
        if (lane == 0)
            lds[wave] = top;
        __syncthreads(); // after it every wave has read `was`
#pragma unroll
        for (int w = 0; w < NW; ++w)
            top = fmaxf(top, lds[w]);
    }
    float s = top / 127.0f;
    s = s < kKvScaleFloor ? 0.0f : s;
    const bool grow = s > was;
    s = grow ? s : was;
    const bool move = off > 0 && grow && was > 0.0f;
    const float ratio = move ? was / s : 1.0f;
    const Scale k = {s, s > 0.0f ? 1.0f / s : 0.0f};
    if (wave == 0 && lane == 0)
        *scale = s;

    if (!VALUES) {
        if (move)
            for (int i = (wave * 64 + lane) * 16; i < off * D; i += NW * 64 * 16) {
                u32x4_t *p = reinterpret_cast<u32x4_t *>(codes + i);
                const u32x4_t c = *p;
                *p = (u32x4_t){rescaled4(c.x, ratio), rescaled4(c.y, ratio), rescaled4(c.z, ratio),
                               rescaled4(c.w, ratio)};
            }
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int i = n * NW * TPW + unit;
            if (i < len) {
                u32x2_t c = {0, 0};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    c[e >> 1] |= (code_of(Act<DT>::lo(raw[n][e]), k) | code_of(Act<DT>::hi(raw[n][e]), k) << 8) << (16 * (e & 1));
                *reinterpret_cast<u32x2_t *>(codes + (int64_t)(off + i) * D + d) = c;
            }
        }
    } else {
        if (MOST == 16 && move)
            for (int lo = unit * 16; lo < first; lo += NW * SPW * 16)
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    u32x4_t *p = reinterpret_cast<u32x4_t *>(codes + (int64_t)(d + v) * block + lo);
                    const u32x4_t c = *p;
                    *p = (u32x4_t){rescaled4(c.x, ratio), rescaled4(c.y, ratio), rescaled4(c.z, ratio),
                                   rescaled4(c.w, ratio)};
                }
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int lo = first + (n * NW * SPW + unit) * 16;
            if (lo >= off + len || (!move && lo + 16 <= off))
                continue;
            int8_t *row0 = codes + (int64_t)d * block + lo, *row1 = row0 + block;
            u32x4_t c0 = {0, 0, 0, 0}, c1 = {0, 0, 0, 0};
            // codes before the run stay (at the new scale); places behind it
            // are not live, and keep what they hold
            if (lo < off || lo + 16 > off + len) {
                c0 = *reinterpret_cast<const u32x4_t *>(row0);
                c1 = *reinterpret_cast<const u32x4_t *>(row1);
                if (move && lo < off) {
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        const uint32_t live = low_bytes(off - lo - 4 * v);
                        c0[v] = (c0[v] & ~live) | (rescaled4(c0[v], ratio) & live);
                        c1[v] = (c1[v] & ~live) | (rescaled4(c1[v], ratio) & live);
                    }
                }
            }
            if (lo + 16 > off) {
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    uint32_t u = 0, w = 0;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        u |= code_of(Act<DT>::lo(raw[n][4 * v + j]), k) << (8 * j);
                        w |= code_of(Act<DT>::hi(raw[n][4 * v + j]), k) << (8 * j);
                    }
                    const uint32_t fresh = low_bytes(off + len - lo - 4 * v) & ~low_bytes(off - lo - 4 * v);
                    c0[v] = (c0[v] & ~fresh) | (u & fresh);
                    c1[v] = (c1[v] & ~fresh) | (w & fresh);
                }
            }
            *reinterpret_cast<u32x4_t *>(row0) = c0;
            *reinterpret_cast<u32x4_t *>(row1) = c1;
        }
    }
}

// Grid: windows of WIN tokens, heads, keys and values.  MOST: the block size,
// or 64 for 32 and 64.  A run within one segment is a wave's work (in decode
// every run is: a token), a longer one the workgroup's.
template <int DT, int D, int WIN, int MOST>
__global__ __launch_bounds__(kThreads) void kv_write_kernel(KvCacheArgs a)
{
    __shared__ float lds[2][kThreads / 64];
    const int lane = __lane_id(), wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int64_t t0 = (int64_t)blockIdx.x * WIN;
    const int head = blockIdx.y;
    const int64_t n_slots = a.num_blocks << a.block_shift;
    const int block = 1 << a.block_shift;

    // A run begins where the slot before is not the one below, or at a block's
    // start.  Slots outside the cache (-1: padding) belong to no run.
    const int64_t mine = t0 + lane;
    const bool here = lane < WIN && mine < a.tokens;
    const int32_t s = here ? a.slots[mine] : -1;
    const int32_t before = here && mine > 0 ? a.slots[mine - 1] : -2;
    const bool live = s >= 0 && s < n_slots;
    const bool leads = live && ((s & (block - 1)) == 0 || before != s - 1);
    const uint64_t leaders = __ballot(leads), breaks = __ballot(leads || !live);

    struct Run {
        int64_t slot;
        int off, len;
        bool brief;
    };
    auto run_at = [&](int l) {
        Run r;
        r.slot = __builtin_amdgcn_readlane(s, l);
        r.off = (int)(r.slot & (block - 1));
        const uint64_t rest = l < 63 ? breaks >> (l + 1) : 0;
        r.len = (rest ? __ffsll((unsigned long long)rest) : 64 - l);
        if (l + r.len >= WIN) { // it may go on behind the window
            const int most = block - r.off;
            for (int i = r.len; i < most; i += 64) {
                const int64_t at = t0 + l + i + lane;
                const bool same = i + lane < most && at < a.tokens && (int64_t)a.slots[at] == r.slot + i + lane;
                const uint64_t b = __ballot(same);
                const int more = ~b ? __ffsll((unsigned long long)~b) - 1 : 64;
                r.len += more;
                if (more < 64)
                    break;
            }
        }
        r.brief = (r.off & 15) + r.len <= 16;
        return r;
    };
    auto write = [&](auto waves, auto most, int l, const Run &r, int w, float *top) {
        if (blockIdx.z == 0)
            write_run<DT, D, decltype(waves)::value, decltype(most)::value, false>(a, t0 + l, r.slot >> a.block_shift, r.off, r.len,
                                                                                    head, w, top);
        else
            write_run<DT, D, decltype(waves)::value, decltype(most)::value, true>(a, t0 + l, r.slot >> a.block_shift, r.off, r.len,
                                                                                   head, w, top);
    };
    uint64_t longer = 0;
    int n = 0;
    for (uint64_t left = leaders; left; left &= left - 1) {
        const int l = __ffsll((unsigned long long)left) - 1;
        const Run r = run_at(l);
        if (MOST > 16 && !r.brief)
            longer |= uint64_t(1) << l;
        else if ((n++ & 3) == wave)
            write(Int<1>(), Int<16>(), l, r, 0, nullptr);
    }
    if constexpr (MOST > 16)
        for (n = 0; longer; longer &= longer - 1, ++n) {
            const int l = __ffsll((unsigned long long)longer) - 1;
            write(Int<kThreads / 64>(), Int<MOST>(), l, run_at(l), wave, lds[n & 1]);
        }
}

// Read: 64 tokens of one head a workgroup.  Key rows are contiguous; the
// codes of the values go through LDS, read with lanes over tokens (the
// contiguous direction in the cache) and written out with lanes over
// channels.  Rows of slots outside the cache are zero.
template <int DT, int D>
__global__ __launch_bounds__(kThreads) void kv_read_kernel(KvCacheArgs a)
{
    constexpr int LPT = D / 8;
    constexpr int PITCH = D + 4; // bytes: an odd number of banks between tokens
    __shared__ __attribute__((aligned(16))) uint8_t tile[64 * PITCH];
    const int tid = threadIdx.x, lane = __lane_id(), wave = tid >> 6;
    const int64_t t0 = (int64_t)blockIdx.x * 64;
    const int head = blockIdx.y;
    const int64_t n_slots = a.num_blocks << a.block_shift;
    const int64_t block = int64_t(1) << a.block_shift;
    const bool values = blockIdx.z != 0;

    if (values) {
        const int64_t t = t0 + lane;
        const int64_t s = t < a.tokens ? a.slots[t] : -1;
        if (s >= 0 && s < n_slots) {
            const int8_t *p = a.v_cache + ((s >> a.block_shift) * a.kv_heads + head) * block * D + (s & (block - 1));
#pragma unroll 8
            for (int d = wave * (D / 4); d < (wave + 1) * (D / 4); ++d)
                tile[lane * PITCH + d] = (uint8_t)p[d * block];
        }
        __syncthreads();
    }
    for (int i = tid / LPT; i < 64; i += kThreads / LPT) {
        const int64_t t = t0 + i;
        if (t >= a.tokens)
            break;
        const int d = (tid & (LPT - 1)) * 8;
        const int64_t s = a.slots[t];
        u32x2_t c = {0, 0};
        float scale = 0.0f;
        if (s >= 0 && s < n_slots) {
            const int64_t bh = (s >> a.block_shift) * a.kv_heads + head;
            scale = (values ? a.v_scales : a.k_scales)[bh];
            if (values) {
                c.x = *reinterpret_cast<const uint32_t *>(tile + i * PITCH + d);
                c.y = *reinterpret_cast<const uint32_t *>(tile + i * PITCH + d + 4);
            } else {
                c = *reinterpret_cast<const u32x2_t *>(a.k_cache + (bh * block + (s & (block - 1))) * D + d);
            }
        }
        float f[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            f[e] = (float)(int8_t)(c.x >> (8 * e) & 0xffu) * scale;
            f[4 + e] = (float)(int8_t)(c.y >> (8 * e) & 0xffu) * scale;
        }
        uint16_t *out = (values ? a.v + t * a.v_stride : a.k + t * a.k_stride) + (int64_t)head * D + d;
        *reinterpret_cast<u32x4_t *>(out) = pack8<DT>(f);
    }
}

template <int DT, int D, int WIN, int MOST>
void write_window(const KvCacheArgs &a, hipStream_t stream)
{
    kv_write_kernel<DT, D, WIN, MOST><<<dim3((unsigned)((a.tokens + WIN - 1) / WIN), (unsigned)a.kv_heads, 2), dim3(kThreads), 0, stream>>>(a);
}

template <int DT, int D, int MOST>
void write_block(const KvCacheArgs &a, hipStream_t stream)
{
    // Small windows suit single tokens, which a workgroup's waves take one after
    // the other, large ones long runs, whose further windows hold nothing to do
    // and cost a workgroup each.  Which of them the slots are the host cannot see;
    // their number says what they are likely to be, and between the two a middle
    // window is best for neither and bad for neither.  With windows of 4, 16 and
    // 64, us: 64 single tokens (2 heads of 128) 4.5, 10.6, 36, and 512 (8 heads) 14.7,
    // 17.1, 41; 2048 (2 heads) 13.0, 15.0, 39, and one prompt of 2000 (8 heads,
    // blocks of 16) 17.9, 6.3, 4.9; four prompts of 4000 (8 heads, blocks of 64) 166,
    // 44, 26.
    if (a.tokens <= 512)
        write_window<DT, D, 4, MOST>(a, stream);
    else if (a.tokens <= 4096)
        write_window<DT, D, 16, MOST>(a, stream);
    else
        write_window<DT, D, 64, MOST>(a, stream);
}

template <int DT, int D>
void write_dim(const KvCacheArgs &a, hipStream_t stream)
{
    if (a.block_shift == 4)
        write_block<DT, D, 16>(a, stream);
    else if (a.block_shift == 7)
        write_block<DT, D, 128>(a, stream);
    else
        write_block<DT, D, 64>(a, stream);
}

template <int DT, int D>
void read_dim(const KvCacheArgs &a, hipStream_t stream)
{
    kv_read_kernel<DT, D><<<dim3((unsigned)((a.tokens + 63) / 64), (unsigned)a.kv_heads, 2), dim3(kThreads), 0, stream>>>(a);
}

} // namespace

hipError_t launch_kv_write(const KvCacheArgs &a, int dtype, hipStream_t stream)
{
    if (a.head_dim == 64)
        dtype == QW_F16 ? write_dim<QW_F16, 64>(a, stream) : write_dim<QW_BF16, 64>(a, stream);
    else if (a.head_dim == 128)
        dtype == QW_F16 ? write_dim<QW_F16, 128>(a, stream) : write_dim<QW_BF16, 128>(a, stream);
    else
        return hipErrorInvalidValue;
    return hipGetLastError();
}

hipError_t launch_kv_read(const KvCacheArgs &a, int dtype, hipStream_t stream)
{
    if (a.head_dim == 64)
        dtype == QW_F16 ? read_dim<QW_F16, 64>(a, stream) : read_dim<QW_BF16, 64>(a, stream);
    else if (a.head_dim == 128)
        dtype == QW_F16 ? read_dim<QW_F16, 128>(a, stream) : read_dim<QW_BF16, 128>(a, stream);
    else
        return hipErrorInvalidValue;
    return hipGetLastError();
}

} // namespace qw
