// ff_api.hip -- the C ABI of the feed-forward operators: argument checks on the
// host, kernel selection, launch on the caller's stream.  Nothing is allocated
// here, and a rejected call launches nothing and writes nothing.
#include <float.h>
#include <math.h>
#include <stdint.h>

#include "ff_internal.h"

namespace {

constexpr int64_t kMaxDim = 0x7fffffff;
constexpr int64_t kSkinnyPartsMaxK = 1 << 30; // (its loads ahead count past k in 32 bits)

bool off16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
bool off4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }

bool meet(const void *a, uint64_t na, const void *b, uint64_t nb)
{
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
    return a && b && na && nb && pa < pb + nb && pb < pa + na;
}

qw_status status_of(hipError_t e) { return e == hipSuccess ? QW_SUCCESS : QW_ERROR_LAUNCH; }

bool known_tile(int tile, bool a8)
{
    return tile == 256256 || tile == 256128 || tile == 256064 || (tile == 128128 && !a8) || tile == 128064;
}

// Parts to split the reduction of a ping-pong grid into: as many as fill the
// CUs, at most 8, where its tiles cover at most half of them and the reduction
// is long.  The accumulators' way to memory and back, and the second launch,
// cost some 20 to 40 us with all CUs at work.  Us, best tile without a split /
// split, n = 4096, k = 4096, 6144, 8192, 13696, 20480: W8A8 256 rows 25 / 33, 37 /
// 31, 61 / 35, 93 / 44, 143 / 61; 512 rows 26 / 45, 39 / 48, 63 / 54, 94 / 57, 146 / 73;
// 2048 rows 57 / 60, 90 / 78, 112 / 92, 173 / 131, 268 / 184; W8A16 256 rows 34 / 36,
// 47 / 36, 70 / 42, 139 / 55, 206 / 75; 512 rows 35 / 44, 56 / 51, 71 / 57, 139 / 75,
// 206 / 96; 2048 rows 82 / 85, 119 / 111, 151 / 137, 245 / 211, 361 / 301.  (Of
// other n nothing was measured; W8A8 with 256 rows and k = 6144 would gain and is
// left out.)
int split_parts(int64_t m, int64_t n, int64_t k, bool gated, bool a8)
{
    const int64_t columns = gated ? n / 2 : n, bn = gated ? 128 : 256;
    const int64_t tiles = ((m + 255) / 256) * ((columns + bn - 1) / bn), cus = qw::device_cu_count();
    if (k < (a8 ? 8192 : 6144) || 2 * tiles > cus)
        return 1;
    return (int)(cus / tiles < 8 ? cus / tiles : 8);
}

// The same for a few rows on the skinny kernel: as many parts as give each CU a
// workgroup of 64 weight rows (gated: 128) that share the activations.  The second
// launch costs about 3 us, and what is saved are reads of all activations for
// every 16 or 32 weight rows, so these decide.  Us without / with parts: fp16, 16
// rows (activations of 256 KB from k = 8192) 4096 x 4096 9 / 10, 2048 x 8192 12.5 /
// 10.3, 8192 x 8192 22 / 18, 4096 x 13696 22 / 19, 8192 x 28672 54 / 43; 8 rows 4096 x
// 13696 16 / 18; 32 rows 4096 x 4096 12.9 / 11.5, 4096 x 13696 33 / 21, gated 16384 x
// 4096 25 / 23; W8A8 32 rows 4096 x 4096 10.1 / 10.4, 4096 x 13696 23 / 20.
int skinny_parts(int64_t m, int64_t n, int64_t k, bool gated, bool a8)
{
    const int64_t wide = gated ? 128 : 64, tiles = (n + wide - 1) / wide, cus = qw::device_cu_count();
    if (m <= 4 || m > 32 || m * k * (a8 ? 1 : 2) < (1 << 18) || k > kSkinnyPartsMaxK || 2 * tiles > cus)
        return 1;
    return (int)(cus / tiles < 8 ? cus / tiles : 8);
}

// The kernel, tile and parts of a linear call: a tuning record of the plain
// product's bucket, else its rule, where the kernel takes the sizes; parts for the
// skinny kernel, and without a record for a ping-pong grid, where they gain.
struct LinearPlan {
    int path, tile, splits;
};

LinearPlan plan_linear(int64_t m, int64_t n, int64_t k, bool gated, bool a8)
{
    const int tuned = qw::tuned_choice(m, n, k, a8);
    LinearPlan p = {tuned >= 0 ? tuned / qw::kChoicePath : qw::auto_path(m, n, k), tuned >= 0 ? tuned % qw::kChoicePath : 0, 1};
    if (p.path == QW_PATH_GEMV && (a8 || !qw::gemv_linear_supported(m, k, gated)))
        p.path = QW_PATH_SKINNY;
    if (p.path == QW_PATH_SKINNY && m > 16 * 65535)
        p.path = QW_PATH_MFMA;
    if (p.path == QW_PATH_MFMA && !qw::mfma_linear_supported(n, k, gated))
        p.path = QW_PATH_SKINNY;
    if (p.path != QW_PATH_MFMA || (p.tile == 256256 && k > qw::kPingPongMaxK) || !known_tile(p.tile, a8))
        p.tile = 0;
    if (p.path == QW_PATH_SKINNY)
        p.splits = skinny_parts(m, n, k, gated, a8);
    // (where rounding m up to 256 rows costs at most a tenth over 64, as for the
    // ping-pong tile without a split.  The split would gain beyond: n = 4096, k =
    // 13696, 64 to 192 rows 90 us, in 8 parts 44 to 47, W8A8 61 and 33)
    const int64_t rows256 = (m + 255) / 256 * 256, rows64 = (m + 63) / 64 * 64;
    if (p.path == QW_PATH_MFMA && p.tile == 0 && k <= qw::kPingPongMaxK && 10 * rows256 <= 11 * rows64) {
        p.splits = split_parts(m, n, k, gated, a8);
        if (p.splits > 1)
            p.tile = 256256;
    }
    return p;
}

int64_t split_bytes(const LinearPlan &p, int64_t m, int64_t n, int64_t k, bool gated)
{
    return p.path == QW_PATH_SKINNY ? qw::skinny_parts_bytes(m, n, k, gated, p.splits) : qw::mfma_split_bytes(m, n, p.splits);
}

int64_t linear_workspace(int64_t m, int64_t n, int64_t k, int gated, bool a8)
{
    if (m < 0 || n < 0 || k <= 0 || (gated != 0 && gated != 1) || (gated && n % 2) || k % 16 != 0 || m > kMaxDim || n > kMaxDim ||
        k > (a8 ? (int64_t)QW_W8A8_MAX_K : kMaxDim))
        return -1;
    if (m == 0 || n == 0)
        return 0;
    const LinearPlan p = plan_linear(m, n, k, gated != 0, a8);
    return p.splits > 1 ? split_bytes(p, m, n, k, gated != 0) : 0;
}

qw_status linear(qw::LinearArgs a, int dtype, int gated, LinearPlan p, void *workspace, int64_t workspace_bytes, void *stream)
{
    const bool a8 = a.sx != nullptr;
    if (p.path != QW_PATH_AUTO && p.path != QW_PATH_MFMA && p.path != QW_PATH_SKINNY && (a8 || p.path != QW_PATH_GEMV))
        return QW_ERROR_INVALID_VALUE;
    if (p.tile != 0 && (p.path != QW_PATH_MFMA || !known_tile(p.tile, a8)))
        return QW_ERROR_INVALID_VALUE;
    if (p.splits < 1 || p.splits > 64 || (p.splits > 1 && p.tile != 256256 && p.path != QW_PATH_SKINNY) || workspace_bytes < 0 ||
        (workspace == nullptr && workspace_bytes > 0))
        return QW_ERROR_INVALID_VALUE;
    if (a.m < 0 || a.n < 0 || a.k <= 0 || (gated != 0 && gated != 1) || (gated && a.n % 2) ||
        a.ep.activation < QW_ACT_NONE || a.ep.activation > QW_ACT_SILU || (dtype != QW_F16 && dtype != QW_BF16))
        return QW_ERROR_INVALID_VALUE;
    if (a.m == 0 || a.n == 0)
        return QW_SUCCESS;
    if (!a.x || !a.q || !a.scales || !a.y)
        return QW_ERROR_INVALID_VALUE;
    if (a.k % 16 != 0 || a.m > kMaxDim || a.n > kMaxDim || a.k > (a8 ? (int64_t)QW_W8A8_MAX_K : kMaxDim))
        return QW_ERROR_UNSUPPORTED;
    if (off16(a.x) || off16(a.sx) || off16(a.q) || off16(a.scales) || off16(a.ep.bias) || off16(a.ep.residual) || off16(a.y))
        return QW_ERROR_MISALIGNED;
    a.gated = gated != 0;
    a.ep.bf16 = dtype == QW_BF16;
    const uint64_t m = (uint64_t)a.m, n = (uint64_t)a.n, k = (uint64_t)a.k;
    const uint64_t ybytes = m * (gated ? n / 2 : n) * 2u;
    if (meet(a.y, ybytes, a.x, m * k * (a8 ? 1u : 2u)) || meet(a.y, ybytes, a.sx, m * 2u) || meet(a.y, ybytes, a.q, n * k) ||
        meet(a.y, ybytes, a.scales, n * 2u) || meet(a.y, ybytes, a.ep.bias, n * 2u) ||
        (a.ep.residual != a.y && meet(a.y, ybytes, a.ep.residual, ybytes)))
        return QW_ERROR_INVALID_VALUE;
    if (p.path == QW_PATH_AUTO) {
        p = plan_linear(a.m, a.n, a.k, a.gated, a8);
        if (p.splits > 1 && workspace == nullptr)
            p.splits = 1, p.tile = 0; // (a caller may do without)
    }
    if (p.splits > 1) {
        const int64_t need = split_bytes(p, a.m, a.n, a.k, a.gated);
        if (workspace == nullptr || workspace_bytes < need)
            return QW_ERROR_INVALID_VALUE;
        if (off16(workspace))
            return QW_ERROR_MISALIGNED;
        const void *used[7] = {a.x, a.sx, a.q, a.scales, a.ep.bias, a.ep.residual, a.y};
        const uint64_t size[7] = {m * k * (a8 ? 1u : 2u), m * 2u, n * k, n * 2u, n * 2u, ybytes, ybytes};
        for (int i = 0; i < 7; ++i)
            if (meet(workspace, (uint64_t)need, used[i], size[i]))
                return QW_ERROR_INVALID_VALUE;
    }
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (p.path == QW_PATH_GEMV) {
        if (!qw::gemv_linear_supported(a.m, a.k, a.gated))
            return QW_ERROR_UNSUPPORTED;
        return status_of(qw::launch_gemv_linear(static_cast<const uint16_t *>(a.x), a.q, a.scales, a.ep, a.gated, a.y, a.m, a.n,
                                                a.k, s));
    }
    if (p.path == QW_PATH_SKINNY) {
        if (a.m > 16 * 65535 || (p.splits > 1 && (a.k < 64 * p.splits || a.k > kSkinnyPartsMaxK)))
            return QW_ERROR_UNSUPPORTED;
        return status_of(p.splits > 1 ? qw::launch_skinny_parts(p.splits, a, workspace, s) : qw::launch_skinny_linear(a, s));
    }
    if (!qw::mfma_linear_supported(a.n, a.k, a.gated) || (p.tile == 256256 && a.k > qw::kPingPongMaxK) ||
        (p.splits > 1 && a.k < 64 * p.splits))
        return QW_ERROR_UNSUPPORTED;
    if (p.splits > 1)
        return status_of(a8 ? qw::launch_mfma_split_a8(p.splits, a, workspace, s) : qw::launch_mfma_split(p.splits, a, workspace, s));
    if (p.tile == 0)
        p.tile = a8 ? qw::w8a8_tile_choice(a.m, a.n, a.k) : qw::mfma_tile_choice(a.m, a.n, a.k);
    return status_of(a8 ? qw::launch_mfma_linear_a8(p.tile, a, s) : qw::launch_mfma_linear(p.tile, a, s));
}

// The tile for a mean number of entries an expert.  A tile's rows belong to one
// expert, so half a tile of each is in vain on average.  Us, 64 experts of 2048
// (gated) by 2048, mean 16 / 64 / 128 / 384: 128 x 64 72 / 86 / 125 / 280, 256 x
// 64 72 / 89 / 116 / 258, 256 x 128 98 / 108 / 125 / 248, 256 x 256 144 / 148 /
// 156 / 272; 128 of 1536 by 2048, mean 16 / 32 / 128 / 256: 91 / 94 / 179 / 291,
// 100 / 104 / 172 / 272, 119 / 119 / 179 / 259; 8 of 8192 by 4096, mean 512 / 2048:
// 256 x 128 350 / 1076, 256 x 256 384 / 1046.  Up to 12 entries the skinny kernel:
// mean 4 / 8 / 12 / 16 of the first 44 / 55 / 65 / 77.
int experts_tile(int64_t mean, int64_t k)
{
    if (mean >= 1536 && k <= qw::kPingPongMaxK)
        return 256256;
    return mean >= 192 ? 256128 : mean >= 96 ? 256064 : 128064;
}

struct Span {
    const void *p;
    uint64_t n;
};
bool meet(Span a, Span b) { return meet(a.p, a.n, b.p, b.n); }

// Rows of k 16-bit elements, `stride` apart.
Span rows_of(const void *p, int64_t stride, int64_t k, int64_t count)
{
    return {p, (uint64_t)((count - 1) * stride + k) * 2u};
}

// Whether rows share an element: rows of one stride may lie between each other
// (the columns of one matrix).
bool rows_meet(const void *a, int64_t a_stride, const void *b, int64_t b_stride, int64_t k, int64_t count)
{
    if (!meet(rows_of(a, a_stride, k, count), rows_of(b, b_stride, k, count)))
        return false;
    if (a_stride != b_stride)
        return true;
    const int64_t bytes = a_stride * 2;
    const int64_t d = (int64_t)(reinterpret_cast<uintptr_t>(b) - reinterpret_cast<uintptr_t>(a));
    const int64_t shift = ((d % bytes) + bytes) % bytes; // b's column from a's
    return shift < k * 2 || shift + k * 2 > bytes;
}

qw_status add_norm(qw::AddNormArgs a, int dtype, double eps, bool codes, void *stream)
{
    if ((dtype != QW_F16 && dtype != QW_BF16) || a.tokens < 0 || a.k <= 0 || !(eps >= 0.0) || !isfinite(eps))
        return QW_ERROR_INVALID_VALUE;
    if ((a.residual == nullptr) != (a.h == nullptr) && a.tokens > 0)
        return QW_ERROR_INVALID_VALUE;
    if (a.tokens == 0)
        return QW_SUCCESS;
    const bool added = a.residual != nullptr;
    if (!added)
        a.residual_stride = a.h_stride = a.x_stride;
    if (!a.x || !a.weight || (codes ? !a.q || !a.scales : !a.y) || a.x_stride < a.k || a.residual_stride < a.k ||
        a.h_stride < a.k)
        return QW_ERROR_INVALID_VALUE;
    if (a.k % 16 != 0 || a.k > QW_QUANTIZE_MAX_K || a.tokens > kMaxDim || a.x_stride % 8 || a.residual_stride % 8 ||
        a.h_stride % 8 || a.x_stride > kMaxDim || a.residual_stride > kMaxDim || a.h_stride > kMaxDim)
        return QW_ERROR_UNSUPPORTED;
    if (off16(a.x) || off16(a.residual) || off16(a.weight) || off16(a.h) || off16(a.y) || off16(a.q) || off16(a.scales))
        return QW_ERROR_MISALIGNED;
    const int64_t T = a.tokens, k = a.k;
    const Span weight = {a.weight, (uint64_t)k * 2u}, x = rows_of(a.x, a.x_stride, k, T);
    const Span res = added ? rows_of(a.residual, a.residual_stride, k, T) : Span{nullptr, 0};
    const Span h = added ? rows_of(a.h, a.h_stride, k, T) : Span{nullptr, 0};
    const Span out = codes ? Span{a.q, (uint64_t)T * (uint64_t)k} : Span{a.y, (uint64_t)T * (uint64_t)k * 2u};
    const Span scales = codes ? Span{a.scales, (uint64_t)T * 2u} : Span{nullptr, 0};
    if (meet(out, x) || meet(out, res) || meet(out, weight) || meet(out, h) || meet(out, scales) || meet(scales, x) ||
        meet(scales, res) || meet(scales, weight) || meet(scales, h) || meet(h, weight))
        return QW_ERROR_INVALID_VALUE;
    if (added) {
        const bool on_x = a.h == a.x && a.h_stride == a.x_stride;
        const bool on_res = a.h == a.residual && a.h_stride == a.residual_stride;
        if ((!on_x && rows_meet(a.h, a.h_stride, a.x, a.x_stride, k, T)) ||
            (!on_res && rows_meet(a.h, a.h_stride, a.residual, a.residual_stride, k, T)))
            return QW_ERROR_INVALID_VALUE;
    }
    // (an eps that binary32 loses still keeps a row of zeros from 0 / 0)
    a.eps = eps > 0.0 && eps < FLT_MIN ? FLT_MIN : (float)eps;
    return status_of(qw::launch_add_rms_norm(a, dtype, static_cast<hipStream_t>(stream)));
}

bool route_sizes_ok(int64_t tokens, int64_t experts, int64_t top_k)
{
    return experts <= QW_MAX_EXPERTS && top_k <= QW_MAX_TOP_K && tokens <= kMaxDim / top_k;
}

int64_t route_blocks(int64_t tokens)
{
    const int64_t per = qw::route_tokens_a_block(tokens);
    return (tokens + per - 1) / per;
}

int64_t route_workspace(int64_t tokens, int64_t experts) { return route_blocks(tokens) * ((experts + 3) / 4) * 16; }

qw_status experts_product(const uint16_t *x, int64_t x_rows, int gather, const int8_t *q, const uint16_t *scales,
                          const uint16_t *bias, int activation, int gated, const int32_t *offsets, const int32_t *rows,
                          int64_t entries, int64_t top_k, void *y, bool f32, int64_t experts, int64_t n, int64_t k, int path,
                          int tile, void *stream)
{
    if ((path != QW_PATH_AUTO && path != QW_PATH_SKINNY && path != QW_PATH_MFMA) ||
        (tile != 0 && (path != QW_PATH_MFMA || !known_tile(tile, false) || tile == 128128)))
        return QW_ERROR_INVALID_VALUE;
    if (x_rows < 0 || entries < 0 || n < 0 || k <= 0 || experts < 1 || top_k < 1 || (gather != 0 && gather != 1) ||
        (!gather && x_rows != entries) || (gated != 0 && gated != 1) || (gated && n % 2) || activation < QW_ACT_NONE ||
        activation > QW_ACT_SILU)
        return QW_ERROR_INVALID_VALUE;
    if (entries == 0 || n == 0)
        return QW_SUCCESS;
    if ((!x && x_rows > 0) || !q || !scales || !offsets || (gather && !rows) || !y)
        return QW_ERROR_INVALID_VALUE;
    if (k % 16 != 0 || experts > QW_MAX_EXPERTS || entries > kMaxDim || x_rows > kMaxDim || n > kMaxDim || top_k > kMaxDim ||
        k > QW_MFMA_MAX_K || n * k >= int64_t(1) << 32 || (gather && (x_rows + 1) * k >= int64_t(1) << 31) ||
        (path == QW_PATH_SKINNY && entries > (1 << 19)) || (tile == 256256 && k > qw::kPingPongMaxK))
        return QW_ERROR_UNSUPPORTED;
    if (off16(x) || off16(q) || off16(scales) || off16(bias) || off16(y) || off4(offsets) || off4(rows))
        return QW_ERROR_MISALIGNED;
    const uint64_t E = (uint64_t)experts, un = (uint64_t)n, uk = (uint64_t)k;
    const Span out = {y, (uint64_t)entries * (gated ? un / 2 : un) * (f32 ? 4u : 2u)};
    if (meet(out, {x, (uint64_t)x_rows * uk * 2u}) || meet(out, {q, E * un * uk}) || meet(out, {scales, E * un * 2u}) ||
        meet(out, {bias, E * un * 2u}) || meet(out, {offsets, (E + 1) * 4u}) || meet(out, {rows, (uint64_t)entries * 4u}))
        return QW_ERROR_INVALID_VALUE;
    const qw::LinearArgs a = {x, nullptr, q, scales, {bias, nullptr, activation, 0}, gated != 0, static_cast<uint16_t *>(y), entries, n, k};
    const qw::Experts ex = {offsets, gather ? rows : nullptr, (int)experts, (int)entries, (int)x_rows, (int)top_k};
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (path == QW_PATH_AUTO)
        path = entries <= 12 * experts && entries <= (1 << 19) ? QW_PATH_SKINNY : QW_PATH_MFMA;
    if (path == QW_PATH_SKINNY)
        return status_of(qw::launch_skinny_experts(a, ex, f32, s));
    if (tile == 0)
        tile = experts_tile(entries / experts, k);
    return status_of(qw::launch_mfma_experts(tile, a, ex, f32, s));
}

qw_status combine(const void *y, bool f32, int64_t entries, const int32_t *places, const float *weights, int64_t tokens,
                  int64_t top_k, const uint16_t *residual, uint16_t *out, int64_t n, void *stream)
{
    if (entries < 0 || tokens < 0 || top_k < 1 || n < 0)
        return QW_ERROR_INVALID_VALUE;
    if (tokens == 0 || n == 0)
        return QW_SUCCESS;
    if ((!y && entries > 0) || !places || !weights || !out)
        return QW_ERROR_INVALID_VALUE;
    if (entries > kMaxDim || tokens > kMaxDim || top_k > kMaxDim || n > kMaxDim || tokens > (int64_t(1) << 40) / n)
        return QW_ERROR_UNSUPPORTED;
    if (off16(y) || off16(residual) || off16(out) || off4(places) || off4(weights))
        return QW_ERROR_MISALIGNED;
    const uint64_t t = (uint64_t)tokens, un = (uint64_t)n;
    const Span to = {out, t * un * 2u};
    if (meet(to, {y, (uint64_t)entries * un * (f32 ? 4u : 2u)}) || meet(to, {places, t * (uint64_t)top_k * 4u}) ||
        meet(to, {weights, t * (uint64_t)top_k * 4u}) || (residual != out && meet(to, {residual, t * un * 2u})))
        return QW_ERROR_INVALID_VALUE;
    const qw::CombineArgs a = {y, places, weights, residual, out, tokens, entries, n, (int)top_k, f32};
    return status_of(qw::launch_experts_combine(a, static_cast<hipStream_t>(stream)));
}

} // namespace

extern "C" {

QW_API qw_status qw_add_rms_norm(const void *x, int64_t x_stride, const void *residual, int64_t residual_stride,
                                 const void *weight, int dtype, int64_t tokens, int64_t k, double eps, void *h,
                                 int64_t h_stride, void *y, void *stream)
{
    qw::AddNormArgs a = {};
    a.x = static_cast<const uint16_t *>(x);
    a.residual = static_cast<const uint16_t *>(residual);
    a.weight = static_cast<const uint16_t *>(weight);
    a.h = static_cast<uint16_t *>(h);
    a.y = static_cast<uint16_t *>(y);
    a.x_stride = x_stride;
    a.residual_stride = residual_stride;
    a.h_stride = h_stride;
    a.tokens = tokens;
    a.k = k;
    return add_norm(a, dtype, eps, false, stream);
}

QW_API qw_status qw_add_rms_norm_quantize(const void *x, int64_t x_stride, const void *residual, int64_t residual_stride,
                                          const void *weight, int dtype, int64_t tokens, int64_t k, double eps, void *h,
                                          int64_t h_stride, int8_t *q, uint16_t *scales, void *stream)
{
    qw::AddNormArgs a = {};
    a.x = static_cast<const uint16_t *>(x);
    a.residual = static_cast<const uint16_t *>(residual);
    a.weight = static_cast<const uint16_t *>(weight);
    a.h = static_cast<uint16_t *>(h);
    a.q = q;
    a.scales = scales;
    a.x_stride = x_stride;
    a.residual_stride = residual_stride;
    a.h_stride = h_stride;
    a.tokens = tokens;
    a.k = k;
    return add_norm(a, dtype, eps, true, stream);
}

QW_API int64_t qw_route_experts_workspace(int64_t tokens, int64_t experts, int64_t top_k)
{
    if (tokens < 0 || experts < 1 || top_k < 1 || !route_sizes_ok(tokens, experts, top_k))
        return -1;
    return route_workspace(tokens, experts);
}

QW_API qw_status qw_route_experts(const void *logits, int dtype, int64_t tokens, int64_t experts, int64_t top_k, int scoring,
                                  const float *bias, int64_t groups, int64_t top_groups, int renormalize, double scale,
                                  int32_t *ids, float *weights, int32_t *offsets, int32_t *rows, int32_t *places,
                                  void *workspace, int64_t workspace_bytes, void *stream)
{
    if (tokens < 0 || experts < 1 || top_k < 1 || groups < 1 || top_groups < 1 || top_groups > groups || experts % groups ||
        (scoring != 0 && scoring != 1) || (renormalize != 0 && renormalize != 1) || !isfinite(scale) ||
        (dtype != QW_F16 && dtype != QW_BF16 && dtype != QW_F32) || workspace_bytes < 0 || !offsets)
        return QW_ERROR_INVALID_VALUE;
    if (tokens > 0 && (!logits || !ids || !weights || !rows || !places || !workspace))
        return QW_ERROR_INVALID_VALUE;
    if (!route_sizes_ok(tokens, experts, top_k) || groups > 64)
        return QW_ERROR_UNSUPPORTED;
    if (workspace_bytes < route_workspace(tokens, experts))
        return QW_ERROR_INVALID_VALUE;
    if (off16(logits) || off16(bias) || off16(workspace) || off4(ids) || off4(weights) || off4(offsets) || off4(rows) ||
        off4(places))
        return QW_ERROR_MISALIGNED;
    const uint64_t entries = (uint64_t)tokens * (uint64_t)top_k * 4u;
    const Span in[2] = {{logits, (uint64_t)tokens * (uint64_t)experts * (dtype == QW_F32 ? 4u : 2u)},
                        {bias, (uint64_t)experts * 4u}};
    const Span out[6] = {{ids, entries}, {weights, entries}, {rows, entries}, {places, entries},
                         {offsets, (uint64_t)(experts + 1) * 4u}, {workspace, (uint64_t)workspace_bytes}};
    for (int i = 0; i < 6; ++i) {
        if (meet(out[i], in[0]) || meet(out[i], in[1]))
            return QW_ERROR_INVALID_VALUE;
        for (int j = i + 1; j < 6; ++j)
            if (meet(out[i], out[j]))
                return QW_ERROR_INVALID_VALUE;
    }
    qw::RouteArgs a = {};
    a.logits = logits;
    a.bias = bias;
    a.tokens = tokens;
    a.experts = (int)experts;
    a.top_k = (int)top_k;
    a.sigmoid = scoring;
    a.groups = (int)groups;
    a.top_groups = (int)top_groups;
    a.renormalize = renormalize;
    a.scale = scale;
    a.ids = ids;
    a.weights = weights;
    a.offsets = offsets;
    a.rows = rows;
    a.places = places;
    a.counts = static_cast<int32_t *>(workspace);
    a.tokens_a_block = (int)qw::route_tokens_a_block(tokens);
    a.blocks = (int)route_blocks(tokens);
    a.counts_stride = (int)((experts + 3) / 4 * 4);
    return status_of(qw::launch_route_experts(a, dtype, static_cast<hipStream_t>(stream)));
}

QW_API qw_status qw_w8a16_experts_path(const uint16_t *x, int64_t x_rows, int gather, const int8_t *q, const uint16_t *scales,
                                       const uint16_t *bias, int activation, int gated, const int32_t *offsets,
                                       const int32_t *rows, int64_t entries, int64_t top_k, uint16_t *y, int64_t experts,
                                       int64_t n, int64_t k, int path, int tile, void *stream)
{
    return experts_product(x, x_rows, gather, q, scales, bias, activation, gated, offsets, rows, entries, top_k, y, false, experts,
                           n, k, path, tile, stream);
}

QW_API qw_status qw_w8a16_experts_f32(const uint16_t *x, int64_t x_rows, int gather, const int8_t *q, const uint16_t *scales,
                                      const uint16_t *bias, int activation, int gated, const int32_t *offsets,
                                      const int32_t *rows, int64_t entries, int64_t top_k, float *y, int64_t experts, int64_t n,
                                      int64_t k, int path, int tile, void *stream)
{
    return experts_product(x, x_rows, gather, q, scales, bias, activation, gated, offsets, rows, entries, top_k, y, true, experts,
                           n, k, path, tile, stream);
}

QW_API qw_status qw_w8a16_experts(const uint16_t *x, int64_t x_rows, int gather, const int8_t *q, const uint16_t *scales,
                                  const uint16_t *bias, int activation, int gated, const int32_t *offsets,
                                  const int32_t *rows, int64_t entries, int64_t top_k, uint16_t *y, int64_t experts, int64_t n,
                                  int64_t k, void *stream)
{
    return qw_w8a16_experts_path(x, x_rows, gather, q, scales, bias, activation, gated, offsets, rows, entries, top_k, y,
                                 experts, n, k, QW_PATH_AUTO, 0, stream);
}

QW_API qw_status qw_experts_combine(const uint16_t *y, int64_t entries, const int32_t *places, const float *weights,
                                    int64_t tokens, int64_t top_k, const uint16_t *residual, uint16_t *out, int64_t n,
                                    void *stream)
{
    return combine(y, false, entries, places, weights, tokens, top_k, residual, out, n, stream);
}

QW_API qw_status qw_experts_combine_f32(const float *y, int64_t entries, const int32_t *places, const float *weights,
                                        int64_t tokens, int64_t top_k, const uint16_t *residual, uint16_t *out, int64_t n,
                                        void *stream)
{
    return combine(y, true, entries, places, weights, tokens, top_k, residual, out, n, stream);
}

QW_API int64_t qw_w8a16_linear_workspace(int64_t m, int64_t n, int64_t k, int gated)
{
    return linear_workspace(m, n, k, gated, false);
}

QW_API int64_t qw_w8a8_linear_workspace(int64_t m, int64_t n, int64_t k, int gated)
{
    return linear_workspace(m, n, k, gated, true);
}

QW_API qw_status qw_w8a16_linear_path(const uint16_t *x, const int8_t *q, const uint16_t *scales, const uint16_t *bias,
                                      int activation, int gated, const uint16_t *residual, uint16_t *y, int64_t m,
                                      int64_t n, int64_t k, int path, int tile, int splits, void *workspace,
                                      int64_t workspace_bytes, void *stream)
{
    const qw::LinearArgs a = {x, nullptr, q, scales, {bias, residual, activation, 0}, false, y, m, n, k};
    return linear(a, QW_F16, gated, {path, tile, splits}, workspace, workspace_bytes, stream);
}

QW_API qw_status qw_w8a16_linear(const uint16_t *x, const int8_t *q, const uint16_t *scales, const uint16_t *bias,
                                 int activation, int gated, const uint16_t *residual, uint16_t *y, int64_t m, int64_t n,
                                 int64_t k, void *workspace, int64_t workspace_bytes, void *stream)
{
    return qw_w8a16_linear_path(x, q, scales, bias, activation, gated, residual, y, m, n, k, QW_PATH_AUTO, 0, 1, workspace,
                                workspace_bytes, stream);
}

QW_API qw_status qw_w8a8_linear_path(const int8_t *qx, const uint16_t *sx, const int8_t *q, const uint16_t *scales,
                                     const void *bias, int activation, int gated, const void *residual, int dtype, void *y,
                                     int64_t m, int64_t n, int64_t k, int path, int tile, int splits, void *workspace,
                                     int64_t workspace_bytes, void *stream)
{
    if (!sx && m != 0 && n != 0)
        return QW_ERROR_INVALID_VALUE;
    // (sx also says which product this is, and the empty ones may have none)
    static const uint16_t empty = 0;
    const qw::LinearArgs a = {qx, sx ? sx : &empty, q, scales,
                              {static_cast<const uint16_t *>(bias), static_cast<const uint16_t *>(residual), activation, 0},
                              false, static_cast<uint16_t *>(y), m, n, k};
    return linear(a, dtype, gated, {path, tile, splits}, workspace, workspace_bytes, stream);
}

QW_API qw_status qw_w8a8_linear(const int8_t *qx, const uint16_t *sx, const int8_t *q, const uint16_t *scales,
                                const void *bias, int activation, int gated, const void *residual, int dtype, void *y,
                                int64_t m, int64_t n, int64_t k, void *workspace, int64_t workspace_bytes, void *stream)
{
    return qw_w8a8_linear_path(qx, sx, q, scales, bias, activation, gated, residual, dtype, y, m, n, k, QW_PATH_AUTO, 0, 1,
                               workspace, workspace_bytes, stream);
}

} // extern "C"
