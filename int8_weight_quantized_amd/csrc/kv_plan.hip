// kv_plan.hip -- the step plan of a paged KV cache: block tables and slot
// maps from request lengths.
//
// With B tokens a block, a request that holds `past` tokens and adds `new`
// owns ceil(past / B) blocks and takes ceil((past + new) / B) -
// ceil(past / B) more, in order, from the list of free ones: the exclusive
// sums over requests of `new` and of that count say where each request's
// tokens and blocks begin.  Everything else is local to a token.
//
// Nothing here moves enough bytes to matter (8 bytes a token): the time is
// the launch and the latency of the sums.  So there is one launch: every
// workgroup forms the sums of all requests itself, in LDS, and then writes
// the positions and slots of its own tokens, finding each token's request
// by bisection.  A new block's table entry is written by the token at its
// offset 0, which is new by construction, so no workgroup waits for
// another's entries.
#include "kv_device.h"
#include "kv_internal.h"

namespace qw {

namespace {

constexpr int kThreads = 256;
constexpr int kTokensPerThread = 4;
constexpr int64_t kIntMax = 0x7fffffff;

__device__ __forceinline__ int64_t nonneg(int32_t v) { return v > 0 ? v : 0; }
__device__ __forceinline__ int64_t min64(int64_t a, int64_t b) { return a < b ? a : b; }

// Inclusive sum over the workgroup's 256 threads, and its total.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t &total, int64_t *wave_sums)
{
    const int lane = __lane_id(), wave = threadIdx.x >> 6;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int64_t o = shfl_up_i64(v, d);
        v += lane >= d ? o : 0;
    }
    if (lane == 63)
        wave_sums[wave] = v;
    __syncthreads();
    int64_t before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w) {
        before += w < wave ? wave_sums[w] : 0;
        total += wave_sums[w];
    }
    __syncthreads();
    return v + before;
}

__global__ __launch_bounds__(kThreads) void kv_plan_kernel(KvPlanArgs a)
{
    extern __shared__ int32_t lds[]; // tokens before request r (requests + 1), then new blocks before it
    __shared__ int64_t wave_sums[kThreads / 64];
    int32_t *cu = lds, *taken = lds + a.requests + 1;
    const bool first = blockIdx.x == 0;
    const int tid = threadIdx.x;
    const int64_t block = int64_t(1) << a.block_shift;

    int64_t tokens = 0, blocks = 0;
    for (int base = 0; base < a.requests; base += kThreads) {
        const int r = base + tid;
        const bool in = r < a.requests;
        const int64_t past = in ? nonneg(a.past[r]) : 0;
        const int64_t want = in ? nonneg(a.fresh[r]) : 0;
        int64_t total;
        const int64_t end = tokens + block_scan(want, total, wave_sums);
        tokens += total;
        // tokens beyond max_tokens are dropped: they get no slot and no block
        const int64_t lo = min64(end - want, a.max_tokens), hi = min64(end, a.max_tokens);
        const int64_t held = (past + block - 1) >> a.block_shift;
        const int64_t holds = (past + (hi - lo) + block - 1) >> a.block_shift;
        const int64_t need = min64(holds, a.table_width) - min64(held, a.table_width);
        const int64_t upto = blocks + block_scan(need, total, wave_sums);
        blocks += total;
        if (in) {
            cu[r] = (int32_t)lo;
            taken[r] = (int32_t)min64(upto - need, kIntMax);
            if (first) {
                a.cu_tokens[r] = (int32_t)lo;
                a.context[r] = (int32_t)min64(past + (hi - lo), kIntMax);
            }
        }
    }
    const int32_t kept = (int32_t)min64(tokens, a.max_tokens);
    if (tid == 0) {
        cu[a.requests] = kept;
        if (first) {
            a.cu_tokens[a.requests] = kept;
            a.counts[0] = (int32_t)min64(blocks, kIntMax);
            a.counts[1] = (int32_t)min64(tokens, kIntMax);
        }
    }
    __syncthreads();

    const int64_t t0 = (int64_t)blockIdx.x * (kThreads * kTokensPerThread) + tid;
#pragma unroll
    for (int i = 0; i < kTokensPerThread; ++i) {
        const int64_t t = t0 + i * kThreads;
        if (t >= a.max_tokens)
            break;
        int32_t position = -1, slot = -1;
        if (t < kept) {
            // the last request that begins at or before t: it is not empty
            int lo = 0, hi = a.requests;
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (cu[mid] <= t)
                    lo = mid;
                else
                    hi = mid;
            }
            const int64_t past = nonneg(a.past[lo]);
            const int64_t pos = past + (t - cu[lo]);
            const int64_t j = pos >> a.block_shift, held = (past + block - 1) >> a.block_shift;
            position = (int32_t)min64(pos, kIntMax);
            if (j < a.table_width) {
                int32_t *entry = a.block_table + (int64_t)lo * a.table_width + j;
                int64_t id;
                if (j < held) {
                    id = *entry;
                } else {
                    const int64_t f = taken[lo] + (j - held);
                    id = f < a.n_free ? a.free_blocks[f] : -1;
                    if ((pos & (block - 1)) == 0)
                        *entry = (int32_t)id;
                }
                const int64_t s = (id << a.block_shift) + (pos & (block - 1));
                slot = id >= 0 && s <= kIntMax ? (int32_t)s : -1;
            }
        }
        a.positions[t] = position;
        a.slots[t] = slot;
    }
}

} // namespace

hipError_t launch_kv_plan(const KvPlanArgs &a, hipStream_t stream)
{
    const int64_t per = kThreads * kTokensPerThread;
    const int64_t grid = a.max_tokens > 0 ? (a.max_tokens + per - 1) / per : 1;
    const size_t lds = (size_t)(2 * a.requests + 1) * sizeof(int32_t);
    kv_plan_kernel<<<dim3((unsigned)grid), dim3(kThreads), lds, stream>>>(a);
    return hipGetLastError();
}

} // namespace qw
