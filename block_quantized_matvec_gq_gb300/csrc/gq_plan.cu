// gq_plan.cu -- the lists of a batch from its requests' lengths (include/gq_plan.h).
//
// Three running sums over the requests (new tokens, pages taken, pages given
// back) say where everything goes; after that every token, every taken page
// and every returned page is one independent item.  One cluster of one to eight
// CTAs plans: every CTA makes the sums for itself (a request list is a few KB in
// L2, an exchange would cost a cluster barrier), and the items are dealt out over
// all CTAs.  kv_len and the ring may be updated in place, so they are written
// after a barrier that all reads of them precede; a barrier inside one cluster
// needs no workspace, so that two plans in flight share nothing.  A page taken in
// this step is read from the ring and not from the table, which another thread is
// writing.  Steps of many tokens leave these to a second kernel of as many CTAs
// as it takes, which reads the finished lists.
//
// What bounds it: latency.  96 requests, one new token each: one CTA, some
// dependent rounds to L2 and the barriers of one scan, 4.9 us; 1000 requests with
// 143830 new tokens 11.3, of which the tokens' kernel is the latter half.
#include "gq_host.h"
#include "gq_internal.cuh"
#include "gq_plan.h"

namespace gq {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCtas = 8;
constexpr int kItemsPerCta = 1024;  // tokens that one CTA takes before another joins
constexpr int kTokenThreads = 256, kTokensPerCta = 1024;

struct Args {
    const int32_t *n_new, *kv_in, *ring_in;
    int32_t *free_pages, *table, *kv_len, *q_start, *ring;
    long long *slot;
    int32_t *position, *sequence;
    int n_pages, max_pages, page_tokens, n_seq, n_tokens;
    int *status;
    uint32_t per, per_mul;  // page_tokens / 16, and 2^32 / per rounded up
};
// x / page_tokens by a product, exact for x <= 2^28: x / 16 * per < 2^32.
__device__ __forceinline__ int page_of(const Args &a, int x)
{
    const uint32_t r = static_cast<uint32_t>(x) >> 4;
    return static_cast<int>(a.per == 1 ? r : __umulhi(r, a.per_mul));
}
__device__ __forceinline__ int pages_of(const Args &a, int tokens) { return tokens > 0 ? page_of(a, tokens - 1) + 1 : 0; }

// Sums stay at kMany, beyond every legal total, once they reach it.
constexpr int kMany = 1 << 29;
struct Sums {
    int tokens, need, back;
};
__device__ __forceinline__ Sums operator+(Sums a, Sums b)
{
    return {min(a.tokens + b.tokens, kMany), min(a.need + b.need, kMany), min(a.back + b.back, kMany)};
}
__device__ __forceinline__ Sums shfl_up(Sums s, int o)
{
    return {__shfl_up_sync(0xffffffffu, s.tokens, o), __shfl_up_sync(0xffffffffu, s.need, o), __shfl_up_sync(0xffffffffu, s.back, o)};
}
__device__ __forceinline__ Sums warp_scan(Sums s)
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Sums up = shfl_up(s, o);
        if ((threadIdx.x & 31) >= o) s = s + up;
    }
    return s;
}

// What request b adds to the sums; `bad` if it cannot be planned.
__device__ __forceinline__ Sums demand(const Args &a, int b, bool &bad)
{
    const int n = __ldg(a.n_new + b), kv = a.kv_in[b];
    const int room = a.max_pages * a.page_tokens;  // at most 2^28
    if (kv < 0 || kv > room) {
        bad = true;
        return {0, 0, 0};
    }
    const int have = pages_of(a, kv);
    if (n < 0) return {0, 0, have};
    if (n > a.n_tokens || n > room - kv) {
        bad = true;
        return {0, 0, 0};
    }
    return {n, pages_of(a, kv + n) - have, 0};
}

// Largest b with at[b] <= x (at[0] = 0, non-decreasing, x < at[n]).
__device__ __forceinline__ int find(const int *at, int n, int x)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (at[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

__device__ __forceinline__ void cluster_barrier()
{
    asm volatile("barrier.cluster.arrive.aligned;\n barrier.cluster.wait.aligned;" ::: "memory");
}

__global__ void __launch_bounds__(kThreads) k_kv_plan(Args a)
{
    extern __shared__ int sh[];
    int *tok_at = sh, *need_at = sh + a.n_seq + 1, *back_at = need_at + a.n_seq + 1;
    __shared__ Sums warp_sum[kWarps];
    __shared__ int s_bad;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int all = gridDim.x * kThreads, me = blockIdx.x * kThreads + tid;
    if (tid == 0) s_bad = 0;
    __syncthreads();
    pdl_launch_dependents();
    pdl_wait();

    // ---- running sums; a thread takes consecutive requests
    const int per = (a.n_seq + kThreads - 1) / kThreads;
    const int b0 = min(tid * per, a.n_seq), b1 = min(b0 + per, a.n_seq);
    bool bad = false;
    Sums mine{0, 0, 0};
    for (int b = b0; b < b1; ++b) mine = mine + demand(a, b, bad);
    const Sums incl = warp_scan(mine);
    if (lane == 31) warp_sum[warp] = incl;
    if (bad) s_bad = 1;
    const int first = a.ring_in[0], count = a.ring_in[1];
    __syncthreads();
    if (warp == 0) warp_sum[lane] = warp_scan(warp_sum[lane]);
    __syncthreads();
    const Sums total = warp_sum[kWarps - 1], none{0, 0, 0}, before = warp ? warp_sum[warp - 1] : none;
    // pages taken and pages returned must not meet in the ring
    bad = s_bad != 0 || total.tokens > a.n_tokens || first < 0 || first >= a.n_pages || count < 0 || count > a.n_pages ||
          total.need > count || total.back > a.n_pages - count;
    if (!bad) {
        Sums at{before.tokens + incl.tokens - mine.tokens, before.need + incl.need - mine.need,
                before.back + incl.back - mine.back};
        for (int b = b0; b < b1; ++b) {
            tok_at[b] = at.tokens;
            need_at[b] = at.need;
            back_at[b] = at.back;
            at = at + demand(a, b, bad);
        }
        if (tid == 0) {
            tok_at[a.n_seq] = total.tokens;
            need_at[a.n_seq] = total.need;
            back_at[a.n_seq] = total.back;
        }
    }
    __syncthreads();

    const int tokens = bad ? 0 : total.tokens;
    const unsigned np = static_cast<unsigned>(a.n_pages);
    auto ring_at = [&](unsigned i) { return i >= np ? i - np : i; };  // i < 2 np
    bool odd_page = false;
    // ---- tokens
    for (int t = me; t < (a.slot || a.position || a.sequence ? a.n_tokens : 0); t += all) {
        int b = -1, pos = -1;
        long long slot = -1;
        if (t < tokens) {
            b = find(tok_at, a.n_seq, t);
            const int kv = a.kv_in[b];
            pos = kv + t - tok_at[b];
            const int j = page_of(a, pos), have = pages_of(a, kv);
            const int page = j < have ? a.table[static_cast<long long>(b) * a.max_pages + j]
                                      : a.free_pages[ring_at(static_cast<unsigned>(first) + need_at[b] + (j - have))];
            if (static_cast<unsigned>(page) < np)
                slot = static_cast<long long>(page) * a.page_tokens + (pos - j * a.page_tokens);
            else
                odd_page = true;
        }
        if (a.slot) a.slot[t] = slot;
        if (a.position) a.position[t] = pos;
        if (a.sequence) a.sequence[t] = b;
    }
    if (!bad) {
        // ---- pages taken and pages returned
        for (int i = me; i < total.need; i += all) {
            const int b = find(need_at, a.n_seq, i);
            const int have = pages_of(a, a.kv_in[b]);
            const int page = a.free_pages[ring_at(static_cast<unsigned>(first) + i)];
            if (static_cast<unsigned>(page) >= np) odd_page = true;
            a.table[static_cast<long long>(b) * a.max_pages + have + (i - need_at[b])] = page;
        }
        for (int i = me; i < total.back; i += all) {
            const int b = find(back_at, a.n_seq, i);
            const int page = a.table[static_cast<long long>(b) * a.max_pages + (i - back_at[b])];
            if (static_cast<unsigned>(page) >= np) odd_page = true;
            a.free_pages[ring_at(ring_at(static_cast<unsigned>(first) + count) + i)] = page;
        }
    }
    if ((odd_page || (bad && me == 0)) && a.status) atomicExch(a.status, GQ_ERR_SHAPE);

    // ---- the lengths, after every thread of the cluster has read them: a CTA's
    // own requests are dealt out by thread, so hold their values over the barrier
    int kv_new[(GQ_MAX_PLAN_SEQ + kThreads - 1) / kThreads];
#pragma unroll
    for (int i = 0; i < (GQ_MAX_PLAN_SEQ + kThreads - 1) / kThreads; ++i) {
        const int b = me + i * all;
        if (b < a.n_seq) {
            const int n = __ldg(a.n_new + b), kv = a.kv_in[b];
            kv_new[i] = bad ? kv : (n < 0 ? 0 : kv + n);
        }
    }
    cluster_barrier();
#pragma unroll
    for (int i = 0; i < (GQ_MAX_PLAN_SEQ + kThreads - 1) / kThreads; ++i) {
        const int b = me + i * all;
        if (b < a.n_seq) a.kv_len[b] = kv_new[i];
    }
    for (int b = me; b <= a.n_seq; b += all) a.q_start[b] = bad ? 0 : tok_at[b];
    if (me == 0) {
        a.ring[0] = bad ? first : static_cast<int>(ring_at(static_cast<unsigned>(first) + static_cast<unsigned>(total.need)));
        a.ring[1] = bad ? count : count - total.need + total.back;
    }
}

// The tokens of a planned step, kTokensPerCta neighbours a CTA.
__global__ void __launch_bounds__(kTokenThreads) k_kv_plan_tokens(Args a)
{
    extern __shared__ int at[];  // q_start
    const int tid = threadIdx.x, lane = tid & 31;
    pdl_launch_dependents();
    pdl_wait();
    for (int b = tid; b <= a.n_seq; b += kTokenThreads) at[b] = __ldcg(a.q_start + b);
    __syncthreads();
    const int tokens = at[a.n_seq];
    bool odd_page = false;
    // a warp takes 128 neighbours, a lane every 32nd: they mostly belong to one request
    const int t0 = blockIdx.x * kTokensPerCta + (tid >> 5) * 128 + lane;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = t0 + 32 * i;
        if (t >= a.n_tokens) break;
        int b = -1, pos = -1;
        long long slot = -1;
        if (t < tokens) {
            b = find(at, a.n_seq, t);
            pos = __ldcg(a.kv_len + b) - at[b + 1] + t;
            const int j = page_of(a, pos), page = __ldcg(a.table + static_cast<long long>(b) * a.max_pages + j);
            if (static_cast<unsigned>(page) < static_cast<unsigned>(a.n_pages))
                slot = static_cast<long long>(page) * a.page_tokens + (pos - j * a.page_tokens);
            else
                odd_page = true;
        }
        if (a.slot) a.slot[t] = slot;
        if (a.position) a.position[t] = pos;
        if (a.sequence) a.sequence[t] = b;
    }
    if (odd_page && a.status) atomicExch(a.status, GQ_ERR_SHAPE);
}

inline bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace
}  // namespace gq

extern "C" int gq_kv_plan(const int32_t *n_new, const int32_t *kv_len_in, const int32_t *ring_in, int32_t *free_pages,
                          int32_t *block_table, int32_t *kv_len, int32_t *q_start, int32_t *ring, int64_t *slot_or_null,
                          int32_t *position_or_null, int32_t *sequence_or_null, int n_pages, int max_pages,
                          int page_tokens, int n_seq, int n_tokens, gq_stream_t stream)
{
    using namespace gq;
    const void *lists[] = {n_new, kv_len_in, ring_in, free_pages, block_table, kv_len, q_start, ring};
    for (const void *p : lists)
        if (!p) return GQ_ERR_NULL;
    for (const void *p : lists)
        if (!aligned4(p)) return GQ_ERR_ALIGN;
    if ((reinterpret_cast<uintptr_t>(slot_or_null) & 7u) != 0 || !aligned4(position_or_null) || !aligned4(sequence_or_null))
        return GQ_ERR_ALIGN;
    if (n_pages < 1 || n_pages > (1 << 28) || page_tokens < 16 || page_tokens % 16 != 0 || page_tokens > 4096 || max_pages < 1 ||
        static_cast<long long>(max_pages) * page_tokens > (1 << 28) || n_seq < 1 || n_seq > GQ_MAX_PLAN_SEQ ||
        n_tokens < 0 || n_tokens > (1 << 28))
        return GQ_ERR_SHAPE;
    // more tokens than the cluster takes at two a thread: a second kernel
    const bool any = slot_or_null || position_or_null || sequence_or_null, second = any && n_tokens > 2 * kMaxCtas * kItemsPerCta;
    const int items = any && !second ? n_tokens : n_tokens / page_tokens + n_seq;  // about as many pages at most
    int ctas = (items + kItemsPerCta - 1) / kItemsPerCta;
    ctas = ctas < 1 ? 1 : (ctas > kMaxCtas ? kMaxCtas : ctas);
    const size_t smem = 3 * (static_cast<size_t>(n_seq) + 1) * sizeof(int);
    // asked for the most requests, whatever their number: the answers are kept, and there is room for some hundreds of
    // different sizes of all kernels together
    constexpr size_t kMostSmem = 3 * (GQ_MAX_PLAN_SEQ + 1) * sizeof(int);
    if (ctas_per_sm(reinterpret_cast<const void *>(k_kv_plan), kThreads, kMostSmem) < 1) return GQ_ERR_CUDA;
    const uint32_t per = static_cast<uint32_t>(page_tokens / 16), per_mul = static_cast<uint32_t>(((1ull << 32) + per - 1) / per);
    Args a{n_new,    kv_len_in, ring_in, free_pages, block_table, kv_len, q_start, ring, nullptr, nullptr, nullptr,
           n_pages,  max_pages, page_tokens, n_seq,  n_tokens,    status_word(), per, per_mul};
    const Args with_tokens{n_new,   kv_len_in, ring_in,     free_pages, block_table,
                           kv_len,  q_start,   ring,        reinterpret_cast<long long *>(slot_or_null),
                           position_or_null, sequence_or_null, n_pages, max_pages, page_tokens, n_seq, n_tokens, a.status, per, per_mul};
    if (!second) a = with_tokens;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    cudaError_t e = cudaLaunchKernelEx(&cfg, k_kv_plan, a);
    if (e == cudaSuccess && second)
        e = launch_pdl(k_kv_plan_tokens, dim3((n_tokens + kTokensPerCta - 1) / kTokensPerCta), dim3(kTokenThreads),
                       (static_cast<size_t>(n_seq) + 1) * sizeof(int), reinterpret_cast<cudaStream_t>(stream), with_tokens);
    return status_from(e);
}
