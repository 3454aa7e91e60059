// gq_kv_attn.cu -- attention of new tokens over the paged Q8_0 cache
// (gq_kv_attention_q8_0), the split form: work divided along the cached
// tokens, for calls with few query rows per sequence and kv head.
//
// An item is one (sequence, kv head, tile of 8 query rows); a query row is
// one (new token, head of the kv head's group), row r of a sequence being
// token r / G and head r % G with G = heads / kv_heads.  Every record of 16
// tokens that an item attends to is one unit of work.  The units of the whole
// call form one line, cut into equal stretches, one per CTA, whatever the
// lengths of the sequences; an item cut by a stretch's end is finished by the
// last of its CTAs to arrive, from partial results in the workspace, in a
// fixed order.
//
// One warp takes one record at a time (a bulk copy of its 34 D bytes into the
// warp's own ring in shared memory, so no warp waits for another inside a
// stretch) and keeps its own softmax state:
//   S = q k~:  mma.sync m16n8k16, f16 x f16 -> f32, A = the 8 query rows as
//     two f16 pieces (rows 0-7 the rounded value, rows 8-15 the remainder, 22
//     bits together), B = the integer codes of 8 tokens, exact in f16.  The
//     products of one 32-block are summed in f32 and scaled by the block's
//     fp16 scale, so a score has f32 accuracy although all operands are f16.
//   O += p v~: A = p times the value's block scale, again as two f16 pieces,
//     B = the value codes.  Four tokens' codes of one element are one word of
//     the layout, so the B fragment is two byte permutes, and the score
//     fragment's columns are assigned to tokens so that a lane's four scores
//     are those of the same four tokens: p never leaves its lane.
// The running reference m is the largest s + log2(largest value scale of the
// token), not the largest s: then p times a scale is at most 1 whatever the
// scales are, and stays in f16's range.  The state is rescaled only when the
// reference would grow by more than 2^8 (one vote per record otherwise).
#include "gq_kv.cuh"
#include "gq_tc.cuh"

namespace gq {
namespace kv {

constexpr int kWarps = 4;
constexpr int kAttnThreads = kWarps * 32;
constexpr int kRows = 8;            // query rows per item
constexpr int kMaxCtas = 1024;      // stretches per call, at most
constexpr float kFloor = -1e30f;    // reference of a row that has seen no token
constexpr float kHead = 6.0f;       // p is kept times 2^6: with the 2^8 slack below 2^15
constexpr float kSlack = 8.0f;

template <int D>
struct SplitCfg {
    static constexpr int kStages = D == 256 ? 3 : 4;
    static constexpr int kRing = kStages * rec_bytes(D);
    // the merge of the warps' states reuses the ring
    static constexpr int kSmem = kWarps * kRing;
    static_assert(kSmem >= kWarps * kRows * (D + 4) * 4, "merge buffers fit in the ring");
};

// Partial results: per CTA two slots of {O[8][D], m[8], l[8]} f32.
__host__ __device__ constexpr size_t slot_floats(int D) { return kRows * (D + 2); }

struct Args {
    const uint8_t *Q, *cache;
    uint8_t *O;
    long long ldq, ldo;  // bytes
    int type, group, window;
    float scale, softcap;
    int *counter;
    float *part;
};

// Records spanned by a sequence's new tokens together, at least one: the
// length of each of its items on the line of work.
struct Span {
    int lo, n;  // first record, records
};
__device__ __forceinline__ Span span_of(const Seq &s, int window)
{
    Span r;
    const int lo = window > 0 ? max(0, s.first - window + 1) : 0;
    r.lo = lo / kRec;
    r.n = max(1, (s.kv + kRec - 1) / kRec - r.lo);
    return r;
}
__device__ __forceinline__ long long cost_of(const Batch &B, const Args &A, int b)
{
    const Seq s = load_seq(B, b);
    const int tiles = (s.n * A.group + kRows - 1) / kRows;
    return static_cast<long long>(tiles) * B.kv_heads * span_of(s, A.window).n;
}

// Lays the sequences on the line: the call's total, and the part [b0, b1) of
// the sequences that this thread looked at with the units before it (all
// threads take part).
template <int THREADS, class Cost>
__device__ __forceinline__ void plan(int n_seq, Cost cost, long long *warp_sum, long long &total, long long &excl, int &b0, int &b1)
{
    const int per = (n_seq + THREADS - 1) / THREADS, lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    b0 = min(static_cast<int>(threadIdx.x) * per, n_seq);
    b1 = min(b0 + per, n_seq);
    long long mine = 0;
    for (int b = b0; b < b1; ++b) mine += cost(b);
    long long inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
    }
    if (lane == 31) warp_sum[w] = inc;
    __syncthreads();
    long long before = 0;
    total = 0;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) {
        if (i < w) before += warp_sum[i];
        total += warp_sum[i];
    }
    excl = before + inc - mine;
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float lg2(float x)
{
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// (a, b) -> f16x2 of the rounded values and of the remainders.
__device__ __forceinline__ void split2(float a, float b, uint32_t &hi, uint32_t &lo)
{
    hi = f2_half2(a, b);
    const float2 r = half2_f2(hi);
    lo = f2_half2(a - r.x, b - r.y);
}
// cap * tanh(x / cap) in f32: tanh|y| = (1 - e) / (1 + e), e = exp(-2|y|).
// For small |y| the difference 1 - e cancels; there the odd series is used.
__device__ __forceinline__ float soft_cap(float x, float cap, float inv_cap)
{
    const float y = x * inv_cap, a = fabsf(y);
    const float e = ex2(-2.885390082f * a);
    const float big = __fdividef(1.0f - e, 1.0f + e);
    const float q = y * y;
    // y - y^3/3 + 2 y^5/15 - 17 y^7/315 + 62 y^9/2835: below 2^-24 relative for |y| < 0.25
    const float small = a * (1.0f + q * (-0.333333333f + q * (0.133333333f + q * (-0.053968254f + q * 0.021869489f))));
    return copysignf(cap * (a < 0.25f ? small : big), y);
}

template <int D>
__global__ void __launch_bounds__(kAttnThreads) k_kv_attn_split(Args A, Batch B)
{
    constexpr int nb = D / 32, kStages = SplitCfg<D>::kStages;
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ __align__(8) uint64_t bars[kWarps * kStages];
    __shared__ long long warp_sum[kWarps];
    __shared__ long long s_at;
    __shared__ int s_seq, s_last;
    __shared__ volatile int s_abort;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    uint8_t *my_ring = ring + warp * SplitCfg<D>::kRing;
    const uint32_t ring_u32 = tcu::smem_u32(my_ring), bar0 = tcu::smem_u32(bars + warp * kStages);
    if (lane == 0)
        for (int i = 0; i < kStages; ++i) tcu::mbar_init(bar0 + 8 * i, 1);
    if (threadIdx.x == 0) s_abort = 0;
    tcu::fence_async_smem();
    pdl_launch_dependents();
    pdl_wait();

    // ---- this CTA's stretch of the line
    long long total, excl;
    int b0, b1;
    auto cost = [&](int b) { return cost_of(B, A, b); };
    plan<kAttnThreads>(B.n_seq, cost, warp_sum, total, excl, b0, b1);
    // at least two records a warp: a shorter stretch would spend more on its merge
    const long long len = max((total + gridDim.x - 1) / gridDim.x, static_cast<long long>(2 * kWarps));
    const long long begin = len * blockIdx.x, end = min(begin + len, total);
    if (begin >= total) return;
    {
        long long at = excl;
        for (int b = b0; b < b1; ++b) {
            const long long c = cost(b);
            if (begin >= at && begin < at + c) {
                s_seq = b;
                s_at = at;
            }
            at += c;
        }
    }
    __syncthreads();
    int b = s_seq;
    long long at = s_at;  // where sequence b begins
    uint32_t fill = 0;    // records this warp has taken so far (ring position and parity)

    for (long long x = begin; x < end;) {
        // ---- the item at x
        Seq s = load_seq(B, b);
        Span sp = span_of(s, A.window);
        const int tiles = (s.n * A.group + kRows - 1) / kRows;
        const long long size = static_cast<long long>(tiles) * B.kv_heads * sp.n;
        if (x >= at + size) {  // next sequence (uniform in the CTA)
            at += size;
            ++b;
            continue;
        }
        const long long item = (x - at) / sp.n;
        const long long item_x = at + item * sp.n;  // its first unit
        const int h = static_cast<int>(item % B.kv_heads), tile = static_cast<int>(item / B.kv_heads);
        const int from = static_cast<int>(x - item_x);
        const int to = static_cast<int>(min(end - item_x, static_cast<long long>(sp.n)));
        x = item_x + to;

        // ---- its rows: lane group g holds row 8 tile + g
        const int r = kRows * tile + g, rows = s.n * A.group;
        const bool live = r < rows;
        const int tok = live ? r / A.group : 0;
        const int pos = s.first + tok;
        const int row_hi = live ? pos : -1;                                        // last visible position
        const int row_lo = A.window > 0 ? max(0, pos - A.window + 1) : 0;          // first
        const int last_tok = min((kRows * tile + kRows - 1) / A.group, s.n - 1), first_tok = kRows * tile / A.group;
        const int item_hi = s.first + last_tok;                                    // over all its rows
        const int item_lo = A.window > 0 ? max(0, s.first + first_tok - A.window + 1) : 0;
        const int all_hi = s.first + first_tok;                                    // visible to every row: [all_lo, all_hi]
        const int all_lo = A.window > 0 ? max(0, s.first + last_tok - A.window + 1) : 0;
        // this CTA's records of the item
        const int rec0 = max(sp.lo + from, item_lo / kRec);
        const int rec1 = item_hi < 0 ? rec0 : min(sp.lo + to, item_hi / kRec + 1);

        // ---- the ring's first records; the pages of 32 records ahead sit one per lane
        const int mine0 = rec0 + warp;
        int pages = -1, pages_base = mine0;
        auto load_pages = [&](int base) {
            const int rec = base + lane * kWarps;
            pages = -1;
            if (rec < rec1) pages = page_of(B, b, rec * kRec);
            pages_base = base;
        };
        load_pages(mine0);
        auto issue = [&](int rec, uint32_t n) {  // n: the ring position's running number
            int k = (rec - pages_base) / kWarps;
            if (k >= 32) {
                load_pages(rec);
                k = 0;
            }
            const int pg = __shfl_sync(0xffffffffu, pages, k);
            if (lane == 0) {
                const uint32_t st = n % kStages, bar = bar0 + 8 * st;
                if (pg >= 0) {
                    tcu::mbar_expect_tx(bar, rec_bytes(D));
                    tcu::bulk_load(ring_u32 + st * rec_bytes(D), A.cache + rec_off(B, pg, h, rec * kRec, D), rec_bytes(D), bar);
                } else {
                    tcu::mbar_arrive(bar);
                }
            }
            return pg >= 0;
        };
        uint32_t good = 0;  // bit n % 32: record number n has a page
        uint32_t ahead = fill;
        {
            int rec = mine0;
#pragma unroll
            for (int i = 0; i < kStages - 1; ++i, rec += kWarps)
                if (rec < rec1) {
                    const bool ok = issue(rec, ahead);
                    good = ok ? good | (1u << (ahead & 31)) : good & ~(1u << (ahead & 31));
                    ++ahead;
                }
        }

        // ---- the query fragments: pieces of q * 2^-e, e from the row's largest magnitude
        uint32_t qf[nb][2][4];
        float zs;  // score = acc * zs
        {
            float amax = 0.f;
            float q[nb][8];
            const uint8_t *p = A.Q + (s.row0 + tok) * A.ldq;
            const int el = type_size(A.type);
            const long long head = static_cast<long long>(h * A.group + (live ? r % A.group : 0)) * D * el;
#pragma unroll
            for (int i = 0; i < nb; ++i) {
                float4 u = make_float4(0.f, 0.f, 0.f, 0.f), v = u;
                if (live) {
                    const uint8_t *e = p + head + (32 * i + 8 * t) * el;
                    if (A.type == GQ_TYPE_F32) {
                        u = load4<GQ_TYPE_F32>(e);
                        v = load4<GQ_TYPE_F32>(e + 16);
                    } else if (A.type == GQ_TYPE_BF16) {
                        u = load4<GQ_TYPE_BF16>(e);
                        v = load4<GQ_TYPE_BF16>(e + 8);
                    } else {
                        u = load4<GQ_TYPE_F16>(e);
                        v = load4<GQ_TYPE_F16>(e + 8);
                    }
                }
                q[i][0] = u.x, q[i][1] = u.y, q[i][2] = u.z, q[i][3] = u.w;
                q[i][4] = v.x, q[i][5] = v.y, q[i][6] = v.z, q[i][7] = v.w;
#pragma unroll
                for (int k = 0; k < 8; ++k) amax = fmaxf(amax, fabsf(q[i][k]));
            }
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            // amax * 2^-e in [2^9, 2^10) (less for rows below 2^-100); both factors are normal
            const int be = static_cast<int>(__float_as_uint(amax) >> 23) - 126;
            const int e = min(max(be, -100), 128) - 10;
            const float f = pow2i(-e);
#pragma unroll
            for (int i = 0; i < nb; ++i)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    split2(q[i][4 * k] * f, q[i][4 * k + 1] * f, qf[i][k][0], qf[i][k][1]);
                    split2(q[i][4 * k + 2] * f, q[i][4 * k + 3] * f, qf[i][k][2], qf[i][k][3]);
                }
            zs = A.scale * pow2i(e);
        }
        const float kLog2e = 1.4426950408889634f;
        const bool capped = A.softcap > 0.f;
        const float inv_cap = capped ? 1.0f / A.softcap : 0.f;
        if (!capped) zs *= kLog2e;

        float o[nb * 4][4];
#pragma unroll
        for (int i = 0; i < nb * 4; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) o[i][k] = 0.f;
        float m = kFloor, l = 0.f;

        // ---- the records
        for (int rec = mine0; rec < rec1; rec += kWarps, ++fill) {
            const int nxt = rec + (kStages - 1) * kWarps;
            if (nxt < rec1) {  // into the stage that the previous record has left
                const bool ok = issue(nxt, ahead);
                good = ok ? good | (1u << (ahead & 31)) : good & ~(1u << (ahead & 31));
                ++ahead;
            }
            const uint32_t st = fill % kStages;
            if (!tcu::wait_warp(bar0 + 8 * st, (fill / kStages) & 1, &s_abort, B.status)) break;
            if (!((good >> (fill & 31)) & 1u)) continue;  // no such page: nothing to attend to
            const uint8_t *R = my_ring + st * rec_bytes(D);

            // scores of tokens 4 t .. 4 t + 3 for row g
            float sc[4] = {0.f, 0.f, 0.f, 0.f};
            const int tk = 4 * (g >> 1) + (g & 1);  // column g of the first half's fragment; + 2 in the second
#pragma unroll
            for (int i = 0; i < nb; ++i) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint2 w = *reinterpret_cast<const uint2 *>(R + k_code_off(tk + 2 * j, i, nb) + 8 * t);
                    float c[4] = {0.f, 0.f, 0.f, 0.f};
                    mma16816(c, qf[i][0][0], qf[i][0][1], qf[i][0][2], qf[i][0][3], codes2(w.x, 0x4140u), codes2(w.x, 0x4342u));
                    mma16816(c, qf[i][1][0], qf[i][1][1], qf[i][1][2], qf[i][1][3], codes2(w.y, 0x4140u), codes2(w.y, 0x4342u));
                    const float d0 = __half2float(*reinterpret_cast<const __half *>(R + k_scale_off(4 * t + 2 * j, i, D)));
                    const float d1 = __half2float(*reinterpret_cast<const __half *>(R + k_scale_off(4 * t + 2 * j + 1, i, D)));
                    sc[2 * j] += (c[0] + c[2]) * d0;
                    sc[2 * j + 1] += (c[1] + c[3]) * d1;
                }
            }
            // value scales of the same four tokens
            uint2 dv[nb];
            uint32_t mx0 = 0, mx1 = 0;
#pragma unroll
            for (int i = 0; i < nb; ++i) {
                dv[i] = *reinterpret_cast<const uint2 *>(R + v_scale_off(4 * t, i, D));
                mx0 = __vmaxu2(mx0, dv[i].x);  // non-negative fp16 order like integers
                mx1 = __vmaxu2(mx1, dv[i].y);
            }
            const float2 da = half2_f2(mx0), db = half2_f2(mx1);
            float lg[4] = {lg2(fmaxf(da.x, 0x1p-24f)), lg2(fmaxf(da.y, 0x1p-24f)), lg2(fmaxf(db.x, 0x1p-24f)),
                           lg2(fmaxf(db.y, 0x1p-24f))};
            const int p0 = rec * kRec;
            const bool edge = p0 < all_lo || p0 + kRec - 1 > all_hi;  // warp-uniform
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                sc[k] *= zs;
                if (capped) sc[k] = soft_cap(sc[k], A.softcap, inv_cap) * kLog2e;
            }
            if (edge) {
                // hidden tokens: what the page holds there is not looked at, their value scales
                // included where no row sees them (0 * NaN would be NaN)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int j = p0 + 4 * t + k;
                    if (j < row_lo || j > row_hi) sc[k] = -INFINITY;
                    if (j < item_lo || j > item_hi) {
                        lg[k] = 0.f;
                        const uint32_t mask = (k & 1) ? 0x0000FFFFu : 0xFFFF0000u;
#pragma unroll
                        for (int i = 0; i < nb; ++i) {
                            if (k < 2) dv[i].x &= mask;
                            else dv[i].y &= mask;
                        }
                    }
                }
            }
            float top = fmaxf(fmaxf(sc[0] + lg[0], sc[1] + lg[1]), fmaxf(sc[2] + lg[2], sc[3] + lg[3]));
            if (__any_sync(0xffffffffu, top > m + kSlack)) {
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const float nm = fmaxf(m, top), f = ex2(m - nm);
                m = nm;
                l *= f;
#pragma unroll
                for (int i = 0; i < nb * 4; ++i)
#pragma unroll
                    for (int k = 0; k < 4; ++k) o[i][k] *= f;
            }
            float p[4];
            const float ref = m - kHead;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                p[k] = ex2(sc[k] - ref);
                l += p[k];
            }
#pragma unroll
            for (int i = 0; i < nb; ++i) {
                const float2 e0 = half2_f2(dv[i].x), e1 = half2_f2(dv[i].y);
                uint32_t a0, a1, a2, a3;
                split2(p[0] * e0.x, p[1] * e0.y, a0, a1);
                split2(p[2] * e1.x, p[3] * e1.y, a2, a3);
                const uint4 w = *reinterpret_cast<const uint4 *>(R + v_chunk_off(t, 8 * i + g, D));
                mma16816(o[4 * i], a0, a1, a2, a3, codes2(w.x, 0x4140u), codes2(w.x, 0x4342u));
                mma16816(o[4 * i + 1], a0, a1, a2, a3, codes2(w.y, 0x4140u), codes2(w.y, 0x4342u));
                mma16816(o[4 * i + 2], a0, a1, a2, a3, codes2(w.z, 0x4140u), codes2(w.z, 0x4342u));
                mma16816(o[4 * i + 3], a0, a1, a2, a3, codes2(w.w, 0x4140u), codes2(w.w, 0x4342u));
            }
            __syncwarp();  // every lane has read the stage before it is filled again
        }
        // after a wait that gave up: let the copies in flight land (bounded again)
        for (; fill != ahead; ++fill) tcu::wait_warp(bar0 + 8 * (fill % kStages), (fill / kStages) & 1, &s_abort, B.status);
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);

        // ---- merge the four warps' states through shared memory (row stride D + 4)
        __syncthreads();
        float *mo = reinterpret_cast<float *>(ring);        // [warp][8][D + 4]; elements D, D + 1 hold m, l
        float *mine = mo + (warp * kRows + g) * (D + 4);
#pragma unroll
        for (int i = 0; i < nb; ++i) {
            // fragment column n of quarter i' is element 32 i + 4 n + i'
            *reinterpret_cast<float4 *>(mine + 32 * i + 8 * t) =
                make_float4(o[4 * i][0] + o[4 * i][2], o[4 * i + 1][0] + o[4 * i + 1][2], o[4 * i + 2][0] + o[4 * i + 2][2],
                            o[4 * i + 3][0] + o[4 * i + 3][2]);
            *reinterpret_cast<float4 *>(mine + 32 * i + 8 * t + 4) =
                make_float4(o[4 * i][1] + o[4 * i][3], o[4 * i + 1][1] + o[4 * i + 1][3], o[4 * i + 2][1] + o[4 * i + 2][3],
                            o[4 * i + 3][1] + o[4 * i + 3][3]);
        }
        if (t == 0) {
            mine[D] = m;
            mine[D + 1] = l;
        }
        __syncthreads();
        const bool whole = from == 0 && to == sp.n;
        constexpr int kQuads = kRows * D / 4;
        float *slot = A.part + (2ll * blockIdx.x + (from == 0 ? 1 : 0)) * slot_floats(D);
        auto store_row = [&](int rr, int d, float4 v, float inv) {
            const int row = kRows * tile + rr;
            if (row >= rows) return;
            v.x *= inv, v.y *= inv, v.z *= inv, v.w *= inv;
            const int el = type_size(A.type);
            uint8_t *dst = A.O + (s.row0 + row / A.group) * A.ldo +
                           (static_cast<long long>(h * A.group + row % A.group) * D + d) * el;
            if (A.type == GQ_TYPE_F32) store4<GQ_TYPE_F32>(dst, v);
            else if (A.type == GQ_TYPE_BF16) store4<GQ_TYPE_BF16>(dst, v);
            else store4<GQ_TYPE_F16>(dst, v);
        };
        for (int i = threadIdx.x; i < kQuads; i += kAttnThreads) {
            const int rr = i / (D / 4), d = 4 * (i % (D / 4));
            float M = kFloor, L = 0.f;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, mo[(w * kRows + rr) * (D + 4) + D]);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float *src = mo + (w * kRows + rr) * (D + 4);
                const float f = ex2(src[D] - M);
                const float4 u = *reinterpret_cast<const float4 *>(src + d);
                L += f * src[D + 1];
                v.x += f * u.x, v.y += f * u.y, v.z += f * u.z, v.w += f * u.w;
            }
            if (whole) {
                store_row(rr, d, v, L == 0.f ? 0.f : 1.0f / L);
            } else {
                *reinterpret_cast<float4 *>(slot + rr * D + d) = v;
                if (d == 0) {
                    slot[kRows * D + rr] = M;
                    slot[kRows * D + kRows + rr] = L;
                }
            }
        }
        if (!whole) {
            // the last of the item's CTAs joins their parts, in the order of the stretches
            const int c0 = static_cast<int>(item_x / len), c1 = static_cast<int>((item_x + sp.n - 1) / len);
            __threadfence();
            __syncthreads();
            if (threadIdx.x == 0) {
                const int old = atomicAdd(A.counter + c0, 1);
                s_last = old == c1 - c0;
                if (old == c1 - c0) A.counter[c0] = 0;
            }
            __syncthreads();
            if (s_last) {
                __threadfence();
                for (int i = threadIdx.x; i < kQuads; i += kAttnThreads) {
                    const int rr = i / (D / 4), d = 4 * (i % (D / 4));
                    float M = kFloor, L = 0.f;
                    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                    for (int c = c0; c <= c1; ++c) {
                        const float *src = A.part + (2ll * c + (c == c0 ? 1 : 0)) * slot_floats(D);
                        const float mc = __ldcg(src + kRows * D + rr), lc = __ldcg(src + kRows * D + kRows + rr);
                        const float4 u = __ldcg(reinterpret_cast<const float4 *>(src + rr * D + d));
                        const float nm = fmaxf(M, mc), f = ex2(M - nm), fc = ex2(mc - nm);
                        M = nm;
                        L = L * f + lc * fc;
                        v.x = v.x * f + u.x * fc, v.y = v.y * f + u.y * fc, v.z = v.z * f + u.z * fc, v.w = v.w * f + u.w * fc;
                    }
                    store_row(rr, d, v, L == 0.f ? 0.f : 1.0f / L);
                }
            }
        }
        __syncthreads();           // the ring is free again
        tcu::fence_async_smem();   // before bulk copies overwrite what generic stores wrote
        if (s_abort) return;       // uniform after the barrier; every part of a cut item stays unfinished
    }
}

template <int D>
static int launch_split(const Args &A, const Batch &B, cudaStream_t s)
{
    const void *k = reinterpret_cast<const void *>(&k_kv_attn_split<D>);
    const int occ = ctas_per_sm(k, kAttnThreads, SplitCfg<D>::kSmem);
    if (occ < 1) return GQ_ERR_CUDA;
    int grid = sm_count() * occ;
    if (grid > kMaxCtas) grid = kMaxCtas;
    return status_from(launch_pdl(k_kv_attn_split<D>, dim3(grid), dim3(kAttnThreads), SplitCfg<D>::kSmem, s, A, B));
}

}  // namespace kv

// Workspace: the split form's counters, the chunk form's, then the partial
// results of whichever runs.
static size_t counter_bytes() { return ((kv::kMaxCtas + kv_chunk_counters()) * sizeof(int) + 127) / 128 * 128; }

size_t kv_attention_workspace_bytes(int head_dim)
{
    const size_t split = 2ull * kv::kMaxCtas * kv::slot_floats(head_dim) * sizeof(float), chunk = kv_chunk_part_bytes(head_dim);
    return counter_bytes() + (split > chunk ? split : chunk);
}

int launch_kv_attention(const void *Q, long long ldq, const uint8_t *cache, const kv::Batch &B, void *O, long long ldo,
                        int type, float scale, float softcap, int window, void *ws, int heads, int head_dim,
                        cudaStream_t s)
{
    int *counter = static_cast<int *>(ws);
    float *part = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + counter_bytes());
    // query rows per sequence and kv head, on average
    const long long rows = static_cast<long long>(B.n_tokens) * (heads / B.kv_heads) / B.n_seq;
    if (type != GQ_TYPE_F32 && rows >= 64)
        return launch_kv_chunk(Q, ldq, cache, B, O, ldo, type, scale, softcap, window, counter + kv::kMaxCtas, part, heads,
                               head_dim, s);
    const int el = kv::type_size(type);
    kv::Args A;
    A.Q = static_cast<const uint8_t *>(Q);
    A.cache = cache;
    A.O = static_cast<uint8_t *>(O);
    A.ldq = ldq * el;
    A.ldo = ldo * el;
    A.type = type;
    A.group = heads / B.kv_heads;
    A.window = window;
    A.scale = scale;
    A.softcap = softcap;
    A.counter = counter;
    A.part = part;
    switch (head_dim) {
    case 64: return kv::launch_split<64>(A, B, s);
    case 128: return kv::launch_split<128>(A, B, s);
    default: return kv::launch_split<256>(A, B, s);
    }
}

}  // namespace gq
