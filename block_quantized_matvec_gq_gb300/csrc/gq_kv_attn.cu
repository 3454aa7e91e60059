// gq_kv_attn.cu -- attention of new tokens over the paged Q8_0 cache
// (gq_kv_attention_q8_0), the split form: work divided along the cached
// tokens, for calls with few query rows per sequence and kv head.
//
// An item is one (sequence, kv head, tile of 8 or 16 query rows); a query row
// is one (new token, head of the kv head's group), row r of a sequence being
// token r / G and head r % G with G = heads / kv_heads.  Every record of 16
// tokens that an item attends to is one unit of work.  The units of the whole
// call form one line, cut into equal stretches, one per CTA, whatever the
// lengths of the sequences; a cut that would fall close to an item's end is
// moved there.  An item that is cut all the same is finished by the last of
// its CTAs to arrive, from partial results in the workspace, in a fixed order.
//
// One warp takes one record at a time (a bulk copy of its 34 D bytes into the
// warp's own ring in shared memory, so no warp waits for another inside a
// stretch) and keeps its own softmax state.  mma.sync m16n8k16 (f16 operands,
// f32 sums), A = query rows or probabilities, B = codes of 8 tokens or
// elements:
//   S = q k~.  A code byte u = code + 128 placed in the low byte of an f16 is
//     the subnormal number u 2^-24, so the B fragment is one byte permute per
//     two codes; adding -128 2^-24 sum q to a 32-block's sum takes the 128s out
//     again.  The sum of a block is scaled by its fp16 scale in f32: no
//     rounding but f32's.
//   O += p v~.  A = p times the value's block scale; B = the exact integer
//     codes (a permute and a subtraction per two codes: here the sum over many
//     tokens would lose too much to a common offset).  Four tokens' codes of
//     one element are one word of the layout, and the score fragment's columns
//     are assigned to tokens so that a lane's four scores are those of the same
//     four tokens: p never leaves its lane.
// With 8 rows both A operands are two f16 pieces, the rounded value in rows
// 0-7 and the remainder in rows 8-15 (22 bits together): f32 accuracy at no
// extra product.  With 16 rows (the 16-bit types, where a call has more than
// eight) the rounded value alone is used.
// What bounds it: the code stream (HBM) for long caches, against the chain of
// one turn (scores, vote, exponentials, conversions, products; about 460
// instructions per record) in three warps a scheduler, which registers (168 a
// thread, 64 of them accumulators) do not let be more: issue is active half of
// the time, the tensor pipe 29 %.  131072 tokens of 8 heads x 128, 4 query
// heads each (285 MB): 66 us, 4.3 TB/s, 0.64 of the measured copy rate, about 9
// us of it beginning and joining; 48 sequences of up to 9000 tokens of 8 x 256
// in f32 (1.1 GB): 192 us, 5.7 TB/s, 0.84.  A short call is latency: looking
// the lists up, the pages, the queries and the first record follow one another
// (5 us), then the record loop, then the join (2-6 us): 129 tokens 7.7 us.  A
// CTA with several pieces goes through that for each, since the merge uses the
// rings: nothing of the next piece is asked for before it (16 sequences with
// five new tokens each and a window of 1024: 27 us, 10.6 for the bytes).
// The running reference m is the largest s + log2(largest value scale of the
// token), not the largest s: then p times a scale is at most 1 whatever the
// scales are, and stays in f16's range.  The state is rescaled only when the
// reference would grow by more than 2^7 (one vote per record otherwise).
#include "gq_kv.cuh"
#include "gq_tc.cuh"

namespace gq {
namespace kv {

constexpr int kWarps = 4;
constexpr int kAttnThreads = kWarps * 32;
constexpr int kMaxCtas = 640;       // stretches per call, at most: four CTAs on each of 160 SMs
constexpr float kFloor = -FLT_MAX;  // reference of a row that has seen no token: below every score
// p is kept times 2^7, and with the slack of 2^7 below 2^15.  Both of 7 so that it
// stays there for scores whose spacing is some octaves: m - 7 is then rounded by
// less than what the spacing keeps a score away from m + 7.
constexpr float kHead = 7.0f;
constexpr float kSlack = 7.0f;


template <int D, int kRows>
struct SplitCfg {
    // records per ring stage: two share one wait, one vote and one loop turn
    static constexpr int kUnit = D == 256 ? 1 : 2;
    static constexpr int kStages = D == 256 ? 3 : (D == 128 ? 2 : 3);
    static constexpr int kStage = kUnit * rec_bytes(D);
    static constexpr int kRing = kStages * kStage;
    // the accumulators take most of the registers, so the query fragments (the
    // same for all warps) lie in shared memory (head_dim 128, 16 rows: 98.6 us
    // with them in registers, 86.5 us here)
    static constexpr bool kQSmem = D >= 128;
    static constexpr int kQ = kQSmem ? (D / 16) * 32 * 16 : 0;
    // the merge of the warps' states, and the weights of an item's parts, reuse the
    // rings; they must not set the size (weights of 1024 parts did at head_dim 64
    // with 16 rows, and cost the fourth CTA of an SM: 76.3 us against 73.3, 16
    // sequences of 16384 tokens, four new ones each)
    static constexpr int kRings = kWarps * kRing;
    static_assert(kWarps * kRows * (D + 4) * 4 <= kRings && kRows * kMaxCtas * 4 <= kRings, "merge and join fit the rings");
    static constexpr int kSmem = kRings + kQ;
};

// Partial results: per CTA two slots of {O[rows][D], m[rows], l[rows]} f32.
__host__ __device__ constexpr size_t slot_floats(int D, int rows) { return static_cast<size_t>(rows) * (D + 2); }

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
__device__ __forceinline__ long long seq_cost(const Seq &s, const Batch &B, const Args &A, int rows)
{
    const int tiles = (s.n * A.group + rows - 1) / rows;
    return static_cast<long long>(tiles) * B.kv_heads * span_of(s, A.window).n;
}
// A cut at x inside an item of n units that begins at x0: moved to the item's
// end if that is closer than `tol`, the units that a CTA streams in the time
// which beginning another piece and joining its part would take it (about 7 us),
// and at most a stretch.
template <int D>
__device__ __forceinline__ int snap_tol(long long len)
{
    return static_cast<int>(min(len, static_cast<long long>(D == 256 ? 12 : 32)));
}
__device__ __forceinline__ long long snap(long long x, long long x0, int n, int tol)
{
    return x - x0 < tol ? x0 : (x0 + n - x < tol ? x0 + n : x);
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
// d = A B
__device__ __forceinline__ void mma16816_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// Code bytes of w as f16 subnormals (u 2^-24): bytes 0, 1 or 2, 3.
__device__ __forceinline__ uint32_t bytes01(uint32_t w) { return __byte_perm(w, 0u, 0x4140u); }
__device__ __forceinline__ uint32_t bytes23(uint32_t w) { return __byte_perm(w, 0u, 0x4342u); }
// About log2 of a value scale (below it by at most 0.09): the upper 24 bits of
// the f32 number count 2^-15 octaves; they are placed under the exponent of
// 2^23.  A scale of 0, a token without a value, counts as 2^-80: its p, which
// only the sum l takes, stays in f32's range (2^94), and the reference is that
// of the tokens with values unless they lie 80 octaves further down.
__device__ __forceinline__ float octaves(float d)
{
    const uint32_t bits = __float_as_uint(fmaxf(d, 0x1p-80f));
    return fmaf(__uint_as_float(__byte_perm(bits, 0x4B000000u, 0x7321u)), 0x1p-15f, -(256.0f + 127.0f));
}
// (a, b) -> f16x2 of the rounded values and of the remainders.
__device__ __forceinline__ void split2(float a, float b, uint32_t &hi, uint32_t &lo)
{
    hi = f2_half2(a, b);
    const float2 r = ffma2(half2_f2(hi), make_float2(-1.f, -1.f), make_float2(a, b));
    lo = f2_half2(r.x, r.y);
}
// kRows = 8: two pieces per operand (any type); 16: the 16-bit types' single
// piece, rows 8-15 of the fragments being query rows.
template <int D, int kRows>
__global__ void __launch_bounds__(kAttnThreads, D == 256 ? 2 : (D == 128 ? 3 : 4)) k_kv_attn_split(Args A, Batch B)
{
    using C = SplitCfg<D, kRows>;
    constexpr int nb = D / 32, kStages = C::kStages, kUnit = C::kUnit;
    constexpr int NR = kRows / 8;         // query rows per lane
    constexpr bool kExact = kRows == 8;
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ __align__(8) uint64_t bars[kWarps * kStages];
    __shared__ long long warp_sum[kWarps];
    __shared__ long long s_begin, s_end, s_at;
    __shared__ int s_seq, s_last;
    __shared__ volatile int s_abort;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    uint8_t *my_ring = ring + warp * C::kRing;
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
    auto cost = [&](int b) { return seq_cost(load_seq(B, b), B, A, kRows); };
    plan<kAttnThreads>(B.n_seq, cost, warp_sum, total, excl, b0, b1);
    // at least two records a warp: a shorter stretch would spend more on its start
    const long long len = max((total + gridDim.x - 1) / gridDim.x, static_cast<long long>(2 * kWarps));
    const long long cut0 = len * blockIdx.x, cut1 = cut0 + len;
    const int tol = snap_tol<D>(len);
    if (cut0 >= total) return;
    {
        long long at = excl;
        for (int b = b0; b < b1; ++b) {
            const Seq s = load_seq(B, b);
            const long long c = seq_cost(s, B, A, kRows);
            const int n = span_of(s, A.window).n;
            if (cut0 >= at && cut0 < at + c) {
                s_begin = snap(cut0, at + (cut0 - at) / n * n, n, tol);
                s_seq = b;
                s_at = at;
            }
            if (cut1 >= at && cut1 < at + c) s_end = snap(cut1, at + (cut1 - at) / n * n, n, tol);
            at += c;
        }
        if (cut1 >= total && threadIdx.x == 0) s_end = total;
    }
    __syncthreads();
    const long long begin = s_begin, end = s_end;
    int b = s_seq;
    long long at = s_at;  // where sequence b begins
    uint32_t fill = 0;    // records this warp has taken so far (ring position and parity)

    for (long long x = begin; x < end;) {
        // ---- the item at x
        const Seq s = load_seq(B, b);
        const Span sp = span_of(s, A.window);
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

        const int rows = s.n * A.group, r0 = kRows * tile;
        const int last_tok = min((r0 + kRows - 1) / A.group, s.n - 1), first_tok = r0 / A.group;
        const int item_hi = min(s.first + last_tok, s.kv - 1);                     // positions that some row sees
        const int item_lo = A.window > 0 ? max(0, s.first + first_tok - A.window + 1) : 0;
        const int all_hi = min(s.first + first_tok, s.kv - 1);                     // and that every row sees
        const int all_lo = A.window > 0 ? max(0, s.first + last_tok - A.window + 1) : 0;
        // this CTA's records of the item
        const int rec0 = max(sp.lo + from, item_lo / kRec);
        const int rec1 = item_hi < 0 ? rec0 : min(sp.lo + to, item_hi / kRec + 1);

        {   // the query rows on their way while the pages are looked up
            const int r = r0 + g < rows ? r0 + g : 0, el = type_size(A.type);
            const uint8_t *p = A.Q + (s.row0 + r / A.group) * A.ldq + (static_cast<long long>(h * A.group + r % A.group) * D + 8 * t) * el;
#pragma unroll
            for (int i = 0; i < nb; ++i) asm volatile("prefetch.global.L1 [%0];" ::"l"(p + 32 * i * el));
        }
        // ---- the ring's first records; the places of the next 32 of this warp's sit one per lane
        const int mine0 = rec0 + warp * kUnit;
        constexpr int kStep = kWarps * kUnit, kAhead = 32 / kUnit;
        long long off = -1;
        int off_base = mine0;
        uint32_t off_ok = 0;
        auto load_offs = [&](int base) {
            const int rec = base + lane / kUnit * kStep + lane % kUnit;
            off = -1;
            if (rec < rec1) {
                const int pg = page_of(B, b, rec);
                if (pg >= 0) off = rec_off(B, pg, h, rec, D);
            }
            off_ok = __ballot_sync(0xffffffffu, off >= 0);
            off_base = base;
        };
        load_offs(mine0);
        uint32_t good = 0;       // bits kUnit (n % 8): which records of stage number n were copied
        uint32_t ahead = fill;   // stages asked for so far
        auto issue = [&](int rec) {
            int k = (rec - off_base) / kStep;
            if (k >= kAhead) {
                load_offs(rec);
                k = 0;
            }
            const uint32_t v = (off_ok >> (k * kUnit)) & ((1u << kUnit) - 1u), sh = (ahead & 7) * kUnit;
            good = (good & ~(((1u << kUnit) - 1u) << sh)) | (v << sh);
            const uint32_t st = ahead % kStages, bar = bar0 + 8 * st;
            if (lane / kUnit == k) {  // the lanes that hold the places
                if (lane % kUnit == 0) {
                    if (v) tcu::mbar_expect_tx(bar, __popc(v) * rec_bytes(D));
                    else tcu::mbar_arrive(bar);
                }
                if (off >= 0)
                    tcu::bulk_load(ring_u32 + st * C::kStage + lane % kUnit * rec_bytes(D), A.cache + off, rec_bytes(D), bar);
            }
            ++ahead;
        };
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i)
            if (mine0 + i * kStep < rec1) issue(mine0 + i * kStep);

        // ---- the rows of this lane, g and g + 8, and their query fragments: q * 2^-e in
        // f16 (and its remainder), e from the row's largest magnitude
        int row_hi[NR], row_lo[NR];   // positions that the row sees
        uint32_t qf[nb][2][4];        // block, K step: {k 0-7: rows g, g + 8, k 8-15: rows g, g + 8}
        float2 bias[NR][nb];          // -128 2^-24 times the block's sum of q, twice
        float zs[NR];                 // score = sum * zs
#pragma unroll
        for (int e = 0; e < NR; ++e) {
            const int r = r0 + g + 8 * e;
            const bool live = r < rows;
            const int tok = live ? r / A.group : 0, pos = s.first + tok;
            row_hi[e] = live ? min(pos, s.kv - 1) : -1;
            row_lo[e] = A.window > 0 ? max(0, pos - A.window + 1) : 0;
            const int el = type_size(A.type);
            const uint8_t *p = A.Q + (s.row0 + tok) * A.ldq +
                               (static_cast<long long>(h * A.group + (live ? r % A.group : 0)) * D + 8 * t) * el;
            float q[nb][8], amax = 0.f;
#pragma unroll
            for (int i = 0; i < nb; ++i) {
                float4 u = make_float4(0.f, 0.f, 0.f, 0.f), v = u;
                if (live) {
                    const uint8_t *w = p + 32 * i * el;
                    if (A.type == GQ_TYPE_F32) {
                        u = load4<GQ_TYPE_F32>(w);
                        v = load4<GQ_TYPE_F32>(w + 16);
                    } else if (A.type == GQ_TYPE_BF16) {
                        u = load4<GQ_TYPE_BF16>(w);
                        v = load4<GQ_TYPE_BF16>(w + 8);
                    } else {
                        u = load4<GQ_TYPE_F16>(w);
                        v = load4<GQ_TYPE_F16>(w + 8);
                    }
                }
                q[i][0] = u.x, q[i][1] = u.y, q[i][2] = u.z, q[i][3] = u.w;
                q[i][4] = v.x, q[i][5] = v.y, q[i][6] = v.z, q[i][7] = v.w;
#pragma unroll
                for (int k = 0; k < 8; ++k) amax = fmaxf(amax, fabsf(q[i][k]));
            }
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            // amax * 2^-e in [2^9, 2^10) for 2^-100 <= amax < 2^102; both factors are normal
            const int be = static_cast<int>(__float_as_uint(amax) >> 23) - 126;
            const int ex = min(max(be, -100), 102) - 10;
            const float f = pow2i(-ex);
#pragma unroll
            for (int i = 0; i < nb; ++i) {
                float sum = 0.f;
#pragma unroll
                for (int k = 0; k < 4; ++k) {  // K step k / 2, half k % 2
                    const float a = q[i][2 * k] * f, c = q[i][2 * k + 1] * f;
                    uint32_t *dst = &qf[i][k >> 1][2 * (k & 1)];
                    if (kExact) {
                        split2(a, c, dst[0], dst[1]);
                        const float2 lo = half2_f2(dst[1]);
                        sum += lo.x + lo.y;
                    } else {
                        dst[e] = f2_half2(a, c);
                    }
                    const float2 hi = half2_f2(dst[e]);
                    sum += hi.x + hi.y;
                }
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                bias[e][i] = make_float2(-0x1p-17f * sum, -0x1p-17f * sum);
            }
            zs[e] = A.scale * pow2i(ex) * 0x1p24f;
        }
        uint4 *qs = reinterpret_cast<uint4 *>(ring + C::kRings) + lane;
        if (C::kQSmem) {
#pragma unroll
            for (int i = 0; i < nb; ++i)
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    if ((2 * i + k) % kWarps == warp)
                        qs[(2 * i + k) * 32] = make_uint4(qf[i][k][0], qf[i][k][1], qf[i][k][2], qf[i][k][3]);
            __syncthreads();
        }
        auto query = [&](int i, int k) {
            if (C::kQSmem) return qs[(2 * i + k) * 32];
            return make_uint4(qf[i][k][0], qf[i][k][1], qf[i][k][2], qf[i][k][3]);
        };
        const float kLog2e = 1.4426950408889634f;
        const bool capped = A.softcap > 0.f;
        const float inv_cap = capped ? inverse_cap(A.softcap) : 0.f;
        if (!capped) {
#pragma unroll
            for (int e = 0; e < NR; ++e) zs[e] *= kLog2e;
        }

        float o[nb * 4][4];
#pragma unroll
        for (int i = 0; i < nb * 4; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) o[i][k] = 0.f;
        float m[NR], l[NR];
#pragma unroll
        for (int e = 0; e < NR; ++e) m[e] = kFloor, l[e] = 0.f;

        // ---- the records
        for (int rec = mine0; rec < rec1; rec += kStep, ++fill) {
            const int nxt = rec + (kStages - 1) * kStep;
            if (nxt < rec1) issue(nxt);  // into the stage that the previous turn has left
            const uint32_t st = fill % kStages;
            if (!tcu::wait_warp(bar0 + 8 * st, (fill / kStages) & 1, &s_abort, B.status)) break;
            const uint32_t have = (good >> ((fill & 7) * kUnit)) & ((1u << kUnit) - 1u);
            if (have == 0) continue;  // no such page: nothing to attend to
            const uint8_t *R = my_ring + st * C::kStage;

            // scores of tokens 4 t .. 4 t + 3 of every record, in pairs
            float2 sc[NR][kUnit][2];
#pragma unroll
            for (int e = 0; e < NR; ++e)
#pragma unroll
                for (int u = 0; u < kUnit; ++u) sc[e][u][0] = sc[e][u][1] = make_float2(0.f, 0.f);
            const int tk = 4 * (g >> 1) + (g & 1);  // column g of the first half's fragment; + 2 in the second
#pragma unroll
            for (int i = 0; i < nb; ++i) {
                const uint4 q0 = query(i, 0), q1 = query(i, 1);
#pragma unroll
                for (int u = 0; u < kUnit; ++u) {
                    const uint8_t *Ru = R + u * rec_bytes(D);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint2 w = *reinterpret_cast<const uint2 *>(Ru + k_code_off(tk + 2 * j, i, nb) + 8 * t);
                        float c[4];
                        mma16816_zero(c, q0.x, q0.y, q0.z, q0.w, bytes01(w.x), bytes23(w.x));
                        mma16816(c, q1.x, q1.y, q1.z, q1.w, bytes01(w.y), bytes23(w.y));
                        const float2 d = make_float2(__half2float(*reinterpret_cast<const __half *>(Ru + k_scale_off(4 * t + 2 * j, i, D))),
                                                     __half2float(*reinterpret_cast<const __half *>(Ru + k_scale_off(4 * t + 2 * j + 1, i, D))));
                        float2 x = __fadd2_rn(make_float2(c[0], c[1]), bias[0][i]);
                        if (kExact) x = __fadd2_rn(x, make_float2(c[2], c[3]));
                        sc[0][u][j] = ffma2(x, d, sc[0][u][j]);
                        if (NR == 2)
                            sc[NR - 1][u][j] = ffma2(__fadd2_rn(make_float2(c[2], c[3]), bias[NR - 1][i]), d,
                                                     sc[NR - 1][u][j]);
                    }
                }
            }
            // value scales of the same tokens: their largest, in octaves
            const int p0 = rec * kRec;
            const bool edge = p0 < all_lo || p0 + kUnit * kRec - 1 > all_hi || have != (1u << kUnit) - 1u;  // warp-uniform
            float z[NR][kUnit][4], top[NR];
#pragma unroll
            for (int e = 0; e < NR; ++e) top[e] = -INFINITY;
#pragma unroll
            for (int u = 0; u < kUnit; ++u) {
                uint32_t mx0 = 0, mx1 = 0;
#pragma unroll
                for (int i = 0; i < nb; ++i) {
                    const uint2 d = *reinterpret_cast<const uint2 *>(R + u * rec_bytes(D) + v_scale_off(4 * t, i, D));
                    mx0 = __vmaxu2(mx0, d.x);  // non-negative fp16 order like integers
                    mx1 = __vmaxu2(mx1, d.y);
                }
                const float2 d01 = half2_f2(mx0), d23 = half2_f2(mx1);
                const float lg[4] = {octaves(d01.x), octaves(d01.y), octaves(d23.x), octaves(d23.y)};
#pragma unroll
                for (int e = 0; e < NR; ++e) {
                    z[e][u][0] = sc[e][u][0].x * zs[e], z[e][u][1] = sc[e][u][0].y * zs[e];
                    z[e][u][2] = sc[e][u][1].x * zs[e], z[e][u][3] = sc[e][u][1].y * zs[e];
                    if (capped) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) z[e][u][k] = soft_cap(z[e][u][k], A.softcap, inv_cap) * kLog2e;
                    }
                    if (edge) {  // hidden tokens: what the page holds there is not looked at
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int j = p0 + u * kRec + 4 * t + k;
                            if (j < row_lo[e] || j > row_hi[e] || !((have >> u) & 1u)) z[e][u][k] = -INFINITY;
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) top[e] = fmaxf(top[e], z[e][u][k] + lg[k]);
                }
            }
            bool grow = false;
#pragma unroll
            for (int e = 0; e < NR; ++e) grow = grow || top[e] > m[e] + kSlack;
            if (__any_sync(0xffffffffu, grow)) {
                float f[2];
#pragma unroll
                for (int e = 0; e < NR; ++e) {
                    top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 1));
                    top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 2));
                    const float nm = fmaxf(m[e], top[e]);
                    f[e] = ex2(m[e] - nm);
                    m[e] = nm;
                    l[e] *= f[e];
                }
                if (NR == 1) f[1] = f[0];  // the remainders' rows
#pragma unroll
                for (int i = 0; i < nb * 4; ++i)
#pragma unroll
                    for (int k = 0; k < 4; ++k) o[i][k] *= f[k >> 1];
            }
#pragma unroll
            for (int u = 0; u < kUnit; ++u) {
                const uint8_t *Ru = R + u * rec_bytes(D);
                float2 p[NR][2];
#pragma unroll
                for (int e = 0; e < NR; ++e) {
                    const float ref = m[e] - kHead;
                    p[e][0] = make_float2(ex2(z[e][u][0] - ref), ex2(z[e][u][1] - ref));
                    p[e][1] = make_float2(ex2(z[e][u][2] - ref), ex2(z[e][u][3] - ref));
                    const float2 sum = __fadd2_rn(p[e][0], p[e][1]);
                    l[e] += sum.x + sum.y;
                }
                // value scales that no row sees count as 0: the page may hold NaN there
                uint32_t keep0 = 0xFFFFFFFFu, keep1 = 0xFFFFFFFFu;
                if (edge) {
                    const int j = p0 + u * kRec + 4 * t;
                    const int lo = (have >> u) & 1u ? item_lo - j : 4, hi = item_hi - j;
                    keep0 = (lo <= 0 && hi >= 0 ? 0x0000FFFFu : 0u) | (lo <= 1 && hi >= 1 ? 0xFFFF0000u : 0u);
                    keep1 = (lo <= 2 && hi >= 2 ? 0x0000FFFFu : 0u) | (lo <= 3 && hi >= 3 ? 0xFFFF0000u : 0u);
                }
#pragma unroll
                for (int i = 0; i < nb; ++i) {
                    const uint2 dv = *reinterpret_cast<const uint2 *>(Ru + v_scale_off(4 * t, i, D));
                    const float2 e0 = half2_f2(dv.x & keep0), e1 = half2_f2(dv.y & keep1);
                    const float2 x0 = __fmul2_rn(p[0][0], e0), x1 = __fmul2_rn(p[0][1], e1);
                    uint32_t a0, a1 = 0u, a2, a3 = 0u;
                    if (kExact) {
                        split2(x0.x, x0.y, a0, a1);
                        split2(x1.x, x1.y, a2, a3);
                    } else {
                        a0 = f2_half2(x0.x, x0.y);
                        a2 = f2_half2(x1.x, x1.y);
                        if (NR == 2) {
                            const float2 y0 = __fmul2_rn(p[NR - 1][0], e0), y1 = __fmul2_rn(p[NR - 1][1], e1);
                            a1 = f2_half2(y0.x, y0.y);
                            a3 = f2_half2(y1.x, y1.y);
                        }
                    }
                    const uint4 w = *reinterpret_cast<const uint4 *>(Ru + v_chunk_off(t, 8 * i + g, D));
                    mma16816(o[4 * i], a0, a1, a2, a3, codes2(w.x, 0x4140u), codes2(w.x, 0x4342u));
                    mma16816(o[4 * i + 1], a0, a1, a2, a3, codes2(w.y, 0x4140u), codes2(w.y, 0x4342u));
                    mma16816(o[4 * i + 2], a0, a1, a2, a3, codes2(w.z, 0x4140u), codes2(w.z, 0x4342u));
                    mma16816(o[4 * i + 3], a0, a1, a2, a3, codes2(w.w, 0x4140u), codes2(w.w, 0x4342u));
                }
            }
            __syncwarp();  // every lane has read the stage before it is filled again
        }
        // after a wait that gave up: let the copies in flight land (bounded again)
        for (; fill != ahead; ++fill) tcu::wait_warp(bar0 + 8 * (fill % kStages), (fill / kStages) & 1, &s_abort, B.status);
#pragma unroll
        for (int e = 0; e < NR; ++e) {
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
        }

        // ---- merge the four warps' states through shared memory (row stride D + 4)
        __syncthreads();
        float *mo = reinterpret_cast<float *>(ring);        // [warp][rows][D + 4]; elements D, D + 1 hold m, l
#pragma unroll
        for (int e = 0; e < NR; ++e) {
            float *mine = mo + (warp * kRows + g + 8 * e) * (D + 4);
#pragma unroll
            for (int i = 0; i < nb; ++i) {
                // fragment column n of quarter i' is element 32 i + 4 n + i'; columns 2 t, 2 t + 1
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float x[4];
#pragma unroll
                    for (int n = 0; n < 4; ++n) x[n] = o[4 * i + n][2 * e + k] + (kExact ? o[4 * i + n][2 + k] : 0.f);
                    *reinterpret_cast<float4 *>(mine + 32 * i + 8 * t + 4 * k) = make_float4(x[0], x[1], x[2], x[3]);
                }
            }
            if (t == 0) {
                mine[D] = m[e];
                mine[D + 1] = l[e];
            }
        }
        __syncthreads();
        const bool whole = from == 0 && to == sp.n;
        constexpr int kQuads = kRows * D / 4;
        float *slot = A.part + (2ll * blockIdx.x + (from == 0 ? 1 : 0)) * slot_floats(D, kRows);
        auto store_row = [&](int rr, int d, float4 v, float inv) {
            const int row = r0 + rr;
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
            // the last of the item's CTAs joins their parts, in the order of the stretches: the first
            // is the one after the last cut that was moved to the item's start, and there is one more
            // for every cut that stayed inside
            const int c0 = static_cast<int>((item_x + min(tol, sp.n) - 1) / len);
            const int c1 = static_cast<int>((item_x + sp.n - tol) / len);
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
                // the parts' weights first, a warp per row, then the rows with every load independent
                auto part = [&](int c) { return A.part + (2ll * c + (c == c0 ? 1 : 0)) * slot_floats(D, kRows); };
                const int np = c1 - c0 + 1;
                float *wt = mo;  // [row][part]: weight of a part divided by the row's sum
                for (int rr = warp; rr < kRows; rr += kWarps) {
                    float M = kFloor, L = 0.f;
                    for (int c = lane; c < np; c += 32) M = fmaxf(M, __ldcg(part(c0 + c) + kRows * D + rr));
#pragma unroll
                    for (int k = 16; k > 0; k >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, k));
                    for (int c = lane; c < np; c += 32) {
                        const float f = ex2(__ldcg(part(c0 + c) + kRows * D + rr) - M);
                        L += f * __ldcg(part(c0 + c) + kRows * D + kRows + rr);
                        wt[rr * np + c] = f;
                    }
#pragma unroll
                    for (int k = 16; k > 0; k >>= 1) L += __shfl_xor_sync(0xffffffffu, L, k);
                    const float inv = L == 0.f ? 0.f : 1.0f / L;
                    for (int c = lane; c < np; c += 32) wt[rr * np + c] *= inv;
                }
                __syncthreads();
                for (int i = threadIdx.x; i < kQuads; i += kAttnThreads) {
                    const int rr = i / (D / 4), d = 4 * (i % (D / 4));
                    if (r0 + rr >= rows) break;
                    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
                    for (int c = 0; c < np; ++c) {
                        const float f = wt[rr * np + c];
                        const float4 u = __ldcg(reinterpret_cast<const float4 *>(part(c0 + c) + rr * D + d));
                        v.x += f * u.x, v.y += f * u.y, v.z += f * u.z, v.w += f * u.w;
                    }
                    store_row(rr, d, v, 1.0f);
                }
            }
        }
        __syncthreads();           // the ring is free again
        tcu::fence_async_smem();   // before bulk copies overwrite what generic stores wrote
        if (s_abort) return;       // uniform after the barrier; every part of a cut item stays unfinished
    }
}

template <int D, int kRows>
static int launch_rows(const Args &A, const Batch &B, cudaStream_t s)
{
    using C = SplitCfg<D, kRows>;
    auto kern = k_kv_attn_split<D, kRows>;
    const int occ = ctas_per_sm(reinterpret_cast<const void *>(kern), kAttnThreads, C::kSmem);
    if (occ < 1) return GQ_ERR_CUDA;
    int grid = sm_count() * occ;
    if (grid > kMaxCtas) grid = kMaxCtas;
    return status_from(launch_pdl(kern, dim3(grid), dim3(kAttnThreads), C::kSmem, s, A, B));
}

// rows: query rows per sequence and kv head, on average
template <int D>
static int launch_split(const Args &A, const Batch &B, long long rows, cudaStream_t s)
{
    return A.type != GQ_TYPE_F32 && rows > 8 ? launch_rows<D, 16>(A, B, s) : launch_rows<D, 8>(A, B, s);
}

}  // namespace kv

// Workspace: the split form's counters, the chunk form's, then the partial
// results of whichever runs.
static size_t counter_bytes() { return ((kv::kMaxCtas + kv_chunk_counters()) * sizeof(int) + 127) / 128 * 128; }

size_t kv_attention_workspace_bytes(int head_dim)
{
    const size_t split = 2ull * kv::kMaxCtas * kv::slot_floats(head_dim, 16) * sizeof(float), chunk = kv_chunk_part_bytes(head_dim);
    return counter_bytes() + (split > chunk ? split : chunk);
}

int launch_kv_attention(const void *Q, long long ldq, const uint8_t *cache, const kv::Batch &B, void *O, long long ldo,
                        int type, float scale, float softcap, int window, void *ws, int heads, int head_dim,
                        cudaStream_t s)
{
    int *counter = static_cast<int *>(ws);
    float *part = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + counter_bytes());
    // Query rows per sequence and kv head, on average.  From 64 on the tensor
    // cores' form is faster: 16 sequences of 4096 tokens, 8 kv heads x 128, 4
    // query heads each, bf16: 32 rows 70 us here and 100 there, 64 rows 110 and
    // 101, 128 rows 202 and 79; f32: 94 and 121, 177 and 123, 336 and 119.  (One
    // sequence of 8192: 64 rows 37 and 43 us, 128 rows 45 and 41.)  These are calls
    // of equal sequences; one kernel serves the whole call, so that in a call of
    // single tokens beside a long chunk one or the other runs in the form that is
    // slower for it.  head_dim 256 in f32 has no form there: both pieces of its
    // query operand do not fit a CTA's shared memory beside keys and values.
    const long long rows = static_cast<long long>(B.n_tokens) * (heads / B.kv_heads) / B.n_seq;
    if (rows >= 64 && (type != GQ_TYPE_F32 || head_dim <= 128))
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
    case 64: return kv::launch_split<64>(A, B, rows, s);
    case 128: return kv::launch_split<128>(A, B, rows, s);
    default: return kv::launch_split<256>(A, B, rows, s);
    }
}

}  // namespace gq
