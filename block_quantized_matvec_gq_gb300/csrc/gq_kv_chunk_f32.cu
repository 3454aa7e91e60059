// gq_kv_chunk_f32.cu -- attention of chunks of new tokens over the paged Q8_0
// cache on tcgen05 tensor cores, for f32 token arrays (head_dim 64 and 128).
//
// The items, the line of work and the joining of cut items are those of the
// 16-bit kernel (gq_kv_chunk.cu) with one 128-row tile per CTA.  Every
// operand is two f16 pieces, the rounded value and the remainder: 22 bits of
// q and p, and all 18 bits of a cached value d * q.  Of the four products the
// one of the two remainders is left out (below 2^-22 relative):
//   S = q1 (k1, k2) + q2 k1.  k1 and k2 of 64 tokens are the 128 rows of one
//     operand tile, so the first two products are one N = 128 MMA per K step
//     (64 cycles; two of N = 64 would take 48 each, A's shared-memory reads
//     being the limit); their sums lie in separate columns, which the softmax
//     adds.
//   O = p1 v1 + p2 v1 + p1 v2.
// The tensor core's f32 sums truncate, so the accumulator of a tile starts
// from 0 and is added, rounded to nearest, into registers: over a long cache
// the bias of thousands of truncated additions into tensor memory would pass
// 1e-5.  With the sum in registers a changed reference costs no pass over
// tensor memory either.
//
// Warpgroups: softmax (a thread per query row), accumulation (a thread per
// row, head_dim sums in registers; the result rows), dequantizers, and
// {producer, mma}.  Tensor memory: two score tiles of 128 columns (p1 and p2
// over them) and two product tiles of head_dim columns.
// What bounds it: per tile of 64 tokens the tensor core takes 8 (64 + 48)
// cycles for S and 12 * 64 for O at head_dim 128, 1664 in all; a tile takes
// about 2500, the rest being waits between the roles and for instructions.  2048
// tokens behind 30720 cached ones, 32 heads over 8 x 128: 2356 us, 452 TFLOP/s
// of the attention's own products (three times that on the tensor cores); 509
// behind 7682: 199 us, of which some 40 are the beginning of the items and the
// joining of cut ones.  (2187 and 179 us before the values' sizes were looked
// at, gq_kv_chunk.cuh; head_dim 64 2050 us before and after.)
#include "gq_kv_chunk.cuh"

namespace gq {
namespace kv {
namespace chunk {

template <int D>
struct CfgF32 {
    static constexpr int kMt = 1;
    static constexpr int kKt = 64;
    static constexpr int kRowsItem = 128;
    static constexpr int kQ = 128 * D * 2;           // one piece of the query operand
    static constexpr int kOp = 2 * kKt * D * 2;      // both pieces of keys or values
    static constexpr int kRecs = kKt / kRec;
    static constexpr int kHalf = 17 * D;
    static constexpr int kRaw = kRecs * kHalf;
    // Four operand tiles: with three, the keys of the next tile could only be
    // converted once this tile's p v had freed its values, just when the tensor
    // core asks for them.
    static constexpr int kOps = 4, kRaws = 3;
    static constexpr int kOffOp = 2 * kQ;
    static constexpr int kOffRaw = kOffOp + kOps * kOp;
    static constexpr int kOffState = kOffRaw + kRaws * kRaw;      // {m, l}[4 tiles][128 rows]
    static constexpr int kOffBar = kOffState + 4 * 128 * 8;
    // raw full/empty, operand full/empty, q full, s full [2], p full [2], o full [2], o empty [2], fixed
    static constexpr int kBars = 2 * kRaws + 2 * kOps + 10;
    static constexpr int kSmem = kOffBar + 8 * kBars;  // and 4.5 KB of static arrays
    static constexpr int kDeqWarp = 8, kDeqWarps = 8, kProdWarp = 16, kMmaWarp = 17, kWarpsAll = 20;
    static constexpr int kThreads = 32 * kWarpsAll;
    // registers per thread after the split; the shares stay within the launch's 640 x 96
    static constexpr int kSoftRegs = 120, kAccRegs = 168, kDeqRegs = 64, kRestRegs = 64;
    static_assert(kSoftRegs + kAccRegs + 2 * kDeqRegs + kRestRegs <= 5 * 96, "register split");
    static_assert(kOffOp % 128 == 0 && kOffRaw % 128 == 0 && kOffState % 16 == 0 && kSmem + 4608 <= 232448, "shared memory layout");
};

// c * d as f16x2 rounded, and the exact remainder (18 bits in two pieces).
__device__ __forceinline__ void pieces(uint32_t c, uint32_t d, uint32_t &hi, uint32_t &lo)
{
    hi = hmul2(c, d);
    const __half2 r = __hfma2(*reinterpret_cast<const __half2 *>(&c), *reinterpret_cast<const __half2 *>(&d),
                              __hneg2(*reinterpret_cast<const __half2 *>(&hi)));
    lo = *reinterpret_cast<const uint32_t *>(&r);
}

// A thread's share of a raw stage, read before the stage before it is
// converted: units of one (token, block) of keys, or of eight tokens of four
// elements of values (as in the 16-bit kernel).
template <int D>
struct RawKeys {
    using C = CfgF32<D>;
    static constexpr int kTh = C::kDeqWarps * 32, kAll = C::kKt * (D / 32), kN = (kAll + kTh - 1) / kTh;
    uint4 w[kN][2];
    uint32_t d[kN];
    __device__ __forceinline__ void load(const uint8_t *raw, int tid)
    {
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int u = tid + i * kTh, tok = u % C::kKt, b = u / C::kKt, t = tok % kRec;
            if (u >= kAll) break;
            const uint8_t *src = raw + tok / kRec * C::kHalf;
            d[i] = *reinterpret_cast<const uint16_t *>(src + k_scale_off(t, b, D));
#pragma unroll
            for (int h = 0; h < 2; ++h)
                w[i][h] = *reinterpret_cast<const uint4 *>(src + k_code_off(t, b, D / 32) + 16 * (h ^ ((t >> 1) & 1)));
        }
    }
    // rows 0-63 the rounded values of 64 tokens, rows 64-127 the remainders
    __device__ __forceinline__ void convert(uint8_t *op, int tid) const
    {
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int u = tid + i * kTh, tok = u % C::kKt, b = u / C::kKt, t = tok % kRec;
            if (u >= kAll) break;
            const uint32_t d2 = d[i] | (d[i] << 16);
            uint8_t *dst = op + (tok >> 3) * 128 + (tok & 7) * 16;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t ww[4] = {w[i][h].x, w[i][h].y, w[i][h].z, w[i][h].w};
                uint8_t *o = dst + (4 * b + 2 * (h ^ ((t >> 1) & 1))) * 2048;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    uint4 hi, lo;
                    pieces(codes2(ww[2 * k], 0x4140u), d2, hi.x, lo.x);
                    pieces(codes2(ww[2 * k], 0x4342u), d2, hi.y, lo.y);
                    pieces(codes2(ww[2 * k + 1], 0x4140u), d2, hi.z, lo.z);
                    pieces(codes2(ww[2 * k + 1], 0x4342u), d2, hi.w, lo.w);
                    *reinterpret_cast<uint4 *>(o + k * 2048) = hi;
                    *reinterpret_cast<uint4 *>(o + k * 2048 + 1024) = lo;
                }
            }
        }
    }
};
template <int D>
struct RawValues {
    using C = CfgF32<D>;
    static constexpr int kTh = C::kDeqWarps * 32, kAll = (C::kKt / 8) * (D / 4), kN = (kAll + kTh - 1) / kTh;
    uint4 w[kN][2], d[kN];
    __device__ __forceinline__ void load(const uint8_t *raw, int tid)
    {
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int u = tid + i * kTh, c = u % (D / 4), t8 = u / (D / 4), g = 2 * (t8 % 2);
            if (u >= kAll) break;
            const uint8_t *src = raw + t8 / 2 * C::kHalf - 17 * D;  // offsets below count from the record
            d[i] = *reinterpret_cast<const uint4 *>(src + v_scale_off(4 * g, c / 8, D));  // eight tokens
            w[i][0] = *reinterpret_cast<const uint4 *>(src + v_chunk_off(g, c, D));
            w[i][1] = *reinterpret_cast<const uint4 *>(src + v_chunk_off(g + 1, c, D));
        }
    }
    // the rounded values' tile, then the remainders'
    __device__ __forceinline__ void convert(uint8_t *op, int tid) const
    {
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int u = tid + i * kTh, c = u % (D / 4), t8 = u / (D / 4);
            if (u >= kAll) break;
            const uint4 s = d[i];
            uint8_t *dst = op + t8 * (D * 16);
            const uint32_t a[4] = {w[i][0].x, w[i][0].y, w[i][0].z, w[i][0].w}, z[4] = {w[i][1].x, w[i][1].y, w[i][1].z, w[i][1].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int n = k * (D / 4) + c;
                uint4 hi, lo;
                pieces(codes2(a[k], 0x4140u), s.x, hi.x, lo.x);
                pieces(codes2(a[k], 0x4342u), s.y, hi.y, lo.y);
                pieces(codes2(z[k], 0x4140u), s.z, hi.z, lo.z);
                pieces(codes2(z[k], 0x4342u), s.w, hi.w, lo.w);
                uint8_t *o = dst + (n >> 3) * 128 + (n & 7) * 16;
                *reinterpret_cast<uint4 *>(o) = hi;
                *reinterpret_cast<uint4 *>(o + C::kKt * D * 2) = lo;
            }
        }
    }
};

__device__ __forceinline__ uint32_t split_lo(float2 x, uint32_t hi)
{
    const float2 r = ffma2(half2_f2(hi), make_float2(-1.f, -1.f), x);
    return f2_half2(r.x, r.y);
}

// This thread's query row, elements * 2^-e (e from its largest magnitude), as
// two pieces; returns 2^e.  A dead row is zeros.
template <int D>
__device__ __forceinline__ float load_query_f32(const float4 *src, bool live, bool negate, uint8_t *op, int row)
{
    float amax = 0.f;
#pragma unroll 8
    for (int i = 0; i < D / 4; ++i) {
        const float4 v = live ? __ldg(src + i) : make_float4(0.f, 0.f, 0.f, 0.f);
        amax = fmaxf(amax, fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w))));
    }
    const int be = static_cast<int>(__float_as_uint(amax) >> 23) - 126;
    const int e = min(max(be, -100), 128) - 10;  // amax * 2^-e in [2^9, 2^10)
    const float f = negate ? -pow2i(-e) : pow2i(-e);
    uint8_t *dst = op + (row >> 3) * 128 + (row & 7) * 16;
#pragma unroll 4
    for (int i = 0; i < D / 8; ++i) {
        const float4 a = live ? __ldg(src + 2 * i) : make_float4(0.f, 0.f, 0.f, 0.f);
        const float4 b = live ? __ldg(src + 2 * i + 1) : make_float4(0.f, 0.f, 0.f, 0.f);
        const float2 x[4] = {make_float2(a.x * f, a.y * f), make_float2(a.z * f, a.w * f), make_float2(b.x * f, b.y * f),
                             make_float2(b.z * f, b.w * f)};
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            hi[k] = f2_half2(x[k].x, x[k].y);
            lo[k] = split_lo(x[k], hi[k]);
        }
        *reinterpret_cast<uint4 *>(dst + i * 2048) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4 *>(dst + CfgF32<D>::kQ + i * 2048) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
    return pow2i(e);
}

template <int D, bool kCap>
__global__ void __launch_bounds__(CfgF32<D>::kThreads, 1) k_kv_attn_chunk_f32(Args A, Batch B)
{
    using C = CfgF32<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ long long s_cost[C::kWarpsAll], s_cut[2];
    __shared__ Walk s_walk;
    __shared__ volatile int s_abort;
    __shared__ uint32_t s_tmem;
    __shared__ uint32_t s_mask[kMaskRing];
    __shared__ __align__(16) float s_dn[kMaskRing * C::kKt];
    __shared__ __align__(16) uint16_t s_scratch[C::kKt];
    __shared__ float2 s_sum[128];
    __shared__ int s_last;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t base = smem_u32(smem);
    const uint32_t raw_full = base + C::kOffBar, raw_empty = raw_full + 8 * C::kRaws, op_full = raw_empty + 8 * C::kRaws,
                   op_empty = op_full + 8 * C::kOps, q_full = op_empty + 8 * C::kOps, s_full = q_full + 8, p_full = s_full + 16,
                   o_full = p_full + 16, o_empty = o_full + 16, fixed = o_empty + 16;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kRaws; ++i) {
            mbar_init(raw_full + 8 * i, 1);
            mbar_init(raw_empty + 8 * i, C::kDeqWarps);
        }
        for (int i = 0; i < C::kOps; ++i) {
            mbar_init(op_full + 8 * i, C::kDeqWarps);
            mbar_init(op_empty + 8 * i, 1);
        }
        mbar_init(q_full, 4);
        mbar_init(fixed, C::kDeqWarps);
        for (int i = 0; i < 2; ++i) {
            mbar_init(s_full + 8 * i, 1);
            mbar_init(p_full + 8 * i, 4);
            mbar_init(o_full + 8 * i, 1);
            mbar_init(o_empty + 8 * i, 4);
        }
        s_abort = 0;
        s_walk.left = 0;
    }
    fence_async_smem();
    if (warp == C::kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    pdl_wait();
    const long long len = find_stretch<C>(B, A, s_cost, s_cut, s_walk);
    Walk w = s_walk;
    volatile int *abort = &s_abort;
    // {m, l} of a tile's rows, from the softmax to the accumulation.  A slot is
    // written again four tiles later: those scores are asked for only after the
    // accumulation has taken this tile's products (o_empty).
    float2 *state = reinterpret_cast<float2 *>(smem + C::kOffState);
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const int row = threadIdx.x & 127;

    if (warp < 4) {
        // ================================================================ softmax: thread = query row
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kSoftRegs));
        const float inv_cap = kCap ? inverse_cap(A.softcap) : 0.f;
        constexpr float kLog2e = 1.4426950408889634f;
        bool ok = true;
        uint32_t n = 0;  // tiles so far
        while (w.left > 0) {
            const Seq s = load_seq(B, w.b);
            const Item it = item_of<C>(s, A, w.st);
            const int to = static_cast<int>(min(static_cast<long long>(it.tiles), w.from + w.left));
            const int r = it.r0 + row;
            const bool live = r < it.rows;
            const int tok = live ? r / A.group : 0, head = w.h * A.group + (live ? r % A.group : 0);
            const int pos = s.first + tok;
            const int row_hi = live ? min(pos, s.kv - 1) : -1;
            const int row_lo = A.window > 0 ? max(0, pos - A.window + 1) : 0;
            // every q k of the piece before is done: its last scores have been taken
            const float f = load_query_f32<D>(
                reinterpret_cast<const float4 *>(A.Q + (s.row0 + tok) * A.ldq) + static_cast<long long>(head) * (D / 4), live,
                A.scale < 0.f, smem, row);
            // a factor of 0 would turn hidden scores (-inf) into NaN
            const float zs = fmaxf(fabsf(A.scale) * f * (kCap ? 1.0f : kLog2e), 1e-37f);
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full);
            float m = kNone, l = 0.f;
            for (int j = w.from; j < to; ++j) {
                const uint32_t buf = n & 1, s_addr = lane_addr + kSCol * buf;
                if (ok) ok = wait_warp(s_full + 8 * buf, (n >> 1) & 1, abort, B.status);
                if (!ok) break;
                tc_fence_after();
                const int p0 = it.base + j * C::kKt;
                const uint32_t word = s_mask[n % kMaskRing], recs = word & ~kMixed;
                const bool edge = __any_sync(0xffffffffu, p0 < row_lo || p0 + C::kKt - 1 > row_hi) || recs != (1u << C::kRecs) - 1u;
                if (kCap) cap_scores<C::kKt, true>(s_addr, zs, A.softcap, inv_cap);
                if (__builtin_expect(word & kMixed, 0))
                    shift_scores<C::kKt, true>(s_addr, kCap ? 1.0f : zs, row_lo - p0, row_hi - p0, recs, s_dn + n % kMaskRing * C::kKt,
                                               s_sum + threadIdx.x);
                float v[C::kKt];
#pragma unroll
                for (int c = 0; c < C::kKt; c += 32) {
                    float x[32], y[32];
                    tmem_ld32_async(s_addr + c, x);
                    tmem_ld32_async(s_addr + C::kKt + c, y);
                    tmem_wait_ld(x);
                    tmem_wait_ld(y);
#pragma unroll
                    for (int k = 0; k < 32; k += 2) {
                        const float2 sum = __fadd2_rn(make_float2(x[k], x[k + 1]), make_float2(y[k], y[k + 1]));
                        v[c + k] = sum.x, v[c + k + 1] = sum.y;
                    }
                }
                if (edge) {
                    const int a = row_lo - p0, b = row_hi - p0;
#pragma unroll
                    for (int k = 0; k < C::kKt; ++k)
                        if (k < a || k > b || !((recs >> (k / kRec)) & 1u)) v[k] = -INFINITY;
                }
                float t0 = v[0], t1 = v[1], t2 = v[2], t3 = v[3];
#pragma unroll
                for (int k = 4; k < C::kKt; k += 4) {
                    t0 = fmaxf(t0, v[k]);
                    t1 = fmaxf(t1, v[k + 1]);
                    t2 = fmaxf(t2, v[k + 2]);
                    t3 = fmaxf(t3, v[k + 3]);
                }
                // the scale (its sign is in q) keeps the order of the scores
                const float zt = fmaxf(fmaxf(t0, t1), fmaxf(t2, t3)) * (kCap ? 1.0f : zs);
                if (__any_sync(0xffffffffu, zt > m + kGrow)) {
                    const float nm = fmaxf(m, zt);
                    l *= ex2(m - nm);
                    m = nm;
                }
                const float2 ref = make_float2(kPHead - m, kPHead - m), zs2 = kCap ? make_float2(1.f, 1.f) : make_float2(zs, zs);
                float2 sum0 = make_float2(0.f, 0.f), sum1 = sum0;
#pragma unroll
                for (int c = 0; c < C::kKt; c += 32) {
                    uint32_t hi[16], lo[16];
#pragma unroll
                    for (int k = 0; k < 32; k += 4) {
                        float2 a = ffma2(make_float2(v[c + k], v[c + k + 1]), zs2, ref);
                        float2 b = ffma2(make_float2(v[c + k + 2], v[c + k + 3]), zs2, ref);
                        a.x = ex2(a.x), a.y = ex2(a.y), b.x = ex2(b.x), b.y = ex2(b.y);
                        sum0 = __fadd2_rn(sum0, a);
                        sum1 = __fadd2_rn(sum1, b);
                        hi[k / 2] = f2_half2(a.x, a.y);
                        hi[k / 2 + 1] = f2_half2(b.x, b.y);
                        lo[k / 2] = split_lo(a, hi[k / 2]);
                        lo[k / 2 + 1] = split_lo(b, hi[k / 2 + 1]);
                    }
                    tmem_st16(s_addr + c / 2, hi);  // over the scores, which are in registers
                    tmem_st16(s_addr + 32 + c / 2, lo);
                }
                float sum = (sum0.x + sum0.y) + (sum1.x + sum1.y);
                if (__builtin_expect(s_mask[n % kMaskRing] & kMixed, 0)) sum = s_sum[threadIdx.x].y * ex2(s_sum[threadIdx.x].x - m);
                l += sum;
                state[(n & 3) * 128 + row] = make_float2(m, l);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full + 8 * buf);
                ++n;
            }
            if (!next_piece<C>(w, B, A, to - w.from)) break;
        }
    } else if (warp < C::kDeqWarp) {
        // ================================================================ accumulation: thread = query row
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kAccRegs));
        bool ok = true;
        uint32_t n = 0;
        while (w.left > 0) {
            const Seq s = load_seq(B, w.b);
            const Item it = item_of<C>(s, A, w.st);
            const int to = static_cast<int>(min(static_cast<long long>(it.tiles), w.from + w.left));
            float acc[D], m = kNone, l = 0.f;
#pragma unroll
            for (int c = 0; c < D; ++c) acc[c] = 0.f;
            for (int j = w.from; j < to; ++j) {
                const uint32_t buf = n & 1;
                if (ok) ok = wait_warp(o_full + 8 * buf, (n >> 1) & 1, abort, B.status);
                if (!ok) break;
                tc_fence_after();
                const float2 ml = state[(n & 3) * 128 + row];
                l = ml.y;
                if (__any_sync(0xffffffffu, ml.x != m)) {
                    const float g = ex2(m - ml.x);
                    m = ml.x;
#pragma unroll
                    for (int c = 0; c < D; c += 2) {
                        const float2 a = __fmul2_rn(make_float2(acc[c], acc[c + 1]), make_float2(g, g));
                        acc[c] = a.x, acc[c + 1] = a.y;
                    }
                }
#pragma unroll
                for (int c = 0; c < D; c += 32) {
                    float x[32];
                    tmem_ld32_async(lane_addr + kOCol + buf * D + c, x);
                    tmem_wait_ld(x);
#pragma unroll
                    for (int k = 0; k < 32; k += 2) {
                        const float2 sum = __fadd2_rn(make_float2(acc[c + k], acc[c + k + 1]), make_float2(x[k], x[k + 1]));
                        acc[c + k] = sum.x, acc[c + k + 1] = sum.y;
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(o_empty + 8 * buf);
                ++n;
            }
            // ---- the piece's result
            const int r = it.r0 + row;
            const bool live = r < it.rows;
            const int tok = live ? r / A.group : 0, head = w.h * A.group + (live ? r % A.group : 0);
            float4 *dst = reinterpret_cast<float4 *>(A.O + (s.row0 + tok) * A.ldo) + static_cast<long long>(head) * (D / 4);
            // column i * D / 4 + c is element 4 c + i
            auto put = [&](const float (&x)[D], float f) {
#pragma unroll
                for (int c = 0; c < D / 4; ++c)
                    dst[c] = make_float4(x[c] * f, x[D / 4 + c] * f, x[D / 2 + c] * f, x[3 * D / 4 + c] * f);
            };
            constexpr int kSlot = 128 * (D + 2);  // floats of a partial: [D][128], m, l
            if (w.from == 0 && to == it.tiles) {
                if (live) put(acc, l == 0.f ? 0.f : 1.0f / l);
            } else {
                float *slot = A.part + (2ll * blockIdx.x + (w.from == 0 ? 1 : 0)) * kSlot;
#pragma unroll
                for (int c = 0; c < D; ++c) slot[c * 128 + row] = acc[c];
                slot[D * 128 + row] = m;
                slot[(D + 1) * 128 + row] = l;
                const long long item_x = w.x - w.from;
                const int c0 = first_cta(item_x, it.tiles, len), c1 = last_cta(item_x, it.tiles, len);
                __threadfence();
                bar_sync(1, 128);
                if (row == 0) {
                    const int old = atomicAdd(A.counter + c0, 1);
                    s_last = old == c1 - c0;
                    if (old == c1 - c0) A.counter[c0] = 0;
                }
                bar_sync(1, 128);
                if (s_last) {
                    __threadfence();
                    auto part = [&](int c) { return A.part + (2ll * c + (c == c0 ? 1 : 0)) * kSlot; };
                    float M = kNone, L = 0.f;
#pragma unroll 4
                    for (int c = c0; c <= c1; ++c) M = fmaxf(M, __ldcg(part(c) + D * 128 + row));
#pragma unroll
                    for (int c = 0; c < D; ++c) acc[c] = 0.f;
                    for (int cc = c0; cc <= c1; ++cc) {
                        const float *src = part(cc);
                        const float g = ex2(__ldcg(src + D * 128 + row) - M);
                        L += g * __ldcg(src + (D + 1) * 128 + row);
#pragma unroll
                        for (int c = 0; c < D; ++c) acc[c] += g * __ldcg(src + c * 128 + row);
                    }
                    if (live) put(acc, L == 0.f ? 0.f : 1.0f / L);
                }
                bar_sync(1, 128);  // s_last may be written again
            }
            if (!next_piece<C>(w, B, A, to - w.from)) break;
        }
    } else if (warp < C::kProdWarp) {
        // ================================================================ dequantizers
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kDeqRegs));
        const int tid = threadIdx.x - 32 * C::kDeqWarp;
        bool ok = true;
        uint32_t n = 0, tile_no = 0;  // operand tiles (keys 2 t, values 2 t + 1 of tile t), key tiles
        uint32_t n_fixed = 0;
        RawKeys<D> keys;
        RawValues<D> vals;
        auto raw_of = [&](uint32_t i) -> const uint8_t * {  // waits for raw stage i
            if (ok) ok = wait_warp(raw_full + 8 * (i % C::kRaws), (i / C::kRaws) & 1, abort, B.status);
            return smem + C::kOffRaw + (i % C::kRaws) * C::kRaw;
        };
        auto op_of = [&](uint32_t i) {  // waits for operand stage i
            if (ok && i >= C::kOps) ok = wait_warp(op_empty + 8 * (i % C::kOps), (i / C::kOps - 1) & 1, abort, B.status);
            return smem + C::kOffOp + (i % C::kOps) * C::kOp;
        };
        // the raw stage is given back only now: an arrival right after the loads
        // would not wait for their data
        auto op_done = [&](uint32_t i) {
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(op_full + 8 * (i % C::kOps));
                mbar_arrive(raw_empty + 8 * (i % C::kRaws));
            }
        };
        while (ok && w.left > 0) {
            const Seq s = load_seq(B, w.b);
            const Item it = item_of<C>(s, A, w.st);
            const int to = static_cast<int>(min(static_cast<long long>(it.tiles), w.from + w.left));
            keys.load(raw_of(n), tid);
            if (!ok) break;
            for (int j = w.from; j < to; ++j, ++tile_no, n += 2) {
                const int p0 = it.base + j * C::kKt;
                raw_of(n + 1);
                if (!ok) break;
                uint8_t *raw = smem + C::kOffRaw + (n + 1) % C::kRaws * C::kRaw;
                ok = fix_scales<D, C>(raw, tid, it.lo - p0, it.hi + 1 - p0, s_mask[tile_no % kMaskRing], s_dn + tile_no % kMaskRing * C::kKt,
                                      fixed, n_fixed, abort, B.status);
                if (!ok) break;
                vals.load(raw, tid);
                uint8_t *op = op_of(n);
                if (!ok) break;
                keys.convert(op, tid);
                op_done(n);
                if (j + 1 < to) keys.load(raw_of(n + 2), tid);
                op = op_of(n + 1);
                if (!ok) break;
                vals.convert(op, tid);
                op_done(n + 1);
            }
            if (!ok || !next_piece<C>(w, B, A, to - w.from)) break;
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRestRegs));
        if (w.left > 0 && (warp == C::kProdWarp || warp == C::kProdWarp + 2)) {
            produce<D, C>(warp != C::kProdWarp, w, B, A, smem, raw_full, raw_empty, s_mask, s_dn, s_scratch, abort);
        } else if (w.left > 0 && warp == C::kMmaWarp && elect_one()) {
            // ============================================================ mma: one thread
            constexpr uint32_t kIdQk1 = idesc_f16(128, 128, false), kIdQk2 = idesc_f16(128, 64, false), kIdPv = idesc_f16(128, D, false);
            bool ok = true;
            uint32_t pieces_done = 0, n = 0, key = 0;  // pieces, tiles, the piece's first operand tile
            auto wait = [&](uint32_t b, uint32_t parity) {
                if (ok) ok = wait_bounded(b, parity, abort, B.status);
                if (ok) tc_fence_after();
                return ok;
            };
            const uint32_t q_lo = desc_lo(base, 2048), k_lo = desc_lo(base + C::kOffOp, 2048), v_lo = desc_lo(base + C::kOffOp, D * 16);
            auto qk = [&](uint32_t os, uint32_t buf) {
                const uint32_t b = k_lo + os * (C::kOp >> 4), d = tmem + kSCol * buf;
#pragma unroll 2  // unrolled wholly it crowds the instruction cache (509 of 8191 tokens 202 -> 217 us)
                for (int k = 0; k < D / 16; ++k) mma_f16(d, desc_of(q_lo + k * 256), desc_of(b + k * 256), kIdQk1, k > 0);
#pragma unroll 2
                for (int k = 0; k < D / 16; ++k)
                    mma_f16(d, desc_of(q_lo + (C::kQ >> 4) + k * 256), desc_of(b + k * 256), kIdQk2, 1);
                mma_commit(s_full + 8 * buf);
                mma_commit(op_empty + 8 * os);
            };
            auto pv = [&](uint32_t os, uint32_t buf) {
                const uint32_t b = v_lo + os * (C::kOp >> 4), d = tmem + kOCol + buf * D, p = tmem + kSCol * buf;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    mma_f16_ts(d, p + 8 * k, desc_of(b + k * 2 * D), kIdPv, k > 0);
                    mma_f16_ts(d, p + 32 + 8 * k, desc_of(b + k * 2 * D), kIdPv, 1);
                    mma_f16_ts(d, p + 8 * k, desc_of(b + ((C::kKt * D * 2) >> 4) + k * 2 * D), kIdPv, 1);
                }
                mma_commit(o_full + 8 * buf);
                mma_commit(op_empty + 8 * os);
            };
            auto op_wait = [&](uint32_t i) { return wait(op_full + 8 * (i % C::kOps), (i / C::kOps) & 1); };
            while (ok) {
                const Seq s = load_seq(B, w.b);
                const Item it = item_of<C>(s, A, w.st);
                const int nt = static_cast<int>(min(static_cast<long long>(it.tiles), w.from + w.left)) - w.from;
                if (!op_wait(key) || !wait(q_full, pieces_done & 1)) break;
                qk(key % C::kOps, n & 1);
                for (int j = 0; j < nt; ++j, ++n) {
                    const uint32_t v = key + 2 * j + 1, buf = n & 1;
                    if (j + 1 < nt) {
                        if (!op_wait(v + 1)) break;
                        qk((v + 1) % C::kOps, buf ^ 1);
                    }
                    if (!wait(p_full + 8 * buf, (n >> 1) & 1) || !op_wait(v)) break;
                    if (n >= 2 && !wait(o_empty + 8 * buf, ((n >> 1) - 1) & 1)) break;
                    pv(v % C::kOps, buf);
                }
                if (!ok) break;
                ++pieces_done;
                key += 2 * nt;
                if (!next_piece<C>(w, B, A, nt)) break;
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    pdl_launch_dependents();
    if (warp == C::kMmaWarp) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    }
}

template <int D, bool kCap>
static int launch_f32(const Args &A, const Batch &B, int max_ctas, cudaStream_t s)
{
    using C = CfgF32<D>;
    auto kern = k_kv_attn_chunk_f32<D, kCap>;
    if (ctas_per_sm(reinterpret_cast<const void *>(kern), C::kThreads, C::kSmem) < 1) return GQ_ERR_CUDA;
    const int grid = sm_count() < max_ctas ? sm_count() : max_ctas;
    return status_from(launch_pdl(kern, dim3(grid), dim3(C::kThreads), C::kSmem, s, A, B));
}

int launch_chunk_f32(const Args &A, const Batch &B, int head_dim, int max_ctas, cudaStream_t s)
{
    if (head_dim == 64) return A.softcap > 0.f ? launch_f32<64, true>(A, B, max_ctas, s) : launch_f32<64, false>(A, B, max_ctas, s);
    return A.softcap > 0.f ? launch_f32<128, true>(A, B, max_ctas, s) : launch_f32<128, false>(A, B, max_ctas, s);
}

}  // namespace chunk
}  // namespace kv
}  // namespace gq
