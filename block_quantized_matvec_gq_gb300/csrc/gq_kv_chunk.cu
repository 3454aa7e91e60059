// gq_kv_chunk.cu -- attention of chunks of new tokens over the paged Q8_0
// cache on tcgen05 tensor cores (gq_kv_attention_q8_0 with 16-bit token
// arrays, for calls with many query rows per sequence and kv head).
//
// An item is one (sequence, kv head, tile of kMt * 128 query rows; row r of a
// sequence is new token r / G, head r % G of the group).  Its cached tokens
// are walked in tiles of kKt; the tiles of all items form one line, cut into
// equal stretches, one per CTA (one CTA per SM), and an item cut by a
// stretch's end is finished by the last of its CTAs to arrive, from partial
// results in the workspace, in a fixed order.
//
// Warp roles (kMt = 2 for head_dim 64 and 128; head_dim 256 has one row tile
// and two score buffers, since its accumulator takes half of tensor memory):
//   softmax      four warps per row tile, a thread per query row: scores from
//                tensor memory, running reference m and sum l, p back to
//                tensor memory as the A operand of p v; the query operand and
//                the result rows.
//   dequantizers eight warps (twelve at head_dim 256): codes and scales of a
//                raw stage -> the f16 operand tile d * q (11 bits, one rounding)
//                in the K-major layout; keys along head_dim, values along the
//                tokens (the cache's words hold four tokens of one element, so
//                neither is transposed).
//   producers    two warps (keys, values): page numbers, and one bulk copy per
//                record half; the first also looks at the values' sizes.
//   mma          one thread.  Per tile of a row tile: p v of this tile, then q k
//                of the next, so the other row tile's softmax runs meanwhile.
// p is kept times 2^7 and the state rescaled only when the row's reference
// would grow by more than 2^8: p stays below 2^15 in f16, and the accumulator
// in tensor memory is touched by the softmax only then (rare after the first
// tiles).  Tensor memory: scores (kKt columns, two buffers; p over them) and
// the accumulators (head_dim columns per row tile).
// What bounds it: per 128 tokens of 256 rows at head_dim 128 the tensor core
// takes 2 x 1024 cycles and one tile takes about 3600.  Without the
// dequantizers it would be 3350, without the exponentials 3520, without both
// 3200: what remains is the chain scores -> p -> p v and q k of one row tile,
// since tensor memory holds one score buffer per row tile beside the
// accumulators.  (Two buffers of 64 columns each took longer: twice the
// waits and N = 64 products.)  A chunk of 2048 tokens behind 30720 cached ones,
// 32 heads over 8 x 128, bf16: 804 us in a graph, 1.32 PFLOP/s, 0.70 of the
// measured bf16 rate (840 us called one by one; 876 on another GB300); head_dim
// 64 712 us, head_dim 256 (16 heads) 1220 us; capped, 2048 of 16384 tokens, 1053.
// Every wait is bounded (gq_tc.cuh).
#include "gq_kv_chunk.cuh"

namespace gq {
namespace kv {
namespace chunk {

template <int D>
struct Cfg {
    static constexpr int kMt = D == 256 ? 1 : 2;
    static constexpr int kKt = D == 256 ? 64 : 128;
    static constexpr int kRowsItem = 128 * kMt;
    static constexpr int kQ = 128 * D * 2;           // query operand of a row tile
    static constexpr int kOp = kKt * D * 2;          // operand tile of keys or values
    static constexpr int kRecs = kKt / kRec;         // records per tile
    static constexpr int kHalf = 17 * D;             // bytes of a record's keys or values
    static constexpr int kRaw = kRecs * kHalf;
    static constexpr int kOps = 3, kRaws = 3;
    static constexpr int kOffOp = kMt * kQ;
    static constexpr int kOffRaw = kOffOp + kOps * kOp;
    static constexpr int kOffBar = kOffRaw + kRaws * kRaw;
    // raw full/empty, operand full/empty, q full [2], s full [2], p full [2], pv done [2], piece done [2], fixed
    static constexpr int kBars = 2 * kRaws + 2 * kOps + 11;
    static constexpr int kOffMisc = kOffBar + 8 * kBars;
    static constexpr int kSmem = kOffMisc + 512;  // and 7.5 KB of static arrays
    // five warpgroups: softmax (one per row tile), dequantizers, {producer, mma}
    static constexpr int kSoftWarps = 4 * kMt;
    static constexpr int kDeqWarps = 16 - kSoftWarps;
    static constexpr int kProdWarp = 16;
    static constexpr int kMmaWarp = 17;
    static constexpr int kWarpsAll = 20;
    static constexpr int kThreads = 32 * kWarpsAll;
    // Registers per thread after the split (a softmax thread holds a whole
    // score row); the shares stay within the launch's 640 x 96.
    static constexpr int kSoftRegs = kMt == 2 ? 168 : 144, kDeqRegs = kMt == 2 ? 48 : 72, kRestRegs = 48;
    static_assert(32 * (kSoftWarps * kSoftRegs + kDeqWarps * kDeqRegs + 4 * kRestRegs) <= kThreads * 96, "register split");
    static_assert(kOffOp % 128 == 0 && kOffRaw % 128 == 0 && kOffBar % 8 == 0 && kSmem + 7680 <= 232448, "shared memory layout");
};
// ---------------------------------------------------------------- dequantizers
// Operand tiles are core matrices of 8 rows x 16 bytes (8 elements of K); row
// group r / 8 at 128 bytes, K group kg at 16 * rows bytes.
// Keys: row = token, K = head_dim.  A unit is one (token, block): 32 codes.
// Neighbouring lanes take neighbouring tokens, so the 16-byte stores of eight
// lanes fill one core matrix; the two halves of the 32 codes are read in an
// order that depends on the token, which with the record's own exclusive or
// spreads eight tokens over all banks.
// `op_free` waits for the operand stage, while the raw stage's words arrive;
// false ends the tile.  The raw stage is given back only after the conversion:
// an arrival right after the loads does not wait for their data, and a refill
// overtook them.
template <int D, class Free>
__device__ __forceinline__ bool dequant_keys(const uint8_t *raw, uint8_t *op, int tid, Free op_free)
{
    using C = Cfg<D>;
    constexpr int nb = D / 32, kTh = C::kDeqWarps * 32, kAll = C::kKt * nb, kN = (kAll + kTh - 1) / kTh;
    uint4 w[kN][2];
    uint32_t d[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) {
        const int u = tid + i * kTh, tok = u % C::kKt, b = u / C::kKt, t = tok % kRec;
        if (kAll % kTh != 0 && u >= kAll) break;
        const uint8_t *src = raw + tok / kRec * C::kHalf;
        d[i] = *reinterpret_cast<const uint16_t *>(src + k_scale_off(t, b, D));
#pragma unroll
        for (int h = 0; h < 2; ++h)
            w[i][h] = *reinterpret_cast<const uint4 *>(src + k_code_off(t, b, nb) + 16 * (h ^ ((t >> 1) & 1)));
    }
    if (!op_free()) return false;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
        const int u = tid + i * kTh, tok = u % C::kKt, b = u / C::kKt, t = tok % kRec;
        if (kAll % kTh != 0 && u >= kAll) break;
        const uint32_t d2 = d[i] | (d[i] << 16);
        uint8_t *dst = op + (tok >> 3) * 128 + (tok & 7) * 16;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint4 x = w[i][h];
            uint4 a, c;
            a.x = hmul2(codes2(x.x, 0x4140u), d2);
            a.y = hmul2(codes2(x.x, 0x4342u), d2);
            a.z = hmul2(codes2(x.y, 0x4140u), d2);
            a.w = hmul2(codes2(x.y, 0x4342u), d2);
            c.x = hmul2(codes2(x.z, 0x4140u), d2);
            c.y = hmul2(codes2(x.z, 0x4342u), d2);
            c.z = hmul2(codes2(x.w, 0x4140u), d2);
            c.w = hmul2(codes2(x.w, 0x4342u), d2);
            uint8_t *o = dst + (4 * b + 2 * (h ^ ((t >> 1) & 1))) * (C::kKt * 16);
            *reinterpret_cast<uint4 *>(o) = a;
            *reinterpret_cast<uint4 *>(o + C::kKt * 16) = c;
        }
    }
    return true;
}
// Values: row n = (e % 4) * D / 4 + e / 4 for element e (neighbouring lanes,
// which take neighbouring 16-byte chunks of four elements, then store to
// neighbouring rows), K = token.  A unit is eight tokens of one chunk.
template <int D, class Free>
__device__ __forceinline__ bool dequant_values(const uint8_t *raw, uint8_t *op, int tid, Free op_free)
{
    using C = Cfg<D>;
    constexpr int kTh = C::kDeqWarps * 32, kAll = (C::kKt / 8) * (D / 4), kN = (kAll + kTh - 1) / kTh;
    uint4 w[kN][2], d[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) {
        const int u = tid + i * kTh, c = u % (D / 4), t8 = u / (D / 4), g = 2 * (t8 % 2);
        if (kAll % kTh != 0 && u >= kAll) break;
        const uint8_t *src = raw + t8 / 2 * C::kHalf - 17 * D;  // offsets below count from the record
        d[i] = *reinterpret_cast<const uint4 *>(src + v_scale_off(4 * g, c / 8, D));  // eight tokens
        w[i][0] = *reinterpret_cast<const uint4 *>(src + v_chunk_off(g, c, D));
        w[i][1] = *reinterpret_cast<const uint4 *>(src + v_chunk_off(g + 1, c, D));
    }
    if (!op_free()) return false;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
        const int u = tid + i * kTh, c = u % (D / 4), t8 = u / (D / 4);
        if (kAll % kTh != 0 && u >= kAll) break;
        const uint4 s = d[i];
        uint8_t *dst = op + t8 * (D * 16);
        const uint32_t a[4] = {w[i][0].x, w[i][0].y, w[i][0].z, w[i][0].w}, z[4] = {w[i][1].x, w[i][1].y, w[i][1].z, w[i][1].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int n = k * (D / 4) + c;
            uint4 o;
            o.x = hmul2(codes2(a[k], 0x4140u), s.x);
            o.y = hmul2(codes2(a[k], 0x4342u), s.y);
            o.z = hmul2(codes2(z[k], 0x4140u), s.z);
            o.w = hmul2(codes2(z[k], 0x4342u), s.w);
            *reinterpret_cast<uint4 *>(dst + (n >> 3) * 128 + (n & 7) * 16) = o;
        }
    }
    return true;
}

// ---------------------------------------------------------------- the query operand
// This thread's row: elements * 2^-e as f16, e from the row's largest
// magnitude; returns 2^e.  A dead row is zeros.  The row is read twice (the
// second time from L1): held in registers it would spill.
template <int D, int TYPE>
__device__ __forceinline__ float load_query(const uint8_t *src, bool live, bool negate, uint8_t *op, int row)
{
    float amax = 0.f;
#pragma unroll 8
    for (int i = 0; i < D / 8; ++i) {
        const uint4 v = live ? __ldg(reinterpret_cast<const uint4 *>(src) + i) : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 x = pair_of<TYPE>(w[k]);
            amax = fmaxf(amax, fmaxf(fabsf(x.x), fabsf(x.y)));
        }
    }
    const int be = static_cast<int>(__float_as_uint(amax) >> 23) - 126;
    const int e = min(max(be, -100), 128) - 10;  // amax * 2^-e in [2^9, 2^10)
    const float f = negate ? -pow2i(-e) : pow2i(-e);
    uint8_t *dst = op + (row >> 3) * 128 + (row & 7) * 16;
#pragma unroll 8
    for (int i = 0; i < D / 8; ++i) {
        const uint4 v = live ? __ldg(reinterpret_cast<const uint4 *>(src) + i) : make_uint4(0u, 0u, 0u, 0u);
        const float2 x0 = pair_of<TYPE>(v.x), x1 = pair_of<TYPE>(v.y), x2 = pair_of<TYPE>(v.z), x3 = pair_of<TYPE>(v.w);
        *reinterpret_cast<uint4 *>(dst + i * 2048) = make_uint4(f2_half2(x0.x * f, x0.y * f), f2_half2(x1.x * f, x1.y * f),
                                                                f2_half2(x2.x * f, x2.y * f), f2_half2(x3.x * f, x3.y * f));
    }
    return pow2i(e);
}

template <int D, bool kCap>
__global__ void __launch_bounds__(Cfg<D>::kThreads, 1) k_kv_attn_chunk(Args A, Batch B)
{
    using C = Cfg<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ long long s_cost[C::kWarpsAll], s_cut[2];
    __shared__ Walk s_walk;
    __shared__ volatile int s_abort;
    __shared__ uint32_t s_tmem;
    __shared__ uint32_t s_mask[kMaskRing];
    __shared__ __align__(16) float s_dn[kMaskRing * C::kKt];
    __shared__ __align__(16) uint16_t s_scratch[C::kKt];
    __shared__ float2 s_sum[128 * C::kMt];
    __shared__ int s_last[2];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t base = smem_u32(smem);
    const uint32_t bar = base + C::kOffBar;
    const uint32_t raw_full = bar, raw_empty = raw_full + 8 * C::kRaws, op_full = raw_empty + 8 * C::kRaws,
                   op_empty = op_full + 8 * C::kOps, q_full = op_empty + 8 * C::kOps, s_full = q_full + 16,
                   p_full = s_full + 16, pv_done = p_full + 16, o_done = pv_done + 16, fixed = o_done + 16;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kRaws; ++i) {
            mbar_init(raw_full + 8 * i, 1);
            mbar_init(raw_empty + 8 * i, C::kDeqWarps);
        }
        for (int i = 0; i < C::kOps; ++i) {
            mbar_init(op_full + 8 * i, C::kDeqWarps);
            mbar_init(op_empty + 8 * i, 1);
        }
        mbar_init(fixed, C::kDeqWarps);
        for (int i = 0; i < 2; ++i) {
            mbar_init(q_full + 8 * i, 4);
            mbar_init(s_full + 8 * i, 1);
            mbar_init(p_full + 8 * i, 4);
            mbar_init(pv_done + 8 * i, 1);
            mbar_init(o_done + 8 * i, 1);
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

    // ---- this CTA's stretch
    const long long len = find_stretch<C>(B, A, s_cost, s_cut, s_walk);
    Walk w = s_walk;
    volatile int *abort = &s_abort;
    // The register split stands at the head of each warpgroup's branch, where
    // the compiler takes it as the limit of what follows.
    if (warp < C::kSoftWarps) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kSoftRegs));
        // ================================================================ softmax: thread = query row
        const int mt = warp >> 2;                       // row tile
        const int row = threadIdx.x & 127;
        const uint32_t lane_addr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const uint32_t o_addr = lane_addr + kOCol + mt * D;
        uint8_t *q_op = smem + mt * C::kQ;
        const float inv_cap = kCap ? inverse_cap(A.softcap) : 0.f;
        constexpr float kLog2e = 1.4426950408889634f;
        bool ok = true;
        uint32_t n_pv = 0;          // tiles of this row tile so far: scores taken, p v products asked for
        uint32_t n_piece = 0;       // pieces of this row tile so far
        uint32_t tile_no = 0;       // key tiles of the CTA so far
        // A piece as this thread sees it; its query row is loaded, and its first
        // scores asked for, before the result of the piece before is written.
        struct Piece {
            int base, tiles, from, to;
            long long x;
            bool tile_live, live;  // any row of the row tile (else the mma warp skips it); this row
            int row_lo, row_hi;    // positions that the row sees
            float zs;              // score = sum * zs
            uint8_t *dst;
        };
        auto begin = [&]() {
            Piece p;
            const Seq s = load_seq(B, w.b);
            const Item it = item_of<C>(s, A, w.st);
            p.base = it.base;
            p.tiles = it.tiles;
            p.from = w.from;
            p.to = static_cast<int>(min(static_cast<long long>(it.tiles), w.from + w.left));
            p.x = w.x;
            const int r = it.r0 + 128 * mt + row;
            p.tile_live = it.r0 + 128 * mt < it.rows;
            p.live = r < it.rows;
            const int tok = p.live ? r / A.group : 0, head = w.h * A.group + (p.live ? r % A.group : 0);
            const int pos = s.first + tok;
            p.row_hi = p.live ? min(pos, s.kv - 1) : -1;
            p.row_lo = A.window > 0 ? max(0, pos - A.window + 1) : 0;
            const long long at = static_cast<long long>(head) * D * 2;
            p.dst = A.O + (s.row0 + tok) * A.ldo + at;
            p.zs = 0.f;
            if (p.tile_live) {
                // every q k of the piece before is done: its last scores have been taken
                const uint8_t *src = A.Q + (s.row0 + tok) * A.ldq + at;
                const float f = A.type == GQ_TYPE_BF16 ? load_query<D, GQ_TYPE_BF16>(src, p.live, A.scale < 0.f, q_op, row)
                                                       : load_query<D, GQ_TYPE_F16>(src, p.live, A.scale < 0.f, q_op, row);
                // a factor of 0 would turn hidden scores (-inf) into NaN
                p.zs = fmaxf(fabsf(A.scale) * f * (kCap ? 1.0f : kLog2e), 1e-37f);
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(q_full + 8 * mt);
            }
            return p;
        };
        bool more = w.left > 0;
        Piece pc = {};
        if (more) pc = begin();
        while (more) {
            float m = kNone, l = 0.f;
            if (pc.tile_live) {
                const float zs = pc.zs;
                for (int j = pc.from; j < pc.to; ++j) {
                    const int buf = C::kMt == 2 ? mt : static_cast<int>(n_pv & 1);
                    const uint32_t s_addr = lane_addr + kSCol * buf;
                    // kMt = 2: one buffer per row tile; kMt = 1: two in turn
                    if (ok) ok = wait_warp(s_full + 8 * buf, (C::kMt == 2 ? n_pv : n_pv >> 1) & 1, abort, B.status);
                    if (!ok) break;
                    tc_fence_after();
                    const int p0 = pc.base + j * C::kKt;
                    const uint32_t slot = (tile_no + (j - pc.from)) % kMaskRing, word = s_mask[slot], recs = word & ~kMixed;
                    // every row of the warp sees the whole tile?
                    const bool edge = __any_sync(0xffffffffu, p0 < pc.row_lo || p0 + C::kKt - 1 > pc.row_hi) ||
                                      recs != (1u << C::kRecs) - 1u;
                    if (kCap) cap_scores<C::kKt, false>(s_addr, zs, A.softcap, inv_cap);
                    if (__builtin_expect(word & kMixed, 0))
                        shift_scores<C::kKt, false>(s_addr, kCap ? 1.0f : zs, pc.row_lo - p0, pc.row_hi - p0, recs, s_dn + slot * C::kKt,
                                                   s_sum + threadIdx.x);
                    float v[C::kKt];
#pragma unroll
                    for (int c = 0; c < C::kKt; c += 32) tmem_ld32_async(s_addr + c, v + c);
                    tmem_wait_ld(v);
                    if (edge) {
                        const int a = pc.row_lo - p0, b = pc.row_hi - p0;
#pragma unroll
                        for (int k = 0; k < C::kKt; ++k)
                            if (k < a || k > b || !((recs >> (k / kRec)) & 1u)) v[k] = -INFINITY;
                    }
                    float t0 = v[0], t1 = v[1], t2 = v[2], t3 = v[3];
#pragma unroll
                    for (int k = 4; k < C::kKt; k += 8) {
                        t0 = fmaxf(t0, fmaxf(v[k], k + 4 < C::kKt ? v[k + 4] : v[k]));
                        t1 = fmaxf(t1, fmaxf(v[k + 1], k + 4 < C::kKt ? v[k + 5] : v[k]));
                        t2 = fmaxf(t2, fmaxf(v[k + 2], k + 4 < C::kKt ? v[k + 6] : v[k]));
                        t3 = fmaxf(t3, fmaxf(v[k + 3], k + 4 < C::kKt ? v[k + 7] : v[k]));
                    }
                    // the scale (its sign is in q) keeps the order of the scores
                    const float zt = fmaxf(fmaxf(t0, t1), fmaxf(t2, t3)) * (kCap ? 1.0f : zs);
                    if (__any_sync(0xffffffffu, zt > m + kGrow)) {
                        const float nm = fmaxf(m, zt), g = ex2(m - nm);
                        m = nm;
                        l *= g;
                        if (j > pc.from) {
                            // the accumulator is at rest once the previous tile's p v is done (the one
                            // before that is: these scores were asked for after it)
                            ok = wait_warp(pv_done + 8 * mt, (n_pv - 1) & 1, abort, B.status);
                            if (!ok) break;
                            tc_fence_after();
#pragma unroll 1
                            for (int c = 0; c < D; c += 8) {
                                uint32_t x[8];
                                tmem_ld8(o_addr + c, x);
#pragma unroll
                                for (int k = 0; k < 8; ++k) x[k] = __float_as_uint(__uint_as_float(x[k]) * g);
                                tmem_st8(o_addr + c, x);
                            }
                            tmem_wait_st();
                        }
                    }
                    const float2 ref = make_float2(kPHead - m, kPHead - m), zs2 = kCap ? make_float2(1.f, 1.f) : make_float2(zs, zs);
                    float2 sum0 = make_float2(0.f, 0.f), sum1 = sum0;
#pragma unroll
                    for (int c = 0; c < C::kKt; c += 32) {
                        uint32_t p[16];
#pragma unroll
                        for (int k = 0; k < 32; k += 4) {
                            float2 a = ffma2(make_float2(v[c + k], v[c + k + 1]), zs2, ref);
                            float2 b = ffma2(make_float2(v[c + k + 2], v[c + k + 3]), zs2, ref);
                            a.x = ex2(a.x), a.y = ex2(a.y), b.x = ex2(b.x), b.y = ex2(b.y);
                            sum0 = __fadd2_rn(sum0, a);
                            sum1 = __fadd2_rn(sum1, b);
                            p[k / 2] = f2_half2(a.x, a.y);
                            p[k / 2 + 1] = f2_half2(b.x, b.y);
                        }
                        tmem_st16(s_addr + c / 2, p);  // over the scores, which are in registers
                    }
                    float sum = (sum0.x + sum0.y) + (sum1.x + sum1.y);
                    if (__builtin_expect(s_mask[(tile_no + (j - pc.from)) % kMaskRing] & kMixed, 0))
                        sum = s_sum[threadIdx.x].y * ex2(s_sum[threadIdx.x].x - m);
                    l += sum;
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(p_full + 8 * buf);
                    ++n_pv;
                }
            }
            const Piece cur = pc;
            tile_no += cur.to - cur.from;
            more = next_piece<C>(w, B, A, cur.to - cur.from);
            if (more) pc = begin();
            if (!cur.tile_live) continue;
            // ---- the piece's result
            if (ok) ok = wait_warp(o_done + 8 * mt, n_piece & 1, abort, B.status);
            ++n_piece;
            tc_fence_after();
            // column i * D / 4 + c is element 4 c + i
            auto put = [&](int c, const float (&x)[32], float inv) {
                uint32_t o[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    // elements 2 k, 2 k + 1 of this group of 32: columns 8 i + cc with i = e % 4, cc = e / 4
                    const float a = x[8 * ((2 * k) & 3) + (2 * k) / 4] * inv, b = x[8 * ((2 * k + 1) & 3) + (2 * k + 1) / 4] * inv;
                    o[k] = A.type == GQ_TYPE_BF16 ? f2_bf162(a, b) : f2_half2(a, b);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    *reinterpret_cast<uint4 *>(cur.dst + (4 * c + 8 * k) * 2) = make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
            };
            const bool whole = cur.from == 0 && cur.to == cur.tiles;
            constexpr int kSlot = 128 * (D + 2);  // floats of one row tile's partial: [D][128], m, l
            float *slot = A.part + ((2ll * blockIdx.x + (cur.from == 0 ? 1 : 0)) * C::kMt + mt) * kSlot;
            const float inv = l == 0.f ? 0.f : 1.0f / l;
#pragma unroll 1
            for (int c = 0; c < D / 4; c += 8) {
                float x[32];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t v[8];
                    tmem_ld8(o_addr + i * (D / 4) + c, v);
#pragma unroll
                    for (int k = 0; k < 8; ++k) x[8 * i + k] = __uint_as_float(v[k]);
                }
                if (whole) {
                    if (cur.live) put(c, x, inv);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int k = 0; k < 8; ++k) slot[(i * (D / 4) + c + k) * 128 + row] = x[8 * i + k];
                }
            }
            // the next piece's first p v overwrites the accumulator only after this warp's next p
            tc_fence_before();
            if (whole) continue;
            slot[D * 128 + row] = m;
            slot[(D + 1) * 128 + row] = l;
            const long long item_x = cur.x - cur.from;
            const int c0 = first_cta(item_x, cur.tiles, len), c1 = last_cta(item_x, cur.tiles, len);
            __threadfence();
            bar_sync(1 + mt, 128);
            if (row == 0) {
                const int old = atomicAdd(A.counter + c0 * C::kMt + mt, 1);
                s_last[mt] = old == c1 - c0;
                if (old == c1 - c0) A.counter[c0 * C::kMt + mt] = 0;
            }
            bar_sync(1 + mt, 128);
            if (s_last[mt]) {
                __threadfence();
                auto part = [&](int c) { return A.part + ((2ll * c + (c == c0 ? 1 : 0)) * C::kMt + mt) * kSlot; };
                float M = kNone, L = 0.f;
#pragma unroll 4
                for (int c = c0; c <= c1; ++c) M = fmaxf(M, __ldcg(part(c) + D * 128 + row));
#pragma unroll 4
                for (int c = c0; c <= c1; ++c) L += ex2(__ldcg(part(c) + D * 128 + row) - M) * __ldcg(part(c) + (D + 1) * 128 + row);
                const float linv = L == 0.f ? 0.f : 1.0f / L;
#pragma unroll 1
                for (int c = 0; c < D / 4; c += 8) {
                    float x[32];
#pragma unroll
                    for (int k = 0; k < 32; ++k) x[k] = 0.f;
#pragma unroll 2
                    for (int cc = c0; cc <= c1; ++cc) {
                        const float *src = part(cc);
                        const float g = ex2(__ldcg(src + D * 128 + row) - M);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int k = 0; k < 8; ++k) x[8 * i + k] += g * __ldcg(src + (i * (D / 4) + c + k) * 128 + row);
                    }
                    if (cur.live) put(c, x, linv);
                }
            }
            bar_sync(1 + mt, 128);  // s_last may be written again
        }
    } else if (warp < C::kProdWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kDeqRegs));
        // ================================================================ dequantizers
        const int tid = threadIdx.x - 32 * C::kSoftWarps;
        bool ok = true;
        uint32_t n = 0, tile_no = 0, n_fixed = 0;  // operand tiles, key tiles
        while (ok && w.left > 0) {
            const Seq s = load_seq(B, w.b);
            const Item it = item_of<C>(s, A, w.st);
            const int to = static_cast<int>(min(static_cast<long long>(it.tiles), w.from + w.left));
            for (int j = w.from; j < to && ok; ++j, ++tile_no) {
                const int p0 = it.base + j * C::kKt;
#pragma unroll 1
                for (int part = 0; part < 2; ++part, ++n) {
                    const uint32_t rs = n % C::kRaws, os = n % C::kOps;
                    ok = wait_warp(raw_full + 8 * rs, (n / C::kRaws) & 1, abort, B.status);
                    if (!ok) break;
                    uint8_t *raw = smem + C::kOffRaw + rs * C::kRaw;
                    uint8_t *op = smem + C::kOffOp + os * C::kOp;
                    auto op_free = [&]() {
                        return n < C::kOps || wait_warp(op_empty + 8 * os, (n / C::kOps - 1) & 1, abort, B.status);
                    };
                    if (part == 0) {
                        ok = dequant_keys<D>(raw, op, tid, op_free);
                    } else {
                        ok = fix_scales<D, C>(raw, tid, it.lo - p0, it.hi + 1 - p0, s_mask[tile_no % kMaskRing],
                                              s_dn + tile_no % kMaskRing * C::kKt, fixed, n_fixed, abort, B.status);
                        if (ok) ok = dequant_values<D>(raw, op, tid, op_free);
                    }
                    if (!ok) break;
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(op_full + 8 * os);
                        mbar_arrive(raw_empty + 8 * rs);
                    }
                }
            }
            if (!ok || !next_piece<C>(w, B, A, to - w.from)) break;
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRestRegs));
    if (w.left > 0 && (warp == C::kProdWarp || warp == C::kProdWarp + 2)) {
        produce<D, C>(warp != C::kProdWarp, w, B, A, smem, raw_full, raw_empty, s_mask, s_dn, s_scratch, abort);
    } else if (w.left > 0 && warp == C::kMmaWarp && elect_one()) {
        // ================================================================ mma: one thread
        constexpr uint32_t kIdQk = idesc_f16(128, C::kKt, false), kIdPv = idesc_f16(128, D, false);
        bool ok = true;
        uint32_t n_q = 0;            // pieces begun
        uint32_t n_q1 = 0;           // pieces with a second row tile begun
        uint32_t n_p0 = 0, n_p1 = 0; // p tiles taken of the two row tiles
        uint32_t key = 0;            // running number of the piece's first operand tile
        auto wait = [&](uint32_t b, uint32_t parity) {
            if (ok) ok = wait_bounded(b, parity, abort, B.status);
            if (ok) tc_fence_after();
            return ok;
        };
        // scores of row tile mt with the keys in operand stage os, into buffer buf
        // The descriptors of successive K steps differ by a constant in their
        // low word: one add per operand and MMA.  (Building each descriptor
        // from its address made this thread the limit: 113 cycles per MMA
        // against the tensor core's 64 for 128 x 128 x 16.)
        const uint32_t q_lo = desc_lo(base, 2048), k_lo = desc_lo(base + C::kOffOp, C::kKt * 16),
                       v_lo = desc_lo(base + C::kOffOp, D * 16);
        auto qk = [&](int mt, uint32_t os, int buf) {
            const uint32_t a = q_lo + mt * (C::kQ >> 4), b = k_lo + os * (C::kOp >> 4);
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
                mma_f16(tmem + kSCol * buf, desc_of(a + k * 256), desc_of(b + k * 2 * C::kKt), kIdQk, k > 0);
            mma_commit(s_full + 8 * buf);
        };
        auto pv = [&](int mt, uint32_t os, int buf, bool first) {
            const uint32_t b = v_lo + os * (C::kOp >> 4);
#pragma unroll
            for (int k = 0; k < C::kKt / 16; ++k)
                mma_f16_ts(tmem + kOCol + mt * D, tmem + kSCol * buf + 8 * k, desc_of(b + k * 2 * D), kIdPv, !first || k > 0);
            mma_commit(pv_done + 8 * mt);
        };
        while (ok) {
            const Seq s = load_seq(B, w.b);
            const Item it = item_of<C>(s, A, w.st);
            const int to = static_cast<int>(min(static_cast<long long>(it.tiles), w.from + w.left));
            const int nt = to - w.from;
            const bool two = C::kMt == 2 && it.r0 + 128 < it.rows;
            // operand tile numbers: keys of the piece's tile j at key + 2 j, values at key + 2 j + 1
            auto op_wait = [&](uint32_t n) { return wait(op_full + 8 * (n % C::kOps), (n / C::kOps) & 1); };
            auto op_free = [&](uint32_t n) { mma_commit(op_empty + 8 * (n % C::kOps)); };
            if (!op_wait(key)) break;
            if (C::kMt == 2) {
                if (!wait(q_full, n_q & 1)) break;
                qk(0, key % C::kOps, 0);
                if (two) {
                    if (!wait(q_full + 8, n_q1 & 1)) break;
                    qk(1, key % C::kOps, 1);
                }
                op_free(key);
                for (int j = 0; j < nt; ++j) {
                    const uint32_t v = key + 2 * j + 1;
                    for (int mt = 0; mt < (two ? 2 : 1); ++mt) {
                        if (!wait(p_full + 8 * mt, (mt == 0 ? n_p0 : n_p1) & 1)) break;
                        if (mt == 0) ++n_p0;
                        else ++n_p1;
                        if (mt == 0 && !op_wait(v)) break;
                        pv(mt, v % C::kOps, mt, j == 0);
                        if (j + 1 == nt) mma_commit(o_done + 8 * mt);
                        if (mt == (two ? 1 : 0)) op_free(v);
                        if (j + 1 < nt) {
                            if (mt == 0 && !op_wait(v + 1)) break;
                            qk(mt, (v + 1) % C::kOps, mt);
                            if (mt == (two ? 1 : 0)) op_free(v + 1);
                        }
                    }
                    if (!ok) break;
                }
            } else {
                if (!wait(q_full, n_q & 1)) break;
                qk(0, key % C::kOps, n_p0 & 1);
                op_free(key);
                for (int j = 0; j < nt; ++j) {
                    const uint32_t v = key + 2 * j + 1;
                    const int buf = n_p0 & 1;
                    if (j + 1 < nt) {
                        if (!op_wait(v + 1)) break;
                        qk(0, (v + 1) % C::kOps, buf ^ 1);
                        op_free(v + 1);
                    }
                    if (!wait(p_full + 8 * buf, (n_p0 >> 1) & 1)) break;
                    ++n_p0;
                    if (!op_wait(v)) break;
                    pv(0, v % C::kOps, buf, j == 0);
                    if (j + 1 == nt) mma_commit(o_done);
                    op_free(v);
                }
            }
            if (!ok) break;
            ++n_q;
            if (two) ++n_q1;
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

// Partials: two slots per CTA and row tile of {O[D][128], m[128], l[128]} f32.
constexpr int kMaxCtas = 160;
constexpr size_t part_floats(int D) { return 2ull * kMaxCtas * (D == 256 ? 1 : 2) * 128 * (D + 2); }

template <int D, bool kCap>
static int launch_cap(const Args &A, const Batch &B, cudaStream_t s)
{
    using C = Cfg<D>;
    if (ctas_per_sm(reinterpret_cast<const void *>(&k_kv_attn_chunk<D, kCap>), C::kThreads, C::kSmem) < 1) return GQ_ERR_CUDA;
    const int grid = sm_count() < kMaxCtas ? sm_count() : kMaxCtas;
    return status_from(launch_pdl(k_kv_attn_chunk<D, kCap>, dim3(grid), dim3(C::kThreads), C::kSmem, s, A, B));
}

template <int D>
static int launch(const Args &A, const Batch &B, cudaStream_t s)
{
    return A.softcap > 0.f ? launch_cap<D, true>(A, B, s) : launch_cap<D, false>(A, B, s);
}

}  // namespace chunk
}  // namespace kv

size_t kv_chunk_part_bytes(int head_dim) { return kv::chunk::part_floats(head_dim) * sizeof(float); }
int kv_chunk_counters() { return 2 * kv::chunk::kMaxCtas; }

int launch_kv_chunk(const void *Q, long long ldq, const uint8_t *cache, const kv::Batch &B, void *O, long long ldo, int type,
                    float scale, float softcap, int window, int *counter, float *part, int heads, int head_dim, cudaStream_t s)
{
    kv::chunk::Args A;
    A.Q = static_cast<const uint8_t *>(Q);
    A.cache = cache;
    A.O = static_cast<uint8_t *>(O);
    A.ldq = ldq * kv::type_size(type);
    A.ldo = ldo * kv::type_size(type);
    A.type = type;
    A.group = heads / B.kv_heads;
    A.window = window;
    A.scale = scale;
    A.softcap = softcap;
    A.counter = counter;
    A.part = part;
    if (type == GQ_TYPE_F32) return kv::chunk::launch_chunk_f32(A, B, head_dim, kv::chunk::kMaxCtas, s);
    switch (head_dim) {
    case 64: return kv::chunk::launch<64>(A, B, s);
    case 128: return kv::chunk::launch<128>(A, B, s);
    default: return kv::chunk::launch<256>(A, B, s);
    }
}

}  // namespace gq
