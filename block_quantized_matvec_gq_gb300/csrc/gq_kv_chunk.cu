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
//   dequantizers four warps (eight for head_dim 256): codes and scales of a raw stage -> the f16 operand
//                tile d * q (11 bits, one rounding) in the K-major layout; keys
//                along head_dim, values along the tokens (the cache's words
//                hold four tokens of one element, so neither is transposed).
//   producer     one warp: page numbers, and one bulk copy per record half.
//   mma          one thread.  Per tile of a row tile: p v of this tile, then q k
//                of the next, so the other row tile's softmax runs meanwhile.
// p is kept times 2^7 and the state rescaled only when the row's reference
// would grow by more than 2^8: p stays below 2^15 in f16, and the accumulator
// in tensor memory is touched by the softmax only then (rare after the first
// tiles).  Tensor memory: scores (kKt columns, two buffers; p over them) and
// the accumulators (head_dim columns per row tile).
// Every wait is bounded (gq_tc.cuh).
#include "gq_kv.cuh"
#include "gq_tc.cuh"

namespace gq {
namespace kv {
namespace chunk {

using namespace tcu;

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
    // raw full/empty, operand full/empty, q full [2], s full [2], p full [2], pv done [2], piece done [2]
    static constexpr int kBars = 2 * kRaws + 2 * kOps + 10;
    static constexpr int kOffMisc = kOffBar + 8 * kBars;
    static constexpr int kSmem = kOffMisc + 512;
    // four warpgroups: softmax (one per row tile), dequantizers, {producer, mma}
    static constexpr int kSoftWarps = 4 * kMt;
    static constexpr int kDeqWarps = 12 - kSoftWarps;
    static constexpr int kProdWarp = 12;
    static constexpr int kMmaWarp = 13;
    static constexpr int kWarpsAll = 16;
    static constexpr int kThreads = 32 * kWarpsAll;
    // Registers per thread after the split; with kKt = 128 a softmax thread
    // holds a whole score row.  The shares add up to the launch's 512 x 128.
    static constexpr int kSoftRegs = kMt == 2 ? 184 : 0, kDeqRegs = 88, kRestRegs = 56;
    static_assert(kMt == 1 || 256 * kSoftRegs + 128 * kDeqRegs + 128 * kRestRegs <= 512 * 128, "register split");
    static_assert(kOffOp % 128 == 0 && kOffRaw % 128 == 0 && kOffBar % 8 == 0 && kSmem <= 232448, "shared memory layout");
};
constexpr int kTmemCols = 512;
constexpr int kSCol = 128;        // column step between score buffers
constexpr int kOCol = 256;        // first accumulator column
constexpr float kNone = -1e30f;   // reference of a row that has seen no token
constexpr float kPHead = 7.0f;
constexpr float kGrow = 8.0f;
constexpr int kMaskRing = 8;

struct Args {
    const uint8_t *Q, *cache;
    uint8_t *O;
    long long ldq, ldo;  // bytes
    int type, group, window;
    float scale, softcap;
    int *counter;  // [grid][kMt]
    float *part;
};

// One item: rows, and the positions they can see.
struct Item {
    Seq s;
    int rows;      // query rows of the sequence
    int r0;        // first row of the item
    int lo, hi;    // positions that some row sees (hi < lo: none)
    int base;      // position of the first tile (whole records)
    int tiles;
};
template <int D>
__device__ __forceinline__ Item item_of(const Seq &s, const Args &A, int st)
{
    using C = Cfg<D>;
    Item it;
    it.s = s;
    it.rows = s.n * A.group;
    it.r0 = st * C::kRowsItem;
    const int t0 = it.r0 / A.group, t1 = min(it.r0 + C::kRowsItem, it.rows) - 1;
    it.hi = s.first + t1 / A.group;
    it.lo = A.window > 0 ? max(0, s.first + t0 - A.window + 1) : 0;
    it.base = it.lo & ~(kRec - 1);
    it.tiles = max(1, (it.hi - it.base + C::kKt) / C::kKt);
    return it;
}

// A warp's walk over the pieces (parts of items) of its CTA's stretch.
struct Walk {
    int b, h, st;
    int from;          // first tile of the piece in its item
    long long left;    // tiles of the stretch still to come, this piece's included
    long long x;       // place of the piece on the line
};

__device__ __forceinline__ int row_tiles(const Seq &s, const Args &A, int rows_item)
{
    return (s.n * A.group + rows_item - 1) / rows_item;
}

// tiles of all items of one kv head of a sequence (every lane gets the sum)
template <int D>
__device__ __forceinline__ long long head_cost(const Seq &s, const Args &A)
{
    const int nst = row_tiles(s, A, Cfg<D>::kRowsItem);
    long long c = 0;
    for (int st = threadIdx.x & 31; st < nst; st += 32) c += item_of<D>(s, A, st).tiles;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
    return c;
}

// Moves to the next piece; false when the stretch is done.
template <int D>
__device__ __forceinline__ bool next_piece(Walk &w, const Batch &B, const Args &A, int tiles_done)
{
    w.left -= tiles_done;
    w.x += tiles_done;
    if (w.left <= 0) return false;
    w.from = 0;
    Seq s = load_seq(B, w.b);
    if (++w.st < row_tiles(s, A, Cfg<D>::kRowsItem)) return true;
    w.st = 0;
    if (++w.h < B.kv_heads) return true;
    w.h = 0;
    do {
        if (++w.b >= B.n_seq) return false;
        s = load_seq(B, w.b);
    } while (s.n == 0);
    return true;
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// cap * tanh(x / cap) in f32 (as in gq_kv_attn.cu)
__device__ __forceinline__ float soft_cap(float x, float cap, float inv_cap)
{
    const float y = x * inv_cap, a = fabsf(y);
    const float e = ex2(-2.885390082f * a);
    const float big = __fdividef(1.0f - e, 1.0f + e);
    const float q = y * y;
    const float small = a * (1.0f + q * (-0.333333333f + q * (0.133333333f + q * (-0.053968254f + q * 0.021869489f))));
    return copysignf(cap * (a < 0.25f ? small : big), y);
}

// ---------------------------------------------------------------- tensor memory
// 32 columns of this thread's lane; tmem_wait_ld has to follow before r is used.
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, float *r)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
          "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]), "=f"(r[16]),
          "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]),
          "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
        : "r"(taddr)
        : "memory");
}
template <int N>
__device__ __forceinline__ void tmem_wait_ld(float (&r)[N])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+f"(r[i]));  // no use of r moves above the wait
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n tcgen05.wait::ld.sync.aligned;"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// A from tensor memory (128 rows, two f16 of K per column), B from shared memory.
__device__ __forceinline__ void mma_f16_ts(uint32_t tmem_d, uint32_t tmem_a, uint64_t bdesc, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(tmem_d),
        "r"(tmem_a), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n selp.u32 %0, 1, 0, q;\n}" : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ void bar_sync(int id, int threads) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory"); }

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b)
{
    const __half2 r = __hmul2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}

// ---------------------------------------------------------------- dequantizers
// Operand tiles are core matrices of 8 rows x 16 bytes (8 elements of K); row
// group r / 8 at 128 bytes, K group kg at 16 * rows bytes.
// Keys: row = token, K = head_dim.  A unit is one (token, block): 32 codes.
// Neighbouring lanes take neighbouring tokens, so the 16-byte stores of eight
// lanes fill one core matrix; the two halves of the 32 codes are read in an
// order that depends on the token, which with the record's own exclusive or
// spreads eight tokens over all banks.
template <int D>
__device__ __forceinline__ void dequant_keys(const uint8_t *raw, uint8_t *op, int tid)
{
    using C = Cfg<D>;
    constexpr int nb = D / 32;
#pragma unroll 2
    for (int u = tid; u < C::kKt * nb; u += C::kDeqWarps * 32) {
        const int tok = u % C::kKt, b = u / C::kKt;  // warp-uniform b
        const int rec = tok / kRec, t = tok % kRec;
        const uint8_t *src = raw + rec * C::kHalf;
        const uint32_t d = *reinterpret_cast<const uint16_t *>(src + k_scale_off(t, b, D));
        const uint32_t d2 = d | (d << 16);
        uint8_t *dst = op + (tok >> 3) * 128 + (tok & 7) * 16;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int half = i ^ ((t >> 1) & 1);
            const uint4 w = *reinterpret_cast<const uint4 *>(src + k_code_off(t, b, nb) + 16 * half);
            uint4 a, c;
            a.x = hmul2(codes2(w.x, 0x4140u), d2);
            a.y = hmul2(codes2(w.x, 0x4342u), d2);
            a.z = hmul2(codes2(w.y, 0x4140u), d2);
            a.w = hmul2(codes2(w.y, 0x4342u), d2);
            c.x = hmul2(codes2(w.z, 0x4140u), d2);
            c.y = hmul2(codes2(w.z, 0x4342u), d2);
            c.z = hmul2(codes2(w.w, 0x4140u), d2);
            c.w = hmul2(codes2(w.w, 0x4342u), d2);
            uint8_t *o = dst + (4 * b + 2 * half) * (C::kKt * 16);
            *reinterpret_cast<uint4 *>(o) = a;
            *reinterpret_cast<uint4 *>(o + C::kKt * 16) = c;
        }
    }
}
// Values: row n = (e % 4) * D / 4 + e / 4 for element e (neighbouring lanes,
// which take neighbouring 16-byte chunks of four elements, then store to
// neighbouring rows), K = token.  A unit is eight tokens of one chunk.
// `seen`: tokens of the tile that some row of the item sees and that have a
// page, as [lo, hi) and a bit per record; the scales of the others count as
// 0, whatever the page holds there (0 * NaN would be NaN).
template <int D>
__device__ __forceinline__ void dequant_values(const uint8_t *raw, uint8_t *op, int tid, int lo, int hi, uint32_t recs)
{
    using C = Cfg<D>;
    const bool edge = lo > 0 || hi < C::kKt || recs != (1u << C::kRecs) - 1u;
#pragma unroll 2
    for (int u = tid; u < (C::kKt / 8) * (D / 4); u += C::kDeqWarps * 32) {
        const int c = u % (D / 4), t8 = u / (D / 4);
        const int rec = t8 / 2, g = 2 * (t8 % 2), b = c / 8;
        const uint8_t *src = raw + rec * C::kHalf - 17 * D;  // offsets below count from the record
        uint4 d = *reinterpret_cast<const uint4 *>(src + v_scale_off(4 * g, b, D));  // eight tokens
        if (edge) {
            uint32_t dw[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int tok = 8 * t8 + k;
                if (tok < lo || tok >= hi || !((recs >> rec) & 1u)) dw[k / 2] &= (k & 1) ? 0x0000FFFFu : 0xFFFF0000u;
            }
            d = make_uint4(dw[0], dw[1], dw[2], dw[3]);
        }
        const uint4 w0 = *reinterpret_cast<const uint4 *>(src + v_chunk_off(g, c, D));
        const uint4 w1 = *reinterpret_cast<const uint4 *>(src + v_chunk_off(g + 1, c, D));
        uint8_t *dst = op + t8 * (D * 16);
        const uint32_t a[4] = {w0.x, w0.y, w0.z, w0.w}, z[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int n = i * (D / 4) + c;
            uint4 o;
            o.x = hmul2(codes2(a[i], 0x4140u), d.x);
            o.y = hmul2(codes2(a[i], 0x4342u), d.y);
            o.z = hmul2(codes2(z[i], 0x4140u), d.z);
            o.w = hmul2(codes2(z[i], 0x4342u), d.w);
            *reinterpret_cast<uint4 *>(dst + (n >> 3) * 128 + (n & 7) * 16) = o;
        }
    }
}

// ---------------------------------------------------------------- the query operand
// This thread's row: elements * 2^-e as f16, e from the row's largest
// magnitude; returns 2^e.  A dead row is zeros.  The row is read twice (the
// second time from L1): held in registers it would spill.
template <int TYPE>
__device__ __forceinline__ float2 pair_of(uint32_t w)
{
    return TYPE == GQ_TYPE_BF16 ? make_float2(bf16_lo(w), bf16_hi(w)) : half2_f2(w);
}
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
    __shared__ long long s_cost[C::kWarpsAll];
    __shared__ Walk s_walk;
    __shared__ volatile int s_abort;
    __shared__ uint32_t s_tmem;
    __shared__ uint32_t s_mask[kMaskRing];
    __shared__ int s_last[2];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t base = smem_u32(smem);
    const uint32_t bar = base + C::kOffBar;
    const uint32_t raw_full = bar, raw_empty = raw_full + 8 * C::kRaws, op_full = raw_empty + 8 * C::kRaws,
                   op_empty = op_full + 8 * C::kOps, q_full = op_empty + 8 * C::kOps, s_full = q_full + 16,
                   p_full = s_full + 16, pv_done = p_full + 16, o_done = pv_done + 16;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kRaws; ++i) {
            mbar_init(raw_full + 8 * i, 1);
            mbar_init(raw_empty + 8 * i, C::kDeqWarps);
        }
        for (int i = 0; i < C::kOps; ++i) {
            mbar_init(op_full + 8 * i, C::kDeqWarps);
            mbar_init(op_empty + 8 * i, 1);
        }
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

    // ---- this CTA's stretch: the sequences' costs, a warp each, twice (the total first)
    long long total = 0, len = 0, begin = 0;
    for (int pass = 0; pass < 2; ++pass) {
        long long at = 0;
        for (int b0 = 0; b0 < B.n_seq; b0 += C::kWarpsAll) {
            if (pass == 0 || B.n_seq > C::kWarpsAll) {
                long long c = 0;
                if (b0 + warp < B.n_seq) {
                    const Seq s = load_seq(B, b0 + warp);
                    c = head_cost<D>(s, A) * B.kv_heads;
                }
                __syncthreads();
                if (lane == 0) s_cost[warp] = c;
                __syncthreads();
            }
            for (int i = 0; i < C::kWarpsAll && b0 + i < B.n_seq; ++i) {
                const long long c = s_cost[i];
                if (pass == 1 && warp == 0 && begin >= at && begin < at + c) {
                    // the item that holds tile `begin`: head, then row tile by a scan over the lanes
                    const Seq s = load_seq(B, b0 + i);
                    const long long hc = c / B.kv_heads;
                    const int h = static_cast<int>((begin - at) / hc);
                    long long rem = begin - at - h * hc;
                    const int nst = row_tiles(s, A, C::kRowsItem);
                    for (int st0 = 0; st0 < nst; st0 += 32) {
                        const int mine = st0 + lane < nst ? item_of<D>(s, A, st0 + lane).tiles : 0;
                        int inc = mine;
#pragma unroll
                        for (int o = 1; o < 32; o <<= 1) {
                            const int v = __shfl_up_sync(0xffffffffu, inc, o);
                            if (lane >= o) inc += v;
                        }
                        if (rem >= inc - mine && rem < inc) {
                            s_walk.b = b0 + i;
                            s_walk.h = h;
                            s_walk.st = st0 + lane;
                            s_walk.from = static_cast<int>(rem) - (inc - mine);
                            s_walk.left = min(len, total - begin);
                            s_walk.x = begin;
                        }
                        const int sum = __shfl_sync(0xffffffffu, inc, 31);
                        if (rem < sum) break;
                        rem -= sum;
                    }
                }
                at += c;
            }
        }
        if (pass == 0) {
            total = at;
            // a stretch of fewer than four tiles would spend more on its join
            len = max((total + gridDim.x - 1) / gridDim.x, 4ll);
            begin = len * blockIdx.x;
        }
    }
    __syncthreads();
    Walk w = s_walk;
    volatile int *abort = &s_abort;
    // The register split stands at the head of each warpgroup's branch, where
    // the compiler takes it as the limit of what follows.
    if (warp < C::kSoftWarps) {
        if (C::kMt == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kMt == 2 ? C::kSoftRegs : 128));
        // ================================================================ softmax: thread = query row
        const int mt = warp >> 2;                       // row tile
        const int row = threadIdx.x & 127;
        const uint32_t lane_addr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const uint32_t o_addr = lane_addr + kOCol + mt * D;
        uint8_t *q_op = smem + mt * C::kQ;
        const float inv_cap = kCap ? 1.0f / A.softcap : 0.f;
        constexpr float kLog2e = 1.4426950408889634f;
        bool ok = true;
        uint32_t n_pv = 0;          // tiles of this row tile so far: scores taken, p v products asked for
        uint32_t n_piece = 0;       // pieces of this row tile so far
        uint32_t tile_no = 0;       // key tiles of the CTA so far
        while (w.left > 0) {
            const Seq s = load_seq(B, w.b);
            const Item it = item_of<D>(s, A, w.st);
            const int to = static_cast<int>(min(static_cast<long long>(it.tiles), w.from + w.left));
            const int r = it.r0 + 128 * mt + row;
            const bool tile_live = it.r0 + 128 * mt < it.rows;  // any row: else the mma warp skips the row tile
            if (tile_live) {
                const bool live = r < it.rows;
                const int tok = live ? r / A.group : 0, head = w.h * A.group + (live ? r % A.group : 0);
                const int pos = s.first + tok;
                const int row_hi = live ? pos : -1;
                const int row_lo = A.window > 0 ? max(0, pos - A.window + 1) : 0;
                const uint8_t *src = A.Q + (s.row0 + tok) * A.ldq + static_cast<long long>(head) * D * 2;
                const float f = A.type == GQ_TYPE_BF16 ? load_query<D, GQ_TYPE_BF16>(src, live, A.scale < 0.f, q_op, row)
                                                       : load_query<D, GQ_TYPE_F16>(src, live, A.scale < 0.f, q_op, row);
                // a factor of 0 would turn hidden scores (-inf) into NaN
                const float zs = fmaxf(fabsf(A.scale) * f * (kCap ? 1.0f : kLog2e), 1e-37f);
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(q_full + 8 * mt);
                float m = kNone, l = 0.f;
                for (int j = w.from; j < to; ++j) {
                    const int buf = C::kMt == 2 ? mt : static_cast<int>(n_pv & 1);
                    const uint32_t s_addr = lane_addr + kSCol * buf;
                    // kMt = 2: one buffer per row tile; kMt = 1: two in turn
                    if (ok) ok = wait_warp(s_full + 8 * buf, (C::kMt == 2 ? n_pv : n_pv >> 1) & 1, abort, B.status);
                    if (!ok) break;
                    tc_fence_after();
                    const int p0 = it.base + j * C::kKt;
                    const uint32_t recs = s_mask[(tile_no + (j - w.from)) % kMaskRing];
                    // every row of the warp sees the whole tile?
                    const bool edge = __any_sync(0xffffffffu, p0 < row_lo || p0 + C::kKt - 1 > row_hi) ||
                                      recs != (1u << C::kRecs) - 1u;
                    float v[C::kKt];
#pragma unroll
                    for (int c = 0; c < C::kKt; c += 32) tmem_ld32_async(s_addr + c, v + c);
                    tmem_wait_ld(v);
                    if (kCap) {
#pragma unroll
                        for (int k = 0; k < C::kKt; ++k) v[k] = soft_cap(v[k] * zs, A.softcap, inv_cap) * kLog2e;
                    }
                    if (edge) {
                        const int a = row_lo - p0, b = row_hi - p0;
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
                        if (j > w.from) {
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
                    l += (sum0.x + sum0.y) + (sum1.x + sum1.y);
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(p_full + 8 * buf);
                    ++n_pv;
                }
                // ---- the piece's result
                if (ok) ok = wait_warp(o_done + 8 * mt, n_piece & 1, abort, B.status);
                ++n_piece;
                tc_fence_after();
                const bool whole = w.from == 0 && to == it.tiles;
                uint8_t *dst = A.O + (s.row0 + tok) * A.ldo + static_cast<long long>(head) * D * 2;
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
                        *reinterpret_cast<uint4 *>(dst + (4 * c + 8 * k) * 2) = make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
                };
                constexpr int kSlot = 128 * (D + 2);  // floats of one row tile's partial: [D][128], m, l
                float *slot = A.part + ((2ll * blockIdx.x + (w.from == 0 ? 1 : 0)) * C::kMt + mt) * kSlot;
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
                        if (live) put(c, x, inv);
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int k = 0; k < 8; ++k) slot[(i * (D / 4) + c + k) * 128 + row] = x[8 * i + k];
                    }
                }
                // the next piece's first p v overwrites the accumulator only after this warp's next p
                tc_fence_before();
                if (!whole) {
                    slot[D * 128 + row] = m;
                    slot[(D + 1) * 128 + row] = l;
                    const long long item_x = w.x - w.from;
                    const int c0 = static_cast<int>(item_x / len), c1 = static_cast<int>((item_x + it.tiles - 1) / len);
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
                        for (int c = c0; c <= c1; ++c) M = fmaxf(M, __ldcg(part(c) + D * 128 + row));
                        for (int c = c0; c <= c1; ++c)
                            L += ex2(__ldcg(part(c) + D * 128 + row) - M) * __ldcg(part(c) + (D + 1) * 128 + row);
                        const float linv = L == 0.f ? 0.f : 1.0f / L;
#pragma unroll 1
                        for (int c = 0; c < D / 4; c += 8) {
                            float x[32];
#pragma unroll
                            for (int k = 0; k < 32; ++k) x[k] = 0.f;
                            for (int cc = c0; cc <= c1; ++cc) {
                                const float *src2 = part(cc);
                                const float g = ex2(__ldcg(src2 + D * 128 + row) - M);
#pragma unroll
                                for (int i = 0; i < 4; ++i)
#pragma unroll
                                    for (int k = 0; k < 8; ++k)
                                        x[8 * i + k] += g * __ldcg(src2 + (i * (D / 4) + c + k) * 128 + row);
                            }
                            if (live) put(c, x, linv);
                        }
                    }
                    bar_sync(1 + mt, 128);  // s_last may be written again
                }
            }
            const int done = to - w.from;
            tile_no += done;
            if (!next_piece<D>(w, B, A, done)) break;
        }
    } else if (warp < C::kProdWarp) {
        if (C::kMt == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kMt == 2 ? C::kDeqRegs : 128));
        // ================================================================ dequantizers
        const int tid = threadIdx.x - 32 * C::kSoftWarps;
        bool ok = true;
        uint32_t n = 0, tile_no = 0;  // operand tiles, key tiles
        while (ok && w.left > 0) {
            const Seq s = load_seq(B, w.b);
            const Item it = item_of<D>(s, A, w.st);
            const int to = static_cast<int>(min(static_cast<long long>(it.tiles), w.from + w.left));
            for (int j = w.from; j < to && ok; ++j, ++tile_no) {
                const int p0 = it.base + j * C::kKt;
#pragma unroll 1
                for (int part = 0; part < 2; ++part, ++n) {
                    const uint32_t rs = n % C::kRaws, os = n % C::kOps;
                    ok = wait_warp(raw_full + 8 * rs, (n / C::kRaws) & 1, abort, B.status);
                    if (!ok) break;
                    if (n >= C::kOps) {
                        ok = wait_warp(op_empty + 8 * os, (n / C::kOps - 1) & 1, abort, B.status);
                        if (!ok) break;
                    }
                    const uint8_t *raw = smem + C::kOffRaw + rs * C::kRaw;
                    uint8_t *op = smem + C::kOffOp + os * C::kOp;
                    if (part == 0) dequant_keys<D>(raw, op, tid);
                    else
                        dequant_values<D>(raw, op, tid, max(it.lo - p0, 0), min(max(it.hi + 1 - p0, 0), C::kKt),
                                          s_mask[tile_no % kMaskRing]);
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(op_full + 8 * os);
                        mbar_arrive(raw_empty + 8 * rs);
                    }
                }
            }
            if (!ok || !next_piece<D>(w, B, A, to - w.from)) break;
        }
    } else {
        if (C::kMt == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kMt == 2 ? C::kRestRegs : 128));
    if (w.left > 0 && warp == C::kProdWarp) {
        // ================================================================ producer: one lane per record
        bool ok = true;
        uint32_t n = 0, tile_no = 0;
        while (ok) {
            const Seq s = load_seq(B, w.b);
            const Item it = item_of<D>(s, A, w.st);
            const int to = static_cast<int>(min(static_cast<long long>(it.tiles), w.from + w.left));
            auto page = [&](int j) {  // this lane's record of tile j: its page, -1 if it is bad, -2 if it is beyond the item
                const int pos = it.base + j * C::kKt + lane * kRec;
                if (lane >= C::kRecs || j >= to || pos > it.hi) return -2;
                return page_of(B, w.b, pos);
            };
            int pg = page(w.from);
            for (int j = w.from; j < to && ok; ++j, ++tile_no) {
                const int pg_next = page(j + 1);
                // records beyond the item are hidden by position; bad pages by this mask
                const uint32_t copied = __ballot_sync(0xffffffffu, pg >= 0);
                const uint32_t bad = __ballot_sync(0xffffffffu, pg == -1);
                const int pos = it.base + j * C::kKt + lane * kRec;
#pragma unroll 1
                for (int part = 0; part < 2; ++part, ++n) {
                    const uint32_t rs = n % C::kRaws;
                    if (n >= C::kRaws) {
                        ok = wait_warp(raw_empty + 8 * rs, (n / C::kRaws - 1) & 1, abort, B.status);
                        if (!ok) break;
                    }
                    if (lane == 0) {
                        if (part == 0) s_mask[tile_no % kMaskRing] = ((1u << C::kRecs) - 1u) & ~bad;
                        const uint32_t bytes = __popc(copied) * C::kHalf;
                        if (bytes) mbar_expect_tx(raw_full + 8 * rs, bytes);
                        else mbar_arrive(raw_full + 8 * rs);
                    }
                    __syncwarp();
                    if (pg >= 0)
                        bulk_load(base + C::kOffRaw + rs * C::kRaw + lane * C::kHalf,
                                  A.cache + rec_off(B, pg, w.h, pos, D) + part * C::kHalf, C::kHalf, raw_full + 8 * rs);
                }
                pg = pg_next;
            }
            if (!ok || !next_piece<D>(w, B, A, to - w.from)) break;
        }
        // copies in flight land before the CTA's memory is given up
        for (uint32_t i = n > C::kRaws ? n - C::kRaws : 0; i < n; ++i)
            wait_warp(raw_full + 8 * (i % C::kRaws), (i / C::kRaws) & 1, abort, B.status);
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
        constexpr uint32_t kHi = (128u >> 4) | (1u << 14);  // 128 bytes between row groups; descriptor version 1
        auto desc_lo = [](uint32_t addr, uint32_t lbo) { return ((addr & 0x3FFFFu) >> 4) | ((lbo >> 4) << 16); };
        auto desc = [](uint32_t lo) {
            uint64_t d;
            asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(kHi));
            return d;
        };
        const uint32_t q_lo = desc_lo(base, 2048), k_lo = desc_lo(base + C::kOffOp, C::kKt * 16),
                       v_lo = desc_lo(base + C::kOffOp, D * 16);
        auto qk = [&](int mt, uint32_t os, int buf) {
            const uint32_t a = q_lo + mt * (C::kQ >> 4), b = k_lo + os * (C::kOp >> 4);
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
                mma_f16(tmem + kSCol * buf, desc(a + k * 256), desc(b + k * 2 * C::kKt), kIdQk, k > 0);
            mma_commit(s_full + 8 * buf);
        };
        auto pv = [&](int mt, uint32_t os, int buf, bool first) {
            const uint32_t b = v_lo + os * (C::kOp >> 4);
#pragma unroll
            for (int k = 0; k < C::kKt / 16; ++k)
                mma_f16_ts(tmem + kOCol + mt * D, tmem + kSCol * buf + 8 * k, desc(b + k * 2 * D), kIdPv, !first || k > 0);
            mma_commit(pv_done + 8 * mt);
        };
        while (ok) {
            const Seq s = load_seq(B, w.b);
            const Item it = item_of<D>(s, A, w.st);
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
            if (!next_piece<D>(w, B, A, nt)) break;
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
    switch (head_dim) {
    case 64: return kv::chunk::launch<64>(A, B, s);
    case 128: return kv::chunk::launch<128>(A, B, s);
    default: return kv::chunk::launch<256>(A, B, s);
    }
}

}  // namespace gq
