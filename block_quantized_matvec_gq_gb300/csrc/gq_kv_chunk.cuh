// gq_kv_chunk.cuh -- what the tensor-core kernels for chunks of new tokens
// share: the items and the line of work, tensor-memory transfers, MMA
// operands, and the query rows.
#pragma once

#include "gq_kv.cuh"
#include "gq_tc.cuh"

namespace gq {
namespace kv {
namespace chunk {

using namespace tcu;

constexpr int kTmemCols = 512;
constexpr int kSCol = 128;        // column step between score buffers
constexpr int kOCol = 256;        // first accumulator column
constexpr float kNone = -FLT_MAX;  // reference of a row that has seen no token: below every score
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
// C: the kernel's configuration (query rows per item kRowsItem, tokens per tile kKt).
template <class C>
__device__ __forceinline__ Item item_of(const Seq &s, const Args &A, int st)
{
    Item it;
    it.s = s;
    it.rows = s.n * A.group;
    it.r0 = st * C::kRowsItem;
    const int t0 = it.r0 / A.group, t1 = min(it.r0 + C::kRowsItem, it.rows) - 1;
    it.hi = min(s.first + t1 / A.group, s.kv - 1);
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
template <class C>
__device__ __forceinline__ long long head_cost(const Seq &s, const Args &A)
{
    const int nst = row_tiles(s, A, C::kRowsItem);
    long long c = 0;
    for (int st = threadIdx.x & 31; st < nst; st += 32) c += item_of<C>(s, A, st).tiles;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
    return c;
}

// Moves to the next piece; false when the stretch is done.
template <class C>
__device__ __forceinline__ bool next_piece(Walk &w, const Batch &B, const Args &A, int tiles_done)
{
    w.left -= tiles_done;
    w.x += tiles_done;
    if (w.left <= 0) return false;
    w.from = 0;
    Seq s = load_seq(B, w.b);
    if (++w.st < row_tiles(s, A, C::kRowsItem)) return true;
    w.st = 0;
    if (++w.h < B.kv_heads) return true;
    w.h = 0;
    do {
        if (++w.b >= B.n_seq) return false;
        s = load_seq(B, w.b);
    } while (s.n == 0);
    return true;
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

// A cut closer than kSnap tiles to an item's end is moved there: joining the
// parts of a cut item costs about as much as that many tiles.
constexpr int kSnap = 4;
__device__ __forceinline__ long long snap(long long x, long long x0, int n)
{
    return x - x0 < kSnap ? x0 : (x0 + n - x < kSnap ? x0 + n : x);
}
// First and last CTA of a cut item of n tiles that begins at x0: the cuts
// moved to its start come before the first, those that stayed inside it
// separate the others.
__device__ __forceinline__ int first_cta(long long x0, int n, long long len) { return static_cast<int>((x0 + min(kSnap, n) - 1) / len); }
__device__ __forceinline__ int last_cta(long long x0, int n, long long len) { return static_cast<int>((x0 + n - kSnap) / len); }

// This CTA's stretch of the line, into `walk` (left = 0 if it has none); all
// threads take part: a warp per sequence for the total, then two warps look
// for the stretch's two cuts.  Returns the length of a stretch.
template <class C>
__device__ __forceinline__ long long find_stretch(const Batch &B, const Args &A, long long *s_cost, long long *s_cut, Walk &s_walk)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    long long total = 0, len = 0, mine = 0;  // mine: this warp's cut
    for (int pass = 0; pass < 2; ++pass) {
        long long at = 0;
        for (int b0 = 0; b0 < B.n_seq; b0 += C::kWarpsAll) {
            if (pass == 0 || B.n_seq > C::kWarpsAll) {
                long long c = 0;
                if (b0 + warp < B.n_seq) c = head_cost<C>(load_seq(B, b0 + warp), A) * B.kv_heads;
                __syncthreads();
                if (lane == 0) s_cost[warp] = c;
                __syncthreads();
            }
            for (int i = 0; i < C::kWarpsAll && b0 + i < B.n_seq; ++i) {
                const long long c = s_cost[i];
                if (pass == 1 && warp < 2 && mine >= at && mine < at + c) {
                    // the item that holds tile `mine`: head, then row tile by a scan over the lanes
                    const Seq s = load_seq(B, b0 + i);
                    const long long hc = c / B.kv_heads;
                    const int h = static_cast<int>((mine - at) / hc);
                    long long rem = mine - at - h * hc;
                    const int nst = row_tiles(s, A, C::kRowsItem);
                    for (int st0 = 0; st0 < nst; st0 += 32) {
                        const int n = st0 + lane < nst ? item_of<C>(s, A, st0 + lane).tiles : 0;
                        int inc = n;
#pragma unroll
                        for (int o = 1; o < 32; o <<= 1) {
                            const int v = __shfl_up_sync(0xffffffffu, inc, o);
                            if (lane >= o) inc += v;
                        }
                        if (rem >= inc - n && rem < inc) {
                            const long long x0 = mine - rem + (inc - n), cut = snap(mine, x0, n);
                            s_cut[warp] = cut;
                            if (warp == 0) {
                                s_walk.b = b0 + i;
                                s_walk.h = h;
                                s_walk.st = st0 + lane;
                                s_walk.from = static_cast<int>(cut - x0);  // = n: the item after it
                                s_walk.x = cut;
                            }
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
            mine = len * (blockIdx.x + warp);
            if (threadIdx.x == 0) s_cut[0] = s_cut[1] = total;
            __syncthreads();
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        Walk w = s_walk;
        w.left = s_cut[0] < total ? s_cut[1] - s_cut[0] : 0;
        if (w.left > 0 && w.from == item_of<C>(load_seq(B, w.b), A, w.st).tiles) next_piece<C>(w, B, A, 0);
        s_walk = w;
    }
    __syncthreads();
    return len;
}

// ---------------------------------------------------------------- the size of a token's values
// p reaches the products in f16, some 32 octaves above whose smallest number a
// strong key's p may stand.  If that key's values are small, the others make
// the result although their p is far smaller.  So a token whose values are much
// smaller (or larger) than most enters with its values times 2^dn and its p
// times 2^-dn, where dn brings its largest value scale to the usual size; the
// reference m is that of the scores less dn, and only the sum l takes p itself.
// The usual size is the mean over the first tile of a piece, or the size before
// where that tile agrees with it (any would do: the products do not depend on
// it); tokens within kNear octaves of it have dn = 0, and a tile of nothing
// else is as if there were no dn.  The others are
// `mixed` and rare.
// Of all this, a tile that is not mixed costs its test alone.  The rest is kept
// short and out of the hot loops, which together fill the SM's instruction
// cache: a second copy of the producer's loop, nothing else changed, took 509 of
// 8191 tokens in f32 from 179 to 245 us (cache misses 0.7 to 4.5 million).  A
// call whose every tile is mixed takes two to three times as long (2048 of 32768
// tokens 817 and 2628 us).
constexpr int kNear = 3;
constexpr int kNoValue = 90;           // in place of 8 - log2 of a scale of 0: its p, 2^105 at most, stays in f32
constexpr int kMostBase = 20;          // values are brought to scales of 2^-12 at least, so that they keep their bits
constexpr uint32_t kMixed = 1u << 31;  // in a tile's word of the mask ring

// 8 - floor(log2 of a largest value scale), from its fp16 bits
__device__ __forceinline__ int value_shift(uint32_t h)
{
    return h == 0 ? kNoValue : 135 - static_cast<int>(__float_as_uint(half2_f2(h).x) >> 23);
}

// The value scales of a tile, as the keys' producer sees them: a lane has
// kTokens neighbouring tokens, two to a word, of every block.
template <int D, class C>
struct TileScales {
    static constexpr int kTokens = C::kKt / 32, kWords = kTokens / 2, nb = D / 32;
    uint32_t w[nb][kWords];
    static __device__ __forceinline__ int record() { return (threadIdx.x & 31) * kTokens / kRec; }
    // off: offset of the lane's record in the cache (lanes below kRecs), negative if it has none
    __device__ __forceinline__ void load(const uint8_t *cache, long long off)
    {
        const long long o = __shfl_sync(0xffffffffu, off, record());
        const uint8_t *src = cache + o + v_scale_off((threadIdx.x & 31) * kTokens % kRec, 0, D);
#pragma unroll
        for (int b = 0; b < nb; ++b) {
            uint2 v = make_uint2(0u, 0u);
            if (o >= 0) {
                if (kWords == 2) v = __ldg(reinterpret_cast<const uint2 *>(src + 2 * kRec * b));
                else v.x = __ldg(reinterpret_cast<const uint32_t *>(src + 2 * kRec * b));
            }
            w[b][0] = v.x;
            if (kWords == 2) w[b][kWords - 1] = v.y;
        }
    }
    // The largest scale of every token
    __device__ __forceinline__ void largest(uint32_t (&m)[kWords]) const
    {
#pragma unroll
        for (int k = 0; k < kWords; ++k) {
            m[k] = w[0][k];
#pragma unroll
            for (int b = 1; b < nb; ++b) m[k] = __vmaxu2(m[k], w[b][k]);
        }
    }
};
// The usual size of a piece and the bounds that it sets, fp16 bits twice.
struct Usual {
    int base;
    uint32_t above, below;  // larger, smaller ones make a tile mixed
};
// Looks at every token of a tile where some scale is out of bounds; at the first
// tile of a piece (`first`) also for the usual size.  scratch: the tokens'
// largest scales; [lo, hi) and recs: the tokens that count.  Writes dn; returns
// the base, and in bit 8 whether the tile is mixed.  Out of line, with loops
// instead of registers.
template <int kKt>
static __device__ __noinline__ int look_closer(const uint16_t *scratch, float *dn, int lo, int hi, uint32_t recs, int base, bool first)
{
    const int lane = threadIdx.x & 31;
    if (first) {
        int sum = 0, n = 0;
#pragma unroll 1
        for (int tok = lane; tok < kKt; tok += 32)
            if (tok >= lo && tok < hi && (recs >> (tok / kRec) & 1u) && scratch[tok] != 0) sum += value_shift(scratch[tok]), ++n;
        sum = __reduce_add_sync(0xffffffffu, sum);
        n = __reduce_add_sync(0xffffffffu, n);
        // a tile without values says nothing
        if (n > 0) base = min(max(__float2int_rn(__fdividef(static_cast<float>(sum), static_cast<float>(n))), 0), kMostBase);
    }
    bool mixed = false;
#pragma unroll 1
    for (int tok = lane; tok < kKt; tok += 32) {
        const int d = value_shift(scratch[tok]) - base;
        const bool far = tok >= lo && tok < hi && (recs >> (tok / kRec) & 1u) && (d < -kNear || d > kNear);
        dn[tok] = far ? static_cast<float>(d) : 0.f;
        mixed = mixed || far;
    }
    return base | (__any_sync(0xffffffffu, mixed) ? 0x100 : 0);
}
// The value scales of a raw stage of values, in place: 0 for tokens outside [lo,
// hi) or without a page (recs), whatever the page holds there (0 * NaN would be
// NaN), times 2^dn in a mixed tile.  All dequantizer threads, which then wait
// for one another at `fixed` (n_fixed: how often so far); false if that gave up.
// Every other tile passes by.
template <int D, class C>
__device__ __forceinline__ bool fix_scales(uint8_t *raw, int tid, int lo, int hi, uint32_t word, const float *dn, uint32_t fixed,
                                           uint32_t &n_fixed, volatile int *abort, int *status)
{
    if (__builtin_expect(lo <= 0 && hi >= C::kKt && word == (1u << C::kRecs) - 1u, 1)) return true;
#pragma unroll 1
    for (int u = tid; u < C::kKt * (D / 32); u += 32 * C::kDeqWarps) {
        const int tok = u % C::kKt;
        __half *d = reinterpret_cast<__half *>(raw + tok / kRec * C::kHalf - 17 * D + v_scale_off(tok % kRec, u / C::kKt, D));
        const float f = word & kMixed ? ex2(dn[tok]) : 1.0f;
        *d = __float2half_rn(tok >= lo && tok < hi && (word >> (tok / kRec) & 1u) ? __half2float(*d) * f : 0.f);
    }
    __syncwarp();
    if ((tid & 31) == 0) mbar_arrive(fixed);
    return wait_warp(fixed, n_fixed++ & 1, abort, status);
}
// The scores of a tile (kSums: two columns each, kKt apart) capped and in octaves,
// in place in tensor memory.  (Unrolled over a row in registers it was 17
// instructions a score, more code than the SM's instruction cache holds.)
template <int kKt, bool kSums>
__device__ __forceinline__ void cap_scores(uint32_t s_addr, float zs, float cap, float inv_cap)
{
#pragma unroll 1
    for (int c = 0; c < kKt; c += 16) {
        float x[16], y[16];
        tmem_ld16(s_addr + c, x);
        if (kSums) tmem_ld16(s_addr + kKt + c, y);
        uint32_t o[16], zero[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const float v = (kSums ? x[k] + y[k] : x[k]) * zs;
            o[k] = __float_as_uint(soft_cap(v, cap, inv_cap) * 1.4426950408889634f);
            zero[k] = 0u;
        }
        tmem_st16(s_addr + c, o);
        if (kSums) tmem_st16(s_addr + kKt + c, zero);
    }
    tmem_wait_st();
}
// A mixed tile's scores (kSums: as above) less dn, in place in tensor memory, for
// the common path to go on with; unit: what it multiplies them by to have
// octaves.  Of the tokens lo .. hi that have a page, into `out`: the largest, in
// octaves, and the sum of p = 2^(score + dn - largest + head), where the products
// take p 2^-dn.
template <int kKt, bool kSums>
__device__ __forceinline__ void shift_scores(uint32_t s_addr, float unit, int lo, int hi, uint32_t recs, const float *dn, float2 *out)
{
    const float back = 1.0f / unit;
    float top = -INFINITY, sum = 0.f;
#pragma unroll 1
    for (int c = 0; c < kKt; c += 8) {
        uint32_t x[8], y[8];
        tmem_ld8(s_addr + c, x);
        if (kSums) tmem_ld8(s_addr + kKt + c, y);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            float v = __uint_as_float(x[k]);
            if (kSums) v += __uint_as_float(y[k]);
            v = fmaf(-dn[c + k], back, v);
            if (c + k >= lo && c + k <= hi && (recs >> (c / kRec) & 1u)) top = fmaxf(top, v);
            x[k] = __float_as_uint(v);
            y[k] = 0u;
        }
        tmem_st8(s_addr + c, x);
        if (kSums) tmem_st8(s_addr + kKt + c, y);
    }
    tmem_wait_st();
    top *= unit;
#pragma unroll 1
    for (int c = 0; c < kKt; c += 8) {
        uint32_t x[8];
        tmem_ld8(s_addr + c, x);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (c + k >= lo && c + k <= hi && (recs >> (c / kRec) & 1u))
                sum = fmaf(ex2(fmaf(__uint_as_float(x[k]), unit, kPHead - top)), ex2(dn[c + k]), sum);
    }
    *out = make_float2(top, sum);
}

// A producer warp: the key halves (part 0) or the value halves (part 1) of a
// tile's records into the ring of raw stages, tile t into stage number 2 t +
// part; a lane per record, one bulk copy each (two warps, because the copies of
// a warp are issued one lane at a time).  Page numbers are fetched a tile ahead
// and looked at only then.  The keys' producer also writes the tile's word of the
// mask ring -- a bit per record, 0 where the page is bad (its tokens are then
// hidden; records beyond the item are hidden by position and not copied), and
// whether the values are mixed -- before the stage can fill: their scales are
// fetched a tile ahead too.  s_dn: [kMaskRing][kKt]; scratch: [kKt].
template <int D, class C>
__device__ __forceinline__ void produce(int part, Walk &w, const Batch &B, const Args &A, uint8_t *smem, uint32_t raw_full,
                                        uint32_t raw_empty, uint32_t *s_mask, float *s_dn, uint16_t *scratch, volatile int *abort)
{
    const int lane = threadIdx.x & 31;
    bool ok = true;
    uint32_t tile_no = 0;
    Usual usual = {12, 0u, ~0u};  // bounds that every tile is outside of, until one has been looked at
    while (ok) {
        const Seq s = load_seq(B, w.b);
        const Item it = item_of<C>(s, A, w.st);
        const int to = static_cast<int>(min(static_cast<long long>(it.tiles), w.from + w.left));
        const int rec0 = it.base / kRec + lane;  // this lane's record of tile 0
        auto wanted = [&](int j) { return lane < C::kRecs && j < to && (rec0 + j * C::kRecs) * kRec <= it.hi; };
        auto entry = [&](int j) { return wanted(j) ? __ldg(page_at(B, w.b, rec0 + j * C::kRecs)) : 0; };
        TileScales<D, C> scales;
        long long off = -1;
        int next = entry(w.from);
        // a turn early: places and scales of the first tile
        for (int j = w.from - 1; j < to; ++j) {
            const long long cur = off;  // of tile j
            const uint32_t n = 2 * tile_no + part, bar = raw_full + 8 * (n % C::kRaws);
            if (j >= w.from) {
                if (n >= C::kRaws) {
                    ok = wait_warp(raw_empty + 8 * (n % C::kRaws), (n / C::kRaws - 1) & 1, abort, B.status);
                    if (!ok) break;
                }
                // the stage is full when these have landed and lane 0 has arrived
                if (cur >= 0) bulk_load(smem_u32(smem) + C::kOffRaw + n % C::kRaws * C::kRaw + lane * C::kHalf, A.cache + cur + part * C::kHalf, C::kHalf, bar);
            }
            // offset of this lane's record of tile j + 1, -1 without one, -2 where the page is bad
            off = -1;
            if (wanted(j + 1)) {
                const int pg = checked_page(B, next);
                off = pg >= 0 ? rec_off(B, pg, w.h, rec0 + (j + 1) * C::kRecs, D) : -2;
            }
            next = entry(j + 2);
            const TileScales<D, C> now = scales;  // of tile j; looked at only after the next ones have been asked for
            if (part == 0) scales.load(A.cache, off);
            if (j < w.from) continue;
            const uint32_t copied = __ballot_sync(0xffffffffu, cur >= 0);
            if (part == 0) {
                uint32_t word = ((1u << C::kRecs) - 1u) & ~__ballot_sync(0xffffffffu, cur == -2);
                const int p0 = it.base + j * C::kKt, lo = it.lo - p0, hi = it.hi + 1 - p0;
                // Whether some scale is out of bounds: of any token of the records here, seen or
                // not, and at a piece's beginning by the last piece's usual size.
                constexpr int kWords = TileScales<D, C>::kWords;
                uint32_t m[kWords], above = usual.above, below = usual.below;
                now.largest(m);
                if (copied >> now.record() & 1u) {
#pragma unroll
                    for (int k = 0; k < kWords; ++k) {
                        above = __vmaxu2(above, m[k]);
                        below = __vminu2(below, m[k]);
                    }
                }
                if (__builtin_expect(__any_sync(0xffffffffu, above != usual.above || below != usual.below), 0)) {
#pragma unroll
                    for (int k = 0; k < kWords; ++k) reinterpret_cast<uint32_t *>(scratch)[kWords * lane + k] = m[k];
                    __syncwarp();
                    const int got = look_closer<C::kKt>(scratch, s_dn + tile_no % kMaskRing * C::kKt, lo, hi, word, usual.base, j == w.from);
                    usual.base = got & 0xFF;
                    const float top = pow2i(9 + kNear - usual.base), low = pow2i(8 - kNear - usual.base);
                    usual.above = f2_half2(top, top) - 0x00010001u;
                    usual.below = f2_half2(low, low);
                    if (got & 0x100) word |= kMixed;
                }
                if (lane == 0) s_mask[tile_no % kMaskRing] = word;
                __syncwarp();
            }
            if (lane == 0) {
                const uint32_t bytes = __popc(copied) * C::kHalf;
                if (bytes) mbar_expect_tx(bar, bytes);
                else mbar_arrive(bar);
            }
            ++tile_no;
        }
        if (!ok || !next_piece<C>(w, B, A, to - w.from)) {
            break;
        }
    }
    // the last copies land before the CTA's memory is given up
    for (uint32_t t = tile_no > C::kRaws ? tile_no - C::kRaws : 0; t < tile_no; ++t) {
        const uint32_t n = 2 * t + part;
        if (n + C::kRaws >= 2 * tile_no + part) wait_warp(raw_full + 8 * (n % C::kRaws), (n / C::kRaws) & 1, abort, B.status);
    }
}

// Shared-memory descriptors of operand tiles in 8 x 16-byte core matrices, 128
// bytes between row groups: the low word of the first K step (lbo: bytes
// between K groups); later steps add a constant to it.
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lbo) { return ((addr & 0x3FFFFu) >> 4) | ((lbo >> 4) << 16); }
__device__ __forceinline__ uint64_t desc_of(uint32_t lo)
{
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"((128u >> 4) | (1u << 14)));
    return d;
}

// Two 16-bit elements of a token array.
template <int TYPE>
__device__ __forceinline__ float2 pair_of(uint32_t w)
{
    return TYPE == GQ_TYPE_BF16 ? make_float2(bf16_lo(w), bf16_hi(w)) : half2_f2(w);
}

// gq_kv_chunk_f32.cu: f32 token arrays, head_dim 64 or 128
int launch_chunk_f32(const Args &A, const Batch &B, int head_dim, int max_ctas, cudaStream_t s);

}  // namespace chunk
}  // namespace kv
}  // namespace gq
