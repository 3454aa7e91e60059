// gq_kv.cu -- writing and reading the paged Q8_0 key/value cache, and the C
// entry points of include/gq_kv.h.
//
// One warp handles one unit: a group of four tokens (one word of the value
// layout) of two neighbouring 32-blocks of one kv head's keys or values.  Lane
// 16 i + 4 j + s holds elements 8 s .. 8 s + 7 of block i of token j.  The
// keys' codes are stored as they are (32 bytes per token and block); the
// values' 4 x 4 byte squares are transposed between lanes j with two
// shuffles, so a lane writes the words of two elements with the four tokens'
// codes.  A group that is only partly new (the ends of a chunk, every decode
// step) writes the new tokens' bytes alone.
//
// What bounds them: long calls stream.  Appending 19008 tokens of 8 heads x 128
// in f32 (197 MB with the codes) takes 35.8 us, 5.5 TB/s, 0.81 of the measured
// copy rate; the instructions of the code rule keep it there (12 a code with
// its tests per element: 59 us; 6 with one test per eight: 35), so bf16 (119 MB)
// takes no less: 39 us.  Narrow caches leave most of a CTA's warps without a
// unit (65536 tokens of 1 x 128: 47 us for 85 MB).  Reading 57410 tokens back
// in bf16 (360 MB) takes 64.3 us, 5.6 TB/s; in f32 90.3 us, 6.6 TB/s.  A decode
// step is launch latency: one token 2.2 us, 64 sequences 3.7.
#include <math.h>

#include "gq_kv.cuh"
#include "gq_q8code.cuh"

namespace gq {
namespace kv {

constexpr int kThreads = 256;

// Slots: sequence b's groups of four positions start at slot
// q_start[b] / 4 + 2 b.  A sequence of n rows touches at most
// floor((n + 6) / 4) <= floor(n / 4) + 2 groups, so the slots of two
// sequences never overlap, and there are n_tokens / 4 + 2 n_seq of them.
// Finds the sequence of `slot` by a 32-way search (every lane of the warp
// takes part) and what the lists say of it: the last step's lanes hold
// neighbouring sequences and load all three numbers at once.
__device__ __forceinline__ Seq find_seq(const Batch &B, long long slot, int &b)
{
    const int lane = threadIdx.x & 31;
    int lo = 0, n = B.n_seq;  // the answer lies in [lo, lo + n)
    while (n > 32) {
        const int step = (n + 31) / 32;
        const int i = lo + lane * step;
        const bool at = i < lo + n && (__ldg(B.q_start + i) >> 2) + 2ll * i <= slot;
        // the starts rise with i: the lanes that hold are a prefix
        const int k = max(__popc(__ballot_sync(0xffffffffu, at)) - 1, 0);
        n = min(step, n - k * step);
        lo += k * step;
    }
    const int i = min(lo + lane, B.n_seq - 1);
    const int r0 = __ldg(B.q_start + i), r1 = __ldg(B.q_start + i + 1), kv = __ldg(B.kv_len + i);
    const bool at = lane < n && (r0 >> 2) + 2ll * i <= slot;
    const int k = max(__popc(__ballot_sync(0xffffffffu, at)) - 1, 0);
    b = lo + k;
    return seq_of(B, __shfl_sync(0xffffffffu, r0, k), __shfl_sync(0xffffffffu, r1, k), __shfl_sync(0xffffffffu, kv, k));
}

// 4 x 4 byte transpose between the lanes j = lane / 4 % 4 that agree elsewhere.
__device__ __forceinline__ uint32_t transpose4(uint32_t x)
{
    const int j = (threadIdx.x >> 2) & 3;
    uint32_t r = __shfl_xor_sync(0xffffffffu, x, 4);
    x = __byte_perm(x, r, (j & 1) ? 0x3715u : 0x6240u);
    r = __shfl_xor_sync(0xffffffffu, x, 8);
    return __byte_perm(x, r, (j & 2) ? 0x3276u : 0x5410u);
}

// max that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// a / 127 rounded to nearest: the product with the rounded reciprocal, corrected
// by its remainder (Markstein's theorem; equal to the division for every f32 in
// a trial over all mantissas).  The product alone is an ulp off often enough
// that the fp16 scale of one block in some millions is another.
__device__ __forceinline__ float over127(float a)
{
    constexpr float r = 1.0f / 127.0f;
    const float q = __fmul_rn(a, r);
    return __fmaf_rn(__fmaf_rn(-127.0f, q, a), r, q);  // NaN for an infinity: fminf takes the other operand
}

// The code bytes (code + 128) of eight elements of a block with scale d:
// the rule of q8_pack4, with its tests made once for all eight.  With r =
// RN(1 / d) and y = RN(e r), RN(e / d) and y round to the same integer n
// unless y is within 2^-15 of a half-integer (gq_q8code.cuh); m = RN(y +
// 1.5 2^23 + 128) holds n + 128 in its low byte, and y - n is exact.  Where an
// element is that close, or not finite, or the clamp could bite (|y| of the
// block's largest beyond 127.4: a scale rounded far down, a saturated block,
// d = 0), the lane takes q8_pack4.
__device__ __forceinline__ uint2 code_bytes8(const float (&e)[8], float d, float amax)
{
    constexpr float kMagic = 12582912.0f + 128.0f;
    const float r = __frcp_rn(d);
    float m[8], off = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float y = __fmul_rn(e[i], r);
        m[i] = __fadd_rn(y, kMagic);
        off = max_nan(off, fabsf(__fsub_rn(y, __fsub_rn(m[i], kMagic))));
    }
    if (off < 0.5f - 0x1p-15f && __fmul_rn(amax, r) < 127.4f) {
        uint32_t w[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint32_t a = __byte_perm(__float_as_uint(m[4 * k]), __float_as_uint(m[4 * k + 1]), 0x0040u);
            const uint32_t b = __byte_perm(__float_as_uint(m[4 * k + 2]), __float_as_uint(m[4 * k + 3]), 0x0040u);
            w[k] = __byte_perm(a, b, 0x5410u);
        }
        return make_uint2(w[0], w[1]);
    }
    const float lo[4] = {e[0], e[1], e[2], e[3]}, hi[4] = {e[4], e[5], e[6], e[7]};
    return make_uint2(q8_pack4(lo, d) ^ 0x80808080u, q8_pack4(hi, d) ^ 0x80808080u);
}

// What a warp's units have in common: the group of four tokens.  Groups are
// aligned in position, so one lies in one record, and wholly inside the table's
// positions or wholly outside (rows there exist only where the lists are
// wrong: they are not written, and read as zeros).
struct Group {
    long long row;  // this lane's token's row
    long long p0;   // the group's first position
    int b;          // sequence
    int t;          // the lane's token's place in the record
    bool mine;      // it is a new token
};
__device__ __forceinline__ Group load_group(const Batch &B, long long slot)
{
    Group g;
    const Seq s = find_seq(B, slot, g.b);
    const long long local = slot - ((static_cast<long long>(s.row0) >> 2) + 2ll * g.b);
    g.p0 = 4ll * ((s.first >> 2) + local);
    const long long pos = g.p0 + ((threadIdx.x >> 2) & 3);
    g.mine = pos >= s.first && pos < s.first + s.n;
    g.row = s.row0 + (pos - s.first);
    g.t = static_cast<int>(pos) & (kRec - 1);
    return g;
}
// Record offset of kv head 0 for the group, -1 if there is none (warp-uniform).
template <int D>
__device__ __forceinline__ long long group_rec(const Batch &B, const Group &g)
{
    if (!__any_sync(0xffffffffu, g.mine)) return -1;
    if (g.p0 < 0 || g.p0 >= static_cast<long long>(B.max_pages) * B.page_tokens) {
        flag_shape(B);
        return -1;
    }
    const int rec = static_cast<int>(g.p0) / kRec, pg = page_of(B, g.b, rec);
    return pg >= 0 ? rec_off(B, pg, 0, rec, D) : -1;
}

// The unit's place: head, first block, keys or values.
struct Unit {
    bool live, isv;
    int h, b;
    int elem;  // first element of this lane in a token's row
};
template <int D>
__device__ __forceinline__ Unit unit_of(int u, int kv_heads)
{
    constexpr int pairs = D / 64;
    Unit x;
    const int half = kv_heads * pairs;
    x.live = u < 2 * half;
    x.isv = u >= half;
    const int hp = x.isv ? u - half : u, lane = threadIdx.x & 31;
    x.h = hp / pairs;
    x.b = 2 * (hp % pairs) + (lane >> 4);
    x.elem = (2 * hp + (lane >> 4)) * 32 + 8 * (lane & 3);
    return x;
}

// kUnits units a warp, all loaded before any is used; the page is looked up
// meanwhile (only the stores need it).
template <int D, int TYPE, int kUnits>
__global__ void __launch_bounds__(kThreads, 4) k_kv_append(const uint8_t *__restrict__ K, long long ldk,
                                                        const uint8_t *__restrict__ V, long long ldv,
                                                        uint8_t *__restrict__ cache, Batch B)
{
    constexpr int nb = D / 32, el = type_size(TYPE);
    pdl_launch_dependents();
    pdl_wait();
    const int j = (threadIdx.x >> 2) & 3, sub = threadIdx.x & 3;
    const Group g = load_group(B, blockIdx.x);
    const int t = g.t, quad = t >> 2;
    const int u0 = (blockIdx.y * (kThreads / 32) + (threadIdx.x >> 5)) * kUnits;
    float4 v[kUnits][2];
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        const Unit u = unit_of<D>(u0 + i, B.kv_heads);
        v[i][0] = v[i][1] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (u.live && g.mine) load8<TYPE>((u.isv ? V + g.row * ldv * el : K + g.row * ldk * el) + u.elem * el, v[i][0], v[i][1]);
    }
    const long long rec0 = group_rec<D>(B, g);
    if (rec0 < 0) return;  // warp-uniform
    const bool whole = __all_sync(0xffffffffu, g.mine);
    const long long head_stride = static_cast<long long>(B.per) * rec_bytes(D);
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        const Unit u = unit_of<D>(u0 + i, B.kv_heads);
        if (!u.live) break;  // warp-uniform
        const float e[8] = {v[i][0].x, v[i][0].y, v[i][0].z, v[i][0].w, v[i][1].x, v[i][1].y, v[i][1].z, v[i][1].w};
        float amax = 0.f;  // so that a block of nothing but NaN has the scale 0
#pragma unroll
        for (int k = 0; k < 8; ++k) amax = fmaxf(amax, fabsf(e[k]));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        const __half dh = __float2half_rn(fminf(over127(amax), kMaxD));
        const uint2 codes = code_bytes8(e, __half2float(dh), amax);
        uint8_t *rec = cache + rec0 + u.h * head_stride;
        if (!u.isv) {
            if (g.mine) {
                *reinterpret_cast<uint2 *>(rec + k_code_off(t, u.b, nb) + 8 * sub) = codes;
                if (sub == 0) *reinterpret_cast<__half *>(rec + k_scale_off(t, u.b, D)) = dh;
            }
        } else {
            const int c = 8 * u.b + 2 * sub;  // this lane's 16-byte chunks of four elements: c and c + 1
            if (whole) {
                // this lane's words: elements 4 c + j and 4 c + 4 + j, the four tokens' codes
                *reinterpret_cast<uint32_t *>(rec + v_chunk_off(quad, c, D) + 4 * j) = transpose4(codes.x);
                *reinterpret_cast<uint32_t *>(rec + v_chunk_off(quad, c + 1, D) + 4 * j) = transpose4(codes.y);
            } else if (g.mine) {
                uint8_t *p = rec + v_chunk_off(quad, c, D) + (t & 3), *q = rec + v_chunk_off(quad, c + 1, D) + (t & 3);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    p[4 * k] = static_cast<uint8_t>(codes.x >> (8 * k));
                    q[4 * k] = static_cast<uint8_t>(codes.y >> (8 * k));
                }
            }
            if (g.mine && sub == 0) *reinterpret_cast<__half *>(rec + v_scale_off(t, u.b, D)) = dh;
        }
    }
}

template <int D, int TYPE, int kUnits>
__global__ void __launch_bounds__(kThreads) k_kv_read(const uint8_t *__restrict__ cache, uint8_t *__restrict__ K,
                                                      long long ldk, uint8_t *__restrict__ V, long long ldv, Batch B)
{
    constexpr int nb = D / 32, el = type_size(TYPE);
    pdl_launch_dependents();
    pdl_wait();
    const int j = (threadIdx.x >> 2) & 3, sub = threadIdx.x & 3;
    const Group g = load_group(B, blockIdx.x);
    const long long rec0 = group_rec<D>(B, g);
    const int t = g.t, quad = t >> 2;
    const int u0 = (blockIdx.y * (kThreads / 32) + (threadIdx.x >> 5)) * kUnits;
    const long long head_stride = static_cast<long long>(B.per) * rec_bytes(D);
    uint2 w[kUnits];
    __half d[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        const Unit u = unit_of<D>(u0 + i, B.kv_heads);
        w[i] = make_uint2(0x80808080u, 0x80808080u);
        d[i] = __float2half_rn(0.0f);
        if (u.live && rec0 >= 0) {
            const uint8_t *rec = cache + rec0 + u.h * head_stride;
            const int c = 8 * u.b + 2 * sub;
            if (u.isv) {
                w[i].x = __ldg(reinterpret_cast<const uint32_t *>(rec + v_chunk_off(quad, c, D) + 4 * j));
                w[i].y = __ldg(reinterpret_cast<const uint32_t *>(rec + v_chunk_off(quad, c + 1, D) + 4 * j));
            } else {
                w[i] = __ldg(reinterpret_cast<const uint2 *>(rec + k_code_off(t, u.b, nb) + 8 * sub));
            }
            d[i] = __ushort_as_half(
                __ldg(reinterpret_cast<const uint16_t *>(rec + (u.isv ? v_scale_off(t, u.b, D) : k_scale_off(t, u.b, D)))));
        }
    }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        const Unit u = unit_of<D>(u0 + i, B.kv_heads);
        if (!u.live) break;  // warp-uniform
        uint2 c = w[i];
        if (u.isv) c = make_uint2(transpose4(c.x), transpose4(c.y));
        if (!g.mine) continue;
        // codes and scales have 7 and 11 significant bits: the f32 products are exact
        const float s = __half2float(d[i]);
        const float2 a = half2_f2(codes2(c.x, 0x4140u)), b = half2_f2(codes2(c.x, 0x4342u));
        const float2 e = half2_f2(codes2(c.y, 0x4140u)), f = half2_f2(codes2(c.y, 0x4342u));
        store8<TYPE>((u.isv ? V + g.row * ldv * el : K + g.row * ldk * el) + u.elem * el,
                     make_float4(a.x * s, a.y * s, b.x * s, b.y * s), make_float4(e.x * s, e.y * s, f.x * s, f.y * s));
    }
}

// Units per warp: one where the call is small (every unit's load is issued at
// once, on as many warps as there are units), kMany where there are warps
// enough to fill the GPU anyway.  Measured with 8 heads x 128 in f32, one unit
// against four: 500 tokens (4 k units) 2.9 and 4.4 us, 1500 5.3 and 5.4, 3000
// (24 k units) 9.7 and 7.7, 12000 36.4 and 23.5 (append); 3.2 and 4.0, 4.8 and
// 5.9, 8.1 and 6.8, 26.8 and 22.0 (read).
constexpr int kMany = 4;
inline int units_per_warp(long long slots, int units)
{
    return slots * units >= 2ll * sm_count() * 64 ? kMany : 1;
}

template <int D, int TYPE>
cudaError_t append_typed(const void *K, long long ldk, const void *V, long long ldv, uint8_t *cache, const Batch &B,
                         cudaStream_t s)
{
    const long long slots = B.n_tokens / 4 + 2ll * B.n_seq;
    const int units = 2 * B.kv_heads * (D / 64), per = units_per_warp(slots, units);
    const dim3 grid(static_cast<unsigned>(slots), static_cast<unsigned>((units + 8 * per - 1) / (8 * per)));
    const uint8_t *k = static_cast<const uint8_t *>(K), *v = static_cast<const uint8_t *>(V);
    if (per == kMany) return launch_pdl(k_kv_append<D, TYPE, kMany>, grid, dim3(kThreads), 0, s, k, ldk, v, ldv, cache, B);
    return launch_pdl(k_kv_append<D, TYPE, 1>, grid, dim3(kThreads), 0, s, k, ldk, v, ldv, cache, B);
}

template <int D, int TYPE>
cudaError_t read_typed(const uint8_t *cache, void *K, long long ldk, void *V, long long ldv, const Batch &B, cudaStream_t s)
{
    const long long slots = B.n_tokens / 4 + 2ll * B.n_seq;
    const int units = 2 * B.kv_heads * (D / 64), per = units_per_warp(slots, units);
    const dim3 grid(static_cast<unsigned>(slots), static_cast<unsigned>((units + 8 * per - 1) / (8 * per)));
    uint8_t *k = static_cast<uint8_t *>(K), *v = static_cast<uint8_t *>(V);
    if (per == kMany) return launch_pdl(k_kv_read<D, TYPE, kMany>, grid, dim3(kThreads), 0, s, cache, k, ldk, v, ldv, B);
    return launch_pdl(k_kv_read<D, TYPE, 1>, grid, dim3(kThreads), 0, s, cache, k, ldk, v, ldv, B);
}

template <int D>
cudaError_t append_dim(int type, const void *K, long long ldk, const void *V, long long ldv, uint8_t *cache, const Batch &B,
                       cudaStream_t s)
{
    switch (type) {
    case GQ_TYPE_F32: return append_typed<D, GQ_TYPE_F32>(K, ldk, V, ldv, cache, B, s);
    case GQ_TYPE_F16: return append_typed<D, GQ_TYPE_F16>(K, ldk, V, ldv, cache, B, s);
    default: return append_typed<D, GQ_TYPE_BF16>(K, ldk, V, ldv, cache, B, s);
    }
}
template <int D>
cudaError_t read_dim(int type, const uint8_t *cache, void *K, long long ldk, void *V, long long ldv, const Batch &B,
                     cudaStream_t s)
{
    switch (type) {
    case GQ_TYPE_F32: return read_typed<D, GQ_TYPE_F32>(cache, K, ldk, V, ldv, B, s);
    case GQ_TYPE_F16: return read_typed<D, GQ_TYPE_F16>(cache, K, ldk, V, ldv, B, s);
    default: return read_typed<D, GQ_TYPE_BF16>(cache, K, ldk, V, ldv, B, s);
    }
}

// ---------------------------------------------------------------- checks of the C entry points
inline bool valid_dim(int D) { return D == 64 || D == 128 || D == 256; }
inline bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

inline int check_cache(int n_pages, int page_tokens, int kv_heads, int head_dim)
{
    if (n_pages < 1 || page_tokens < kRec || page_tokens % kRec != 0 || page_tokens > 4096 || kv_heads < 1 ||
        kv_heads > 65536 / head_dim)
        return GQ_ERR_SHAPE;
    return GQ_OK;
}

// A token array: n_tokens rows of `width` elements, `ld` apart.  Without rows it
// may be null, as an empty tensor's address is.
inline int check_rows(const void *p, long long ld, int width, int type, int n_tokens)
{
    if (!p && n_tokens > 0) return GQ_ERR_NULL;
    if (!aligned16(p)) return GQ_ERR_ALIGN;
    if (ld < width) return GQ_ERR_SHAPE;
    return ld * type_size(type) % 16 == 0 ? GQ_OK : GQ_ERR_ALIGN;
}

inline int check_batch(const void *cache, const int32_t *block_table, const int32_t *kv_len, const int32_t *q_start,
                       int type, int n_pages, int max_pages, int page_tokens, int kv_heads, int head_dim, int n_seq,
                       int n_tokens)
{
    if (type != GQ_TYPE_F32 && type != GQ_TYPE_F16 && type != GQ_TYPE_BF16) return GQ_ERR_FORMAT;
    if (!cache || !block_table || !kv_len || !q_start) return GQ_ERR_NULL;
    if (!aligned16(cache) || !aligned4(block_table) || !aligned4(kv_len) || !aligned4(q_start)) return GQ_ERR_ALIGN;
    if (!valid_dim(head_dim) || check_cache(n_pages, page_tokens, kv_heads, head_dim) != GQ_OK) return GQ_ERR_SHAPE;
    // positions and rows are 32-bit numbers in the kernels
    if (max_pages < 1 || static_cast<long long>(max_pages) * page_tokens > (1 << 28) || n_seq < 1 || n_seq > (1 << 24) ||
        n_tokens < 0 || n_tokens > (1 << 28))
        return GQ_ERR_SHAPE;
    return GQ_OK;
}

}  // namespace kv
}  // namespace gq

using namespace gq;
using namespace gq::kv;

extern "C" {

size_t gq_kv_cache_bytes(int n_pages, int page_tokens, int kv_heads, int head_dim)
{
    if (!valid_dim(head_dim) || check_cache(n_pages, page_tokens, kv_heads, head_dim) != GQ_OK) return 0;
    return static_cast<size_t>(n_pages) * kv_heads * (page_tokens / kRec) * rec_bytes(head_dim);
}

int gq_kv_append_q8_0(const void *K, long long ldk, const void *V, long long ldv, int type, void *cache,
                      const int32_t *block_table, const int32_t *kv_len, const int32_t *q_start, int n_pages,
                      int max_pages, int page_tokens, int kv_heads, int head_dim, int n_seq, int n_tokens,
                      gq_stream_t stream)
{
    int st = check_batch(cache, block_table, kv_len, q_start, type, n_pages, max_pages, page_tokens, kv_heads, head_dim,
                         n_seq, n_tokens);
    if (st == GQ_OK) st = check_rows(K, ldk, kv_heads * head_dim, type, n_tokens);
    if (st == GQ_OK) st = check_rows(V, ldv, kv_heads * head_dim, type, n_tokens);
    if (st != GQ_OK) return st;
    if (n_tokens == 0) return GQ_OK;
    const Batch B = make_batch(block_table, kv_len, q_start, n_pages, max_pages, page_tokens, kv_heads, n_seq, n_tokens,
                               status_word());
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    uint8_t *c = static_cast<uint8_t *>(cache);
    switch (head_dim) {
    case 64: return status_from(append_dim<64>(type, K, ldk, V, ldv, c, B, s));
    case 128: return status_from(append_dim<128>(type, K, ldk, V, ldv, c, B, s));
    default: return status_from(append_dim<256>(type, K, ldk, V, ldv, c, B, s));
    }
}

int gq_kv_read_q8_0(const void *cache, const int32_t *block_table, const int32_t *kv_len, const int32_t *q_start,
                    void *K, long long ldk, void *V, long long ldv, int type, int n_pages, int max_pages,
                    int page_tokens, int kv_heads, int head_dim, int n_seq, int n_tokens, gq_stream_t stream)
{
    int st = check_batch(cache, block_table, kv_len, q_start, type, n_pages, max_pages, page_tokens, kv_heads, head_dim,
                         n_seq, n_tokens);
    if (st == GQ_OK) st = check_rows(K, ldk, kv_heads * head_dim, type, n_tokens);
    if (st == GQ_OK) st = check_rows(V, ldv, kv_heads * head_dim, type, n_tokens);
    if (st != GQ_OK) return st;
    if (n_tokens == 0) return GQ_OK;
    const Batch B = make_batch(block_table, kv_len, q_start, n_pages, max_pages, page_tokens, kv_heads, n_seq, n_tokens,
                               status_word());
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const uint8_t *c = static_cast<const uint8_t *>(cache);
    switch (head_dim) {
    case 64: return status_from(read_dim<64>(type, c, K, ldk, V, ldv, B, s));
    case 128: return status_from(read_dim<128>(type, c, K, ldk, V, ldv, B, s));
    default: return status_from(read_dim<256>(type, c, K, ldk, V, ldv, B, s));
    }
}

size_t gq_kv_attention_workspace_bytes(int heads, int kv_heads, int head_dim)
{
    if (!valid_dim(head_dim) || kv_heads < 1 || heads < kv_heads || heads % kv_heads != 0 || heads > 65536 / head_dim)
        return 0;
    return kv_attention_workspace_bytes(head_dim);
}

int gq_kv_attention_q8_0(const void *Q, long long ldq, const void *cache, const int32_t *block_table,
                         const int32_t *kv_len, const int32_t *q_start, void *O, long long ldo, int type, float scale,
                         float softcap, int window, void *workspace, size_t workspace_bytes, int heads, int n_pages,
                         int max_pages, int page_tokens, int kv_heads, int head_dim, int n_seq, int n_tokens,
                         gq_stream_t stream)
{
    int st = check_batch(cache, block_table, kv_len, q_start, type, n_pages, max_pages, page_tokens, kv_heads, head_dim,
                         n_seq, n_tokens);
    if (st != GQ_OK) return st;
    const size_t need = gq_kv_attention_workspace_bytes(heads, kv_heads, head_dim);
    if (need == 0 || window < 0 || !isfinite(scale) || !isfinite(softcap)) return GQ_ERR_SHAPE;
    st = check_rows(Q, ldq, heads * head_dim, type, n_tokens);
    if (st == GQ_OK) st = check_rows(O, ldo, heads * head_dim, type, n_tokens);
    if (st != GQ_OK) return st;
    if (!workspace || workspace_bytes < need) return GQ_ERR_WORKSPACE;
    if (!aligned16(workspace)) return GQ_ERR_ALIGN;
    if (n_tokens == 0) return GQ_OK;
    // A row's window begins at position - window + 1, a 32-bit number in the
    // kernels, and a row may lie up to 2^28 positions before 0: windows beyond
    // every position are all the same.
    if (window > kMaxWindow) window = kMaxWindow;
    const Batch B = make_batch(block_table, kv_len, q_start, n_pages, max_pages, page_tokens, kv_heads, n_seq, n_tokens,
                               status_word());
    return launch_kv_attention(Q, ldq, static_cast<const uint8_t *>(cache), B, O, ldo, type, scale, softcap, window,
                               workspace, heads, head_dim, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
