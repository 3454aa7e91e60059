// gq_kv.cu -- writing and reading the paged Q8_0 key/value cache, and the C
// entry points of include/gq_kv.h.
//
// One warp handles one unit: a group of four tokens (one word of the value
// layout) of one 32-block of one kv head's keys or values.  Lane 8 j + s
// holds elements 4 s .. 4 s + 3 of token j, as in the activation quantizer.
// The keys' codes are stored as they are (32 bytes per token and block); the
// values' 4 x 4 byte squares are transposed between lanes j with two
// shuffles, so a lane writes the word of one element with the four tokens'
// codes.  A group that is only partly new (the ends of a chunk, every decode
// step) writes the new tokens' bytes alone.
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
// takes part).
__device__ __forceinline__ int find_seq(const Batch &B, long long slot)
{
    const int lane = threadIdx.x & 31;
    int lo = 0, n = B.n_seq;  // the answer lies in [lo, lo + n)
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int b = lo + lane * step;
        const bool at = b < lo + n && (__ldg(B.q_start + b) >> 2) + 2ll * b <= slot;
        // the starts rise with b: the lanes that hold are a prefix
        const int k = max(__popc(__ballot_sync(0xffffffffu, at)) - 1, 0);
        n = min(step, n - k * step);
        lo += k * step;
    }
    return lo;
}

// 4 x 4 byte transpose between the lanes j = lane / 8 that share lane % 8.
__device__ __forceinline__ uint32_t transpose4(uint32_t x)
{
    const int j = (threadIdx.x >> 3) & 3;
    uint32_t r = __shfl_xor_sync(0xffffffffu, x, 8);
    x = __byte_perm(x, r, (j & 1) ? 0x3715u : 0x6240u);
    r = __shfl_xor_sync(0xffffffffu, x, 16);
    return __byte_perm(x, r, (j & 2) ? 0x3276u : 0x5410u);
}

// What a warp's units have in common: the group of four tokens.  Groups are
// aligned in position, so one lies in one record, and wholly below position 0
// or wholly above (rows below it exist only where the lists disagree).
struct Group {
    long long row;  // this lane's token's row
    int t;          // its place in the record
    bool mine;      // it is a new token
    bool whole;     // all four are (warp-uniform)
    long long rec;  // record offset of kv head 0, -1 if there is none (warp-uniform)
};
template <int D>
__device__ __forceinline__ Group load_group(const Batch &B, long long slot)
{
    Group g;
    const int b = find_seq(B, slot);
    const Seq s = load_seq(B, b);
    const long long local = slot - ((static_cast<long long>(s.row0) >> 2) + 2ll * b);
    const long long p0 = 4ll * ((s.first >> 2) + local), pos = p0 + ((threadIdx.x >> 3) & 3);
    g.mine = pos >= s.first && pos < s.kv;
    g.row = s.row0 + (pos - s.first);
    g.t = static_cast<int>(pos) & (kRec - 1);
    g.whole = __all_sync(0xffffffffu, g.mine);
    g.rec = -1;
    if (__any_sync(0xffffffffu, g.mine)) {
        if (p0 < 0) {
            flag_shape(B);
        } else {
            const int pg = page_of(B, b, static_cast<int>(p0));
            if (pg >= 0) g.rec = rec_off(B, pg, 0, static_cast<int>(p0), D);
        }
    }
    return g;
}

// kUnits units a warp, all loaded before any is used.
template <int D, int TYPE, int kUnits>
__global__ void __launch_bounds__(kThreads) k_kv_append(const uint8_t *__restrict__ K, long long ldk,
                                                        const uint8_t *__restrict__ V, long long ldv,
                                                        uint8_t *__restrict__ cache, Batch B)
{
    constexpr int nb = D / 32, el = type_size(TYPE);
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, j = lane >> 3, sub = lane & 7;
    const Group g = load_group<D>(B, blockIdx.x);
    if (g.rec < 0) return;  // warp-uniform
    const long long row = g.row;
    const int t = g.t, quad = t >> 2;
    const int units = 2 * B.kv_heads * nb;
    const int u0 = (blockIdx.y * (kThreads / 32) + (threadIdx.x >> 5)) * kUnits;
    const long long head_stride = static_cast<long long>(B.page_tokens / kRec) * rec_bytes(D);
    float4 v[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        const int u = u0 + i;
        v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (u < units && g.mine) {
            const bool isv = u >= units / 2;
            const int hb = isv ? u - units / 2 : u;  // head * nb + block: 32 hb is the element's place in the row
            v[i] = load4<TYPE>((isv ? V + row * ldv * el : K + row * ldk * el) + (hb * 32 + sub * 4) * el);
        }
    }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        const int u = u0 + i;
        if (u >= units) break;  // warp-uniform
        const bool isv = u >= units / 2;
        const int hb = isv ? u - units / 2 : u;
        const int h = hb / nb, b = hb % nb;
        // from 0, so that a block of nothing but NaN has the scale 0
        float amax = fmaxf(fmaxf(fmaxf(0.f, fabsf(v[i].x)), fabsf(v[i].y)), fmaxf(fabsf(v[i].z), fabsf(v[i].w)));
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        const __half dh = __float2half_rn(fminf(__fmul_rn(amax, 1.0f / 127.0f), kMaxD));
        const float e[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
        const uint32_t codes = q8_pack4(e, __half2float(dh)) ^ 0x80808080u;
        uint8_t *rec = cache + g.rec + h * head_stride;
        if (!isv) {
            if (g.mine) {
                *reinterpret_cast<uint32_t *>(rec + k_code_off(t, b, nb) + 4 * sub) = codes;
                if (sub == 0) *reinterpret_cast<__half *>(rec + k_scale_off(t, b, D)) = dh;
            }
        } else {
            if (g.whole) {
                // this lane's word: element 4 sub + j of the block, the four tokens' codes
                *reinterpret_cast<uint32_t *>(rec + v_chunk_off(quad, 8 * b + sub, D) + 4 * j) = transpose4(codes);
            } else if (g.mine) {
                uint8_t *p = rec + v_chunk_off(quad, 8 * b + sub, D) + (t & 3);
#pragma unroll
                for (int k = 0; k < 4; ++k) p[4 * k] = static_cast<uint8_t>(codes >> (8 * k));
            }
            if (g.mine && sub == 0) *reinterpret_cast<__half *>(rec + v_scale_off(t, b, D)) = dh;
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
    const int lane = threadIdx.x & 31, j = lane >> 3, sub = lane & 7;
    const Group g = load_group<D>(B, blockIdx.x);
    const long long row = g.row;
    const int t = g.t, quad = t >> 2;
    const int units = 2 * B.kv_heads * nb;
    const int u0 = (blockIdx.y * (kThreads / 32) + (threadIdx.x >> 5)) * kUnits;
    const long long head_stride = static_cast<long long>(B.page_tokens / kRec) * rec_bytes(D);
    uint32_t w[kUnits];
    __half d[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        const int u = u0 + i;
        w[i] = 0x80808080u;
        d[i] = __float2half_rn(0.0f);
        if (u < units && g.rec >= 0) {
            const bool isv = u >= units / 2;
            const int hb = isv ? u - units / 2 : u;
            const int h = hb / nb, b = hb % nb;
            const uint8_t *rec = cache + g.rec + h * head_stride;
            w[i] = __ldg(reinterpret_cast<const uint32_t *>(
                rec + (isv ? v_chunk_off(quad, 8 * b + sub, D) + 4 * j : k_code_off(t, b, nb) + 4 * sub)));
            d[i] = __ushort_as_half(__ldg(reinterpret_cast<const uint16_t *>(rec + (isv ? v_scale_off(t, b, D) : k_scale_off(t, b, D)))));
        }
    }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        const int u = u0 + i;
        if (u >= units) break;  // warp-uniform
        const bool isv = u >= units / 2;
        const int hb = isv ? u - units / 2 : u;
        uint32_t c = w[i];
        if (isv) c = transpose4(c);
        if (!g.mine) continue;
        const float s = __half2float(d[i]);
        const float2 a = half2_f2(codes2(c, 0x4140u)), z = half2_f2(codes2(c, 0x4342u));
        // codes and scales have 7 and 11 significant bits: the f32 products are exact
        store4<TYPE>((isv ? V + row * ldv * el : K + row * ldk * el) + (hb * 32 + sub * 4) * el,
                     make_float4(a.x * s, a.y * s, z.x * s, z.y * s));
    }
}

// Units per warp: one where the call is small (a decode step: every unit's
// load is issued at once, on as many warps as there are units), four where
// there are enough warps to fill the GPU anyway.
inline int units_per_warp(long long slots, int units)
{
    return slots * units >= 4ll * sm_count() * 64 ? 4 : 1;
}

template <int D, int TYPE>
cudaError_t append_typed(const void *K, long long ldk, const void *V, long long ldv, uint8_t *cache, const Batch &B,
                         cudaStream_t s)
{
    const long long slots = B.n_tokens / 4 + 2ll * B.n_seq;
    const int units = 2 * B.kv_heads * (D / 32), per = units_per_warp(slots, units);
    const dim3 grid(static_cast<unsigned>(slots), static_cast<unsigned>((units + 8 * per - 1) / (8 * per)));
    const uint8_t *k = static_cast<const uint8_t *>(K), *v = static_cast<const uint8_t *>(V);
    if (per == 4) return launch_pdl(k_kv_append<D, TYPE, 4>, grid, dim3(kThreads), 0, s, k, ldk, v, ldv, cache, B);
    return launch_pdl(k_kv_append<D, TYPE, 1>, grid, dim3(kThreads), 0, s, k, ldk, v, ldv, cache, B);
}

template <int D, int TYPE>
cudaError_t read_typed(const uint8_t *cache, void *K, long long ldk, void *V, long long ldv, const Batch &B, cudaStream_t s)
{
    const long long slots = B.n_tokens / 4 + 2ll * B.n_seq;
    const int units = 2 * B.kv_heads * (D / 32), per = units_per_warp(slots, units);
    const dim3 grid(static_cast<unsigned>(slots), static_cast<unsigned>((units + 8 * per - 1) / (8 * per)));
    uint8_t *k = static_cast<uint8_t *>(K), *v = static_cast<uint8_t *>(V);
    if (per == 4) return launch_pdl(k_kv_read<D, TYPE, 4>, grid, dim3(kThreads), 0, s, cache, k, ldk, v, ldv, B);
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

// A token array: rows of `width` elements, `ld` apart.
inline int check_rows(const void *p, long long ld, int width, int type)
{
    if (!p) return GQ_ERR_NULL;
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
    if (max_pages < 1 || static_cast<long long>(max_pages) * page_tokens > (1 << 30) || n_seq < 1 || n_seq > (1 << 24) ||
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
    if (st == GQ_OK) st = check_rows(K, ldk, kv_heads * head_dim, type);
    if (st == GQ_OK) st = check_rows(V, ldv, kv_heads * head_dim, type);
    if (st != GQ_OK) return st;
    if (n_tokens == 0) return GQ_OK;
    const Batch B = {block_table, kv_len, q_start, n_pages, max_pages, page_tokens, kv_heads, n_seq, n_tokens, status_word()};
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
    if (st == GQ_OK) st = check_rows(K, ldk, kv_heads * head_dim, type);
    if (st == GQ_OK) st = check_rows(V, ldv, kv_heads * head_dim, type);
    if (st != GQ_OK) return st;
    if (n_tokens == 0) return GQ_OK;
    const Batch B = {block_table, kv_len, q_start, n_pages, max_pages, page_tokens, kv_heads, n_seq, n_tokens, status_word()};
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
    st = check_rows(Q, ldq, heads * head_dim, type);
    if (st == GQ_OK) st = check_rows(O, ldo, heads * head_dim, type);
    if (st != GQ_OK) return st;
    if (!workspace || workspace_bytes < need) return GQ_ERR_WORKSPACE;
    if (!aligned16(workspace)) return GQ_ERR_ALIGN;
    if (n_tokens == 0) return GQ_OK;
    const Batch B = {block_table, kv_len, q_start, n_pages, max_pages, page_tokens, kv_heads, n_seq, n_tokens, status_word()};
    return launch_kv_attention(Q, ldq, static_cast<const uint8_t *>(cache), B, O, ldo, type, scale, softcap, window,
                               workspace, heads, head_dim, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
