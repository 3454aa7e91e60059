// gq_kv.cuh -- the paged Q8_0 key/value cache: its record layout, the batch
// description that the kernels take, and the code conversions they share.
// The layout and the batch are specified in include/gq_kv.h.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <float.h>

#include "gq_host.h"
#include "gq_internal.cuh"
#include "gq_kv.h"

namespace gq {
namespace kv {

constexpr int kRec = 16;          // tokens per record
constexpr int kMaxWindow = 1 << 30;
constexpr float kMaxD = 515.5f;   // largest block scale: 127 * 515.5 = 65468.5 is finite in fp16

// The batch and the cache as the kernels see them.
struct Batch {
    const int32_t *table, *kv_len, *q_start;
    int n_pages, max_pages, page_tokens, kv_heads, n_seq, n_tokens;
    int *status;             // device status word
    uint32_t per, per_mul;   // records per page, and 2^32 / per rounded up
};
inline Batch make_batch(const int32_t *table, const int32_t *kv_len, const int32_t *q_start, int n_pages, int max_pages,
                        int page_tokens, int kv_heads, int n_seq, int n_tokens, int *status)
{
    const uint32_t per = static_cast<uint32_t>(page_tokens / kRec);
    return Batch{table, kv_len, q_start, n_pages, max_pages, page_tokens, kv_heads, n_seq, n_tokens, status, per,
                 static_cast<uint32_t>(((1ull << 32) + per - 1) / per)};
}

__host__ __device__ __forceinline__ constexpr int rec_bytes(int D) { return 34 * D; }
// Byte offset of block b of token t's key codes in a record, of token t's key
// scale, of a value word's 16-byte chunk c of token group g, and of a value
// scale.
__host__ __device__ __forceinline__ constexpr int k_key(int t, int nb)
{
    return nb > 2 ? ((t & 1) | ((t >> 1) & 2)) : ((t >> 2) & 1);
}
__host__ __device__ __forceinline__ constexpr int k_code_off(int t, int b, int nb)
{
    return 32 * (t * nb + (b ^ k_key(t, nb)));
}
__host__ __device__ __forceinline__ constexpr int k_scale_off(int t, int b, int D) { return 16 * D + 2 * (t * (D / 32) + b); }
__host__ __device__ __forceinline__ constexpr int v_chunk_off(int g, int c, int D) { return 17 * D + 4 * D * g + 16 * (c ^ (2 * g)); }
__host__ __device__ __forceinline__ constexpr int v_scale_off(int t, int b, int D) { return 33 * D + 2 * (b * 16 + t); }

__device__ __forceinline__ void flag_shape(const Batch &B)
{
    if (B.status) atomicExch(B.status, GQ_ERR_SHAPE);
}

// One sequence of the batch: what the lists say, brought into bounds.  Rows and
// cached tokens outside are cut off; the rows that stay keep the positions that
// the lists give them (some of these below 0 or at kv and beyond if the lists
// disagree with each other or with the sizes).
struct Seq {
    int row0;   // first token row
    int n;      // new tokens (rows)
    int kv;     // cached tokens
    int first;  // position of row0
};
constexpr int kFar = 1 << 30;  // beyond every position, and far from overflow
__device__ __forceinline__ Seq seq_of(const Batch &B, int r0, int r1, int kv)
{
    Seq s;
    s.row0 = min(max(r0, 0), B.n_tokens);
    const int r1c = min(max(r1, s.row0), B.n_tokens);
    s.n = r1c - s.row0;
    const long long room = static_cast<long long>(B.max_pages) * B.page_tokens;
    s.kv = kv < 0 ? 0 : (kv > room ? static_cast<int>(room) : kv);
    const long long first = static_cast<long long>(kv) - r1 + s.row0;
    s.first = static_cast<int>(first < -kFar ? -kFar : (first > kFar ? kFar : first));
    if (s.row0 != r0 || r1c != r1 || s.kv != kv) flag_shape(B);
    return s;
}
__device__ __forceinline__ Seq load_seq(const Batch &B, int b)
{
    const int r0 = __ldg(B.q_start + b), r1 = __ldg(B.q_start + b + 1), kv = __ldg(B.kv_len + b);
    return seq_of(B, r0, r1, kv);
}

// Entry of a sequence's table that holds record `rec` (16 tokens), by a
// product: exact for rec * per < 2^32, which the checked range (2^28 tokens,
// 256 records a page) keeps.
__device__ __forceinline__ int page_entry(const Batch &B, int rec)
{
    return B.per == 1 ? rec : static_cast<int>(__umulhi(static_cast<uint32_t>(rec), B.per_mul));
}
__device__ __forceinline__ const int32_t *page_at(const Batch &B, int b, int rec)
{
    return B.table + static_cast<long long>(b) * B.max_pages + page_entry(B, rec);
}
// A table entry, or -1 (flagged) if it names no page.
__device__ __forceinline__ int checked_page(const Batch &B, int pg)
{
    if (static_cast<unsigned>(pg) < static_cast<unsigned>(B.n_pages)) return pg;
    flag_shape(B);
    return -1;
}
__device__ __forceinline__ int page_of(const Batch &B, int b, int rec) { return checked_page(B, __ldg(page_at(B, b, rec))); }

// Byte offset of head h's record `rec` of the sequence in page pg.
__device__ __forceinline__ long long rec_off(const Batch &B, int pg, int h, int rec, int D)
{
    return ((static_cast<long long>(pg) * B.kv_heads + h) * B.per + (rec - page_entry(B, rec) * static_cast<int>(B.per))) * rec_bytes(D);
}

// ---------------------------------------------------------------- element types
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ float2 half2_f2(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2 *>(&w)); }
__device__ __forceinline__ uint32_t f2_half2(float a, float b)
{
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t f2_bf162(float a, float b)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
// Four consecutive elements at p (16-byte aligned for f32, 8-byte for the 16-bit types).
template <int TYPE>
__device__ __forceinline__ float4 load4(const void *p)
{
    if (TYPE == GQ_TYPE_F32) return __ldg(static_cast<const float4 *>(p));
    const uint2 w = __ldg(static_cast<const uint2 *>(p));
    if (TYPE == GQ_TYPE_BF16) return make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
    const float2 a = half2_f2(w.x), b = half2_f2(w.y);
    return make_float4(a.x, a.y, b.x, b.y);
}
template <int TYPE>
__device__ __forceinline__ void store4(void *p, float4 v)
{
    if (TYPE == GQ_TYPE_F32) {
        *static_cast<float4 *>(p) = v;
    } else if (TYPE == GQ_TYPE_BF16) {
        *static_cast<uint2 *>(p) = make_uint2(f2_bf162(v.x, v.y), f2_bf162(v.z, v.w));
    } else {
        *static_cast<uint2 *>(p) = make_uint2(f2_half2(v.x, v.y), f2_half2(v.z, v.w));
    }
}
// Eight consecutive elements at p (16-byte aligned).
template <int TYPE>
__device__ __forceinline__ void load8(const void *p, float4 &a, float4 &b)
{
    if (TYPE == GQ_TYPE_F32) {
        a = __ldg(static_cast<const float4 *>(p));
        b = __ldg(static_cast<const float4 *>(p) + 1);
        return;
    }
    const uint4 w = __ldg(static_cast<const uint4 *>(p));
    if (TYPE == GQ_TYPE_BF16) {
        a = make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
        b = make_float4(bf16_lo(w.z), bf16_hi(w.z), bf16_lo(w.w), bf16_hi(w.w));
    } else {
        const float2 x = half2_f2(w.x), y = half2_f2(w.y), z = half2_f2(w.z), u = half2_f2(w.w);
        a = make_float4(x.x, x.y, y.x, y.y);
        b = make_float4(z.x, z.y, u.x, u.y);
    }
}
template <int TYPE>
__device__ __forceinline__ void store8(void *p, float4 a, float4 b)
{
    if (TYPE == GQ_TYPE_F32) {
        static_cast<float4 *>(p)[0] = a;
        static_cast<float4 *>(p)[1] = b;
    } else if (TYPE == GQ_TYPE_BF16) {
        *static_cast<uint4 *>(p) = make_uint4(f2_bf162(a.x, a.y), f2_bf162(a.z, a.w), f2_bf162(b.x, b.y), f2_bf162(b.z, b.w));
    } else {
        *static_cast<uint4 *>(p) = make_uint4(f2_half2(a.x, a.y), f2_half2(a.z, a.w), f2_half2(b.x, b.y), f2_half2(b.z, b.w));
    }
}
__host__ __device__ __forceinline__ constexpr int type_size(int type) { return type == GQ_TYPE_F32 ? 4 : 2; }

// Code bytes 0, 1 (sel 0x4140) or 2, 3 (sel 0x4342) of w -> f16x2, exact: a
// byte u placed under the exponent of 1024 is 1024 + u, and the code is
// u - 128.
__device__ __forceinline__ uint32_t codes2(uint32_t w, uint32_t sel)
{
    const uint32_t m = __byte_perm(w, 0x64646464u, sel);
    const __half2 r = __hsub2(*reinterpret_cast<const __half2 *>(&m), __float2half2_rn(1152.0f));
    return *reinterpret_cast<const uint32_t *>(&r);
}

// ---------------------------------------------------------------- what the attention kernels share
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 1 / cap, finite also for a subnormal cap (0 times an infinity would be NaN)
__device__ __forceinline__ float inverse_cap(float cap) { return fminf(1.0f / cap, FLT_MAX); }
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

}  // namespace kv

// gq_kv_attn.cu
int launch_kv_attention(const void *Q, long long ldq, const uint8_t *cache, const kv::Batch &B, void *O, long long ldo,
                        int type, float scale, float softcap, int window, void *ws, int heads, int head_dim,
                        cudaStream_t s);
size_t kv_attention_workspace_bytes(int head_dim);
// gq_kv_chunk.cu: the tensor-core form for many query rows (16-bit types);
// `counter` and `part` are its parts of the workspace.
size_t kv_chunk_part_bytes(int head_dim);
int kv_chunk_counters();
int launch_kv_chunk(const void *Q, long long ldq, const uint8_t *cache, const kv::Batch &B, void *O, long long ldo, int type,
                    float scale, float softcap, int window, int *counter, float *part, int heads, int head_dim, cudaStream_t s);

}  // namespace gq
