// gq_embed.cu -- rows of a packed table by token id (include/gq_embed.h).
//
// A warp takes a token's row, or a part of it where there are fewer tokens than
// warps: 256 consecutive weights at a time, eight per lane.  A lane's codes are
// one load of 4 or 8 bytes, its scales one or two short ones that its neighbours
// share, its result one or two 16-byte stores; two such pieces are loaded before
// the first is stored.
//
// What bounds it: issue (70 %; 13.6 instructions a weight, as every lane unpacks its
// sub-block's scale and minimum anew for eight weights) beside the writes.  8192 rows of 5376 from a Q4_K
// table to bf16 (24 MB read, 88 MB written) take 23.7 us, 4.7 TB/s; one row 1.5.
#include <math.h>

#include "gq_embed.h"
#include "gq_host.h"
#include "gq_internal.cuh"
#include "gq_kv.cuh"

namespace gq {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float half_f(uint16_t h) { return __half2float(__ushort_as_half(h)); }

// A whole number below 2^23, less `off`, as f32: put under the exponent of 2^23 it
// needs no conversion.
__device__ __forceinline__ float whole(uint32_t q, float off = 0.f) { return __uint_as_float(0x4B000000u | q) - (8388608.0f + off); }

// Where row r's parts lie: codes, (Q6_K) top bits and sub-scales, scales or records.
struct Row {
    const uint8_t *codes, *top, *sub, *scales;
};
template <int FORMAT>
__device__ __forceinline__ Row row_at(const uint8_t *W, long long rows, int K, long long r)
{
    const long long nb = K / 32, ns = K / 256;
    if (FORMAT == GQ_FORMAT_Q8_0) return {W + r * nb * 32, nullptr, nullptr, W + rows * nb * 32 + r * nb * 2};
    if (FORMAT == GQ_FORMAT_Q4_0) return {W + r * nb * 16, nullptr, nullptr, W + rows * nb * 16 + r * nb * 2};
    if (FORMAT == GQ_FORMAT_Q4_K) return {W + r * ns * 128, nullptr, nullptr, W + (rows * 128 + r * 16) * ns};
    return {W + r * ns * 128, W + (rows * 128 + r * 64) * ns, W + (rows * 192 + r * 16) * ns, W + (rows * 208 + r * 2) * ns};
}

// What eight weights are made of, as it is loaded; and the weights e0 .. e0 + 7 (e0 a multiple of 8) from it.
struct Raw {
    uint4 rec;
    uint32_t c0, c1;
};
template <int FORMAT>
__device__ __forceinline__ void load8(const Row &r, int e0, Raw &x)
{
    auto u16 = [&](const uint8_t *p, int i) { return static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t *>(p) + i)); };
    if (FORMAT == GQ_FORMAT_Q8_0) {
        const uint2 c = __ldg(reinterpret_cast<const uint2 *>(r.codes + e0));
        x.c0 = c.x, x.c1 = c.y;
        x.rec.x = u16(r.scales, e0 / 32);
        return;
    }
    x.c0 = __ldg(reinterpret_cast<const uint32_t *>(r.codes + e0 / 2));
    if (FORMAT == GQ_FORMAT_Q4_0) {
        x.rec.x = u16(r.scales, e0 / 32);
    } else if (FORMAT == GQ_FORMAT_Q4_K) {
        x.rec = __ldg(reinterpret_cast<const uint4 *>(r.scales) + e0 / 256);
    } else {
        x.c1 = __ldg(reinterpret_cast<const uint32_t *>(r.top) + e0 / 16);
        x.rec.x = u16(r.scales, e0 / 256);
        x.rec.y = __ldg(r.sub + e0 / 16);
    }
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// Nibbles i and i + 4 of c as f32, less `off`: masked in place they are units under the exponent of 2^(23 - 4 i).
template <int I>
__device__ __forceinline__ float2 nibbles(uint32_t c, float off)
{
    constexpr uint32_t kOne = 0x4B000000u - 0x02000000u * I;  // bits of 2^(23 - 4 I)
    const uint32_t lo = (c & 15u << (4 * I)) | kOne, hi = (c >> 16 & 15u << (4 * I)) | kOne;
    return __fadd2_rn(make_float2(__uint_as_float(lo), __uint_as_float(hi)), both(-(static_cast<float>(1 << (23 - 4 * I)) + off)));
}
template <int FORMAT>
__device__ __forceinline__ void decode8(const Raw &x, int e0, float scale, float (&y)[8])
{
    float2 p[4];  // weights i and i + 4
    if (FORMAT == GQ_FORMAT_Q8_0) {
        const float2 d = both(half_f(static_cast<uint16_t>(x.rec.x)));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 q = make_float2(__uint_as_float(__byte_perm(x.c0, 0x4B000000u, 0x7440 | i)),
                                         __uint_as_float(__byte_perm(x.c1, 0x4B000000u, 0x7440 | i)));
            p[i] = __fmul2_rn(__fadd2_rn(q, both(-8388736.0f)), d);
        }
    } else if (FORMAT == GQ_FORMAT_Q4_0) {
        const float2 d = both(half_f(static_cast<uint16_t>(x.rec.x)));
        p[0] = __fmul2_rn(nibbles<0>(x.c0, 8.f), d);
        p[1] = __fmul2_rn(nibbles<1>(x.c0, 8.f), d);
        p[2] = __fmul2_rn(nibbles<2>(x.c0, 8.f), d);
        p[3] = __fmul2_rn(nibbles<3>(x.c0, 8.f), d);
    } else if (FORMAT == GQ_FORMAT_Q4_K) {
        const float d = half_f(static_cast<uint16_t>(x.rec.x)), dmin = half_f(static_cast<uint16_t>(x.rec.x >> 16));
        // bytes 0-3: scales 0-3 in 6 bits, 4-7: minima 0-3, 8-11: the low four bits of both of 4-7, whose top two
        // bits are those of the first eight bytes
        const int s = (e0 & 255) / 32, sh = 8 * (s & 3);
        const uint32_t lo = x.rec.y >> sh, mi = x.rec.z >> sh, hi = x.rec.w >> sh;
        const uint32_t sc = s < 4 ? lo & 63u : (hi & 15u) | (lo >> 2 & 48u);
        const uint32_t mn = s < 4 ? mi & 63u : (hi >> 4 & 15u) | (mi >> 2 & 48u);
        const float2 dsc = both(d * whole(sc)), m = both(-dmin * whole(mn));
        p[0] = __ffma2_rn(nibbles<0>(x.c0, 0.f), dsc, m);
        p[1] = __ffma2_rn(nibbles<1>(x.c0, 0.f), dsc, m);
        p[2] = __ffma2_rn(nibbles<2>(x.c0, 0.f), dsc, m);
        p[3] = __ffma2_rn(nibbles<3>(x.c0, 0.f), dsc, m);
    } else {
        const float2 d = both(half_f(static_cast<uint16_t>(x.rec.x)) * static_cast<float>(static_cast<int8_t>(x.rec.y)));
        const uint32_t t = x.c1 >> ((e0 & 8) ? 16 : 0);  // elements 4 a + i of the word, a = 0, 1 or 2, 3
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            auto q = [&](int e, int at) { return whole((x.c0 >> (4 * e) & 15u) | (t >> at & 3u) << 4, 32.f); };
            p[i] = __fmul2_rn(make_float2(q(i, 4 * i), q(i + 4, 4 * i + 2)), d);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = __fmul2_rn(p[i], both(scale));
        y[i] = v.x;
        y[i + 4] = v.y;
    }
}

template <int FORMAT, int TYPE>
__global__ void __launch_bounds__(kThreads, 8)
    k_embed(const uint8_t *__restrict__ W, const int32_t *__restrict__ ids, float scale, uint8_t *__restrict__ Y,
            long long row_bytes, int rows, int K, int M, int parts, int part_elems, int *status)
{
    constexpr int kBatch = 2;
    const int lane = threadIdx.x & 31;
    const unsigned warp = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int t = static_cast<int>(warp / static_cast<unsigned>(parts)), part = static_cast<int>(warp - t * static_cast<unsigned>(parts));
    pdl_launch_dependents();
    pdl_wait();
    if (t >= M) return;
    const int id = __ldg(ids + t);
    const int end = min(K, (part + 1) * part_elems);
    const bool have = id >= 0 && id < rows;
    if (id >= rows && part == 0 && lane == 0 && status) atomicExch(status, GQ_ERR_SHAPE);
    const Row r = row_at<FORMAT>(W, rows, K, have ? id : 0);
    uint8_t *y = Y + t * row_bytes;
    for (int e0 = part * part_elems + 8 * lane; e0 < end; e0 += kBatch * 256) {
        Raw w[kBatch];
        if (have) {
#pragma unroll
            for (int q = 0; q < kBatch; ++q)
                if (e0 + 256 * q < end) load8<FORMAT>(r, e0 + 256 * q, w[q]);
        }
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
            if (e0 + 256 * q >= end) continue;
            float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (have) decode8<FORMAT>(w[q], e0, scale, x);
            kv::store8<TYPE>(y + static_cast<long long>(e0 + 256 * q) * kv::type_size(TYPE),
                             make_float4(x[0], x[1], x[2], x[3]), make_float4(x[4], x[5], x[6], x[7]));
        }
    }
}

template <int FORMAT>
cudaError_t launch(const uint8_t *W, const int32_t *ids, float scale, void *Y, long long ldy, int type, int rows, int K,
                   int M, cudaStream_t s)
{
    // three times the warps that the SMs hold, so that the last ones to finish are a small part
    const int pieces = (K + 255) / 256;
    const long long warps = sm_count() * 64 * 3;
    int parts = static_cast<int>((warps + M - 1) / M);  // (the sum of two ints may pass 31 bits)
    if (parts > pieces) parts = pieces;
    const int part_elems = (pieces + parts - 1) / parts * 256;
    parts = (K + part_elems - 1) / part_elems;
    const long long ctas = (static_cast<long long>(M) * parts + kThreads / 32 - 1) / (kThreads / 32);
    if (ctas > 0x7FFFFFFF || static_cast<long long>(M) * parts > 0xFFFFFF00ll) return cudaErrorInvalidConfiguration;
    const dim3 grid(static_cast<unsigned>(ctas)), block(kThreads);
    uint8_t *y = static_cast<uint8_t *>(Y);
    const long long row_bytes = ldy * kv::type_size(type);
    switch (type) {
    case GQ_TYPE_F32:
        return launch_pdl(k_embed<FORMAT, GQ_TYPE_F32>, grid, block, 0, s, W, ids, scale, y, row_bytes, rows, K, M,
                          parts, part_elems, status_word());
    case GQ_TYPE_F16:
        return launch_pdl(k_embed<FORMAT, GQ_TYPE_F16>, grid, block, 0, s, W, ids, scale, y, row_bytes, rows, K, M,
                          parts, part_elems, status_word());
    default:
        return launch_pdl(k_embed<FORMAT, GQ_TYPE_BF16>, grid, block, 0, s, W, ids, scale, y, row_bytes, rows, K, M,
                          parts, part_elems, status_word());
    }
}

}  // namespace
}  // namespace gq

extern "C" int gq_embed(int format, const void *W, const int32_t *ids, float scale, void *Y, long long ldy, int type,
                        int rows, int K, int M, gq_stream_t stream)
{
    using namespace gq;
    if (format != GQ_FORMAT_Q4_0 && format != GQ_FORMAT_Q8_0 && format != GQ_FORMAT_Q4_K && format != GQ_FORMAT_Q6_K)
        return GQ_ERR_FORMAT;
    if (type != GQ_TYPE_F32 && type != GQ_TYPE_F16 && type != GQ_TYPE_BF16) return GQ_ERR_FORMAT;
    if (!W || (M > 0 && (!ids || !Y))) return GQ_ERR_NULL;
    if (!aligned16(W) || !aligned16(Y) || (reinterpret_cast<uintptr_t>(ids) & 3u) != 0) return GQ_ERR_ALIGN;
    if (M < 0 || K > (1 << 24) || !isfinite(scale) || gq_packed_bytes(format, rows, K) == 0 || ldy < K) return GQ_ERR_SHAPE;
    if (ldy * kv::type_size(type) % 16 != 0) return GQ_ERR_ALIGN;
    if (M == 0) return GQ_OK;
    const uint8_t *w = static_cast<const uint8_t *>(W);
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    switch (format) {
    case GQ_FORMAT_Q4_0: return status_from(launch<GQ_FORMAT_Q4_0>(w, ids, scale, Y, ldy, type, rows, K, M, s));
    case GQ_FORMAT_Q8_0: return status_from(launch<GQ_FORMAT_Q8_0>(w, ids, scale, Y, ldy, type, rows, K, M, s));
    case GQ_FORMAT_Q4_K: return status_from(launch<GQ_FORMAT_Q4_K>(w, ids, scale, Y, ldy, type, rows, K, M, s));
    default: return status_from(launch<GQ_FORMAT_Q6_K>(w, ids, scale, Y, ldy, type, rows, K, M, s));
    }
}
