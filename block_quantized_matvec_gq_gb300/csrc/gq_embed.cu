// gq_embed.cu -- rows of a packed table by token id (include/gq_embed.h).
//
// A warp takes a token's row, or a part of it where there are fewer tokens than
// warps: 256 consecutive weights at a time, eight per lane.  A lane's codes are
// one load of 4 or 8 bytes, its scales one or two short ones that its neighbours
// share, its result one or two 16-byte stores; four such pieces are loaded before
// the first is stored.
//
// What bounds it: the writes.
#include <math.h>

#include "gq_embed.h"
#include "gq_host.h"
#include "gq_internal.cuh"
#include "gq_kv.cuh"

namespace gq {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float half_f(uint16_t h) { return __half2float(__ushort_as_half(h)); }

// The eight weights e0 .. e0 + 7 of row r (e0 a multiple of 8).
template <int FORMAT>
__device__ __forceinline__ void decode8(const uint8_t *__restrict__ W, long long rows, int K, long long r, int e0,
                                        float (&w)[8])
{
    if (FORMAT == GQ_FORMAT_Q8_0) {
        const long long nb = K / 32, blk = r * nb + e0 / 32;
        const uint2 c = __ldg(reinterpret_cast<const uint2 *>(W + blk * 32 + (e0 & 31)));
        const float d = half_f(__ldg(reinterpret_cast<const uint16_t *>(W + rows * nb * 32) + blk));
#pragma unroll
        for (int i = 0; i < 8; ++i)
            w[i] = d * static_cast<float>(static_cast<int>((i < 4 ? c.x : c.y) >> (8 * (i & 3)) & 255u) - 128);
    } else if (FORMAT == GQ_FORMAT_Q4_0) {
        const long long nb = K / 32, blk = r * nb + e0 / 32;
        const uint32_t c = __ldg(reinterpret_cast<const uint32_t *>(W + blk * 16 + (e0 & 31) / 2));
        const float d = half_f(__ldg(reinterpret_cast<const uint16_t *>(W + rows * nb * 16) + blk));
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = d * static_cast<float>(static_cast<int>(c >> (4 * i) & 15u) - 8);
    } else if (FORMAT == GQ_FORMAT_Q4_K) {
        const long long ns = K / 256, sb = r * ns + e0 / 256;
        const int s = (e0 & 255) / 32;
        const uint32_t c = __ldg(reinterpret_cast<const uint32_t *>(W + sb * 128 + (e0 & 255) / 2));
        const uint4 rec = __ldg(reinterpret_cast<const uint4 *>(W + rows * ns * 128) + sb);
        const float d = half_f(static_cast<uint16_t>(rec.x)), dmin = half_f(static_cast<uint16_t>(rec.x >> 16));
        // bytes 0-3: scales 0-3 in 6 bits, 4-7: minima 0-3, 8-11: the low four bits of both of 4-7, whose top two
        // bits are those of the first eight bytes
        const int sh = 8 * (s & 3);
        const uint32_t lo = rec.y >> sh & 255u, mi = rec.z >> sh & 255u, hi = rec.w >> sh & 255u;
        const uint32_t sc = s < 4 ? lo & 63u : (hi & 15u) | (lo >> 6) << 4;
        const uint32_t mn = s < 4 ? mi & 63u : hi >> 4 | (mi >> 6) << 4;
        const float dsc = d * static_cast<float>(sc), m = dmin * static_cast<float>(mn);
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = fmaf(dsc, static_cast<float>(c >> (4 * i) & 15u), -m);
    } else {
        const long long ns = K / 256, sb = r * ns + e0 / 256;
        const int e = e0 & 255;
        const uint8_t *top = W + rows * ns * 128, *sub = top + rows * ns * 64;
        const uint32_t c = __ldg(reinterpret_cast<const uint32_t *>(W + sb * 128 + e / 2));
        const uint32_t t = __ldg(reinterpret_cast<const uint32_t *>(top + sb * 64) + e / 16);
        const float sc = static_cast<float>(static_cast<int8_t>(__ldg(sub + sb * 16 + e / 16)));
        const float d = half_f(__ldg(reinterpret_cast<const uint16_t *>(sub + rows * ns * 16) + sb)) * sc;
        const int a0 = (e & 8) / 4;  // elements 4 a + i of the word, a from a0
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int p = (a0 ? 16 : 0) + (i < 4 ? 0 : 2) + 4 * (i & 3);
            const int q = static_cast<int>(c >> (4 * i) & 15u) + static_cast<int>((t >> p & 3u) << 4) - 32;
            w[i] = d * static_cast<float>(q);
        }
    }
}

template <int FORMAT, int TYPE>
__global__ void __launch_bounds__(kThreads)
    k_embed(const uint8_t *__restrict__ W, const int32_t *__restrict__ ids, float scale, uint8_t *__restrict__ Y,
            long long row_bytes, int rows, int K, int M, int parts, int part_elems, int *status)
{
    constexpr int kBatch = 4;
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
    uint8_t *y = Y + t * row_bytes;
    for (int e0 = part * part_elems + 8 * lane; e0 < end; e0 += kBatch * 256) {
        float w[kBatch][8];
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
            if (have && e0 + 256 * q < end) {
                decode8<FORMAT>(W, rows, K, id, e0 + 256 * q, w[q]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) w[q][i] = 0.f;
            }
        }
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
            if (e0 + 256 * q >= end) continue;
            const float *x = w[q];
            kv::store8<TYPE>(y + static_cast<long long>(e0 + 256 * q) * kv::type_size(TYPE),
                             make_float4(x[0] * scale, x[1] * scale, x[2] * scale, x[3] * scale),
                             make_float4(x[4] * scale, x[5] * scale, x[6] * scale, x[7] * scale));
        }
    }
}

template <int FORMAT>
cudaError_t launch(const uint8_t *W, const int32_t *ids, float scale, void *Y, long long ldy, int type, int rows, int K,
                   int M, cudaStream_t s)
{
    // six times the warps that an SM holds, so that the last ones to finish are a small part
    const int pieces = (K + 255) / 256, warps = sm_count() * 48 * 6;
    int parts = (warps + M - 1) / M;
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
