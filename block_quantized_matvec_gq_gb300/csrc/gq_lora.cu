// gq_lora.cu -- low-rank adapters of a batch's requests (include/gq_lora.h).
//
//   v = A_a x (rank numbers a token), then Y = Y0 + scale_a B_a v.
//
// Two kernels: `shrink` writes v to the workspace, `expand` adds.  Both work on
// neighbouring tokens; an adapter's weights touch only its own tokens' results.
//
//   decode batches, whose neighbours differ: tiles of 8 tokens, the width of the
//     matrix instruction.  A tile's distinct adapters (its groups) are found with
//     one warp vote, each multiplied with the whole tile in a CTA of its own and
//     kept for its own tokens; every lane copies the pieces of weights and
//     activations that it multiplies (cp.async), so that no thread waits for another.
//   prompts: units of up to 32 and 16 tokens of one adapter, found by a kernel in
//     front; `shrink` shares a step's copies between its warps, `expand` moves Y by
//     bulk copies.
//
// The products run on mma.sync.  Weights are operands as they are (16 bits).  So
// are Q8_0 codes, whose scale is applied to each 32-block's sum; f32 numbers are
// three pieces of bf16, or two of f16 where they can be scaled into its range (v),
// or two of tf32 (activations beside f16 weights): 22 bits or more.  The order of
// the contraction is free, so a lane takes 8 consecutive elements of a row, one
// 16-byte load, as its operands of two instructions.  Sums of more than 32
// products are added in f32 registers, because the tensor core truncates its own.
//
// tcgen05 is not used: the contraction is 8 to 128 deep, so the work is the
// bytes of Y (and, for few tokens, of the adapters), not the products.
//
// What bounds them: 4096 tokens of rank 16 beside 21504 rows (732 MB) take 126 us,
// 5.8 TB/s: the memory (a plain copy in the same order takes 114 for Y alone).  1531
// tokens of rank 64 (112 MB) take 46, of which finding the units and shrink are the
// first 20; 64 tokens of 48 adapters of rank 32 (84 MB) 25.2.  One token: 4.5, the
// latency of two kernels.
#include "gq_host.h"
#include "gq_internal.cuh"
#include "gq_kv.cuh"
#include "gq_lora.h"
#include "gq_tc.cuh"

namespace gq {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRowBlock = 32;  // output rows of a warp's step

struct Batch {
    const int32_t *adapter, *sequence;
    const float *scale;
    int n_adapters, n_seq, M;
    int *status;
};

__device__ __forceinline__ void mma_tf32(float (&d)[4], const float (&a)[4], float b0, float b1)
{
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(__float_as_uint(a[0])), "r"(__float_as_uint(a[1])), "r"(__float_as_uint(a[2])),
                   "r"(__float_as_uint(a[3])), "r"(__float_as_uint(b0)), "r"(__float_as_uint(b1)));
}

// The two 16-bit weights of a word, exact.
template <bool BF16>
__device__ __forceinline__ float2 weights2(uint32_t w)
{
    if (BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}

template <bool BF16>
__device__ __forceinline__ void mma_16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    if (BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The 11 leading bits of x; the rest, x - head(x), is exact and tf32 keeps 11 bits of it.
__device__ __forceinline__ float head(float x) { return __uint_as_float(__float_as_uint(x) & 0xFFFFE000u); }

// A pair of numbers as 16-bit ones, and what that leaves of them (exact).  The first piece of a number above the largest
// bf16 stays at that instead of becoming infinite; what is infinite stays so in the second.  (f16: such numbers have been
// scaled into the range, or are codes.)
template <bool BF16>
__device__ __forceinline__ uint32_t round2(float &a, float &b, bool first)
{
    uint32_t w;
    if (!BF16)
        w = kv::f2_half2(a, b);
    else if (first)
        asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(b), "f"(a));
    else
        w = kv::f2_bf162(a, b);
    const float2 r = weights2<BF16>(w);
    a -= r.x;
    b -= r.y;
    return w;
}
// Pieces of 16 bits that hold an f32 number to 22 bits or more.
template <bool BF16>
constexpr int kPiecesOf = BF16 ? 3 : 2;

// One 32-element chunk of v = A x: acc += A x for 16 MT rows and 8 NT tokens.
// `a(m, h)` gives the lane's 8 weights of row 16 m + 8 h + g, `x(q, v)` its 8
// activations of token 8 q + g (codes as whole numbers for Q8), `d(q, i)` the scale
// of token 8 q + 2 t + i.  The order of the contraction is free: step s takes
// elements 4 s .. 4 s + 3 of every lane.  16-bit weights are operands as they are;
// codes are exact in either type, f32 numbers are three pieces of bf16.  f16 has
// not the range for f32 numbers: there both are tf32, the numbers in two pieces.
template <int MT, int NT, bool BF16, bool Q8, class GetA, class GetX, class GetD>
__device__ __forceinline__ void multiply_chunk(float (&acc)[MT][NT][4], GetA &&a, GetX &&x, GetD &&d)
{
    constexpr bool k16 = Q8 || BF16;
    constexpr int P = Q8 ? 1 : kPiecesOf<BF16>;
    uint32_t b[k16 ? P : 1][NT][4];
    float v[k16 ? 1 : NT][8];
#pragma unroll
    for (int q = 0; q < NT; ++q) {
        if (k16) {
            float y[8];
            x(q, y);
#pragma unroll
            for (int p = 0; p < P; ++p)
#pragma unroll
                for (int e = 0; e < 4; ++e) b[p][q][e] = round2<BF16>(y[2 * e], y[2 * e + 1], p == 0);
        } else {
            x(q, v[q]);
        }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const uint4 lo4 = a(m, 0), hi4 = a(m, 1);
        const uint32_t lo[4] = {lo4.x, lo4.y, lo4.z, lo4.w}, hi[4] = {hi4.x, hi4.y, hi4.z, hi4.w};
        float af[4][4];
        if (!k16) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 l = weights2<BF16>(lo[e]), h = weights2<BF16>(hi[e]);
                af[e][0] = l.x, af[e][1] = h.x, af[e][2] = l.y, af[e][3] = h.y;
            }
        }
#pragma unroll
        for (int q = 0; q < NT; ++q) {
            float r[4] = {0.f, 0.f, 0.f, 0.f};
            if (k16) {
#pragma unroll
                for (int p = P - 1; p >= 0; --p)
#pragma unroll
                    for (int s = 0; s < 2; ++s)
                        mma_16<BF16>(r, lo[2 * s], hi[2 * s], lo[2 * s + 1], hi[2 * s + 1], b[p][q][2 * s], b[p][q][2 * s + 1]);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    mma_tf32(r, af[e], v[q][2 * e] - head(v[q][2 * e]), v[q][2 * e + 1] - head(v[q][2 * e + 1]));
#pragma unroll
                for (int e = 0; e < 4; ++e) mma_tf32(r, af[e], head(v[q][2 * e]), head(v[q][2 * e + 1]));
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[m][q][e] = Q8 ? fmaf(d(q, e & 1), r[e], acc[m][q][e]) : acc[m][q][e] + r[e];
        }
    }
}
// Eight codes as whole numbers: a code's byte + 128 as the low bits of 2^23.
__device__ __forceinline__ void codes8(uint2 c, float (&x)[8])
{
#pragma unroll
    for (int e = 0; e < 8; ++e)
        x[e] = __uint_as_float(__byte_perm((e < 4 ? c.x : c.y) ^ 0x80808080u, 0x4B000000u, 0x7440 | (e & 3))) - 8388736.0f;
}

// Tokens of a tile: which group (distinct adapter, by first appearance) each
// belongs to, -1 for none, and the groups' adapters.  All threads take part.
struct Tile {
    int group[32], adapter[32];
    int groups;
};
template <int TT>
__device__ __forceinline__ void find_groups(Tile &tile, const Batch &B, int t0)
{
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x, t = t0 + lane;
        int a = -1;
        if (lane < TT && t < B.M) {
            const int b = B.sequence ? __ldg(B.sequence + t) : t;
            if (b >= 0 && b < B.n_seq) a = __ldg(B.adapter + b);
            if ((b >= B.n_seq || a >= B.n_adapters) && B.status) atomicExch(B.status, GQ_ERR_SHAPE);
            if (a < 0 || a >= B.n_adapters) a = -1;
        }
        const unsigned same = __match_any_sync(0xffffffffu, a);
        const int first = __ffs(same) - 1;
        const unsigned leaders = __ballot_sync(0xffffffffu, a >= 0 && first == lane);
        const int g = __popc(leaders & ((1u << first) - 1u));
        tile.group[lane] = a >= 0 ? g : -1;
        if (a >= 0 && first == lane) tile.adapter[g] = a;
        if (lane == 0) tile.groups = __popc(leaders);
    }
    __syncthreads();
}

// Asynchronous copy of 16, 8 or 4 bytes to shared memory.
template <int BYTES>
__device__ __forceinline__ void cp_async(void *to, const void *from)
{
    const uint32_t s = static_cast<uint32_t>(__cvta_generic_to_shared(to));
    if (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(s), "l"(from) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(s), "l"(from), "n"(BYTES) : "memory");
}

// ---------------------------------------------------------------- v = A x
// A chunk of 32 elements: a warp's weights, and activations (f32, or codes and scales).  Stages: what two CTAs per SM
// have room for, at least two.
__host__ __device__ constexpr int shrink_stage(int mt, int nt, bool q8) { return 1024 * mt + (q8 ? 512 : 1024) * nt; }
__host__ __device__ constexpr int shrink_stages(int mt, int nt, bool q8)
{
    const int n = (108 << 10) / (8 * shrink_stage(mt, nt, q8));
    return n > 6 ? 6 : (n < 2 ? 2 : n);
}
// CTA: a tile of 8 tokens, one slice of K.  The warps take the slice's
// 32-element chunks in turn, each for all of rank (16 MT), and add up in
// shared memory; the slices' sums are added by `expand`.
template <int MT, bool BF16, bool Q8>
__global__ void __launch_bounds__(kThreads)
    k_lora_shrink(const uint16_t *__restrict__ A, Batch B, const float *__restrict__ X, long long ldx,
                  const int8_t *__restrict__ Xq, const float *__restrict__ dx, float *__restrict__ V, int rank, int K,
                  int slice_chunks)
{
    extern __shared__ __align__(16) float red[];  // [kWarps][16 MT][8 NT], and before that the warps' rings
    __shared__ Tile tile;
    constexpr int NT = 1, TT = 8 * NT, kOut = 16 * MT * TT, kStage = shrink_stage(MT, NT, Q8), kStages = shrink_stages(MT, NT, Q8);
    struct Raw {  // the lane's part of a chunk
        uint4 a[MT][2];
        uint2 q[NT];
        float4 x[NT][2];
        float d[NT][2];
    };
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int t0 = blockIdx.x * TT, chunks = K / 32;
    char *const ring = reinterpret_cast<char *>(red) + (threadIdx.x >> 5) * kStages * kStage;
    const int c0 = blockIdx.y * slice_chunks, c1 = min(c0 + slice_chunks, chunks);
    pdl_wait();
    // only now: what the next kernel reads before its own wait is complete then
    pdl_launch_dependents();
    find_groups<TT>(tile, B, t0);
    for (int j = blockIdx.z; j < tile.groups; j += gridDim.z) {
        const uint16_t *a = A + static_cast<long long>(tile.adapter[j]) * rank * K;
        float acc[MT][NT][4];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.f;
        bool in[NT], col_in[NT][2];  // whether the lane's tokens belong to the group: as operand (column g), as results
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            in[n] = tile.group[8 * n + g] == j;
            col_in[n][0] = tile.group[8 * n + 2 * t] == j;
            col_in[n][1] = tile.group[8 * n + 2 * t + 1] == j;
        }
        // Chunks come through a ring in shared memory; every lane copies what it reads itself.
        auto fetch = [&](int i) {
            const int c = c0 + warp + kWarps * i;
            if (c < c1) {
                char *to = ring + (i % kStages) * kStage + lane * 16;
                const int k = 32 * c + 8 * t;
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int r = 16 * m + 8 * h + g;
                        if (r < rank) cp_async<16>(to + (2 * m + h) * 512, a + static_cast<long long>(r) * K + k);
                    }
                to += 1024 * MT;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const long long tok = t0 + 8 * n + g;
                    if (Q8) {
                        if (in[n]) cp_async<8>(to + n * 512 - lane * 8, Xq + tok * K + k);
#pragma unroll
                        for (int x = 0; x < 2; ++x)
                            if (col_in[n][x])
                                cp_async<4>(to + n * 512 + 256 + x * 128 - lane * 12, dx + static_cast<long long>(t0 + 8 * n + 2 * t + x) * chunks + c);
                    } else if (in[n]) {
                        cp_async<16>(to + n * 1024, X + tok * ldx + k);
                        cp_async<16>(to + n * 1024 + 512, X + tok * ldx + k + 4);
                    }
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        auto load = [&](Raw &w, int i) {
            const char *from = ring + (i % kStages) * kStage + lane * 16;
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(from + (2 * m + h) * 512);
                    w.a[m][h] = 16 * m + 8 * h + g < rank ? v : make_uint4(0, 0, 0, 0);
                }
            from += 1024 * MT;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                if (Q8) {
                    const uint2 v = *reinterpret_cast<const uint2 *>(from + n * 512 - lane * 8);
                    w.q[n] = in[n] ? v : make_uint2(0, 0);
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const float d = *reinterpret_cast<const float *>(from + n * 512 + 256 + x * 128 - lane * 12);
                        w.d[n][x] = col_in[n][x] ? d : 0.f;
                    }
                } else {
                    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const float4 v = *reinterpret_cast<const float4 *>(from + n * 1024 + x * 512);
                        w.x[n][x] = in[n] ? v : zero;
                    }
                }
            }
        };
        auto multiply = [&](const Raw &w) {
            multiply_chunk<MT, NT, BF16, Q8>(
                acc, [&](int m, int h) { return w.a[m][h]; },
                [&](int q, float(&v)[8]) {
                    if (Q8) {
                        codes8(w.q[q], v);
                    } else {
                        v[0] = w.x[q][0].x, v[1] = w.x[q][0].y, v[2] = w.x[q][0].z, v[3] = w.x[q][0].w;
                        v[4] = w.x[q][1].x, v[5] = w.x[q][1].y, v[6] = w.x[q][1].z, v[7] = w.x[q][1].w;
                    }
                },
                [&](int q, int i) { return w.d[q][i]; });
        };
        const int mine_n = c0 + warp < c1 ? (c1 - c0 - warp + kWarps - 1) / kWarps : 0;
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) fetch(i);
#pragma unroll 1
        for (int i = 0; i < mine_n; ++i) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
            Raw now;
            load(now, i);
            multiply(now);
            fetch(i + kStages - 1);
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();  // the sums take the rings' place
        float *mine = red + warp * kOut;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    mine[(8 * n + 2 * t + (i & 1)) * 16 * MT + 16 * m + g + 8 * (i >> 1)] = acc[m][n][i];
        __syncthreads();
        float *out = V + static_cast<long long>(blockIdx.y) * B.M * rank;
        for (int i = threadIdx.x; i < kOut; i += kThreads) {
            const int tok = i / (16 * MT), r = i - tok * 16 * MT;
            if (r < rank && tile.group[tok] == j) {
                float s = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) s += red[w * kOut + i];
                out[static_cast<long long>(t0 + tok) * rank + r] = s;
            }
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------- the same for prompts
// Units: neighbouring tokens of one adapter (or of none), at most 32 or 16.  A tile
// at fixed places would hold two requests' ends here and there, and its CTA would
// take twice as long as the others and keep the call waiting (1531 tokens of seven
// prompts: 60 us, 47 with units and the kernel that finds them; 4096 of four
// prompts: 152 and 132).  [0] is their number, then first tokens and adapters,
// behind the last M.
constexpr int kUnitThreads = 1024, kUnitTokens = 4;  // tokens of a thread in a round
__host__ __device__ constexpr long long unit_words(long long M) { return M + 2; }
__device__ __forceinline__ int adapter_of(const Batch &B, int t)
{
    const int b = __ldg(B.sequence + t);
    if (b < 0) return -1;
    const int a = b < B.n_seq ? __ldg(B.adapter + b) : B.n_adapters;
    if (a >= B.n_adapters) {
        if (B.status) atomicExch(B.status, GQ_ERR_SHAPE);
        return -1;
    }
    return a < 0 ? -1 : a;
}
__global__ void __launch_bounds__(kUnitThreads) k_lora_units(Batch B, int2 *__restrict__ of32, int2 *__restrict__ of16)
{
    __shared__ int starts[2][kUnitThreads / 32];
    __shared__ unsigned counts[2][kUnitThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int n32 = 0, n16 = 0, start = 0;  // units so far, and where the last run began
    pdl_wait();
    pdl_launch_dependents();
    for (int t0 = 0, round = 0; t0 < B.M; t0 += kUnitThreads * kUnitTokens, round ^= 1) {
        const int t = t0 + tid * kUnitTokens;
        int a[kUnitTokens + 1];  // and the token in front
#pragma unroll
        for (int i = 0; i <= kUnitTokens; ++i) a[i] = t + i - 1 >= 0 && t + i - 1 < B.M ? adapter_of(B, t + i - 1) : -2;
        // the run's first token: the greatest at or in front of the thread's
        int from[kUnitTokens], mine = -1;
#pragma unroll
        for (int i = 0; i < kUnitTokens; ++i) from[i] = mine = a[i + 1] != a[i] ? t + i : mine;
        int before = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, before, o);
            if (lane >= o) before = max(before, up);
        }
        if (lane == 31) starts[round][warp] = before;
        before = __shfl_up_sync(0xffffffffu, before, 1);
        if (lane == 0) before = -1;
        __syncthreads();
        const int others = starts[round][lane];
        before = max(max(before, start), __reduce_max_sync(0xffffffffu, lane < warp ? others : -1));
        start = max(start, __reduce_max_sync(0xffffffffu, others));
        unsigned is16 = 0, is32 = 0;
#pragma unroll
        for (int i = 0; i < kUnitTokens; ++i) {
            const int at = t + i - max(from[i], before);
            if (t + i < B.M) {
                is16 |= (at % 16 == 0 ? 1u : 0u) << i;
                is32 |= (at % 32 == 0 ? 1u : 0u) << i;
            }
        }
        const unsigned own = __popc(is16) << 16 | __popc(is32);  // at most 4096 of each in a round
        unsigned incl = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned up = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += up;
        }
        if (lane == 31) counts[round][warp] = incl;
        __syncthreads();
        const unsigned sums = counts[round][lane];
        incl += __reduce_add_sync(0xffffffffu, lane < warp ? sums : 0u) - own;
        int to16 = n16 + static_cast<int>(incl >> 16), to32 = n32 + static_cast<int>(incl & 0xFFFFu);
#pragma unroll
        for (int i = 0; i < kUnitTokens; ++i) {
            const int2 unit = make_int2(t + i, a[i + 1]);
            if (is16 >> i & 1u) of16[1 + to16++] = unit;
            if (is32 >> i & 1u) of32[1 + to32++] = unit;
        }
        const unsigned all = __reduce_add_sync(0xffffffffu, sums);
        n16 += static_cast<int>(all >> 16);
        n32 += static_cast<int>(all & 0xFFFFu);
    }
    if (tid == 0) {
        of16[0] = make_int2(n16, 0);
        of32[0] = make_int2(n32, 0);
        of16[1 + n16] = of32[1 + n32] = make_int2(B.M, -1);
    }
}

// CTA: a unit of up to 32 tokens and one slice of K, in steps: all threads copy a step's
// weights and activations, and each warp takes one 32-element chunk of 16 MT ranks.
// Above rank 32 the warps divide the ranks into MH parts, so that a step is 128 or
// 64 elements instead of 256 and more steps are on their way.  Rows are padded so
// that the operands' loads meet no bank twice.  (Bulk copies, one per row, took 58 us where this then took 25 for 4096 tokens of rank
// 16: they cost some 60 cycles each, and the rows are 256 and 512 bytes.)
constexpr int kTileTokens = 32;
__host__ __device__ constexpr int step_of(int mh) { return kWarps / mh * 32; }
__host__ __device__ constexpr int step_a(int mh) { return 2 * step_of(mh) + 64; }
__host__ __device__ constexpr int step_x(int mh, bool q8) { return q8 ? step_of(mh) + 32 : 4 * step_of(mh) + 16; }
__host__ __device__ constexpr int step_d(int mh) { return 4 * (kWarps / mh) + 4; }
__host__ __device__ constexpr int step_bytes(int rank, int mh, bool q8)
{
    return rank * step_a(mh) + kTileTokens * (step_x(mh, q8) + (q8 ? step_d(mh) : 0));
}
inline int step_stages(int rank, int mh, bool q8)
{
    const int n = (104 << 10) / step_bytes(rank, mh, q8);
    return n > 4 ? 4 : (n < 2 ? 2 : n);
}

template <int MT, int MH, bool BF16, bool Q8>
__global__ void __launch_bounds__(kThreads, 2)
    k_lora_shrink_tile(const uint16_t *__restrict__ A, const int2 *__restrict__ units, int M, const float *__restrict__ X,
                       long long ldx, const int8_t *__restrict__ Xq, const float *__restrict__ dx, float *__restrict__ V, int rank,
                       int K, int slice_steps, int stages)
{
    extern __shared__ __align__(16) char raw[];  // stages; after the last step the warps' sums [kWarps][tokens][16 MT]
    constexpr int TT = kTileTokens, NT = TT / 8, kOut = 16 * MT * TT, kChunks = kWarps / MH, kStep = 32 * kChunks;
    constexpr int kPieces = kStep * (Q8 ? 1 : 4) / 16, kPiecesA = 2 * kStep / 16;  // 16-byte pieces of a token's step, of a rank's
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3, chunk = warp % kChunks, m0 = warp / kChunks * MT;
    const int chunks = K / 32, steps = (K + kStep - 1) / kStep;
    const int s0 = blockIdx.y * slice_steps, n = min(slice_steps, steps - s0);
    const int stage_bytes = step_bytes(rank, MH, Q8), off_x = rank * step_a(MH), off_d = off_x + TT * step_x(MH, Q8);
    pdl_wait();
    // only now: what the next kernel reads before its own wait is complete then
    pdl_launch_dependents();
    const int n_units = __ldcg(units).x;
    for (int j = blockIdx.x; j < n_units; j += gridDim.x) {
        const int2 unit = __ldcg(units + 1 + j);
        const int t0 = unit.x, tokens = __ldcg(units + 2 + j).x - t0;
        if (unit.y < 0) continue;
        const uint16_t *a = A + static_cast<long long>(unit.y) * rank * K;
        auto fetch = [&](int i, int slot) {
            if (i < n) {
                const int k0 = (s0 + i) * kStep, count = min(kStep, K - k0);
                char *to = raw + slot * stage_bytes;
                {
                    constexpr int kRanks = kThreads / kPiecesA;  // ranks copied at once
                    const int c = tid % kPiecesA;
                    const uint16_t *from = a + static_cast<long long>(tid / kPiecesA) * K + k0 + 8 * c;
                    if (8 * c < count)
                        for (int r = tid / kPiecesA; r < rank; r += kRanks, from += static_cast<long long>(kRanks) * K)
                            cp_async<16>(to + r * step_a(MH) + 16 * c, from);
                }
                constexpr int kRows = kThreads / kPieces;  // tokens copied at once
                const int c = tid % kPieces;
                if (c * (Q8 ? 16 : 4) < count) {
#pragma unroll
                    for (int r0 = 0; r0 < TT; r0 += kRows) {
                        const int r = r0 + tid / kPieces;
                        if (r < tokens) {
                            const void *from = Q8 ? static_cast<const void *>(Xq + static_cast<long long>(t0 + r) * K + k0 + 16 * c)
                                                  : static_cast<const void *>(X + (t0 + r) * ldx + k0 + 4 * c);
                            cp_async<16>(to + off_x + r * step_x(MH, Q8) + 16 * c, from);
                        }
                    }
                }
                if (Q8) {
                    const int r = tid / kChunks, x = tid % kChunks, at = k0 / 32 + x;
                    if (r < tokens && at < chunks)
                        cp_async<4>(to + off_d + r * step_d(MH) + 4 * x, dx + static_cast<long long>(t0 + r) * chunks + at);
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        float acc[MT][NT][4];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int q = 0; q < NT; ++q)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[m][q][i] = 0.f;
        unsigned in = 0, col = 0;  // whether the lane's tokens belong to the unit: as operand (column g), as results
#pragma unroll
        for (int q = 0; q < NT; ++q) {
            in |= (8 * q + g < tokens ? 1u : 0u) << q;
            col |= (8 * q + 2 * t < tokens ? 1u : 0u) << (2 * q);
            col |= (8 * q + 2 * t + 1 < tokens ? 1u : 0u) << (2 * q + 1);
        }
        for (int i = 0; i < stages - 1; ++i) fetch(i, i);
        int slot = 0, next = stages - 1;
        for (int i = 0; i < n; ++i) {
            // this step's copies; the later ones, stages - 2 of them, may be on their way
            if (stages == 2)
                asm volatile("cp.async.wait_group 0;" ::: "memory");
            else if (stages == 3)
                asm volatile("cp.async.wait_group 1;" ::: "memory");
            else
                asm volatile("cp.async.wait_group 2;" ::: "memory");
            __syncthreads();
            fetch(i + stages - 1, next);
            if ((s0 + i) * kChunks + chunk < chunks) {
                const char *from = raw + slot * stage_bytes + chunk * 64 + t * 16;
                const char *xs = raw + slot * stage_bytes + off_x + (chunk * 32 + t * 8) * (Q8 ? 1 : 4);
                const char *ds = raw + slot * stage_bytes + off_d + chunk * 4;
                multiply_chunk<MT, NT, BF16, Q8>(
                    acc,
                    [&](int m, int h) {
                        const int r = 16 * (m0 + m) + 8 * h + g;
                        return r < rank ? *reinterpret_cast<const uint4 *>(from + r * step_a(MH)) : make_uint4(0, 0, 0, 0);
                    },
                    [&](int q, float(&v)[8]) {
                        const char *p = xs + (8 * q + g) * step_x(MH, Q8);
                        const bool have = in >> q & 1u;
                        if (Q8) {
                            const uint2 c = *reinterpret_cast<const uint2 *>(p);
                            codes8(have ? c : make_uint2(0, 0), v);
                        } else {
                            const float4 u = reinterpret_cast<const float4 *>(p)[0], w = reinterpret_cast<const float4 *>(p)[1];
                            const float y[8] = {u.x, u.y, u.z, u.w, w.x, w.y, w.z, w.w};
#pragma unroll
                            for (int e = 0; e < 8; ++e) v[e] = have ? y[e] : 0.f;
                        }
                    },
                    [&](int q, int i) { return col >> (2 * q + i) & 1u ? *reinterpret_cast<const float *>(ds + (8 * q + 2 * t + i) * step_d(MH)) : 0.f; });
            }
            if (++slot == stages) slot = 0;
            if (++next == stages) next = 0;
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();  // the sums take the stages' place
        float *mine = reinterpret_cast<float *>(raw) + warp * kOut;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int q = 0; q < NT; ++q)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    mine[(8 * q + 2 * t + (i & 1)) * 16 * MT + 16 * m + g + 8 * (i >> 1)] = acc[m][q][i];
        __syncthreads();
        const float *sums = reinterpret_cast<const float *>(raw);
        float *out = V + static_cast<long long>(blockIdx.y) * M * rank;
        for (int i = tid; i < MH * kOut; i += kThreads) {
            const int tok = i / (16 * MT * MH), r = i % (16 * MT * MH);
            if (r < rank && tok < tokens) {
                const float *part = sums + r / (16 * MT) * kChunks * kOut + tok * 16 * MT + r % (16 * MT);
                float v = 0.f;
#pragma unroll
                for (int w = 0; w < kChunks; ++w) v += part[w * kOut];
                out[static_cast<long long>(t0 + tok) * rank + r] = v;
            }
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------- Y = Y0 + scale B v
// v in shared memory as pieces of 16 bits: kPiecesOf rows of TOKENS x pitch bytes,
// then (f16) the factors that undo the scaling.  f16 has not v's range: a token's
// v is scaled so that its largest lies in [2^13, 2^14), an exact power of two.  The
// second piece ends at f16's smallest step: half of it, 2^-25, is 2^-38 of the largest.
__host__ __device__ constexpr int v_pitch(int depth) { return 2 * depth + (2 * depth % 128 == 0 ? 64 : 0); }  // (banks)
__host__ __device__ constexpr int v_bytes(int depth, int tokens) { return 3 * tokens * v_pitch(depth) + 4 * tokens; }

// A lane takes four numbers of a token, a warp as many tokens as that makes; slices
// are added up.  `member` says which tokens have a v.
template <int TOKENS, bool BF16, class Member>
__device__ __forceinline__ void stage_v(char *vs, const float *__restrict__ V, long long t0, int M, int rank, int depth, int slices,
                                        float scale, Member &&member)
{
    const int pitch = v_pitch(depth), shift = depth > 64 ? 5 : depth > 32 ? 4 : depth > 16 ? 3 : 2;  // lanes a token
    const int lane = threadIdx.x & 31 & ((1 << shift) - 1);
#pragma unroll 1
    for (int tok = threadIdx.x >> shift; tok < TOKENS; tok += kThreads >> shift) {
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
        if (4 * lane < rank && member(tok)) {
            const float *p = V + (t0 + tok) * rank + 4 * lane;
#pragma unroll 8
            for (int c = 0; c < slices; ++c) {
                const float4 x = __ldcg(reinterpret_cast<const float4 *>(p + static_cast<long long>(c) * M * rank));
                sum.x += x.x, sum.y += x.y, sum.z += x.z, sum.w += x.w;
            }
        }
        float y[4] = {sum.x * scale, sum.y * scale, sum.z * scale, sum.w * scale};
        if (!BF16) {
            float most = fmaxf(fmaxf(fabsf(y[0]), fabsf(y[1])), fmaxf(fabsf(y[2]), fabsf(y[3])));
            uint32_t bits = __float_as_uint(most);
            for (int o = 1 << shift >> 1; o > 0; o >>= 1) bits = max(bits, __shfl_xor_sync(0xffffffffu, bits, o));
            most = __uint_as_float(bits);
            const int e = static_cast<int>(__float_as_uint(most) >> 23) - 127;  // 128: not finite, and so v stays
            const int k = e == 128 ? 0 : min(13 - e, 126);
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] *= pow2i(k);
            if (lane == 0) reinterpret_cast<float *>(vs + 3 * TOKENS * pitch)[tok] = pow2i(-k);
        }
        if (4 * lane < depth) {
#pragma unroll
            for (int p = 0; p < kPiecesOf<BF16>; ++p) {
                const uint32_t a = round2<BF16>(y[0], y[1], p == 0), b = round2<BF16>(y[2], y[3], p == 0);
                *reinterpret_cast<uint2 *>(vs + (p * TOKENS + tok) * pitch + 8 * lane) = make_uint2(a, b);
            }
        }
    }
}
// The lane's part of a chunk of v, for 8 NT tokens; and two instructions' rows (m)
// times that: weights are operands as they lie.
template <int KC, int NT, bool BF16>
struct Fragment {
    uint32_t w[kPiecesOf<BF16>][NT][KC / 8];
    __device__ __forceinline__ void load(const char *vs, int pitch, int k0, int g, int t)
    {
#pragma unroll
        for (int p = 0; p < kPiecesOf<BF16>; ++p)
#pragma unroll
            for (int q = 0; q < NT; ++q) {
                const char *from = vs + (p * 8 * NT + 8 * q + g) * pitch + 2 * k0 + KC / 2 * t;
                if (KC == 32) {
                    const uint4 x = *reinterpret_cast<const uint4 *>(from);
                    w[p][q][0] = x.x, w[p][q][1] = x.y, w[p][q][KC / 8 - 2] = x.z, w[p][q][KC / 8 - 1] = x.w;
                } else {
                    const uint2 x = *reinterpret_cast<const uint2 *>(from);
                    w[p][q][0] = x.x, w[p][q][1] = x.y;
                }
            }
    }
    __device__ __forceinline__ void multiply(float (&acc)[NT][2][4], const uint32_t (&x)[2][2][KC / 8], bool first) const
    {
#pragma unroll
        for (int q = 0; q < NT; ++q)
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int p = kPiecesOf<BF16> - 1; p >= 0; --p)
#pragma unroll
                    for (int s = 0; s < KC / 16; ++s)
                        mma_16<BF16>(d, x[m][0][2 * s], x[m][1][2 * s], x[m][0][2 * s + 1], x[m][1][2 * s + 1], w[p][q][2 * s], w[p][q][2 * s + 1]);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[q][m][e] = first ? d[e] : acc[q][m][e] + d[e];
            }
    }
};

constexpr int kStages = 3;
// Four rows of weights (16 bytes a lane, 8 where a chunk is 16 deep) and the lane's results of 8 NT tokens.
__host__ __device__ constexpr int expand_stage(int kc, int nt) { return 64 * kc + 1024 * nt; }
// What a CTA does in the time that a tile's beginning takes (groups, v, the first
// copies: some 4 us), in row blocks.  CTAs that pass from one tile to the next get
// so much less (64 tokens of rank 32: 26.4 us, 25.2 with it).
__host__ __device__ constexpr int tile_start(int rank) { return (128 << 10) / (64 * rank + 512); }
// CTA: a range of row blocks of tiles of 8 tokens, which its warps take in
// turn.  Row slots are dealt so that a lane's four results of a token are four
// consecutive rows: slot g (+ 8) of instruction m is row 4 g + 2 m (+ 1).
// KC = 16: a rank of up to 16, where a lane's chunk is four elements.
// kOne: the rank is one chunk, whose v then stays in registers.
template <int KC, bool kOne, bool BF16>
__global__ void __launch_bounds__(kThreads, 2)
    k_lora_expand(const uint16_t *__restrict__ W, Batch B, const float *__restrict__ V, const float *Y0, long long ldy0,
                  float *Y, long long ldy, int rank, int rows, int slices, long long cta_blocks, long long total_blocks)
{
    extern __shared__ __align__(16) char raw[];
    __shared__ Tile tile;
    constexpr int NT = 1, TT = 8 * NT, E = KC / 4;  // E: elements of a lane's chunk
    constexpr int kStageBytes = expand_stage(KC, NT);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    constexpr int kRowPieces = KC / 8, kPieces = kRowPieces;  // 16-byte pieces of a row's chunk, and of a lane
    // where piece c of row r lies: the pieces of a 128-byte line turned by the row group 4 g that reads it
    auto place = [](int r, int c) { return (r * kRowPieces + c) ^ (kRowPieces == 2 ? (r >> 2 & 3) * 2 : (r >> 2 & 1) * 4); };
    char *const ring = raw + warp * kStages * kStageBytes;
    char *const vs = raw + kWarps * kStages * kStageBytes;
    const int depth = kOne ? KC : (rank + KC - 1) / KC * KC, pitch = v_pitch(depth);
    pdl_launch_dependents();
    bool waited = false;
    // a range of all tiles' row blocks in one row, `start` in front of every tile's standing for what beginning it costs
    const int start = tile_start(rank), tile_blocks = start + (rows + kRowBlock - 1) / kRowBlock;
    long long at = start + blockIdx.x * cta_blocks;
    const long long last = min(at + cta_blocks, total_blocks);
    while (at < last) {
        const int tile_no = static_cast<int>(at / tile_blocks), from = static_cast<int>(at - static_cast<long long>(tile_no) * tile_blocks);
        const int to = static_cast<int>(min(static_cast<long long>(tile_blocks), from + (last - at)));
        at += to - from;
        const int rb0 = max(from - start, 0), rb1 = to - start;
        if (rb1 <= rb0) continue;
        const int t0 = tile_no * TT;
        // the lists, Y0 and the weights were complete before `shrink` let this
        // kernel begin; v is complete after the wait
        find_groups<TT>(tile, B, t0);
        const int groups = tile.groups;
        for (int j = blockIdx.z; j < max(groups, 1); j += gridDim.z) {
            const bool product = j < groups;
            // tokens whose rows this pass writes: the group's, and with the first group those without an adapter, if
            // their rows have to be copied
            bool put[NT][2], add[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int tok = 8 * n + 2 * t + i;
                    add[n][i] = product && tile.group[tok] == j;
                    put[n][i] = add[n][i] || (j == 0 && tile.group[tok] < 0 && t0 + tok < B.M && Y != Y0);
                }
            const uint16_t *w = W + static_cast<long long>(product ? tile.adapter[j] : 0) * rows * rank;
            // Steps: a warp's row blocks, each in nk chunks of the rank.  A step's weights, and with a block's last chunk its
            // part of Y0, come through a ring of kStages steps in shared memory.  Of Y0 every lane copies what it reads itself;
            // the weights are copied as they lie (a rank of 16 or 32: 1 or 2 KB without a gap; copied by the lanes that read
            // them they cost three times their bytes), the 16-byte pieces placed so that no two lanes meet on a bank.
            const int nk = depth / KC, blocks = rb0 + warp < rb1 ? (rb1 - rb0 - warp + kWarps - 1) / kWarps : 0, steps = blocks * nk;
            const int row0 = (rb0 + warp) * kRowBlock;
            int fetched = 0, fetch_row = row0, fetch_k = 0;
            char *to = ring;
            const uint16_t *from_w = w + static_cast<long long>(row0 + lane / kRowPieces) * rank + lane % kRowPieces * 8;
            const float *from_y = Y0 + static_cast<long long>(t0 + 2 * t) * ldy0 + row0 + 4 * g;
            auto fetch = [&] {
                if (fetched < steps) {
                    if (product && fetch_k + lane % kRowPieces * 8 < rank) {
#pragma unroll
                        for (int i = 0; i < kPieces; ++i) {
                            constexpr int kRows = 32 / kRowPieces;  // rows that the warp copies at once
                            if (fetch_row + lane / kRowPieces + i * kRows < rows)
                                cp_async<16>(to + 16 * place(lane / kRowPieces + i * kRows, lane % kRowPieces),
                                             from_w + fetch_k + static_cast<long long>(i * kRows) * rank);
                        }
                    }
                    if ((fetch_k += KC) == depth) {
                        if (fetch_row + 4 * g < rows) {
#pragma unroll
                            for (int n = 0; n < NT; ++n)
#pragma unroll
                                for (int i = 0; i < 2; ++i)
                                    if (put[n][i]) cp_async<16>(to + 256 * E + (2 * n + i) * 512 + lane * 16, from_y + (8 * n + i) * ldy0);
                        }
                        fetch_k = 0;
                        fetch_row += kWarps * kRowBlock;
                        from_w += static_cast<long long>(kWarps * kRowBlock) * rank;
                        from_y += kWarps * kRowBlock;
                    }
                    ++fetched;
                    to = to == ring + (kStages - 1) * kStageBytes ? ring : to + kStageBytes;
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
            };
#pragma unroll
            for (int i = 0; i < kStages - 1; ++i) fetch();
            // v is complete after the wait; the copies above were let go before
            if (!waited) pdl_wait();
            waited = true;
            const float scale = product ? __ldg(B.scale + tile.adapter[j]) : 0.f;
            stage_v<TT, BF16>(vs, V, t0, B.M, rank, depth, slices, scale, [&](int tok) { return tile.group[tok] == j; });
            __syncthreads();
            Fragment<KC, NT, BF16> v;  // of all of the rank, where that is one chunk
            if (kOne) v.load(vs, pitch, 0, g, t);
            float undo[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) undo[n][i] = BF16 ? 1.f : reinterpret_cast<const float *>(vs + 3 * TT * pitch)[8 * n + 2 * t + i];
            int row = row0 + 4 * g, k0 = 0;
            const char *from = ring;
            float *y_to = Y + static_cast<long long>(t0 + 2 * t) * ldy + row;
            float acc[NT][2][4];
#pragma unroll 1
            for (int step = 0; step < steps; ++step) {
                asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
                __syncwarp();  // the other lanes' copies as well; and they have read the step before, whose place is next
                if (product) {
                    uint32_t x[2][2][E / 2];
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const char *q = from + 16 * place(4 * g + 2 * m + h, E * t / 8) + (E * t % 8) * 2;
                            if (E == 8) {
                                const uint4 y = *reinterpret_cast<const uint4 *>(q);
                                x[m][h][0] = y.x, x[m][h][1] = y.y, x[m][h][E / 2 - 2] = y.z, x[m][h][E / 2 - 1] = y.w;
                            } else {
                                const uint2 y = *reinterpret_cast<const uint2 *>(q);
                                x[m][h][0] = y.x, x[m][h][1] = y.y;
                            }
                        }
                    if (rank < depth && k0 + E * t >= rank) {  // what lies there was not copied
#pragma unroll
                        for (int e = 0; e < E / 2; ++e) x[0][0][e] = x[0][1][e] = x[1][0][e] = x[1][1][e] = 0u;
                    }
                    if (!kOne) v.load(vs, pitch, k0, g, t);
                    v.multiply(acc, x, kOne || k0 == 0);
                }
                if ((k0 += KC) == depth) {
                    if (row < rows) {
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                if (put[n][i]) {
                                    float4 y = *reinterpret_cast<const float4 *>(from + 256 * E + (2 * n + i) * 512 + lane * 16);
                                    if (add[n][i]) {
                                        y.x = fmaf(acc[n][0][i], undo[n][i], y.x);
                                        y.y = fmaf(acc[n][0][2 + i], undo[n][i], y.y);
                                        y.z = fmaf(acc[n][1][i], undo[n][i], y.z);
                                        y.w = fmaf(acc[n][1][2 + i], undo[n][i], y.w);
                                    }
                                    *reinterpret_cast<float4 *>(y_to + (8 * n + i) * ldy) = y;
                                }
                    }
                    k0 = 0;
                    row += kWarps * kRowBlock;
                    y_to += kWarps * kRowBlock;
                }
                from = from == ring + (kStages - 1) * kStageBytes ? ring : from + kStageBytes;
                fetch();
            }
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            __syncthreads();
        }
        __syncthreads();
    }
    if (!waited) pdl_wait();
}

// ---------------------------------------------------------------- the same for prompts
// Tiles of 16 tokens by 256 rows as bulk copies: a producer warp brings Y0's 16
// stretches of 1 KB and the rows' weights into a stage, eight warps add B v in
// place, and the producer sends the stretches to Y.  Copied by the threads that
// hold the results, in 128-byte pieces of four tokens an instruction, the same
// bytes took 168 us where this then took 136 (4096 tokens, 21504 rows, rank 16:
// 705 MB); long stretches are what the memory is fast at, and the copies cost the
// multiplying warps no instructions.
constexpr int kBulkThreads = kThreads + 32, kBulkTokens = 16, kBulkRows = 256, kPitch = 4 * kBulkRows + 16;
__host__ __device__ constexpr int bulk_stage(int rank) { return kBulkTokens * kPitch + 2 * kBulkRows * rank; }
__host__ __device__ constexpr int unit_start(int rank) { return (128 << 10) / (2 * kBulkRows * rank + 2048 * kBulkTokens); }
inline int bulk_stages(int rank)
{
    const int n = (104 << 10) / bulk_stage(rank);
    return n > 6 ? 6 : (n < 2 ? 2 : n);
}
__device__ __forceinline__ void bulk_store(void *to, uint32_t from, uint32_t bytes)
{
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(to), "r"(from), "r"(bytes) : "memory");
}

template <int KC, bool kOne, bool BF16>
__global__ void __launch_bounds__(kBulkThreads, 2)
    k_lora_expand_bulk(const uint16_t *__restrict__ W, const int2 *__restrict__ units, const float *__restrict__ scales, int M,
                       int *status, const float *__restrict__ V, const float *Y0, long long ldy0, float *Y, long long ldy, int rank,
                       int rows, int slices, int stages)
{
    extern __shared__ __align__(16) char raw[];
    __shared__ __align__(8) uint64_t bars[2 * 6];  // filled, and multiplied
    __shared__ int abort;
    constexpr int E = KC / 4, NT = 2;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int depth = kOne ? KC : (rank + KC - 1) / KC * KC, pitch = v_pitch(depth);
    const int stage_bytes = bulk_stage(rank);
    char *const vs = raw + stages * stage_bytes;
    const uint32_t base = tcu::smem_u32(raw), full = tcu::smem_u32(bars), done = full + 8 * 6;
    volatile int *const abort_flag = &abort;
    if (threadIdx.x == 0) {
        for (int i = 0; i < stages; ++i) {
            tcu::mbar_init(full + 8 * i, 1);
            tcu::mbar_init(done + 8 * i, kWarps);
        }
        abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    pdl_launch_dependents();
    bool waited = false;
    int stage = 0, phase = 0;  // of the next item
    auto next_stage = [&](int &s, int &ph) {
        if (++s == stages) {
            s = 0;
            ph ^= 1;
        }
    };
    // The items of all units in one row, `start` in front of every unit's as in the other form, dealt out evenly.  The
    // units, Y0 and the weights were complete before `shrink` let this kernel begin; v is complete after the wait.
    const int start = unit_start(rank), unit_items = start + (rows + kBulkRows - 1) / kBulkRows;
    const long long total_items = static_cast<long long>(__ldcg(units).x) * unit_items;
    const long long cta_items = (total_items - start + gridDim.x - 1) / gridDim.x;
    long long at = start + blockIdx.x * cta_items;
    const long long last = min(at + cta_items, total_items);
    while (at < last) {
        const int unit_no = static_cast<int>(at / unit_items), from = static_cast<int>(at - static_cast<long long>(unit_no) * unit_items);
        const int to = static_cast<int>(min(static_cast<long long>(unit_items), from + (last - at)));
        at += to - from;
        const int i0 = max(from - start, 0), n = to - start - i0;
        if (n <= 0) continue;
        const int2 unit = __ldcg(units + 1 + unit_no);
        const int t0 = unit.x, tokens = __ldcg(units + 2 + unit_no).x - t0;
        const bool product = unit.y >= 0;
        if (!product && Y == Y0) continue;
        const uint16_t *w = W + static_cast<long long>(product ? unit.y : 0) * rows * rank;
        if (warp == kWarps) {
            // ---- the producer: lane i < 16 copies token i, lane 16 the weights
            const bool mine = lane < tokens;
            const float *y0 = Y0 + (t0 + lane) * ldy0;
            float *y = Y + (t0 + lane) * ldy;
            int ls = stage, lp = phase, issued = 0;
            auto load = [&](int i) {
                const int row = (i0 + i) * kBulkRows, count = min(kBulkRows, rows - row);
                const uint32_t to = base + ls * stage_bytes, bar = full + 8 * ls;
                if (lane == 0) tcu::mbar_expect_tx(bar, tokens * count * 4 + (product ? count * rank * 2 : 0));
                __syncwarp();
                if (mine) tcu::bulk_load(to + lane * kPitch, y0 + row, count * 4, bar);
                if (lane == kBulkTokens && product)
                    tcu::bulk_load(to + kBulkTokens * kPitch, w + static_cast<long long>(row) * rank, count * rank * 2, bar);
                next_stage(ls, lp);
                ++issued;
            };
            for (int i = 0; i < stages - 1 && i < n; ++i) load(i);
            int s = stage, ph = phase, i = 0;
            for (; i < n; ++i) {
                if (i + stages - 1 < n) {
                    // into the stage of the item before, once its results have been read
                    asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                    __syncwarp();
                    load(i + stages - 1);
                }
                if (!tcu::wait_warp(done + 8 * s, ph, abort_flag, status)) break;
                const int row = (i0 + i) * kBulkRows, count = min(kBulkRows, rows - row);
                if (mine) bulk_store(y + row, base + s * stage_bytes + lane * kPitch, count * 4);
                asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                next_stage(s, ph);
            }
            if (i < n) {  // gave up: its copies have to arrive before the CTA may end
                int ws = stage, wp = phase;
                for (int x = 0; x < issued; ++x, next_stage(ws, wp)) {
                    abort = 0;
                    tcu::wait_warp(full + 8 * ws, wp, abort_flag, status);
                }
                abort = 1;
            }
            asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        } else {
            // ---- the multiplying warps: 32 rows each
            if (!waited) pdl_wait();
            const float scale = product ? __ldg(scales + unit.y) : 0.f;
            if (product)
                stage_v<kBulkTokens, BF16>(vs, V, t0, M, rank, depth, slices, scale, [&](int tok) { return tok < tokens; });
            asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory");
            Fragment<KC, NT, BF16> v;  // of all of the rank, where that is one chunk
            if (kOne) v.load(vs, pitch, 0, g, t);
            float undo[NT][2];
#pragma unroll
            for (int q = 0; q < NT; ++q)
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    undo[q][x] = BF16 ? 1.f : reinterpret_cast<const float *>(vs + 3 * kBulkTokens * pitch)[8 * q + 2 * t + x];
            int s = stage, ph = phase;
            for (int i = 0; i < n; ++i) {
                if (!tcu::wait_warp(full + 8 * s, ph, abort_flag, status)) break;
                char *const from = raw + s * stage_bytes;
                if (product) {
                    float acc[NT][2][4];
                    for (int k0 = 0; k0 < depth; k0 += KC) {
                        const int k = k0 + E * t;
                        uint32_t x[2][2][E / 2];
#pragma unroll
                        for (int m = 0; m < 2; ++m)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const char *q = from + kBulkTokens * kPitch + ((32 * warp + 16 * m + 8 * h + g) * rank + k) * 2;
                                if (E == 8) {
                                    const uint4 y = *reinterpret_cast<const uint4 *>(q);
                                    x[m][h][0] = y.x, x[m][h][1] = y.y, x[m][h][E / 2 - 2] = y.z, x[m][h][E / 2 - 1] = y.w;
                                } else {
                                    const uint2 y = *reinterpret_cast<const uint2 *>(q);
                                    x[m][h][0] = y.x, x[m][h][1] = y.y;
                                }
#pragma unroll
                                for (int e = 0; e < E / 2; ++e) x[m][h][e] = k < rank ? x[m][h][e] : 0u;
                            }
                        if (!kOne) v.load(vs, pitch, k0, g, t);
                        v.multiply(acc, x, kOne || k0 == 0);
                    }
#pragma unroll
                    for (int q = 0; q < NT; ++q)
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const int tok = 8 * q + 2 * t + x;
                            float *y = reinterpret_cast<float *>(from + tok * kPitch) + 32 * warp + g;
                            if (tok < tokens) {
#pragma unroll
                                for (int m = 0; m < 2; ++m)
#pragma unroll
                                    for (int h = 0; h < 2; ++h) y[16 * m + 8 * h] = fmaf(acc[q][m][2 * h + x], undo[q][x], y[16 * m + 8 * h]);
                            }
                        }
                    tcu::fence_async_smem();  // before the bulk copies read it
                }
                __syncwarp();
                if (lane == 0) tcu::mbar_arrive(done + 8 * s);
                next_stage(s, ph);
            }
        }
        waited = true;
        for (int i = 0; i < n; ++i) next_stage(stage, phase);
        __syncthreads();
        if (*abort_flag) return;
    }
    if (!waited) pdl_wait();
}

// ---------------------------------------------------------------- host
// Slices of K: some three CTAs per SM for a decode batch's tiles of 8 tokens; for a
// prompt's, of 32, as many CTAs as run at once, at most two per SM.  A slice
// has 256 elements or more, a chunk for every warp.
constexpr int kWantCtas = 456, kWantTiles = 304;
int bounded_slices(long long n, int K)
{
    const int by_k = (K + 255) / 256;
    return n < 1 ? 1 : (n < by_k ? static_cast<int>(n) : by_k);
}
int decode_slices(int K, long long tiles) { return bounded_slices((kWantCtas + tiles - 1) / tiles, K); }
// Rows of slices' sums that calls of up to M tokens write: the most of slices x tokens, so that the workspace of the
// largest batch serves the smaller ones.  A decode batch has at most ceil(kWantCtas / tiles of 8) slices, which times
// its tokens is at most 8 (kWantCtas - 1) + M; a prompt's at most kWantTiles / (tiles of 32), or one.
long long sum_rows(int K, int M)
{
    const long long by_k = static_cast<long long>((K + 255) / 256) * M, few = 8ll * (kWantCtas - 1) + M,
                    many = M > 32 * kWantTiles ? M : 32 * kWantTiles, most = few > many ? few : many;
    return by_k < most ? by_k : most;
}

struct Call {
    const uint16_t *A, *W;
    Batch B;
    const float *X;
    long long ldx;
    const int8_t *Xq;
    const float *dx;
    const float *Y0;
    long long ldy0;
    float *Y;
    long long ldy;
    float *V;
    int rank, rows, K;
    cudaStream_t s;
    int2 *of32 = nullptr, *of16 = nullptr;
};

template <int MT, bool BF16, bool Q8>
cudaError_t shrink(const Call &c, int tiles, int groups, int slices, int slice_chunks)
{
    constexpr int NT = 1;
    auto kern = k_lora_shrink<MT, BF16, Q8>;
    const size_t sums = sizeof(float) * kWarps * 16 * MT * 8 * NT, rings = kWarps * shrink_stages(MT, NT, Q8) * shrink_stage(MT, NT, Q8);
    const size_t smem = sums > rings ? sums : rings;
    if (ctas_per_sm(reinterpret_cast<const void *>(kern), kThreads, smem) < 1) return cudaErrorInvalidConfiguration;
    return launch_pdl(kern, dim3(tiles, slices, groups), dim3(kThreads), smem, c.s, c.A, c.B, c.X, c.ldx, c.Xq, c.dx, c.V,
                      c.rank, c.K, slice_chunks);
}
template <int MT>
cudaError_t shrink_typed(const Call &c, bool bf16, int tiles, int groups, int slices, int slice_chunks)
{
    if (c.Xq)
        return bf16 ? shrink<MT, true, true>(c, tiles, groups, slices, slice_chunks)
                    : shrink<MT, false, true>(c, tiles, groups, slices, slice_chunks);
    return bf16 ? shrink<MT, true, false>(c, tiles, groups, slices, slice_chunks)
                : shrink<MT, false, false>(c, tiles, groups, slices, slice_chunks);
}
cudaError_t shrink_rank(const Call &c, bool bf16, int tiles, int groups, int slices, int slice_chunks)
{
    if (c.rank <= 16) return shrink_typed<1>(c, bf16, tiles, groups, slices, slice_chunks);
    if (c.rank <= 32) return shrink_typed<2>(c, bf16, tiles, groups, slices, slice_chunks);
    if (c.rank <= 64) return shrink_typed<4>(c, bf16, tiles, groups, slices, slice_chunks);
    return shrink_typed<8>(c, bf16, tiles, groups, slices, slice_chunks);
}

template <int MT, int MH, bool BF16, bool Q8>
cudaError_t shrink_tile(const Call &c, int *slices)
{
    auto kern = k_lora_shrink_tile<MT, MH, BF16, Q8>;
    // as many CTAs as there can be units, if every request's tokens lie together
    const int tiles = (c.B.M + kTileTokens - 1) / kTileTokens + c.B.n_seq, steps = (c.K + step_of(MH) - 1) / step_of(MH);
    const int stages = step_stages(c.rank, MH, Q8);
    const size_t rings = static_cast<size_t>(stages) * step_bytes(c.rank, MH, Q8), sums = sizeof(float) * kWarps * 16 * MT * kTileTokens;
    const size_t smem = rings > sums ? rings : sums;
    const int per_sm = ctas_per_sm(reinterpret_cast<const void *>(kern), kThreads, smem);
    if (per_sm < 1) return cudaErrorInvalidConfiguration;
    const int at_once = per_sm * sm_count();
    const int want = bounded_slices((at_once < kWantTiles ? at_once : kWantTiles) / tiles, c.K), slice_steps = (steps + want - 1) / want;
    *slices = (steps + slice_steps - 1) / slice_steps;
    return launch_pdl(kern, dim3(tiles, *slices), dim3(kThreads), smem, c.s, c.A, static_cast<const int2 *>(c.of32), c.B.M, c.X, c.ldx, c.Xq, c.dx, c.V, c.rank, c.K,
                      slice_steps, stages);
}
template <int MT, int MH>
cudaError_t shrink_tile_typed(const Call &c, bool bf16, int *slices)
{
    if (c.Xq) return bf16 ? shrink_tile<MT, MH, true, true>(c, slices) : shrink_tile<MT, MH, false, true>(c, slices);
    return bf16 ? shrink_tile<MT, MH, true, false>(c, slices) : shrink_tile<MT, MH, false, false>(c, slices);
}
cudaError_t shrink_tile_rank(const Call &c, bool bf16, int *slices)
{
    if (c.rank <= 16) return shrink_tile_typed<1, 1>(c, bf16, slices);
    if (c.rank <= 32) return shrink_tile_typed<2, 1>(c, bf16, slices);
    if (c.rank <= 64) return shrink_tile_typed<2, 2>(c, bf16, slices);
    return shrink_tile_typed<2, 4>(c, bf16, slices);
}

template <int KC, bool kOne, bool BF16>
cudaError_t expand(const Call &c, int tiles, int groups, int slices)
{
    constexpr int NT = 1;
    auto kern = k_lora_expand<KC, kOne, BF16>;
    const int depth = (c.rank + KC - 1) / KC * KC;
    const size_t smem = v_bytes(depth, 8 * NT) + kWarps * kStages * expand_stage(KC, NT);
    if (ctas_per_sm(reinterpret_cast<const void *>(kern), kThreads, smem) < 1) return cudaErrorInvalidConfiguration;
    // two CTAs per SM at once, the row blocks of all tiles dealt out evenly: no SM is left with less at the end
    const long long total = static_cast<long long>(tiles) * (tile_start(c.rank) + (c.rows + kRowBlock - 1) / kRowBlock);
    const int ctas = (2 * sm_count() + groups - 1) / groups;
    const long long work = total - tile_start(c.rank);  // the first tile's beginning is every CTA's own
    long long per = (work + ctas - 1) / ctas;
    if (per < kWarps) per = kWarps;
    return launch_pdl(kern, dim3(static_cast<unsigned>((work + per - 1) / per), 1, groups), dim3(kThreads), smem, c.s, c.W, c.B, c.V,
                      c.Y0, c.ldy0, c.Y, c.ldy, c.rank, c.rows, slices, per, total);
}
cudaError_t expand_rank(const Call &c, bool bf16, int tiles, int groups, int slices)
{
    if (c.rank <= 16)
        return bf16 ? expand<16, true, true>(c, tiles, groups, slices) : expand<16, true, false>(c, tiles, groups, slices);
    if (c.rank <= 32)
        return bf16 ? expand<32, true, true>(c, tiles, groups, slices) : expand<32, true, false>(c, tiles, groups, slices);
    return bf16 ? expand<32, false, true>(c, tiles, groups, slices) : expand<32, false, false>(c, tiles, groups, slices);
}

template <int KC, bool kOne, bool BF16>
cudaError_t expand_bulk(const Call &c, int slices)
{
    auto kern = k_lora_expand_bulk<KC, kOne, BF16>;
    const int depth = (c.rank + KC - 1) / KC * KC, stages = bulk_stages(c.rank);
    const size_t smem = v_bytes(depth, kBulkTokens) + static_cast<size_t>(stages) * bulk_stage(c.rank);
    const int per_sm = ctas_per_sm(reinterpret_cast<const void *>(kern), kBulkThreads, smem);
    if (per_sm < 1) return cudaErrorInvalidConfiguration;
    const long long most = ((c.B.M + kBulkTokens - 1ll) / kBulkTokens + c.B.n_seq) * ((c.rows + kBulkRows - 1) / kBulkRows);
    const long long ctas = static_cast<long long>(per_sm) * sm_count();
    return launch_pdl(kern, dim3(static_cast<unsigned>(ctas < most ? ctas : most)), dim3(kBulkThreads), smem, c.s, c.W,
                      static_cast<const int2 *>(c.of16), c.B.scale, c.B.M, c.B.status, c.V, c.Y0, c.ldy0, c.Y, c.ldy, c.rank, c.rows,
                      slices, stages);
}
cudaError_t expand_bulk_rank(const Call &c, bool bf16, int slices)
{
    if (c.rank <= 16) return bf16 ? expand_bulk<16, true, true>(c, slices) : expand_bulk<16, true, false>(c, slices);
    if (c.rank <= 32) return bf16 ? expand_bulk<32, true, true>(c, slices) : expand_bulk<32, true, false>(c, slices);
    return bf16 ? expand_bulk<32, false, true>(c, slices) : expand_bulk<32, false, false>(c, slices);
}

int run(Call c, int type)
{
    const bool bf16 = type == GQ_TYPE_BF16;
    int slices = 0;
    // Neighbouring tokens of one request share their adapter: the prompts' form where requests have 8 tokens or more on
    // average, or 4 in a large batch.  5376 x 5376, us in this form and in the other: 8 requests of 4, 8 and 16 tokens,
    // rank 16: 11.1 and 8.3, 11.2 and 9.8, 12.0 and 17.3; rank 64: 16.4 and 13.0, 16.7 and 17.7, 17.4 and 36.0; 64
    // requests of 2, 4 and 8, rank 16: 20.4 and 14.6, 20.5 and 24.5, 22.9 and 50.9.
    if (c.B.sequence != nullptr && c.B.M / (c.B.M < 256 ? 8 : 4) >= c.B.n_seq) {
        c.of32 = reinterpret_cast<int2 *>(c.V + sum_rows(c.K, c.B.M) * c.rank);
        c.of16 = c.of32 + unit_words(c.B.M);
        cudaError_t e = launch_pdl(k_lora_units, dim3(1), dim3(kUnitThreads), 0, c.s, c.B, c.of32, c.of16);
        if (e == cudaSuccess) e = shrink_tile_rank(c, bf16, &slices);
        if (e == cudaSuccess) e = expand_bulk_rank(c, bf16, slices);
        return status_from(e);
    }
    constexpr int kTokens = 8;
    int groups = kTokens;  // at most, in a tile
    if (groups > c.B.n_adapters) groups = c.B.n_adapters;
    if (groups > c.B.M) groups = c.B.M;
    const int tiles = (c.B.M + kTokens - 1) / kTokens, chunks = c.K / 32;
    slices = decode_slices(c.K, static_cast<long long>(tiles) * groups);
    const int slice_chunks = (chunks + slices - 1) / slices;
    slices = (chunks + slice_chunks - 1) / slice_chunks;
    cudaError_t e = shrink_rank(c, bf16, tiles, groups, slices, slice_chunks);
    if (e == cudaSuccess) e = expand_rank(c, bf16, tiles, groups, slices);
    return status_from(e);
}

inline bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

int check_and_run(Call c, int type, size_t workspace_bytes)
{
    const Batch &B = c.B;
    if (type != GQ_TYPE_F16 && type != GQ_TYPE_BF16) return GQ_ERR_FORMAT;
    if (B.M < 0 || B.n_adapters < 1 || B.n_seq < 1 || c.rows < 4 || c.rows % 4 != 0 || c.rows > (1 << 24)) return GQ_ERR_SHAPE;
    if (B.M == 0) return GQ_OK;
    const size_t need = gq_lora_workspace_bytes(c.rank, c.K, B.M);
    if (need == 0) return GQ_ERR_SHAPE;
    const bool q8 = c.ldx < 0;
    if (!c.A || !c.W || !B.scale || !B.adapter || !c.Y0 || !c.Y || (q8 ? !c.Xq || !c.dx : !c.X)) return GQ_ERR_NULL;
    if (!aligned16(c.A) || !aligned16(c.W) || !aligned16(c.X) || !aligned16(c.Xq) || !aligned16(c.dx) || !aligned16(c.Y0) ||
        !aligned16(c.Y) || !aligned4(B.scale) || !aligned4(B.adapter) || !aligned4(B.sequence))
        return GQ_ERR_ALIGN;
    if (!B.sequence && B.M > B.n_seq) return GQ_ERR_SHAPE;
    if ((!q8 && c.ldx < c.K) || c.ldy0 < c.rows || c.ldy < c.rows || (c.Y == c.Y0 && c.ldy != c.ldy0)) return GQ_ERR_SHAPE;
    if ((!q8 && c.ldx % 4 != 0) || c.ldy0 % 4 != 0 || c.ldy % 4 != 0) return GQ_ERR_ALIGN;
    if (!c.V || workspace_bytes < need) return GQ_ERR_WORKSPACE;
    if (!aligned16(c.V)) return GQ_ERR_ALIGN;
    c.B.status = status_word();
    if (!c.B.status) return GQ_ERR_CUDA;
    return run(c, type);
}

}  // namespace
}  // namespace gq

using namespace gq;

extern "C" {

size_t gq_lora_workspace_bytes(int rank, int K, int M)
{
    if (rank < 8 || rank % 8 != 0 || rank > GQ_MAX_LORA_RANK || K < 32 || K % 32 != 0 || K > (1 << 24) || M < 1 || M > (1 << 28))
        return 0;
    // A x of every slice; and the units, from the fewest tokens on that take the prompts' form
    return static_cast<size_t>(sum_rows(K, M)) * rank * sizeof(float) + (M < 8 ? 0 : 2 * unit_words(M) * sizeof(int2));
}

int gq_lora_add(const void *A, const void *B, int type, const float *scale, const int32_t *adapter,
                const int32_t *sequence_or_null, const float *X, long long ldx, const float *Y0, long long ldy0,
                float *Y, long long ldy, void *workspace, size_t workspace_bytes, int n_adapters, int rank, int rows,
                int K, int n_seq, int M, gq_stream_t stream)
{
    if (ldx < 0) return GQ_ERR_SHAPE;
    const Call c{static_cast<const uint16_t *>(A), static_cast<const uint16_t *>(B),
                 Batch{adapter, sequence_or_null, scale, n_adapters, n_seq, M, nullptr}, X, ldx, nullptr, nullptr, Y0, ldy0, Y,
                 ldy, static_cast<float *>(workspace), rank, rows, K, reinterpret_cast<cudaStream_t>(stream)};
    return check_and_run(c, type, workspace_bytes);
}

int gq_lora_add_q8act(const void *A, const void *B, int type, const float *scale, const int32_t *adapter,
                      const int32_t *sequence_or_null, const int8_t *Xq, const float *dx, const float *Y0,
                      long long ldy0, float *Y, long long ldy, void *workspace, size_t workspace_bytes,
                      int n_adapters, int rank, int rows, int K, int n_seq, int M, gq_stream_t stream)
{
    const Call c{static_cast<const uint16_t *>(A), static_cast<const uint16_t *>(B),
                 Batch{adapter, sequence_or_null, scale, n_adapters, n_seq, M, nullptr}, nullptr, -1, Xq, dx, Y0, ldy0, Y, ldy,
                 static_cast<float *>(workspace), rank, rows, K, reinterpret_cast<cudaStream_t>(stream)};
    return check_and_run(c, type, workspace_bytes);
}

}  // extern "C"
