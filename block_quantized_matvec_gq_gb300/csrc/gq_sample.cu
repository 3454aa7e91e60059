// gq_sample.cu -- temperature, top-k, top-p and min-p sampling (include/gq_sample.h).
//
// Every limit keeps a beginning of one order (falling logit, then rising
// index), and the drawn token is the first of that order whose running weight
// exceeds a target.  So the whole operator is: sums of weights, and "the first
// element at which a running count or weight reaches X".  Nothing sorts a row.
//
// Weights are whole numbers of 2^-43 of about the largest weight, w = M 2^(A - 31)
// with A = rint(l log2(e) / T) and a 32-bit M: A and M depend on the logit and T
// alone, so sums are integers, the same in any order, and a slice can be summed
// before the row's largest logit is known.  A slice's sum is in units of its own
// largest; brought to the row's, their total is up to a unit an element above the
// running weights' last, and goes by how the row was cut.
//
//   scan   streams the row once, a slice per CTA held in registers: largest
//          logit, sum of weights, and a list of the slice's leading elements.
//          The list's threshold is the want-th largest of the threads' own
//          maxima, found by bisection with a vote of the CTA per step: at least
//          `want` elements reach it, and few more.
//   pick   one CTA per row (where a row is one slice, the same CTA): the lists
//          above the slices' highest threshold hold every element above it, some
//          hundreds.  They are sorted, and where the limits and the draw fall
//          among them, which they do for a language model's usual rows, the row
//          is done.
//   deep   the other rows (flat ones, a large top_k), a cluster of 16 CTAs each: a
//          histogram of the row over 2048 equal steps of the exponent, counts and
//          exact weights, gives the step in which X is reached; the step's
//          elements are collected and sorted.  A step with too many elements is
//          divided further, by the bits of (logit, index), which no two elements
//          share.
//
// What bounds it.  160 rows of 262144 f32 logits (168 MB), settings of all kinds,
// 101 us: the scan 55 (issue; 30 instructions an element on average: 10 to read it
// and find the largest, 11 for the list, 22 for the weight where weights are summed),
// the pick some 13, the search of the four to seven rows that need it 25: the pass
// over the row 6, joining the histograms 4.6, and rounds over little data, barriers
// of the cluster, and fetching code that runs once (unrolled passes took 16 us more
// in all).
#include <cooperative_groups.h>
#include <limits.h>
#include <math.h>
#include <stddef.h>

#include "gq_host.h"
#include "gq_internal.cuh"
#include "gq_kv.cuh"
#include "gq_sample.h"

namespace gq {
namespace {

namespace cg = cooperative_groups;
using u64 = unsigned long long;

constexpr int kScanThreads = 256, kSmallThreads = 512;  // of a slice of 8192 and of 4096 elements
constexpr int kPickThreads = 512;
constexpr int kDeepThreads = 1024;
constexpr int kDeepCtas = 16;
constexpr int kDeepClusters = 64;
constexpr int kList = 2048;  // elements that are sorted at once
constexpr int kSumFrom = 512;  // a top_k from here on may lie behind the list: the slices' sums bound its weight
constexpr int kBins = 2048;
constexpr uint32_t kNone = 0x007FFFFFu;        // key of -infinity: no candidate
constexpr uint32_t kUnknown = 0xFFFFFFFFu;     // threshold of a slice whose list is empty
constexpr float kRound = 12582912.0f;          // 1.5 * 2^23: adding it rounds to a whole number
constexpr float kFarDown = -2097152.0f;        // exponents below give no weight
constexpr float kFarUp = 1048576.0f;

struct Settings {
    const float *temperature;
    const int32_t *top_k;
    const float *top_p, *min_p, *u;
};

// What `scan` says of a slice.
struct __align__(16) Header {
    u64 sum;         // weights in units of 2^(exp - 43)
    u64 best;        // the first of the order
    uint32_t lowest, theta;  // smallest candidate's key; every element with a key of theta or more is listed
    int exp, count, cands, pad[3];
};
static_assert(sizeof(Header) == 48, "read as three 16-byte words");

struct Rows {
    const uint8_t *logits;
    long long row_bytes;
    int vocab, slices, cap, cap_log2;
    Header *head;
    u64 *list;
    int *deep;  // rows for the last kernel
};

// Order-preserving bits of a logit that is not a NaN; -0 is 0.
__device__ __forceinline__ uint32_t key_of(float v)
{
    const uint32_t b = __float_as_uint(v + 0.f);
    return b ^ (b >> 31 ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t k) { return __uint_as_float(k ^ (k >> 31 ? 0x80000000u : 0xFFFFFFFFu)); }
// (logit, index) as one number: larger is earlier in the order, 0 is nothing.
__device__ __forceinline__ u64 rank_of(uint32_t key, int index) { return static_cast<u64>(key) << 32 | ~static_cast<uint32_t>(index); }
__device__ __forceinline__ int index_of(u64 rank) { return static_cast<int>(~static_cast<uint32_t>(rank)); }

// ---------------------------------------------------------------- weights
// The exponent of a logit is (l - base) * (ch + cl), ch + cl = log2(e) / T to 47
// bits.  `base` is 0 unless the row's exponents are too large for the rounding
// below; then it is the largest logit, next to which differences are exact.
struct Scale {
    float ch, cl, base;
    bool infinite;  // the largest logit is +infinity
};
__device__ __forceinline__ Scale scale_of(float T)
{
    const float t = fmaxf(T, 7.888609052e-31f);  // 2^-100
    const float hi = 1.44269502f, lo = 1.92596299e-8f;  // log2(e)
    Scale s{0.f, 0.f, 0.f, false};
    if (t < INFINITY) {
        s.ch = __fdiv_rn(hi, t);
        s.cl = __fdiv_rn(__fadd_rn(fmaf(-s.ch, t, hi), lo), t);
    }
    return s;
}
__device__ __forceinline__ Scale scale_of(float T, float largest)
{
    Scale s = scale_of(T);
    s.infinite = largest == INFINITY;
    if (!(fabsf(largest * s.ch) <= kFarUp)) s.base = largest;
    return s;
}

// Exponent A (rounded) and mantissa M in [2^30.5, 2^31.5]: weight M 2^(A - 31).
// 2^f - 1 = f P(f) for |f| <= 1/2, P of degree 5 through the values at the six
// Chebyshev points of the interval (2^-27.5 from it), its leading coefficient
// in two parts: M is within 2^-24.9 of the weight, 2^-33 on average.
constexpr float kP5 = 1.545316336e-04f, kP4 = 1.339086331e-03f, kP3 = 9.618083015e-03f, kP2 = 5.550356954e-02f,
                kP1 = 2.402265072e-01f, kP0 = 6.931471825e-01f, kP0Low = 5.561629e-09f;
__device__ __forceinline__ void split(const Scale &s, float l, int &A, uint32_t &M)
{
    const float d = l - s.base;
    const float r = fmaxf(d * s.ch, kFarDown) + kRound;
    A = __float_as_int(r) - __float_as_int(kRound);
    const float f = fmaf(d, s.cl, fmaf(d, s.ch, kRound - r));
    float p = fmaf(kP5, f, kP4);
    p = fmaf(p, f, kP3);
    p = fmaf(p, f, kP2);
    p = fmaf(p, f, kP1);
    p = fmaf(p, f, kP0Low);
    const float e = fmaf(f, kP0, f * p);
    M = 0x80000000u + static_cast<uint32_t>(__float2int_rn(e * 2147483648.0f));
}
__device__ __forceinline__ u64 shifted(uint32_t M, unsigned sh) { return sh < 64 ? (static_cast<u64>(M) << 12) >> sh : 0ull; }
// sum += M 2^(12 - sh) cut off to a whole number, as `shifted` does: M shifted down or multiplied up, one wide
// multiply-add.
__device__ __forceinline__ void add_shifted(u64 &sum, uint32_t M, int sh)
{
    const int down = max(sh - 12, 0);
    const uint32_t up = 1u << (12 - sh + down);  // 2^(12 - sh), or 1
    sum += static_cast<u64>(__funnelshift_rc(M, 0u, down)) * up;
}
// Two weights for base = 0, the same operations in pairs.
__device__ __forceinline__ void add_weights(u64 &sum, const Scale &s, float a, float b, int top)
{
    const float2 ch = make_float2(s.ch, s.ch), cl = make_float2(s.cl, s.cl), l = make_float2(a, b),
                 round = make_float2(kRound, kRound);
    float2 r = __fmul2_rn(l, ch);
    r = __fadd2_rn(make_float2(fmaxf(r.x, kFarDown), fmaxf(r.y, kFarDown)), round);
    const float2 n = __ffma2_rn(r, make_float2(-1.f, -1.f), round);
    const float2 f = __ffma2_rn(l, cl, __ffma2_rn(l, ch, n));
    float2 p = __ffma2_rn(make_float2(kP5, kP5), f, make_float2(kP4, kP4));
    p = __ffma2_rn(p, f, make_float2(kP3, kP3));
    p = __ffma2_rn(p, f, make_float2(kP2, kP2));
    p = __ffma2_rn(p, f, make_float2(kP1, kP1));
    p = __ffma2_rn(p, f, make_float2(kP0Low, kP0Low));
    const float2 e = __ffma2_rn(f, make_float2(kP0, kP0), __fmul2_rn(f, p));
    const float2 x = __fmul2_rn(e, make_float2(2147483648.0f, 2147483648.0f));
    const int from = top + __float_as_int(kRound);  // less the bits of r: the weight's distance below `top`
    add_shifted(sum, 0x80000000u + static_cast<uint32_t>(__float2int_rn(x.x)), from - __float_as_int(r.x));
    add_shifted(sum, 0x80000000u + static_cast<uint32_t>(__float2int_rn(x.y)), from - __float_as_int(r.y));
}
// Weight in units of 2^(top - 43).
__device__ __forceinline__ u64 weight(const Scale &s, float l, int top)
{
    int A;
    uint32_t M;
    split(s, l, A, M);
    return shifted(M, static_cast<unsigned>(top - A));
}
__device__ __forceinline__ int exponent(const Scale &s, float l)
{
    int A;
    uint32_t M;
    split(s, l, A, M);
    return A;
}
// The same for a row whose largest logit may be infinite: those share the weight.
__device__ __forceinline__ u64 row_weight(const Scale &s, float l, int top)
{
    if (s.infinite) return l == INFINITY ? 1ull << 43 : 0ull;
    return weight(s, l, top);
}

// floor(f * z) for 0 <= f < 1, z < 2^64, and whether something was cut off.
__device__ __forceinline__ u64 part_of(float f, u64 z, bool &rest)
{
    const uint32_t b = __float_as_uint(f);
    const int ex = b >> 23;
    const u64 m = ex ? (b & 0x7FFFFFu) | 0x800000u : b & 0x7FFFFFu;
    const int s = ex ? 150 - ex : 149;  // f = m 2^-s, s >= 24
    const u64 hi = __umul64hi(z, m), lo = z * m;
    if (s < 64) {
        rest = (lo << (64 - s)) != 0;
        return (hi << (64 - s)) | (lo >> s);
    }
    if (s == 64) {
        rest = lo != 0;
        return hi;
    }
    if (s < 128) {
        rest = lo != 0 || (hi << (128 - s)) != 0;
        return hi >> (s - 64);
    }
    rest = (hi | lo) != 0;
    return 0;
}
// The running weight that top_p asks for, and the one that the draw asks for.
__device__ __forceinline__ u64 nucleus(float p, u64 z)
{
    if (!(p > 0.f)) return 1;
    bool rest;
    const u64 x = part_of(p, z, rest);
    return max(x + (rest ? 1 : 0), 1ull);
}
__device__ __forceinline__ u64 drawn(float u, u64 z)
{
    const float f = fmaxf(u, 0.f);  // NaN: 0
    if (f >= 1.f) return z;
    bool rest;
    return min(part_of(f, z, rest) + 1, z);
}
__device__ __forceinline__ float ratio(u64 w, u64 z) { return __fdiv_rn(__ull2float_rn(w), __ull2float_rn(z)); }

// ---------------------------------------------------------------- reading a row
// A row begins anywhere: 16-byte units from the boundary at or below it, the
// first and the last read element by element.
template <int TYPE>
struct Reader {
    static constexpr int kVec = TYPE == GQ_TYPE_F32 ? 4 : 8;
    const uint8_t *base;
    int shift, vocab, units;
    __device__ __forceinline__ Reader(const uint8_t *row, int n)
    {
        const int size = kv::type_size(TYPE);
        shift = static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15u) / size);
        base = row - shift * size;
        vocab = n;
        units = (n + shift + kVec - 1) / kVec;
    }
    __device__ __forceinline__ int index(int unit, int i) const { return unit * kVec + i - shift; }
    __device__ __forceinline__ bool inside(int unit) const { return index(unit, 0) >= 0 && index(unit, kVec) <= vocab; }
    __device__ __forceinline__ uint4 word(int unit) const
    {
        return __ldg(reinterpret_cast<const uint4 *>(base + static_cast<long long>(unit) * 16));
    }
    // The numbers as they are.
    __device__ __forceinline__ void raw(uint4 w, float (&v)[kVec]) const
    {
        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (TYPE == GQ_TYPE_F32) {
                v[i] = __uint_as_float(x[i]);
            } else {
                const float2 f = TYPE == GQ_TYPE_F16 ? kv::half2_f2(x[i]) : make_float2(kv::bf16_lo(x[i]), kv::bf16_hi(x[i]));
                v[2 * i % kVec] = f.x;
                v[(2 * i + 1) % kVec] = f.y;
            }
        }
    }
    // Candidates as they are, NaN and what lies outside as -infinity.
    __device__ __forceinline__ void values(uint4 w, float (&v)[kVec]) const
    {
        raw(w, v);
#pragma unroll
        for (int i = 0; i < kVec; ++i) v[i] = fmaxf(v[i], -INFINITY);
    }
    // A unit that the row's beginning or end cuts, element by element.
    __device__ __forceinline__ void edge(int unit, float (&v)[kVec]) const
    {
        const uint8_t *p = base + static_cast<long long>(unit) * 16;
        const int first = index(unit, 0);
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            v[i] = -INFINITY;
            if (unit < units && first + i >= 0 && first + i < vocab) {
                if (TYPE == GQ_TYPE_F32)
                    v[i] = __ldg(reinterpret_cast<const float *>(p) + i);
                else if (TYPE == GQ_TYPE_F16)
                    v[i] = __half2float(__ushort_as_half(__ldg(reinterpret_cast<const uint16_t *>(p) + i)));
                else
                    v[i] = __uint_as_float(static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t *>(p) + i)) << 16);
                v[i] = fmaxf(v[i], -INFINITY);
            }
        }
    }
    // NaN is left in whole units.
    __device__ __forceinline__ void load(int unit, float (&v)[kVec]) const
    {
        if (unit < units && inside(unit))
            raw(word(unit), v);
        else
            edge(unit, v);
    }
};

__device__ __forceinline__ float temperature(const Settings &s, int row) { return s.temperature ? __ldg(s.temperature + row) : 1.f; }
__device__ __forceinline__ int top_k(const Settings &s, int row, int vocab)
{
    const int k = s.top_k ? __ldg(s.top_k + row) : 0;
    return k > 0 && k < vocab ? k : 0;
}

__device__ __forceinline__ u64 warp_sum(u64 v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
// Sum over the CTA, in every thread.  `sh` has one word per warp; a barrier on both sides.
template <int THREADS>
__device__ __forceinline__ u64 cta_sum(u64 v, u64 *sh)
{
    v = warp_sum(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    return warp_sum(lane < THREADS / 32 ? sh[lane] : 0ull);
}

// ---------------------------------------------------------------- sorted lists
// Falling bitonic sort of n (a power of two, 64 .. kList) numbers.  Steps of 32
// or less stay within a warp's own 64 numbers.
template <int THREADS>
__device__ __forceinline__ void bitonic_down(u64 *a, int n)
{
    for (int size = 2; size <= n; size <<= 1)
        for (int step = size >> 1; step > 0; step >>= 1) {
            for (int t = threadIdx.x; t < n / 2; t += THREADS) {
                const int i = 2 * t - (t & (step - 1)), j = i + step;
                const u64 x = a[i], y = a[j];
                const bool down = (i & size) == 0;
                if ((x < y) == down) {
                    a[i] = y;
                    a[j] = x;
                }
            }
            if (step > 32 || (step == 1 && size >= 64))
                __syncthreads();
            else
                __syncwarp();
        }
    __syncthreads();
}
// Falling sort of the n numbers of `list` (distinct, none above `first` or below
// `last`), with `tmp` as long: dealt into kSteps equal steps of the value, then
// every number finds its place among its step's few.  Numbers of one value are
// dealt by their bits.  The bitonic sort remains for lists with more than kCrowd
// in one step (ties, far outliers).  Loops are not unrolled: this code runs once
// in a kernel, and what it costs is latency and fetching instructions.
constexpr int kSteps = 1024, kCrowd = 256, kFew = 256;
struct SortShared {
    unsigned count[kSteps + 1];
    unsigned short pos[kList];
    unsigned sh[32];
};
template <int THREADS>
__device__ __forceinline__ void sort_down(u64 *list, u64 *tmp, SortShared &Q, int n, u64 first, u64 last)
{
    constexpr int kPer = kSteps / THREADS;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (n <= kFew) {  // every number finds its place among all
        const u64 x = tid < n ? list[tid] : 0ull;
        int place = 0;
        if (tid < n)
#pragma unroll 4
            for (int j = 0; j < n; ++j) place += list[j] > x ? 1 : 0;
        __syncthreads();
        if (tid < n) list[place] = x;
        __syncthreads();
        return;
    }
    const float high = value_of(static_cast<uint32_t>(first >> 32)), low = value_of(static_cast<uint32_t>(last >> 32));
    const float per = (kSteps - 1) / fmaxf(high - low, 1e-30f);
    const bool ties = !(high > low);
    const int shift = max(0, 54 - __clzll(static_cast<long long>(first - last)));
    auto step_of = [&](u64 r) {
        if (ties) return static_cast<int>((first - r) >> shift);
        const float x = (high - value_of(static_cast<uint32_t>(r >> 32))) * per;
        return max(0, min(kSteps - 1, __float2int_rz(x)));
    };
#pragma unroll
    for (int i = 0; i < kPer; ++i) Q.count[tid + i * THREADS] = 0;
    __syncthreads();
    unsigned most = 0;
#pragma unroll 1
    for (int x = tid; x < n; x += THREADS) {
        const unsigned pos = atomicAdd(&Q.count[step_of(list[x])], 1u);
        Q.pos[x] = static_cast<unsigned short>(pos);
        most = max(most, pos + 1);
    }
    __syncthreads();
    // running counts, in place: count[s] = numbers in front of step s
    unsigned c[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) sum += c[i] = Q.count[tid * kPer + i];
    unsigned incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
    }
    if (lane == 31) Q.sh[warp] = incl;
    const bool crowded = __syncthreads_or(most > kCrowd);
    if (crowded) {
        int P = 64;
        while (P < n) P <<= 1;
        for (int i = n + tid; i < P; i += THREADS) list[i] = 0ull;
        __syncthreads();
        bitonic_down<THREADS>(list, P);
        return;
    }
    unsigned at = incl - sum + __reduce_add_sync(0xffffffffu, lane < warp ? Q.sh[lane] : 0u);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        Q.count[tid * kPer + i] = at;
        at += c[i];
    }
    if (tid == 0) Q.count[kSteps] = n;
    __syncthreads();
#pragma unroll 1
    for (int x = tid; x < n; x += THREADS) {
        const u64 r = list[x];
        tmp[Q.count[step_of(r)] + Q.pos[x]] = r;
    }
    __syncthreads();
#pragma unroll 1
    for (int x = tid; x < n; x += THREADS) {
        const u64 r = tmp[x];
        const int s = step_of(r);
        int place = Q.count[s];
        const int to = Q.count[s + 1];
        for (int j = place; j < to; ++j) place += tmp[j] > r ? 1 : 0;
        list[place] = r;
    }
    __syncthreads();
}

// F[i] = before + the weights of list[0 .. i], for the n sorted numbers; a thread
// takes consecutive ones.
template <int THREADS>
__device__ __forceinline__ void running_weights(const u64 *list, u64 *F, int n, u64 before, const Scale &sc, int top, u64 *sh)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, per = (n + THREADS - 1) / THREADS, i0 = threadIdx.x * per,
              i1 = min(i0 + per, n);
    u64 mine = 0;
#pragma unroll 1
    for (int i = i0; i < i1; ++i) {
        mine += row_weight(sc, value_of(static_cast<uint32_t>(list[i] >> 32)), top);
        F[i] = mine;
    }
    u64 incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
    }
    if (lane == 31) sh[warp] = incl;
    __syncthreads();
    const u64 at = before + incl - mine + warp_sum(lane < warp ? sh[lane] : 0ull);
#pragma unroll 1
    for (int i = i0; i < i1; ++i) F[i] += at;
    __syncthreads();
}
// The first i < kList from which on `reaches` holds, the last i if it nowhere does.
// One warp's work, a look at every 64th and at those of one such part (a CTA's look
// at all, with its barriers, took 0.65 us, all warps at a binary search 0.9).
template <class Reaches>
__device__ __forceinline__ int search(Reaches &&reaches)
{
    static_assert(kList == 64 * 32, "a lane a part");
    const int lane = threadIdx.x & 31;
    auto vote = [&](int i) { return __ballot_sync(0xffffffffu, reaches(i)); };
    const unsigned part = vote(64 * lane + 63);
    const int i = 64 * (part ? __ffs(part) - 1 : 31);
    const unsigned lo = vote(i + lane), hi = vote(i + 32 + lane);
    return i + (lo ? __ffs(lo) - 1 : hi ? 31 + __ffs(hi) : 63);
}
// First i with F[i] >= x, n if there is none; a warp's.
__device__ __forceinline__ int reach(const u64 *F, int n, u64 x)
{
    return F[n - 1] >= x ? search([&](int i) { return i >= n - 1 || F[i] >= x; }) : n;
}

// What the slices' headers say of a row.
struct RowHead {
    u64 best;
    uint32_t lowest, theta;
    int cands, most;  // most: the longest list
};
__device__ __forceinline__ Header load_header(const Header *h)
{
    Header r;
    const uint4 *p = reinterpret_cast<const uint4 *>(h);
    uint4 *q = reinterpret_cast<uint4 *>(&r);
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(Header) / 16); ++i) q[i] = __ldcg(p + i);
    return r;
}
// The CTA's rows of headers, joined in every thread; `sh` has one entry per warp.
__device__ __forceinline__ RowHead warp_join(RowHead r)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) r.best = max(r.best, __shfl_xor_sync(0xffffffffu, r.best, o));
    r.lowest = __reduce_min_sync(0xffffffffu, r.lowest);
    r.theta = __reduce_max_sync(0xffffffffu, r.theta);
    r.cands = __reduce_add_sync(0xffffffffu, r.cands);
    r.most = __reduce_max_sync(0xffffffffu, r.most);
    return r;
}
template <int THREADS>
__device__ __forceinline__ RowHead join_heads(RowHead r, RowHead *sh)
{
    const int lane = threadIdx.x & 31;
    r = warp_join(r);
    if (lane == 0) sh[threadIdx.x >> 5] = r;
    __syncthreads();
    const RowHead none{0ull, kUnknown, 0u, 0, 0};
    return warp_join(lane < THREADS / 32 ? sh[lane] : none);
}
__device__ __forceinline__ void add_head(RowHead &r, const Header &h)
{
    if (h.cands == 0) return;
    r.best = max(r.best, h.best);
    r.lowest = min(r.lowest, h.lowest);
    r.theta = max(r.theta, h.theta);
    r.cands += h.cands;
    r.most = max(r.most, h.count);
}

// ---------------------------------------------------------------- pick
struct PickShared {
    u64 list[kList], F[kList], sh[32];
    SortShared sort;
    RowHead heads[32];
    int count;
};

// The row from its slices' headers and lists; false where they do not settle it.  Of
// use in the first warp.
template <int THREADS>
__device__ __forceinline__ bool settle(const Rows &R, const Settings &S, int row, PickShared &P, int &tok, float &pr, bool &refused)
{
    const int tid = threadIdx.x, lane = tid & 31;
    const Header *head = R.head + static_cast<long long>(row) * R.slices;
    const float T = temperature(S, row), p = S.top_p ? __ldg(S.top_p + row) : 1.f, mp = S.min_p ? __ldg(S.min_p + row) : 0.f,
                u = __ldg(S.u + row);
    const int k = top_k(S, row, R.vocab);
    tok = -1;
    pr = 0.f;
    refused = isnan(T) || isnan(p) || isnan(mp);
    if (refused) return true;
    RowHead h{0ull, kUnknown, 0u, 0, 0};
#pragma unroll 1
    for (int s = tid; s < R.slices; s += THREADS) add_head(h, load_header(head + s));
    if (tid == 0) P.count = 0;
    h = join_heads<THREADS>(h, P.heads);  // (a barrier in it)
    if (h.best == 0) return true;
    const float largest = value_of(static_cast<uint32_t>(h.best >> 32));
    if (!(T > 0.f)) {
        tok = index_of(h.best);
        pr = 1.f;
        return true;
    }
    if (h.theta == kUnknown) return false;
    const Scale sc = scale_of(T, largest);
    const int top = exponent(sc, largest);
    const bool summed = (k == 0 || k >= kSumFrom) && sc.base == 0.f && !sc.infinite;
    // the row's weight from the slices', each in units of its own largest; and their lists, 2^g threads a slice
    u64 total = 0;
    const u64 *lists = R.list + (static_cast<long long>(row) * R.slices << R.cap_log2);
    int g = 0;
    while ((R.slices << (g + 1)) <= THREADS) ++g;
    constexpr int kBatch = 8;
#pragma unroll 1
    for (int s0 = 0; s0 < R.slices; s0 += THREADS >> g) {
        const int s = s0 + (tid >> g), e0 = tid & ((1 << g) - 1);
        int n = 0;
        if (s < R.slices) {
            const Header x = load_header(head + s);
            n = x.count;
            const unsigned shift = static_cast<unsigned>(top - x.exp);
            if (summed && e0 == 0 && x.cands > 0 && shift < 64) total += x.sum >> shift;
        }
#pragma unroll 1
        for (int e = 0; e < h.most; e += kBatch << g) {
            u64 x[kBatch];
#pragma unroll
            for (int q = 0; q < kBatch; ++q) {
                const int i = e + e0 + (q << g);
                x[q] = i < n ? __ldcg(lists + (static_cast<long long>(s) << R.cap_log2) + i) : 0ull;
            }
            unsigned mine = 0;
#pragma unroll
            for (int q = 0; q < kBatch; ++q) mine += static_cast<uint32_t>(x[q] >> 32) >= h.theta ? 1u : 0u;
            unsigned incl = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned up = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += up;
            }
            int to = 0;
            if (lane == 31 && incl) to = atomicAdd(&P.count, static_cast<int>(incl));
            to = __shfl_sync(0xffffffffu, to, 31) + static_cast<int>(incl - mine);
#pragma unroll
            for (int q = 0; q < kBatch; ++q)
                if (static_cast<uint32_t>(x[q] >> 32) >= h.theta) {
                    if (to < kList) P.list[to] = x[q];
                    ++to;
                }
        }
    }
    total = cta_sum<THREADS>(total, P.sh);
    const int n = P.count;
    if (n == 0 || n > kList) return false;
    const bool all = n == h.cands;  // every candidate is in the list
    sort_down<THREADS>(P.list, P.F, P.sort, n, h.best, rank_of(max(h.theta, h.lowest), R.vocab - 1));
    running_weights<THREADS>(P.list, P.F, n, 0ull, sc, top, P.sh);
    if (threadIdx.x >= 32) return false;  // the first warp has the rest to itself
    const u64 *F = P.F;
    const u64 listed = F[n - 1], last = n > 1 ? listed - F[n - 2] : listed;
    // the weight of what top_k keeps, between z and most
    u64 z, most;
    if (k > 0 && k <= n) {
        z = most = F[k - 1];
    } else if (all || last == 0) {  // nothing of weight lies beyond the list
        z = most = listed;
    } else if (k == 0) {
        if (!summed) return false;
        z = most = max(total, listed);
    } else {
        z = listed;
        most = summed ? max(total, listed) : ~0ull;
        if (last < (1ull << 43)) most = min(most, listed + static_cast<u64>(k - n) * last);
    }
    // the first element where top_p is reached, and the weight that min_p keeps, where they are in the list
    int from = n, to = n;
    if (p < 1.f) {
        from = to = reach(F, n, nucleus(p, z));
        if (most != z) to = reach(F, n, nucleus(p, most));
    }
    u64 least = ~0ull;
    if (mp > 0.f) {
        bool rest = false;
        const u64 thr = mp < 1.f ? part_of(mp, F[0], rest) + (rest ? 1 : 0) : F[0];
        // first of the list below the threshold; the list falls
        auto w = [&](int i) { return F[i] - (i ? F[i - 1] : 0ull); };
        const int lo = w(n - 1) < thr ? search([&](int i) { return i >= n - 1 || w(i) < thr; }) : n;
        if (lo < n)
            least = F[max(lo, 1) - 1];
        else if (all)
            least = listed;
    }
    u64 kept;
    if (least != ~0ull && (from == n || least <= F[from]))
        kept = least;
    else if (from < n && from == to)
        kept = F[from];
    else if (p < 1.f || mp > 0.f || most != z)
        return false;
    else
        kept = z;
    kept = min(kept, z);
    const int j = reach(F, n, drawn(u, kept));
    if (j == n) return false;
    tok = index_of(P.list[j]);
    pr = ratio(j ? F[j] - F[j - 1] : F[0], kept);
    return true;
}

template <int THREADS>
__device__ __forceinline__ void pick(const Rows &R, const Settings &S, int row, PickShared &P, int32_t *token, float *prob, int *status)
{
    int tok;
    float pr;
    bool refused;
    const bool settled = settle<THREADS>(R, S, row, P, tok, pr, refused);
    if (threadIdx.x == 0) {
        if (settled) {
            token[row] = tok;
            if (prob) prob[row] = pr;
        }
        R.deep[row] = settled ? 0 : 1;
        if (refused && status) atomicExch(status, GQ_ERR_SHAPE);
    }
}

// ---------------------------------------------------------------- scan
// kOne: a row is one slice, and the CTA goes on to pick the token.
template <int TYPE, int EPT, int THREADS, bool kOne>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS)
    k_sample_scan(Rows R, Settings S, int want, int32_t *token, float *prob, int *status)
{
    constexpr int kVec = Reader<TYPE>::kVec, kUnits = EPT / kVec, kWarps = THREADS / 32;
    __shared__ u64 s_sum[kWarps];
    __shared__ uint32_t s_hi[kWarps], s_lo[kWarps];
    __shared__ int s_cands[kWarps], s_count, s_first;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, row = blockIdx.y, slice = blockIdx.x;
    if (tid == 0) {
        s_count = 0;
        s_first = INT_MAX;
    }
    pdl_wait();
    pdl_launch_dependents();
    const Reader<TYPE> in(R.logits + row * R.row_bytes, R.vocab);
    const int u0 = slice * THREADS * kUnits + tid;
    float v[kUnits][kVec];
#pragma unroll
    for (int j = 0; j < kUnits; ++j) in.load(u0 + j * THREADS, v[j]);
    const float T = temperature(S, row);
    const int k = top_k(S, row, R.vocab);
    // per unit the largest; of all the largest and the smallest; and whether all are finite (0 v is not a NaN)
    float most[kUnits], hi = -INFINITY, lo = INFINITY;
    float2 zero = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < kUnits; ++j) {
        most[j] = -INFINITY;
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            most[j] = fmaxf(most[j], v[j][i]);
            lo = fminf(lo, v[j][i]);
        }
#pragma unroll
        for (int i = 0; i < kVec; i += 2) zero = __ffma2_rn(make_float2(v[j][i], v[j][i + 1]), make_float2(0.f, 0.f), zero);
        hi = fmaxf(hi, most[j]);
    }
    int cands = EPT;
    if (!(zero.x + zero.y == 0.f)) {  // masked tokens, or the row's ends
        lo = INFINITY;
        cands = 0;
#pragma unroll
        for (int j = 0; j < kUnits; ++j)
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                v[j][i] = fmaxf(v[j][i], -INFINITY);  // a NaN is no candidate
                if (v[j][i] > -INFINITY) {
                    lo = fminf(lo, v[j][i]);
                    ++cands;
                }
            }
    }
    const uint32_t mine = key_of(hi);
    {
        const uint32_t a = __reduce_max_sync(0xffffffffu, mine), b = __reduce_min_sync(0xffffffffu, lo < INFINITY ? key_of(lo) : kUnknown);
        const int c = __reduce_add_sync(0xffffffffu, cands);
        if (lane == 0) {
            s_hi[warp] = a;
            s_lo[warp] = b;
            s_cands[warp] = c;
        }
    }
    __syncthreads();
    Header h{};
    uint32_t top = 0;
    h.lowest = kUnknown;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        top = max(top, s_hi[w]);
        h.lowest = min(h.lowest, s_lo[w]);
        h.cands += s_cands[w];
    }
    const float best = value_of(top);
    if (mine == top) {  // the slice's first of the order: the lowest index among its largest
        int first = INT_MAX;
#pragma unroll
        for (int j = kUnits - 1; j >= 0; --j)
#pragma unroll
            for (int i = kVec - 1; i >= 0; --i)
                if (v[j][i] == best) first = in.index(u0 + j * THREADS, i);
        atomicMin(&s_first, first);
    }
    h.theta = kUnknown;
    if (T > 0.f && top > kNone) {  // otherwise the first of the order is all that is asked for
        const Scale sc = scale_of(T);
        if (k == 0 || k >= kSumFrom) {
            h.exp = exponent(sc, best);
            u64 sum = 0;
#pragma unroll
            for (int j = 0; j < kUnits; ++j)
#pragma unroll
                for (int i = 0; i < kVec; i += 2) add_weights(sum, sc, v[j][i], v[j][i + 1], h.exp);
            sum = warp_sum(sum);
            if (lane == 0) s_sum[warp] = sum;
        }
        uint32_t a = kNone + 1;
        if (h.cands > R.cap) {
            // a threshold that `w` threads reach and few elements more
            const int threads = __syncthreads_count(mine > kNone);
            const int w = max(1, min(k > 0 ? min(want, 2 * k / static_cast<int>(gridDim.x) + 8) : want, threads / 2));
            uint32_t b = top;  // w threads reach a; look in a .. b
            if (threads == THREADS) {  // all threads reach the least of their maxima
                uint32_t m = __reduce_min_sync(0xffffffffu, mine);
                if (lane == 0) s_lo[warp] = m;
                __syncthreads();
                a = b;
#pragma unroll
                for (int x = 0; x < kWarps; ++x) a = min(a, s_lo[x]);
            }
            while (a < b) {
                const uint32_t mid = a + (b - a) / 2 + 1;
                const int n = __syncthreads_count(mine >= mid);
                if (n >= w)
                    a = mid;
                else
                    b = mid - 1;
                if (n >= w && n <= w + w / 4) break;
            }
        }
        u64 *list = R.list + (static_cast<long long>(row) * R.slices + slice) * R.cap;
        auto put = [&](uint32_t least) {  // the elements from `least` on, as far as there is room
            if (mine < least) return;
            const float from = value_of(least);
#pragma unroll
            for (int j = 0; j < kUnits; ++j) {
                if (most[j] < from) continue;
#pragma unroll
                for (int i = 0; i < kVec; ++i)
                    if (v[j][i] >= from) {
                        const int at = atomicAdd(&s_count, 1);
                        if (at < R.cap) list[at] = rank_of(key_of(v[j][i]), in.index(u0 + j * THREADS, i));
                    }
            }
        };
        put(a);
        __syncthreads();
        h.count = s_count;
        if (h.count <= R.cap) {
            h.theta = a;
        } else {  // many equal ones at the threshold: leave them out
            __syncthreads();
            if (tid == 0) s_count = 0;
            __syncthreads();
            if (a < top) put(a + 1);
            __syncthreads();
            h.count = s_count;
            if (a < top && h.count <= R.cap)
                h.theta = a + 1;
            else
                h.count = 0;
        }
        if (k == 0 || k >= kSumFrom)
#pragma unroll
            for (int w = 0; w < kWarps; ++w) h.sum += s_sum[w];
    }
    __syncthreads();
    if (tid == 0) {
        h.best = top > kNone ? rank_of(top, s_first) : 0ull;
        R.head[static_cast<long long>(row) * R.slices + slice] = h;
    }
    if (kOne) {
        __shared__ PickShared P;
        __syncthreads();
        pick<THREADS>(R, S, row, P, token, prob, status);
    }
}

__global__ void __launch_bounds__(kPickThreads) k_sample_pick(Rows R, Settings S, int32_t *token, float *prob, int *status)
{
    __shared__ PickShared P;
    pdl_wait();
    pdl_launch_dependents();
    pick<kPickThreads>(R, S, blockIdx.x, P, token, prob, status);
}

// ---------------------------------------------------------------- deep
// What stands in all steps up to each, and its weight with that in front of the first.
struct Level {
    unsigned count[kBins];
    u64 weight[kBins];
};
struct DeepShared {
    u64 list[kList], F[kList];
    SortShared sort;
    alignas(16) unsigned hist[kBins], low[kBins], high[kBins];  // this CTA's counts, and weights as two words
    Level fine, coarse;
    u64 sh[kDeepThreads / 32], sh2[kDeepThreads / 32];
    unsigned sh32[kDeepThreads / 32];
    RowHead heads[kDeepThreads / 32];
    u64 least[kDeepCtas];  // weights that min_p keeps
    u64 rank, reached;          // what a search found: the element, and the running weight at it
    u64 limits[2];              // the running weights where top_k ends, and top_p
    int from[3], to[3];         // the steps that are collected for top_k, top_p and the draw
    int found, fit;
    unsigned listed, local;
};

template <int TYPE>
__global__ void __launch_bounds__(kDeepThreads) __cluster_dims__(kDeepCtas, 1, 1)
    k_sample_deep(Rows R, Settings S, int n_rows, int32_t *token, float *prob)
{
    extern __shared__ __align__(16) unsigned char raw[];
    DeepShared &D = *reinterpret_cast<DeepShared *>(raw);
    constexpr int kVec = Reader<TYPE>::kVec, kPer = kBins / kDeepThreads;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    auto cluster = cg::this_cluster();
    const int me = static_cast<int>(cluster.block_rank());
    pdl_launch_dependents();
    pdl_wait();
#pragma unroll 1
    for (int row = blockIdx.y; row < n_rows; row += gridDim.y) {
        if (R.deep[row] == 0) continue;  // the whole cluster
        const float T = temperature(S, row), p = S.top_p ? __ldg(S.top_p + row) : 1.f, mp = S.min_p ? __ldg(S.min_p + row) : 0.f,
                    u = __ldg(S.u + row);
        const int k = top_k(S, row, R.vocab);
        RowHead h{0ull, kUnknown, 0u, 0, 0};
        for (int i = tid; i < R.slices; i += kDeepThreads) add_head(h, load_header(R.head + static_cast<long long>(row) * R.slices + i));
        h = join_heads<kDeepThreads>(h, D.heads);
        const float largest = value_of(static_cast<uint32_t>(h.best >> 32));
        const Scale sc = scale_of(T, largest);
        const int top = exponent(sc, largest);
        // equal steps of the exponent; everything 50 octaves down is one step
        // (the products rounded alike: fused with the difference they would leave the largest's rounding, of either sign)
        auto exponent_of = [&](float v) { return __fmul_rn(v - sc.base, sc.ch); };
        const float t_top = exponent_of(largest);
        const float range = fminf(fmaxf(t_top - exponent_of(value_of(h.lowest)), 0.001f), 50.f), per = kBins / range;
        auto step_of = [&](float v) { return max(0, min(kBins - 1, __float2int_rz((t_top - exponent_of(v)) * per))); };

        const Reader<TYPE> in(R.logits + row * R.row_bytes, R.vocab);
        const int cta_units = (in.units + kDeepCtas - 1) / kDeepCtas, first = me * cta_units, end = min(first + cta_units, in.units);
        // This CTA's part of the row, a 16-byte unit at a time, the next one on its way.  Not unrolled: the kernel runs
        // once over little data, and fetching long code is what it would wait for.
        auto each = [&](auto &&f) {
            int q = first + tid;
            uint4 w = make_uint4(0, 0, 0, 0);
            if (q < end && in.inside(q)) w = in.word(q);
#pragma unroll 1
            for (; q < end; q += kDeepThreads) {
                const int next = q + kDeepThreads;
                uint4 after = make_uint4(0, 0, 0, 0);
                if (next < end && in.inside(next)) after = in.word(next);
                float v[kVec];
                in.values(w, v);
                if (!in.inside(q)) in.edge(q, v);
                f(v, in.index(q, 0));
                w = after;
            }
        };
        auto clear = [&] {
#pragma unroll
            for (int i = 0; i < kPer; ++i) D.hist[tid + i * kDeepThreads] = D.low[tid + i * kDeepThreads] = D.high[tid + i * kDeepThreads] = 0;
            __syncthreads();
        };
        // One element in step b.  Its weight is added to two words, the carry found from the word's old value.
        auto add = [&](int b, u64 w) {
            atomicAdd(&D.hist[b], 1u);
            const unsigned lo = static_cast<unsigned>(w), old = atomicAdd(&D.low[b], lo);
            const unsigned hi = static_cast<unsigned>(w >> 32) + (old + lo < old ? 1u : 0u);
            if (hi) atomicAdd(&D.high[b], hi);
        };
        // The CTAs' histograms, added up and summed over the steps, in every CTA's L; `base` in front.  `between` is done
        // between the two barriers of the cluster: the first is also the one that says that all its CTAs run, before
        // which none may touch another's memory.
        auto merge = [&](Level &L, u64 base, auto &&between) {
            // A CTA sums a share of the steps: two warps fetch each CTA's part of it, 128 bytes an access (single words of
            // many CTAs cost ten times that), and bring the sums to one CTA each.
            constexpr int kShare = kBins / kDeepCtas, kHalf = kShare / 2;
            static_assert(kDeepThreads == 64 * kDeepCtas && kShare == 128, "two warps a CTA, two steps a lane");
            unsigned *const part = reinterpret_cast<unsigned *>(D.list);  // [3][kDeepCtas][kShare]: list and F, which are free
            static_assert(3 * kDeepCtas * kShare * sizeof(unsigned) <= sizeof(D.list) + sizeof(D.F), "room for the parts");
            cluster.sync();
            between();
            {
                const int c = warp >> 1, x = (warp & 1) * kHalf + lane;
                const unsigned *from[3] = {cluster.map_shared_rank(D.hist, c), cluster.map_shared_rank(D.low, c),
                                           cluster.map_shared_rank(D.high, c)};
                unsigned v[3][2];
#pragma unroll
                for (int k = 0; k < 3; ++k)
#pragma unroll
                    for (int i = 0; i < 2; ++i) v[k][i] = from[k][me * kShare + x + 32 * i];
#pragma unroll
                for (int k = 0; k < 3; ++k)
#pragma unroll
                    for (int i = 0; i < 2; ++i) part[(k * kDeepCtas + c) * kShare + x + 32 * i] = v[k][i];
            }
            __syncthreads();
            if (tid < kShare) {
                unsigned n = 0;
                u64 w = 0;
#pragma unroll 4
                for (int c = 0; c < kDeepCtas; ++c) {
                    n += part[c * kShare + tid];
                    w += part[(kDeepCtas + c) * kShare + tid] + (static_cast<u64>(part[(2 * kDeepCtas + c) * kShare + tid]) << 32);
                }
                L.count[me * kShare + tid] = n;
                L.weight[me * kShare + tid] = w;
            }
            __syncthreads();
            {
                Level *to = cluster.map_shared_rank(&L, warp >> 1);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int b = me * kShare + (warp & 1) * kHalf + lane + 32 * i;
                    if ((warp >> 1) != me) {
                        to->count[b] = L.count[b];
                        to->weight[b] = L.weight[b];
                    }
                }
            }
            cluster.sync();
            unsigned n[kPer], ns = 0;
            u64 w[kPer], ws = 0;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                ns += n[i] = L.count[tid * kPer + i];
                ws += w[i] = L.weight[tid * kPer + i];
            }
            unsigned ni = ns;
            u64 wi = ws;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned a = __shfl_up_sync(0xffffffffu, ni, o);
                const u64 b = __shfl_up_sync(0xffffffffu, wi, o);
                if (lane >= o) {
                    ni += a;
                    wi += b;
                }
            }
            if (lane == 31) {
                D.sh32[warp] = ni;
                D.sh2[warp] = wi;
            }
            __syncthreads();
            ni += __reduce_add_sync(0xffffffffu, lane < warp ? D.sh32[lane] : 0u) - ns;
            wi += warp_sum(lane < warp ? D.sh2[lane] : 0ull) + base - ws;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                L.count[tid * kPer + i] = ni += n[i];
                L.weight[tid * kPer + i] = wi += w[i];
            }
            __syncthreads();
        };

        // ---- the row's steps
        bool rest = false;
        const u64 w0 = row_weight(sc, largest, top);
        const u64 thr = mp < 1.f ? (mp > 0.f ? part_of(mp, w0, rest) + (rest ? 1 : 0) : 0ull) : w0;
        u64 least = 0;
        if (tid == 0) D.listed = 0;
        clear();
        each([&](const float (&v)[kVec], int) {
#pragma unroll
            for (int i = 0; i < kVec; ++i)
                if (v[i] > -INFINITY) {
                    const u64 w = row_weight(sc, v[i], top);
                    add(step_of(v[i]), w);
                    least += w >= thr ? w : 0ull;
                }
        });
        least = cta_sum<kDeepThreads>(least, D.sh);
        merge(D.coarse, 0ull, [&] {
            if (tid < kDeepCtas) cluster.map_shared_rank(D.least, tid)[me] = least;
        });
        least = 0;
        for (int c = 0; c < kDeepCtas; ++c) least += D.least[c];

        // The first step in which a running weight or count reaches X; it holds an element.
        static_assert(kBins == kList, "as `search` looks");
        auto first_step = [&](const Level &L, bool by_count, u64 X, unsigned skip) {
            return search([&](int b) { return by_count ? L.count[b] + skip >= X : L.weight[b] >= X; });
        };
        // This CTA's list sorted, and its running weights with `front` in front; how many they are.
        auto sort_list = [&](u64 front) {
            const int n = min(static_cast<int>(D.listed), kList);
            u64 most = 0, fewest = ~0ull;
            if (n > kFew) {
#pragma unroll 1
                for (int i = tid; i < n; i += kDeepThreads) {
                    most = max(most, D.list[i]);
                    fewest = min(fewest, D.list[i]);
                }
                auto extremes = [&] {
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) {
                        most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
                        fewest = min(fewest, __shfl_xor_sync(0xffffffffu, fewest, o));
                    }
                };
                extremes();
                if (lane == 0) {
                    D.sh[warp] = most;
                    D.sh2[warp] = fewest;
                }
                __syncthreads();
                most = D.sh[lane];  // (32 warps)
                fewest = D.sh2[lane];
                extremes();
            }
            sort_down<kDeepThreads>(D.list, D.F, D.sort, n, most, fewest);
            running_weights<kDeepThreads>(D.list, D.F, n, front, sc, top, D.sh);
            return n;
        };
        auto finish = [&](u64 rank, u64 kept) {
            token[row] = index_of(rank);
            if (prob) prob[row] = ratio(row_weight(sc, value_of(static_cast<uint32_t>(rank >> 32)), top), kept);
        };

        // ---- three times the first element at which a running count or weight reaches X: the last that top_k keeps,
        // the last that top_p keeps, the drawn one.  Each X follows from the one before, but the step that holds that
        // bounds it: the steps between the bounds are collected for all three at once and sorted by a CTA each, which
        // leaves a look-up to be done in turn (160 rows of 262144: 102 us, one after the other 109).
        const u64 total = D.coarse.weight[kBins - 1];
        const bool limited = k > 0 && static_cast<unsigned>(k) < D.coarse.count[kBins - 1];
        auto front_of = [&](int b) { return b ? D.coarse.weight[b - 1] : 0ull; };
        auto count_in_front = [&](int b) { return b ? D.coarse.count[b - 1] : 0u; };
        if (warp == 0) {
            int from[3] = {kBins, kBins, kBins}, to[3] = {-1, -1, -1};  // none if there is no such limit
            u64 lo = total, hi = total;  // bounds of the weight kept so far
            if (limited) {
                from[0] = to[0] = first_step(D.coarse, true, static_cast<u64>(k), 0u);
                lo = front_of(to[0]);
                hi = D.coarse.weight[to[0]];
            }
            if (p < 1.f) {
                from[1] = first_step(D.coarse, false, nucleus(p, lo), 0u);
                to[1] = first_step(D.coarse, false, nucleus(p, hi), 0u);
                lo = min(lo, front_of(from[1]));
                hi = min(hi, D.coarse.weight[to[1]]);
            }
            if (mp > 0.f) {
                lo = min(lo, least);
                hi = min(hi, least);
            }
            from[2] = first_step(D.coarse, false, drawn(u, lo), 0u);
            to[2] = first_step(D.coarse, false, drawn(u, hi), 0u);
            bool fit = true;
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                fit &= to[i] < 0 || D.coarse.count[to[i]] - count_in_front(from[i]) <= kList;
                if (lane == i) {
                    D.from[i] = from[i];
                    D.to[i] = to[i];
                }
            }
            if (lane == 0) {
                D.fit = fit ? 1 : 0;
                D.local = 0;
            }
        }
        __syncthreads();
        if (D.fit != 0) {  // the whole cluster
            const int from[3] = {D.from[0], D.from[1], D.from[2]}, to[3] = {D.to[0], D.to[1], D.to[2]};
            // Here first, then to the CTAs that sort them: a count in another CTA's memory takes a microsecond.  Which
            // lists an element belongs to stands above its index.
            static_assert(GQ_MAX_VOCAB <= 1 << 28, "room above the index");
            constexpr unsigned kLocal = 3 * kList;
            u64 *const local = reinterpret_cast<u64 *>(D.hist);  // and `fine`, which are free
            static_assert(offsetof(DeepShared, coarse) - offsetof(DeepShared, hist) >= kLocal * sizeof(u64), "room for all three");
            u64 *const list[3] = {cluster.map_shared_rank(D.list, 0), cluster.map_shared_rank(D.list, 1), cluster.map_shared_rank(D.list, 2)};
            unsigned *const listed[3] = {cluster.map_shared_rank(&D.listed, 0), cluster.map_shared_rank(&D.listed, 1),
                                         cluster.map_shared_rank(&D.listed, 2)};
            auto send = [&](bool have, u64 r, unsigned in) {  // a warp's
                unsigned mask[3], at[3];
#pragma unroll
                for (int c = 0; c < 3; ++c) {
                    mask[c] = __ballot_sync(0xffffffffu, have && (in >> c & 1u));
                    at[c] = 0;
                    if (lane == 0 && mask[c]) at[c] = atomicAdd(listed[c], static_cast<unsigned>(__popc(mask[c])));
                }
#pragma unroll
                for (int c = 0; c < 3; ++c) {
                    const unsigned place = __shfl_sync(0xffffffffu, at[c], 0) + __popc(mask[c] & ((1u << lane) - 1u));
                    if (mask[c] >> lane & 1u && place < kList) list[c][place] = r;
                }
            };
            each([&](const float (&v)[kVec], int index) {
#pragma unroll
                for (int i = 0; i < kVec; ++i) {
                    if (!(v[i] > -INFINITY)) continue;
                    const int b = step_of(v[i]);
                    const unsigned in = (b >= from[0] && b <= to[0] ? 1u : 0u) | (b >= from[1] && b <= to[1] ? 2u : 0u) |
                                        (b >= from[2] && b <= to[2] ? 4u : 0u);
                    if (in) {
                        const unsigned at = atomicAdd(&D.local, 1u);
                        if (at < kLocal) local[at] = rank_of(key_of(v[i]), index + i) ^ in << 28;
                    }
                }
            });
            __syncthreads();
#pragma unroll 1
            for (unsigned x = warp * 32; x < D.local; x += kDeepThreads) {
                const u64 r = x + lane < D.local ? local[x + lane] : 0ull;
                const unsigned in = ~static_cast<uint32_t>(r) >> 28;
                send(x + lane < D.local, r | 0xF0000000ull, in);
            }
            cluster.sync();
            int n = 0;
            const int mine = me < 3 ? D.from[me] : kBins;
            if (mine < kBins) n = sort_list(front_of(mine));
            // the first of the list whose running weight reaches X
            auto first_of = [&](u64 X) { return n > 0 ? min(reach(D.F, n, X), n - 1) : 0; };
            u64 kept = total;
            if (limited) {
                if (me == 0) {
                    const int at = max(min(k - static_cast<int>(count_in_front(mine)), n) - 1, 0);
                    if (tid > 0 && tid < 3) cluster.map_shared_rank(D.limits, tid)[0] = D.F[at];
                }
                cluster.sync();
                kept = D.limits[0];
            }
            if (p < 1.f) {
                if (me == 1 && warp == 0) {
                    const int at = first_of(nucleus(p, kept));
                    if (lane == 0) cluster.map_shared_rank(D.limits, 2)[1] = D.F[at];
                }
                cluster.sync();
                kept = min(kept, D.limits[1]);
            }
            if (mp > 0.f) kept = min(kept, least);
            if (me == 2 && warp == 0) {
                const int at = first_of(drawn(u, kept));
                if (lane == 0) finish(D.list[at], kept);
            }
            cluster.sync();  // no CTA goes on while another reads its memory
            continue;
        }
        // ---- a step with too many elements: one after the other, dividing such steps further
        u64 z = total, kept = z;
#pragma unroll 1
        for (int phase = 0; phase < 3; ++phase) {
            const bool by_count = phase == 0;
            u64 X;
            if (phase == 0) {
                if (!limited) continue;
                X = static_cast<u64>(k);
            } else if (phase == 1) {
                if (mp > 0.f) kept = min(kept, least);
                if (!(p < 1.f)) continue;
                X = nucleus(p, z);
            } else {
                X = drawn(u, kept);
            }
            const Level *L = &D.coarse;
            unsigned skip = 0;      // elements in front of the level's first step
            u64 base = 0;           // and their weight
            u64 high = 0, low = 0;  // ranks that the level divides (below the first level)
            int shift = 0;
#pragma unroll 1
            while (true) {
                if (warp == 0) {
                    const int x = first_step(*L, by_count, X, skip);
                    if (lane == 0) D.found = x;
                }
                __syncthreads();
                const int b = D.found;
                const unsigned in_front = b ? L->count[b - 1] : 0u, in_step = L->count[b] - in_front;
                const u64 weight_in_front = b ? L->weight[b - 1] : base;
                const bool divided = L != &D.coarse;
                if (in_step <= kList) {
                    // its elements, to the first CTA, which sorts them
                    unsigned *counter = cluster.map_shared_rank(&D.listed, 0);
                    u64 *list = cluster.map_shared_rank(D.list, 0);
                    each([&](const float (&v)[kVec], int index) {
#pragma unroll
                        for (int i = 0; i < kVec; ++i) {
                            if (!(v[i] > -INFINITY)) continue;
                            const u64 r = rank_of(key_of(v[i]), index + i);
                            const bool here = divided ? r <= high && r >= low && static_cast<int>((high - r) >> shift) == b : step_of(v[i]) == b;
                            if (here) {
                                const unsigned at = atomicAdd(counter, 1u);
                                if (at < kList) list[at] = r;
                            }
                        }
                    });
                    cluster.sync();
                    if (me == 0) {
                        const int n = sort_list(weight_in_front);
                        if (warp == 0) {
                            int at = by_count ? static_cast<int>(X - skip - in_front) - 1 : n > 0 ? reach(D.F, n, X) : 0;
                            at = max(min(at, n - 1), 0);
                            if (lane < kDeepCtas) {
                                *cluster.map_shared_rank(&D.rank, lane) = D.list[at];
                                *cluster.map_shared_rank(&D.reached, lane) = D.F[at];
                            }
                        }
                        if (tid == 0) D.listed = 0;
                    }
                    cluster.sync();
                    break;
                }
                // too many: divide it by the bits of (logit, index), which no two elements share
                if (!divided) {
                    // the smallest number in the step and the largest, by bisection of all numbers in their order
                    uint32_t lo = kNone + 1, hi = static_cast<uint32_t>(h.best >> 32);
                    while (lo < hi) {
                        const uint32_t mid = lo + (hi - lo) / 2;
                        if (step_of(value_of(mid)) <= b)
                            hi = mid;
                        else
                            lo = mid + 1;
                    }
                    low = rank_of(lo, R.vocab - 1);
                    hi = static_cast<uint32_t>(h.best >> 32);
                    while (lo < hi) {
                        const uint32_t mid = hi - (hi - lo) / 2;
                        if (step_of(value_of(mid)) >= b)
                            lo = mid;
                        else
                            hi = mid - 1;
                    }
                    high = rank_of(lo, 0);
                } else {
                    high -= static_cast<u64>(b) << shift;
                    low = max(low, high - ((1ull << shift) - 1));
                }
                skip += in_front;
                base = weight_in_front;
                shift = max(0, 53 - __clzll(static_cast<long long>(high - low)));
                clear();
                each([&](const float (&v)[kVec], int index) {
#pragma unroll
                    for (int i = 0; i < kVec; ++i) {
                        if (!(v[i] > -INFINITY)) continue;
                        const u64 r = rank_of(key_of(v[i]), index + i);
                        if (r <= high && r >= low) add(static_cast<int>((high - r) >> shift), row_weight(sc, v[i], top));
                    }
                });
                merge(D.fine, base, [] {});
                L = &D.fine;
            }
            if (phase == 0)
                z = kept = D.reached;
            else if (phase == 1)
                kept = min(kept, D.reached);
            else if (me == 0 && tid == 0)
                finish(D.rank, kept);
        }
        cluster.sync();  // no CTA goes on while another reads its memory
    }
}

// ---------------------------------------------------------------- host
// Slices of 4096 elements while they all fit the GPU at once, of 8192 else: a
// small batch is latency, and a large one wants long streams per CTA.
struct Plan {
    int ept, slices, cap_log2, want;
};
constexpr int kFineSlices = 304;
int fine_slices(int vocab) { return (vocab + 7 + 4095) / 4096; }
Plan plan_for(int vocab, int n_rows)
{
    Plan p;
    p.ept = static_cast<long long>(fine_slices(vocab)) * n_rows <= kFineSlices ? 8 : 32;
    const int threads = p.ept == 8 ? kSmallThreads : kScanThreads, per = threads * p.ept;
    p.slices = (vocab + 7 + per - 1) / per;
    // lists of some 1024 elements a row in all, with room for two to four times as many
    p.cap_log2 = 5;
    while (p.cap_log2 < 11 && (p.slices << (p.cap_log2 + 1)) <= 4096) ++p.cap_log2;
    const int want = 1024 / p.slices;
    p.want = want < 4 ? 4 : (want > threads / 2 ? threads / 2 : want);
    return p;
}
size_t up16(size_t n) { return (n + 15) & ~static_cast<size_t>(15); }
size_t bytes_for(int vocab, int n_rows)
{
    const Plan p = plan_for(vocab, n_rows);
    const size_t slices = static_cast<size_t>(p.slices) * n_rows;
    return slices * sizeof(Header) + (slices << p.cap_log2) * sizeof(u64) + up16(static_cast<size_t>(n_rows) * sizeof(int));
}

template <int TYPE>
cudaError_t launch(Rows R, const Settings &S, const Plan &p, int n_rows, int32_t *token, float *prob, cudaStream_t s)
{
    auto deep = k_sample_deep<TYPE>;
    if (ctas_per_sm(reinterpret_cast<const void *>(deep), kDeepThreads, sizeof(DeepShared)) < 1) return cudaErrorInvalidConfiguration;
    static std::once_flag once[64];  // clusters of 16 are asked for, once a device
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::call_once(once[dev], [&] { cudaFuncSetAttribute(deep, cudaFuncAttributeNonPortableClusterSizeAllowed, 1); });
    const dim3 grid(p.slices, n_rows);
    int *status = status_word();
    auto scan = [&](auto kern, int threads) { return launch_pdl(kern, grid, dim3(threads), 0, s, R, S, p.want, token, prob, status); };
    const bool one = p.slices == 1;
    cudaError_t e;
    if (p.ept == 8)
        e = one ? scan(k_sample_scan<TYPE, 8, kSmallThreads, true>, kSmallThreads) : scan(k_sample_scan<TYPE, 8, kSmallThreads, false>, kSmallThreads);
    else
        e = one ? scan(k_sample_scan<TYPE, 32, kScanThreads, true>, kScanThreads) : scan(k_sample_scan<TYPE, 32, kScanThreads, false>, kScanThreads);
    if (e == cudaSuccess && !one) e = launch_pdl(k_sample_pick, dim3(n_rows), dim3(kPickThreads), 0, s, R, S, token, prob, status);
    // a row whose every candidate is in the list is always settled
    if (e == cudaSuccess && !(one && R.vocab <= R.cap))
        e = launch_pdl(deep, dim3(kDeepCtas, n_rows < kDeepClusters ? n_rows : kDeepClusters), dim3(kDeepThreads), sizeof(DeepShared), s, R,
                       S, n_rows, token, prob);
    return e;
}

inline bool aligned_to(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

}  // namespace
}  // namespace gq

using namespace gq;

extern "C" {

size_t gq_sample_workspace_bytes(int vocab, int n_rows)
{
    if (vocab < 1 || vocab > GQ_MAX_VOCAB || n_rows < 1 || n_rows > GQ_MAX_SAMPLE_ROWS) return 0;
    // of either size of slices the larger the more rows: the most of up to n_rows is that of all, or of the most
    // that take the small slices
    const int few = kFineSlices / fine_slices(vocab);
    const size_t most = few >= 1 && few < n_rows ? bytes_for(vocab, few) : 0, all = bytes_for(vocab, n_rows);
    return most > all ? most : all;
}

int gq_sample(const void *logits, long long ldl, int type, const float *temperature, const int32_t *top_k,
              const float *top_p, const float *min_p, const float *u, int32_t *token, float *prob_or_null,
              void *workspace, size_t workspace_bytes, int vocab, int n_rows, gq_stream_t stream)
{
    if (type != GQ_TYPE_F32 && type != GQ_TYPE_F16 && type != GQ_TYPE_BF16) return GQ_ERR_FORMAT;
    if (vocab < 1 || vocab > GQ_MAX_VOCAB || n_rows < 0 || n_rows > GQ_MAX_SAMPLE_ROWS || ldl < vocab || ldl > (1ll << 40)) return GQ_ERR_SHAPE;
    if (n_rows == 0) return GQ_OK;
    if (!logits || !u || !token) return GQ_ERR_NULL;
    if (!aligned_to(logits, kv::type_size(type)) || !aligned_to(temperature, 4) || !aligned_to(top_k, 4) || !aligned_to(top_p, 4) ||
        !aligned_to(min_p, 4) || !aligned_to(u, 4) || !aligned_to(token, 4) || !aligned_to(prob_or_null, 4))
        return GQ_ERR_ALIGN;
    if (!workspace || workspace_bytes < gq_sample_workspace_bytes(vocab, n_rows)) return GQ_ERR_WORKSPACE;
    if (!aligned16(workspace)) return GQ_ERR_ALIGN;
    const Plan p = plan_for(vocab, n_rows);
    const size_t slices = static_cast<size_t>(p.slices) * n_rows;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    uint8_t *const heads = ws, *const lists = heads + slices * sizeof(Header);
    const Rows R{static_cast<const uint8_t *>(logits),
                 ldl * kv::type_size(type),
                 vocab,
                 p.slices,
                 1 << p.cap_log2,
                 p.cap_log2,
                 reinterpret_cast<Header *>(heads),
                 reinterpret_cast<u64 *>(lists),
                 reinterpret_cast<int *>(lists + (slices << p.cap_log2) * sizeof(u64))};
    const Settings S{temperature, top_k, top_p, min_p, u};
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    switch (type) {
    case GQ_TYPE_F32: return status_from(launch<GQ_TYPE_F32>(R, S, p, n_rows, token, prob_or_null, s));
    case GQ_TYPE_F16: return status_from(launch<GQ_TYPE_F16>(R, S, p, n_rows, token, prob_or_null, s));
    default: return status_from(launch<GQ_TYPE_BF16>(R, S, p, n_rows, token, prob_or_null, s));
    }
}

}  // extern "C"
