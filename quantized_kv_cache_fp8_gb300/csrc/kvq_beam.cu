// kvq_beam.cu — beam search's selection over beams and vocabulary (kvq_beam_select).
//
// With x the logits of a beam, its candidates have the values score + x_t - log sum_u exp(x_u).  One pass
// over the logits: a CTA takes a chunk of one beam's row into registers and leaves its maximum, its sum of
// exponentials and its n_out best tokens; a second kernel, a CTA a request, joins the chunks' sums to each beam's
// logarithm and picks the n_out best of all chunks' candidates.  The logits' bytes are the floor, and an exponential
// takes 0.7 of the time of a bfloat16's two.  512 rows of 128000 bfloat16, 16 of each request's 8 beams kept, take
// 40.2 us (35 the chunks, the join the rest) against 19 for the bytes: a warp spends 940 instructions on a chunk, 65% of the
// issue slots; the rest goes to waits for a chunk's loads and between its barriers, with half of the SM's warps (64
// registers) to fill them.
//
// Best k of the values that a CTA holds: k of its threads' maxima reach some level, so that nothing below it can be
// among the best k (put_floor).  What reaches it (little more than k, unless many values are equal) is gathered and
// ranked by counting.  Where it does not fit the buffer, the best are taken one by one instead (constant rows: 645 us
// for the same; maxima that many share, logits rounded to integers, 48; 300 tokens that are not -inf, side by side, 57).
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "kvq_internal.cuh"

namespace kvq {

namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxBeam = 64, kMaxOut = 128, kMaxVocab = 1 << 24;
constexpr int kBuffer = 1024;            // gathered candidates
constexpr int kVectors = 512;            // gathered vectors
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLarge = 0x1p13f;        // logits from here on are subtracted before they are scaled

struct BeamArgs {
    kvq_beam_problem p;
    int n_chunk;
    float* part_m;                       // [n_req * n_beam][n_chunk]: the chunk's largest logit
    float2* part_s;                      // [n_req * n_beam][n_chunk]: sum of exp(x - that) in two floats; NaN: not finite
    uint64_t* part_key;                  // [n_req * n_beam][n_chunk][n_out]: candidates, 0: none
    uint32_t* status;
};

// floats as unsigned integers of the same order (equal values alike: -0 is +0); never 0 for a number
__device__ __forceinline__ uint32_t ordered(float x)
{
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b ^ ((int32_t)b < 0 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t k) { return __uint_as_float(k ^ ((int32_t)k < 0 ? 0x80000000u : 0xffffffffu)); }
__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// the r-th largest of the warp's keys, counted with their multiplicity (0 if fewer are not 0)
__device__ __forceinline__ uint32_t rth_largest(uint32_t key, int r)
{
    uint32_t m = 0;
    for (int i = 0; i < r; ++i) {
        m = __reduce_max_sync(kFull, key);
        const unsigned who = __ballot_sync(kFull, key == m);
        if ((threadIdx.x & 31) == __ffs(who) - 1) key = 0;
    }
    return m;
}

// A level that k of the CTA's keys reach, one a thread (0, if fewer than k are not 0).  Up to 16: the k-th largest of the
// maxima of 32 groups of eight lanes, which little more than k keys reach.  More: the least of the warps' (k / warps)-th
// largest.  s: 32 entries, 16-byte aligned.  put_floor, a barrier, make_floor, a barrier: s[0].
__device__ __forceinline__ void put_floor(uint32_t key, int k, uint32_t* s)
{
    const int warp = threadIdx.x >> 5;
    if (k <= 16) {
#pragma unroll
        for (int o = 4; o >= 1; o >>= 1) key = max(key, __shfl_xor_sync(kFull, key, o));
        if (threadIdx.x % 8 == 0) s[threadIdx.x / 8] = key;
    } else {
        const uint32_t m = rth_largest(key, (k + kWarps - 1) / kWarps);
        if ((threadIdx.x & 31) == 0) s[warp] = m;
    }
}
__device__ __forceinline__ void make_floor(int k, uint32_t* s)
{
    if (threadIdx.x >= 32) return;                          // (the others' issue slots are for other CTAs)
    uint32_t least;
    if (k <= 16) {
        // the least of the values with fewer than k above them
        const uint32_t v = s[threadIdx.x];
        int above = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint4 q = reinterpret_cast<const uint4*>(s)[i];
            above += (q.x > v) + (q.y > v) + (q.z > v) + (q.w > v);
        }
        least = __reduce_min_sync(kFull, above < k ? v : ~0u);
    } else {
        least = __reduce_min_sync(kFull, threadIdx.x < kWarps ? s[threadIdx.x] : ~0u);
    }
    __syncwarp();
    if (threadIdx.x == 0) s[0] = least;
}

// s += x, what the addition rounds off gathered in lo (exact whichever is the larger: Knuth, 1969)
__device__ __forceinline__ void add_exact(float& s, float& lo, float x)
{
    const float t = __fadd_rn(s, x), z = __fsub_rn(t, s);
    lo += __fadd_rn(__fsub_rn(s, __fsub_rn(t, z)), __fsub_rn(x, z));
    s = t;
}

// sum += (x + lo_x) f, in two floats
__device__ __forceinline__ void add_scaled(float& sum, float& lo, float2 x, float f)
{
    const float y = x.x * f;
    lo += fmaf(x.x, f, -y) + x.y * f;
    add_exact(sum, lo, y);
}

// the warp's sum of (sum + lo), in two floats
__device__ __forceinline__ void warp_sum(float& sum, float& lo)
{
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        const float s2 = __shfl_xor_sync(kFull, sum, o), l2 = __shfl_xor_sync(kFull, lo, o);
        add_exact(sum, lo, s2);
        lo += l2;
    }
}

// score - log(s.x + s.y) in two floats, s.x > 0 finite.  The logarithm is e log 2 + 2 atanh u, u = (f - 1) / (f + 1),
// for s = 2^e f, f in [1/sqrt 2, sqrt 2): u to two floats, then 2 (u + u^3 / 3 + u^5 / 5 + ...) with the powers from the
// third on in one (|u| < 0.172: they are below 2^-8 of u, and seven terms leave 2^-37).  64-bit arithmetic takes 16
// times as long here.
__device__ __forceinline__ float2 less_log(float score, float2 s)
{
    int e = (int)(__float_as_uint(s.x) >> 23) - 127;
    float f = __uint_as_float((__float_as_uint(s.x) & 0x7FFFFFu) | 0x3F800000u);       // (sums are 1 or more, not subnormal)
    if (f > 1.41421354f) {
        f *= 0.5f;
        ++e;
    }
    const float fl = s.y * __uint_as_float((uint32_t)(127 - e) << 23);
    const float num = f - 1.0f, den = f + 1.0f;             // num is exact
    const float den_lo = (f - (den - 1.0f)) + fl;
    const float u = __fdividef(num, den);
    const float ul = __fdividef(fmaf(-u, den, num) + fl - u * den_lo, den);
    const float q = u * u;
    const float tail = u * q * fmaf(q, fmaf(q, fmaf(q, fmaf(q, fmaf(q, 1.0f / 13.0f, 1.0f / 11.0f), 1.0f / 9.0f), 1.0f / 7.0f), 0.2f), 1.0f / 3.0f);
    float hi = score, lo = 0.0f;
    add_exact(hi, lo, (float)-e * 0x1.62e4p-1f);            // log 2 = 0x1.62e4p-1 (15 bits: the product is exact) + the rest
    add_exact(hi, lo, -2.0f * u);
    lo -= fmaf((float)e, 0x1.7f7d1cp-20f, 2.0f * (fmaf(ul, q, ul) + tail));
    const float r = hi + lo;
    return make_float2(r, (hi - r) + lo);
}

// how many j below n have on(j), counted by eight lanes (a candidate a warp, counted by ballots: 41.2 us instead of 39.8)
template <typename F>
__device__ __forceinline__ int eight_sum(int n, F on)
{
    int sum = 0;
    for (int j = threadIdx.x % 8; j < n; j += 8) sum += on(j) ? 1 : 0;
#pragma unroll
    for (int o = 4; o >= 1; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
    return sum;
}

// whether beam b of request r has candidates of its own logits
__device__ __forceinline__ bool reads_logits(const kvq_beam_problem& p, int64_t row)
{
    const float s = p.score[row];
    return s > -INFINITY && s < INFINITY && !(p.finished && p.finished[row]);
}

// 16 bytes of a row as values
template <typename X>
struct Vec;
template <>
struct __align__(16) Vec<float> {
    static constexpr int kN = 4;
    uint32_t w[4];
    __device__ float get(int i) const { return __uint_as_float(w[i]); }
    __device__ void set(int i, float x) { w[i] = __float_as_uint(x); }
    __device__ float largest() const { return fmaxf(fmaxf(get(0), get(1)), fmaxf(get(2), get(3))); }
    static __device__ float load(const float* p) { return *p; }
    // elements at .. of a row of n, -inf for those outside
    __device__ void fill(const float* row, int at, int n)
    {
#pragma unroll
        for (int e = 0; e < kN; ++e) set(e, at + e >= 0 && at + e < n ? row[at + e] : -INFINITY);
    }
};
template <>
struct __align__(16) Vec<__nv_bfloat16> {
    static constexpr int kN = 8;
    uint32_t w[4];
    __device__ float get(int i) const { return __uint_as_float(i % 2 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16); }
    __device__ void set(int i, float x)                     // (a bfloat16's value)
    {
        const uint32_t b = __float_as_uint(x);
        w[i / 2] = i % 2 ? (w[i / 2] & 0xFFFFu) | (b & 0xFFFF0000u) : (w[i / 2] & 0xFFFF0000u) | b >> 16;
    }
    __device__ float largest() const                        // packed maxima pass over NaNs, as fmaxf does
    {
        uint32_t a, b;
        asm("max.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(w[0]), "r"(w[1]));
        asm("max.bf16x2 %0, %1, %2;" : "=r"(b) : "r"(w[2]), "r"(w[3]));
        asm("max.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(a), "r"(b));
        return fmaxf(__uint_as_float(a << 16), __uint_as_float(a & 0xFFFF0000u));
    }
    static __device__ float load(const __nv_bfloat16* p) { return __bfloat162float(*p); }
    __device__ void fill(const __nv_bfloat16* row, int at, int n)
    {
#pragma unroll
        for (int e = 0; e < kN; ++e) set(e, at + e >= 0 && at + e < n ? load(row + at + e) : -INFINITY);
    }
};

// sum over a vector, in two chains (packed pairs of fp32 gain 1%): of 2^(x l - c), or of 2^((x - c) l)
template <bool LARGE, typename V>
__device__ __forceinline__ float exp_sum(const V& v, float c)
{
    float acc[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < V::kN; ++i) {
        const float t = ex2(LARGE ? (v.get(i) - c) * kLog2e : fmaf(v.get(i), kLog2e, -c));
        acc[i & 1] = i < 2 ? t : acc[i & 1] + t;
    }
    return acc[0] + acc[1];
}

// 16 bytes from byte `lead` of a on, which b continues
template <typename V>
__device__ __forceinline__ V shifted(const V& a, const uint32_t (&b)[4], int lead)
{
    const bool two = lead & 8, one = lead & 4;
    uint32_t c[6], d[5];
#pragma unroll
    for (int i = 0; i < 6; ++i) c[i] = two ? (i < 2 ? a.w[i + 2] : b[i - 2 < 4 ? i - 2 : 3]) : i < 4 ? a.w[i] : b[i - 4];
#pragma unroll
    for (int i = 0; i < 5; ++i) d[i] = one ? c[i + 1] : c[i];
    V r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.w[i] = __funnelshift_r(d[i], d[i + 1], (lead & 3) * 8);
    return r;
}

// NV vectors of 16 bytes a thread, counted from the row's beginning wherever that lies, so that equal rows have equal
// sums to the last bit.  ODD: of a row that does not begin at a multiple of 16 bytes the pieces that do are loaded, and
// a vector put together from a lane's piece and the next lane's.
// The CTAs go over the rows' chunks in turn; a next chunk's vectors are on their way while this one's best are ranked.
template <typename X, int NV, bool ODD>
__global__ void __launch_bounds__(kThreads, 4) beam_chunk_kernel(const BeamArgs a)
{
    using V = Vec<X>;
    constexpr int kE = V::kN, kChunk = kThreads * NV * kE;
    __shared__ __align__(16) uint32_t s_floor[32];
    __shared__ float s_m[kWarps];
    __shared__ float2 s_sum[kWarps];
    __shared__ int2 s_count[2];                             // vectors and elements gathered, of this chunk and the next
    __shared__ uint64_t s_best[kWarps];
    __shared__ uint64_t s_key[kBuffer];
    __shared__ V s_vec[kVectors];
    __shared__ int s_at[kVectors];
    const kvq_beam_problem& p = a.p;
    grid_dependency_wait();
    grid_dependents_launch();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int k = p.n_out;
    const int rows = p.n_req * p.n_beam;

    // the chunk at hand, chunk `chunk` of row `row`: element c0 + at_of(j) begins vector j of a thread, which lies `lead`
    // bytes behind x[j] where lead is not 0 (then `after` is lane 0's piece behind the warp's last)
    V x[NV];
    uint32_t after[4];
    int lead = 0;
    auto at_of = [&](int j) { return (ODD ? (warp * NV + j) * 32 + lane : j * kThreads + tid) * kE; };
    int row = blockIdx.x / a.n_chunk, chunk = blockIdx.x - row * a.n_chunk;
    const int row_step = gridDim.x / a.n_chunk, chunk_step = gridDim.x - row_step * a.n_chunk;
    const X* src = nullptr;
    int c0 = 0;
    auto advance = [&]() {
        row += row_step;
        chunk += chunk_step;
        if (chunk >= a.n_chunk) {
            chunk -= a.n_chunk;
            ++row;
        }
    };
    // the next chunk with logits to be read, from this one on; its vectors
    auto fetch = [&]() {
        while (row < rows && !reads_logits(p, row)) advance();
        if (row >= rows) return;
        src = static_cast<const X*>(p.logits) + (int64_t)row * p.ld;
        if constexpr (ODD) lead = (int)((uintptr_t)src % 16);
        c0 = chunk * kChunk;
        const uint4* const from = reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(src) - lead);
        auto take = [](uint32_t (&w)[4], const uint4* q) {
            const uint4 v = __ldcs(q);
            w[0] = v.x;
            w[1] = v.y;
            w[2] = v.z;
            w[3] = v.w;
        };
        if (c0 + kChunk <= p.vocab && lead == 0) {
#pragma unroll
            for (int j = 0; j < NV; ++j) take(x[j].w, from + (c0 + at_of(j)) / kE);
            return;
        }
        // (pieces that lie in the row as a whole)
        auto inside = [&](int piece) { return (piece > 0 || lead == 0) && (piece + 1) * kE - lead / (int)sizeof(X) <= p.vocab; };
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int piece = (c0 + at_of(j)) / kE;
            if (inside(piece)) take(x[j].w, from + piece);
            else if (lead == 0) x[j].fill(src, c0 + at_of(j), p.vocab);
        }
        const int behind = (c0 + at_of(NV - 1)) / kE + 32;
        if (ODD && lead != 0 && lane == 0 && inside(behind)) take(after, from + behind);
    };
    auto put_together = [&](const X* row_at, int from) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            uint32_t next[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                next[i] = __shfl_sync(kFull, lane > 0 ? x[j].w[i] : j + 1 < NV ? x[j + 1 < NV ? j + 1 : j].w[i] : after[i], (lane + 1) & 31);
            // (whole, and of pieces that are)
            const int at = from + at_of(j);
            if (at > 0 && at + 2 * kE - lead / (int)sizeof(X) <= p.vocab) x[j] = shifted(x[j], next, lead);
            else x[j].fill(row_at, at, p.vocab);
        }
    };
    if (tid == 0) s_count[0] = make_int2(0, 0);
    fetch();
    for (int turn = 0; row < rows; turn ^= 1) {
        const X* const this_src = src;
        const int this_c0 = c0;
        const int64_t this_at = (int64_t)row * a.n_chunk + chunk;
        if (ODD && lead != 0) put_together(src, c0);
        float most[NV], mine = -INFINITY;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            most[j] = x[j].largest();
            mine = fmaxf(mine, most[j]);
        }
        const uint32_t my_key = mine > -INFINITY ? ordered(mine) : 0u;
        const uint32_t wm = __reduce_max_sync(kFull, my_key);
        put_floor(my_key, k, s_floor);

        // exp(y - m), m the warp's largest, as 2^(y l - c), one fused multiply-add: l = log2 e in fp32, c = m l rounded.
        // What the rounding of c took is the same factor for all and is put back below.
        const float m = wm ? unordered(wm) : -INFINITY;
        float sum = 0.0f, low = 0.0f;
        if (fabsf(m) < kLarge) {
            const float c = __fmul_rn(m, kLog2e);
#pragma unroll
            for (int j = 0; j < NV; j += 2) add_exact(sum, low, exp_sum<false>(x[j], c) + exp_sum<false>(x[j + 1], c));
        } else {
            // (without a maximum there is nothing, or a NaN)
            const float c = m == -INFINITY ? 0.0f : m;
#pragma unroll
            for (int j = 0; j < NV; j += 2) add_exact(sum, low, exp_sum<true>(x[j], c) + exp_sum<true>(x[j + 1], c));
        }
        warp_sum(sum, low);
        if (lane == 0) {
            s_m[warp] = m;
            s_sum[warp] = make_float2(sum, low);
        }
        __syncthreads();

        make_floor(k, s_floor);
        if (warp == kWarps - 1) {                               // the chunk's sum, a warp's a lane
            const float mw = lane < kWarps ? s_m[lane] : -INFINITY;
            float2 sw = lane < kWarps ? s_sum[lane] : make_float2(0.0f, 0.0f);
            float all = mw;
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) all = fmaxf(all, __shfl_xor_sync(kFull, all, o));
            // What the rounding of c took is exact as a fused multiply-add.  It is below 2^-11 in nats, so its exponential is its
            // series (to 2^-35).  The largest term is 1: it is taken out as the instruction gave it and put back, so that
            // a beam with one token left has a sum of 1.
            if (fabsf(mw) < kLarge) {
                const float r = fmaf(mw, kLog2e, -__fmul_rn(mw, kLog2e)), off = -0.6931471805599453f * r;
                add_exact(sw.x, sw.y, -ex2(r));
                sw.y = fmaf(sw.x, off * fmaf(0.5f, off, 1.0f), sw.y);
                add_exact(sw.x, sw.y, 1.0f);
            }
            float t = 0.0f, lo = 0.0f;
            // (a sum of 0 has no maximum; that of the maximum's warp stays as it is)
            if (sw.x != 0.0f) add_scaled(t, lo, sw, mw == all ? 1.0f : expf(mw - all));
            warp_sum(t, lo);
            if (lane == 0) {
                a.part_m[this_at] = all;
                a.part_s[this_at] = make_float2(t, lo);
            }
        }
        __syncthreads();

        // vectors with something at or above the floor (few): their elements are looked at together, further down
        const uint32_t floor_key = s_floor[0];
        const float least = floor_key ? unordered(floor_key) : -0x1.fffffep127f;       // (all but -inf)
        if (mine >= least) {
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (most[j] >= least) {
                    const int i = atomicAdd(&s_count[turn].x, 1);
                    if (i < kVectors) {
                        s_vec[i] = x[j];
                        s_at[i] = this_c0 + at_of(j);
                    }
                }
        }
        if (tid == 0) s_count[turn ^ 1] = make_int2(0, 0);      // (nobody counts for the next chunk yet)
        advance();
        fetch();
        __syncthreads();
        const int vecs = s_count[turn].x;
        for (int i = tid; i < min(vecs, kVectors) * kE; i += kThreads) {
            const float y = s_vec[i / kE].get(i % kE);
            if (y >= least) {
                const int at = atomicAdd(&s_count[turn].y, 1);
                if (at < kBuffer) s_key[at] = (uint64_t)ordered(y) << 32 | (uint32_t)~(s_at[i / kE] + i % kE);
            }
        }
        __syncthreads();
        const int n = s_count[turn].y;
        uint64_t* out = a.part_key + this_at * k;
        if (vecs <= kVectors && n <= kBuffer) {
            for (int i0 = 0; i0 < n; i0 += kThreads / 8) {      // eight lanes count what is above one
                const int i = i0 + tid / 8;
                const uint64_t key = s_key[min(i, n - 1)];
                const int rank = eight_sum(n, [&](int j) { return s_key[j] > key; });
                if (i < n && rank < k && tid % 8 == 0) out[rank] = key;
            }
            for (int i = n + tid; i < k; i += kThreads) out[i] = 0;
            continue;
        }
        // too many equal values: the best one by one, of a thread's elements read again
        uint64_t last = ~0ull, best = 0;
        bool stale = true;
        for (int i = 0; i < k; ++i) {
            if (stale) {
                best = 0;
                for (int t = this_c0 + tid; t < min(this_c0 + kChunk, p.vocab); t += kThreads) {
                    const float y = V::load(this_src + t);
                    const uint64_t key = y > -INFINITY ? (uint64_t)ordered(y) << 32 | (uint32_t)~t : 0;
                    if (key < last && key > best) best = key;
                }
            }
            uint64_t b = best;
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) b = max(b, (uint64_t)__shfl_xor_sync(kFull, (unsigned long long)b, o));
            __syncthreads();
            if (lane == 0) s_best[warp] = b;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < kWarps; ++w) b = max(b, s_best[w]);
            if (tid == 0) out[i] = b;
            last = b;
            stale = best == b;
        }
    }
}

// A candidate of any beam: value (as two floats, ordered), then beam (ascending), logit (descending), token (ascending)
struct Cand {
    uint64_t v, t;
};
__device__ __forceinline__ bool above(const Cand& a, const Cand& b) { return a.v > b.v || (a.v == b.v && a.t > b.t); }

__global__ void __launch_bounds__(kThreads) beam_merge_kernel(const BeamArgs a)
{
    __shared__ float2 s_base[kMaxBeam];                     // sum of exp(x - the largest logit), then score - its logarithm
    __shared__ float s_max[kMaxBeam];                       // the largest logit
    __shared__ uint8_t s_live[kMaxBeam];                    // 0: no candidates; 1: its tokens; 2: finished
    __shared__ __align__(16) uint32_t s_floor[32];
    __shared__ int s_n;
    __shared__ Cand s_best[kWarps];
    __shared__ Cand s_c[kBuffer];
    const kvq_beam_problem& p = a.p;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t row0 = (int64_t)blockIdx.x * p.n_beam;
    const int k = p.n_out, per_beam = a.n_chunk * k;
    if (tid == 0) s_n = 0;
    // (the scores and flags too: the step before this one may have written them in place)
    grid_dependency_wait();
    grid_dependents_launch();
    // A list is what a chunk left, descending; `share` threads (a power of two) take its places in turn, so that each
    // one's first is its largest.  That one is read here already (of a dead beam it is not used, and may be anything).
    // List l is chunk l / n_beam of beam l % n_beam: where one beam has all the best, they are in many groups of lanes.
    const int lists = p.n_beam * a.n_chunk;
    int share = 1;
    while (share < 32 && 2 * share * lists <= kThreads) share *= 2;
    const int list_step = kThreads / share, first = tid % list_step, place0 = tid / list_step;
    const int b_first = first % p.n_beam;
    auto key_at = [&](int l, int b, int place) { return a.part_key + (row0 + b) * per_beam + (int64_t)(l / p.n_beam) * k + place; };
    const uint64_t head_key = first < lists && place0 < k ? *key_at(first, b_first, place0) : 0;
    // the lane's first chunk of the warp's first beam likewise
    const bool one = lane < a.n_chunk;
    const int64_t at_warp = (row0 + warp) * a.n_chunk + lane;
    const float m_warp = one && warp < p.n_beam ? a.part_m[at_warp] : -INFINITY;
    const float2 s_warp = one && warp < p.n_beam ? a.part_s[at_warp] : make_float2(0.0f, 0.0f);
    float score = 0.0f;                                     // of beam `tid`
    int live = 0;
    if (tid < p.n_beam) {
        score = p.score[row0 + tid];
        const bool done = p.finished && p.finished[row0 + tid] != 0;
        if (score > -INFINITY && score < INFINITY) live = done ? 2 : 1;
        s_base[tid] = make_float2(score, 0.0f);
        s_live[tid] = (uint8_t)live;
        if (!(score < INFINITY) && a.status) atomicOr(a.status, (unsigned)KVQ_DEV_BAD_VALUE);      // NaN or +inf
    }
    __syncthreads();
    for (int b = warp; b < p.n_beam; b += kWarps) {
        if (s_live[b] != 1) continue;
        const int64_t at = (row0 + b) * a.n_chunk;
        float m0 = m_warp;
        float2 sc0 = s_warp;
        if (b != warp) {
            m0 = one ? a.part_m[at + lane] : -INFINITY;
            sc0 = one ? a.part_s[at + lane] : make_float2(0.0f, 0.0f);
        }
        float m = m0;
        for (int c = lane + 32; c < a.n_chunk; c += 32) m = fmaxf(m, a.part_m[at + c]);
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
        float s = 0.0f, lo = 0.0f;
        // (the chunk of the maximum as it is, the others by an fp32 exponential as all terms are)
        if (sc0.x != 0.0f) add_scaled(s, lo, sc0, m0 == m ? 1.0f : expf(m0 - m));
        for (int c = lane + 32; c < a.n_chunk; c += 32) {
            const float2 sc = a.part_s[at + c];
            const float mc = a.part_m[at + c];
            if (sc.x != 0.0f) add_scaled(s, lo, sc, mc == m ? 1.0f : expf(mc - m));
        }
        warp_sum(s, lo);
        if (lane == 0) {
            s_max[b] = m;
            s_base[b] = make_float2(s, lo);
        }
    }
    __syncthreads();
    if (tid < p.n_beam && s_live[tid] == 1) {
        const float2 s = s_base[tid];
        if (s.x > 0.0f) {
            s_base[tid] = less_log(score, s);
        } else {
            s_live[tid] = 0;
            if (s.x != s.x && a.status) atomicOr(a.status, (unsigned)KVQ_DEV_BAD_VALUE);
        }
    }
    __syncthreads();

    // a candidate of beam b from the key that its chunk left (a finished beam's, whatever the key: its one)
    auto candidate = [&](int b, uint64_t key) {
        Cand c{0, 0};
        const uint64_t beam = (uint64_t)(kMaxBeam - 1 - b) << 56;
        if (s_live[b] == 2) {
            c.v = (uint64_t)ordered(s_base[b].x) << 32 | ordered(0.0f);
            c.t = beam;
        } else if (key) {
            float v = unordered((uint32_t)(key >> 32)), lo = s_base[b].y;
            add_exact(v, lo, -s_max[b]);                    // (first: the largest ones' difference is small, wherever they lie)
            add_exact(v, lo, s_base[b].x);
            float hi = v + lo;                              // (both normalised: their pairs order as their sums)
            lo = (v - hi) + lo;
            if (!(hi > -INFINITY)) {                        // (beyond fp32: its parts may be NaN)
                hi = -INFINITY;
                lo = 0.0f;
            }
            c.v = (uint64_t)ordered(hi) << 32 | ordered(lo);
            c.t = beam | (key >> 32) << 24 | ((uint32_t)key & (kMaxVocab - 1));
        }
        return c;
    };
    auto item = [&](int l, int b, int place) {
        if (s_live[b] == 2) return place == 0 && l == b ? candidate(b, 0) : Cand{0, 0};
        return candidate(b, s_live[b] == 1 && place < k ? *key_at(l, b, place) : 0);
    };
    const Cand head = first >= lists ? Cand{0, 0}
                      : s_live[b_first] == 2 ? item(first, b_first, place0)
                                             : candidate(b_first, s_live[b_first] == 1 ? head_key : 0);
    uint32_t mine = (uint32_t)(head.v >> 32);               // the upper half of this thread's largest value
    for (int l = first + list_step; l < lists; l += list_step) mine = max(mine, (uint32_t)(item(l, l % p.n_beam, place0).v >> 32));
    put_floor(mine, k, s_floor);
    __syncthreads();
    make_floor(k, s_floor);
    __syncthreads();
    const uint32_t floor_key = s_floor[0];
    if (mine != 0 && mine >= floor_key) {
        for (int l = first; l < lists; l += list_step) {
            const int b = l == first ? b_first : l % p.n_beam;
            for (int i = place0; i < k; i += share) {
                const Cand c = l == first && i == place0 ? head : item(l, b, i);
                if (!c.v || (uint32_t)(c.v >> 32) < floor_key) break;
                const int at = atomicAdd(&s_n, 1);
                if (at < kBuffer) s_c[at] = c;
            }
        }
    }
    __syncthreads();
    const int64_t out0 = (int64_t)blockIdx.x * k;
    auto write = [&](int i, const Cand& c) {
        const int64_t at = out0 + i;
        if (!c.v) {
            p.out_score[at] = -INFINITY;
            p.out_token[at] = -1;
            p.out_parent[at] = -1;
            if (p.out_finished) p.out_finished[at] = 0;
            return;
        }
        const int b = kMaxBeam - 1 - (int)(c.t >> 56);
        const bool done = s_live[b] == 2;
        const int token = done ? p.pad : (int)(~(uint32_t)c.t & (kMaxVocab - 1));
        p.out_score[at] = unordered((uint32_t)(c.v >> 32));
        p.out_token[at] = token;
        p.out_parent[at] = (int)(row0 + b);
        if (p.out_finished) p.out_finished[at] = done || (p.eos >= 0 && token == p.eos);
    };
    const int n = s_n;
    if (n <= kBuffer) {
        for (int i0 = 0; i0 < n; i0 += kThreads / 8) {      // eight lanes count what is above one
            const int i = i0 + tid / 8;
            const Cand c = s_c[min(i, n - 1)];
            const int rank = eight_sum(n, [&](int j) { return above(s_c[j], c); });
            if (i < n && rank < k && tid % 8 == 0) write(rank, c);
        }
        for (int i = n + tid; i < k; i += kThreads) write(i, Cand{0, 0});
        return;
    }
    Cand last{~0ull, ~0ull}, best{0, 0};
    bool stale = true;
    for (int i = 0; i < k; ++i) {
        if (stale) {
            best = Cand{0, 0};
            for (int l = first; l < lists; l += list_step)
                for (int i = place0; i < k; i += share) {
                    const Cand c = item(l, l % p.n_beam, i);
                    if (above(last, c) && above(c, best)) best = c;
                }
        }
        Cand b = best;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) {
            const Cand u{__shfl_xor_sync(kFull, (unsigned long long)b.v, o), __shfl_xor_sync(kFull, (unsigned long long)b.t, o)};
            if (above(u, b)) b = u;
        }
        __syncthreads();
        if (lane == 0) s_best[warp] = b;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            if (above(s_best[w], b)) b = s_best[w];
        if (tid == 0) write(i, b);
        last = b;
        stale = best.v == b.v && best.t == b.t;
    }
}

struct BeamPlan {
    int nv = 1, n_chunk = 1;
    size_t off_s = 0, off_key = 0, bytes = 0;
};

BeamPlan plan_beam(const kvq_beam_problem& p)
{
    BeamPlan q;
    const int64_t rows = (int64_t)p.n_req * p.n_beam;
    const int e = p.x_type == KVQ_WEIGHT_BF16 ? 8 : 4;
    // large chunks where they fill the GPU, else small ones
    const auto chunks = [&](int nv) { return ((int64_t)p.vocab + kThreads * nv * e - 1) / (kThreads * nv * e); };
    q.nv = rows * chunks(8) >= 2 * (int64_t)sm_count() ? 8 : 2;
    q.n_chunk = (int)chunks(q.nv);
    const size_t n = (size_t)rows * q.n_chunk;
    q.off_s = (n * 4 + 255) / 256 * 256;
    q.off_key = (q.off_s + n * 8 + 255) / 256 * 256;
    q.bytes = q.off_key + n * p.n_out * 8;
    return q;
}

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

int check_problem(const kvq_beam_problem* p, const char* E)
{
    if (!p) return set_last_error(KVQ_EINVAL, "%s: NULL problem", E);
    if (p->x_type != KVQ_WEIGHT_F32 && p->x_type != KVQ_WEIGHT_BF16) return set_last_error(KVQ_EINVAL, "%s: x_type %d", E, p->x_type);
    if (p->n_req < 0 || p->n_req > 65535 || p->n_beam < 1 || p->n_beam > kMaxBeam || p->n_out < 1 || p->n_out > kMaxOut)
        return set_last_error(KVQ_EINVAL, "%s: n_req, n_beam or n_out outside [0, 65535], [1, 64], [1, 128]", E);
    if (p->vocab < 1 || p->vocab > kMaxVocab) return set_last_error(KVQ_EINVAL, "%s: vocab outside [1, 2^24]", E);
    if (p->eos < -1) return set_last_error(KVQ_EINVAL, "%s: eos < -1", E);
    if (p->ld < p->vocab) return set_last_error(KVQ_EINVAL, "%s: ld smaller than vocab", E);
    if (p->n_req == 0) return KVQ_OK;
    if (!p->logits || !p->score || !p->out_score || !p->out_token || !p->out_parent)
        return set_last_error(KVQ_EINVAL, "%s: NULL pointer", E);
    if (p->n_out != p->n_beam && (p->out_score == p->score || (p->finished && p->out_finished == p->finished)))
        return set_last_error(KVQ_EINVAL, "%s: a step in place needs n_out == n_beam", E);
    if (!aligned(p->logits, p->x_type == KVQ_WEIGHT_BF16 ? 2 : 4)) return set_last_error(KVQ_EALIGN, "%s: logits misaligned", E);
    for (const void* q : {(const void*)p->score, (const void*)p->finished, (const void*)p->out_score, (const void*)p->out_token,
                          (const void*)p->out_parent, (const void*)p->out_finished})
        if (!aligned(q, 4)) return set_last_error(KVQ_EALIGN, "%s: an array is not 4-byte aligned", E);
    return KVQ_OK;
}

template <typename X>
cudaError_t launch_chunks(const BeamArgs& a, int nv, cudaStream_t s)
{
    const int64_t items = (int64_t)a.p.n_req * a.p.n_beam * a.n_chunk;
    // (a CTA a chunk up to many: the finished beams' make the work uneven, and the GPU levels it)
    const unsigned grid = (unsigned)std::min<int64_t>(items, 64 * (int64_t)sm_count());
    const bool odd = !aligned(a.p.logits, 16) || a.p.ld * (int64_t)sizeof(X) % 16 != 0;
    const auto kernel = nv == 8 ? odd ? beam_chunk_kernel<X, 8, true> : beam_chunk_kernel<X, 8, false>
                                : odd ? beam_chunk_kernel<X, 2, true> : beam_chunk_kernel<X, 2, false>;
    return launch_dependent(kernel, dim3(grid), dim3(kThreads), 0, s, a);
}

}  // namespace

}  // namespace kvq

extern "C" {

size_t kvq_beam_select_workspace(const kvq_beam_problem* p)
{
    using namespace kvq;
    if (check_problem(p, "kvq_beam_select_workspace") != KVQ_OK || p->n_req == 0) return 0;
    return plan_beam(*p).bytes;
}

int kvq_beam_select(const kvq_beam_problem* p, void* workspace, size_t ws_bytes, uint32_t* dev_status,
                    kvq_stream_t stream)
{
    using namespace kvq;
    const char* E = "kvq_beam_select";
    if (int st = fault_injected(E)) return st;
    if (int st = check_problem(p, E)) return st;
    if (p->n_req == 0) return KVQ_OK;
    if (!aligned(dev_status, 4)) return set_last_error(KVQ_EALIGN, "%s: dev_status misaligned", E);
    const BeamPlan q = plan_beam(*p);
    if (!workspace || ws_bytes < q.bytes)
        return set_last_error(KVQ_EWORKSPACE, "%s: workspace of %zu bytes, need %zu", E, workspace ? ws_bytes : (size_t)0, q.bytes);
    if (!aligned(workspace, 256)) return set_last_error(KVQ_EALIGN, "%s: workspace not 256-byte aligned", E);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    BeamArgs a{*p, q.n_chunk, reinterpret_cast<float*>(ws), reinterpret_cast<float2*>(ws + q.off_s),
               reinterpret_cast<uint64_t*>(ws + q.off_key), dev_status};
    const cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e = p->x_type == KVQ_WEIGHT_BF16 ? launch_chunks<__nv_bfloat16>(a, q.nv, s) : launch_chunks<float>(a, q.nv, s);
    if (e == cudaSuccess) e = launch_dependent(beam_merge_kernel, dim3((unsigned)p->n_req), dim3(kThreads), 0, s, a);
    return e == cudaSuccess ? KVQ_OK : set_last_error(KVQ_ECUDA, "%s: %s", E, cudaGetErrorString(e));
}

}  // extern "C"
