// kvq_beam.cu — beam search's selection over beams and vocabulary (kvq_beam_select).
//
// With x the logits of a beam, its candidates have the values score + x_t - log sum_u exp(x_u).  One pass
// over the logits: a CTA takes a chunk of one beam's row into registers and leaves its maximum, its sum of
// exponentials and its n_out best tokens; a second kernel, a CTA a request, joins the chunks' sums to each beam's
// logarithm and picks the n_out best of all chunks' candidates.  Bound by the logits' bytes, with an exponential an
// element not far behind (two bytes at the copy's rate take as long as 0.6 of a MUFU operation).
//
// Best k of the values that a CTA holds: each warp finds the r-th largest of its threads' maxima,
// r = ceil(k / warps); at least k values reach the least of these, so that nothing below it can be among the best k.
// What reaches it (a few times k, unless many values are equal) is gathered and ranked by counting.  Where it does
// not fit the buffer, the best are taken one by one instead.
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
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLarge = 1e30f;          // logits from here on are subtracted before they are scaled

struct BeamArgs {
    kvq_beam_problem p;
    int n_chunk;
    float* part_m;                       // [n_req * n_beam][n_chunk]: the chunk's largest logit
    double* part_s;                      // [n_req * n_beam][n_chunk]: sum of exp(x - that), up to the rounding of that times log2 e; NaN: not finite
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
__device__ __forceinline__ uint64_t ordered(double x)
{
    const uint64_t b = (uint64_t)__double_as_longlong(x + 0.0);
    return b ^ ((int64_t)b < 0 ? ~0ull : 1ull << 63);
}
__device__ __forceinline__ double unordered(uint64_t k)
{
    return __longlong_as_double((long long)(k ^ ((int64_t)k < 0 ? 1ull << 63 : ~0ull)));
}

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

// whether beam b of request r has candidates of its own logits
__device__ __forceinline__ bool reads_logits(const kvq_beam_problem& p, int64_t row)
{
    const float s = p.score[row];
    return s > -INFINITY && s < INFINITY && !(p.finished && p.finished[row]);
}

template <typename X>
__device__ __forceinline__ float widen(X x);
template <>
__device__ __forceinline__ float widen(float x) { return x; }
template <>
__device__ __forceinline__ float widen(__nv_bfloat16 x) { return __bfloat162float(x); }

// VPT values a thread; VEC: rows are 16-byte aligned
template <typename X, int VPT, bool VEC>
__global__ void __launch_bounds__(kThreads) beam_chunk_kernel(const BeamArgs a)
{
    constexpr int kE = VEC ? 16 / (int)sizeof(X) : 1;       // consecutive elements a load
    constexpr int kChunk = kThreads * VPT;
    __shared__ uint32_t s_t[kWarps];
    __shared__ float s_m[kWarps];
    __shared__ double s_sum[kWarps];
    __shared__ int s_n;
    __shared__ uint64_t s_best[kWarps];
    __shared__ uint64_t s_key[kBuffer];
    const kvq_beam_problem& p = a.p;
    const int64_t row = blockIdx.x;
    grid_dependents_launch();
    if (!reads_logits(p, row)) return;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int c0 = blockIdx.y * kChunk;
    const X* src = static_cast<const X*>(p.logits) + row * p.ld;
    const int k = p.n_out;

    float x[VPT];
#pragma unroll
    for (int j = 0; j < VPT / kE; ++j) {
        const int at = c0 + (j * kThreads + tid) * kE;
        if constexpr (VEC) {
            if (at + kE <= p.vocab) {
                const uint4 w = __ldcs(reinterpret_cast<const uint4*>(src + at));
                const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if constexpr (sizeof(X) == 2) {
                        x[j * kE + 2 * e] = __uint_as_float(u[e] << 16);
                        x[j * kE + 2 * e + 1] = __uint_as_float(u[e] & 0xFFFF0000u);
                    } else {
                        x[j * kE + e] = __uint_as_float(u[e]);
                    }
                }
                continue;
            }
        }
#pragma unroll
        for (int e = 0; e < kE; ++e) x[j * kE + e] = at + e < p.vocab ? widen(src[at + e]) : -INFINITY;
    }
    auto index_of = [&](int v) { return c0 + ((v / kE) * kThreads + tid) * kE + v % kE; };

    float mine = -INFINITY;
#pragma unroll
    for (int v = 0; v < VPT; ++v) mine = fmaxf(mine, x[v]);
    const uint32_t my_key = mine > -INFINITY ? ordered(mine) : 0u;
    const uint32_t wt = rth_largest(my_key, (k + kWarps - 1) / kWarps);
    const uint32_t wm = __reduce_max_sync(kFull, my_key);
    if (lane == 0) {
        s_t[warp] = wt;
        s_m[warp] = wm ? unordered(wm) : -INFINITY;
    }
    if (tid == 0) s_n = 0;
    __syncthreads();
    uint32_t floor_key = s_t[0];
    float m = s_m[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) {
        floor_key = min(floor_key, s_t[w]);
        m = fmaxf(m, s_m[w]);
    }

    // exp(x - m) as 2^(x l - c), one fused multiply-add: l = log2 e in fp32, c = m l rounded; what the
    // rounding of c took is the same factor for all and is put back by the merge
    float sum = 0.0f;
    if (fabsf(m) < kLarge) {
        const float c = __fmul_rn(m, kLog2e);
#pragma unroll
        for (int v = 0; v < VPT; ++v) sum += ex2(fmaf(x[v], kLog2e, -c));
    } else if (m != -INFINITY) {                            // (m l may not be finite)
#pragma unroll
        for (int v = 0; v < VPT; ++v) sum += ex2((x[v] - m) * kLog2e);
    } else {
#pragma unroll
        for (int v = 0; v < VPT; ++v) sum += x[v] == -INFINITY ? 0.0f : x[v];      // nothing, or NaN
    }
    double ds = sum;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) ds += __shfl_xor_sync(kFull, ds, o);
    if (lane == 0) s_sum[warp] = ds;

    if (my_key != 0 && my_key >= floor_key) {
        const float low = floor_key ? unordered(floor_key) : -INFINITY;
#pragma unroll
        for (int v = 0; v < VPT; ++v)
            if (x[v] >= low && x[v] > -INFINITY) {
                const int i = atomicAdd(&s_n, 1);
                if (i < kBuffer) s_key[i] = (uint64_t)ordered(x[v]) << 32 | (uint32_t)~index_of(v);
            }
    }
    __syncthreads();
    const int n = s_n;
    const int64_t at = row * a.n_chunk + blockIdx.y;
    if (tid == 0) {
        double t = 0.0;
        for (int w = 0; w < kWarps; ++w) t += s_sum[w];
        a.part_m[at] = m;
        a.part_s[at] = t;
    }
    uint64_t* out = a.part_key + at * k;
    if (n <= kBuffer) {
        for (int i = tid; i < n; i += kThreads) {
            const uint64_t key = s_key[i];
            int rank = 0;
            for (int j = 0; j < n; ++j) rank += s_key[j] > key;
            if (rank < k) out[rank] = key;
        }
        for (int i = n + tid; i < k; i += kThreads) out[i] = 0;
        return;
    }
    // too many equal values: the best one by one
    uint64_t last = ~0ull, best = 0;
    bool stale = true;
    for (int i = 0; i < k; ++i) {
        if (stale) {
            best = 0;
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                const uint64_t key = x[v] > -INFINITY ? (uint64_t)ordered(x[v]) << 32 | (uint32_t)~index_of(v) : 0;
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

// A candidate of any beam: value, then beam (ascending), logit (descending), token (ascending)
struct Cand {
    uint64_t v, t;
};
__device__ __forceinline__ bool above(const Cand& a, const Cand& b) { return a.v > b.v || (a.v == b.v && a.t > b.t); }

__global__ void __launch_bounds__(kThreads) beam_merge_kernel(const BeamArgs a)
{
    __shared__ double s_base[kMaxBeam];                     // score - log sum exp
    __shared__ uint8_t s_live[kMaxBeam];                    // 0: no candidates; 1: its tokens; 2: finished
    __shared__ uint32_t s_t[kWarps];
    __shared__ int s_n;
    __shared__ Cand s_best[kWarps];
    __shared__ Cand s_c[kBuffer];
    const kvq_beam_problem& p = a.p;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t row0 = (int64_t)blockIdx.x * p.n_beam;
    const int k = p.n_out, per_beam = a.n_chunk * k;
    if (tid == 0) s_n = 0;
    grid_dependency_wait();
    for (int b = warp; b < p.n_beam; b += kWarps) {
        const int64_t row = row0 + b;
        const float score = p.score[row];
        bool bad = !(score < INFINITY);                     // NaN or +inf
        int live = 0;
        double base = score;
        if (!bad && score > -INFINITY) {
            if (p.finished && p.finished[row]) {
                live = 2;
            } else {
                float m = -INFINITY;
                for (int c = lane; c < a.n_chunk; c += 32) m = fmaxf(m, a.part_m[row * a.n_chunk + c]);
#pragma unroll
                for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
                double s = 0.0;
                for (int c = lane; c < a.n_chunk; c += 32) {
                    const double sc = a.part_s[row * a.n_chunk + c];
                    const float mc = a.part_m[row * a.n_chunk + c];
                    // (the product of two floats is exact in 64 bits, and so is the rounding that it shows)
                    const double off = fabsf(mc) < kLarge ? (double)__fmul_rn(mc, kLog2e) - (double)mc * (double)kLog2e : 0.0;
                    s += sc == 0.0 ? 0.0 : sc * exp(((double)mc - (double)m) + off * 0.6931471805599453);
                }
#pragma unroll
                for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
                bad = s != s;
                live = !bad && s > 0.0;
                if (live) base = (double)score - ((double)m + log(s));
            }
        }
        if (lane == 0) {
            s_base[b] = base;
            s_live[b] = (uint8_t)live;
            if (bad && a.status) atomicOr(a.status, (unsigned)KVQ_DEV_BAD_VALUE);
        }
    }
    __syncthreads();

    // candidate i: the chunks' of beam i / per_beam; a finished beam's first place is its one candidate
    const int total = p.n_beam * per_beam;
    auto candidate = [&](int i) {
        const int b = i / per_beam;
        Cand c{0, 0};
        const int live = s_live[b];
        const uint64_t beam = (uint64_t)(kMaxBeam - 1 - b) << 56;
        if (live == 1) {
            const uint64_t key = a.part_key[row0 * per_beam + i];
            if (key) {
                c.v = ordered((double)unordered((uint32_t)(key >> 32)) + s_base[b]);
                c.t = beam | (key >> 32) << 24 | ((uint32_t)key & (kMaxVocab - 1));
            }
        } else if (live == 2 && i == b * per_beam) {
            c.v = ordered(s_base[b]);
            c.t = beam;
        }
        return c;
    };
    Cand mine{0, 0};
    for (int i = tid; i < total; i += kThreads) {
        const Cand c = candidate(i);
        if (above(c, mine)) mine = c;
    }
    const uint32_t wt = rth_largest((uint32_t)(mine.v >> 32), (k + kWarps - 1) / kWarps);
    if (lane == 0) s_t[warp] = wt;
    __syncthreads();
    uint32_t floor_key = s_t[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) floor_key = min(floor_key, s_t[w]);
    if ((uint32_t)(mine.v >> 32) >= floor_key && mine.v) {
        for (int i = tid; i < total; i += kThreads) {
            const Cand c = candidate(i);
            if (c.v && (uint32_t)(c.v >> 32) >= floor_key) {
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
        p.out_score[at] = (float)unordered(c.v);
        p.out_token[at] = token;
        p.out_parent[at] = (int)(row0 + b);
        if (p.out_finished) p.out_finished[at] = done || (p.eos >= 0 && token == p.eos);
    };
    const int n = s_n;
    if (n <= kBuffer) {
        for (int i = tid; i < n; i += kThreads) {
            const Cand c = s_c[i];
            int rank = 0;
            for (int j = 0; j < n; ++j) rank += above(s_c[j], c);
            if (rank < k) write(rank, c);
        }
        for (int i = n + tid; i < k; i += kThreads) write(i, Cand{0, 0});
        return;
    }
    Cand last{~0ull, ~0ull}, best{0, 0};
    bool stale = true;
    for (int i = 0; i < k; ++i) {
        if (stale) {
            best = Cand{0, 0};
            for (int j = tid; j < total; j += kThreads) {
                const Cand c = candidate(j);
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
    int vpt = 8, n_chunk = 1;
    size_t off_s = 0, off_key = 0, bytes = 0;
};

BeamPlan plan_beam(const kvq_beam_problem& p)
{
    BeamPlan q;
    const int64_t rows = (int64_t)p.n_req * p.n_beam;
    const int64_t big = (p.vocab + kThreads * 32 - 1) / (kThreads * 32);
    if (rows * big >= 2 * (int64_t)sm_count()) q.vpt = 32;
    q.n_chunk = (p.vocab + kThreads * q.vpt - 1) / (kThreads * q.vpt);
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

template <typename X, bool VEC>
void launch_chunks(const BeamArgs& a, int vpt, cudaStream_t s)
{
    const dim3 grid((unsigned)(a.p.n_req * a.p.n_beam), (unsigned)a.n_chunk);     // (chunks: at most 2^24 / 2048)
    if (vpt == 32) beam_chunk_kernel<X, 32, VEC><<<grid, kThreads, 0, s>>>(a);
    else beam_chunk_kernel<X, 8, VEC><<<grid, kThreads, 0, s>>>(a);
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
    BeamArgs a{*p, q.n_chunk, reinterpret_cast<float*>(ws), reinterpret_cast<double*>(ws + q.off_s),
               reinterpret_cast<uint64_t*>(ws + q.off_key), dev_status};
    const cudaStream_t s = (cudaStream_t)stream;
    const bool bf16 = p->x_type == KVQ_WEIGHT_BF16;
    const bool vec = aligned(p->logits, 16) && p->ld % (bf16 ? 8 : 4) == 0;
    if (bf16) vec ? launch_chunks<__nv_bfloat16, true>(a, q.vpt, s) : launch_chunks<__nv_bfloat16, false>(a, q.vpt, s);
    else vec ? launch_chunks<float, true>(a, q.vpt, s) : launch_chunks<float, false>(a, q.vpt, s);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) e = launch_dependent(beam_merge_kernel, dim3((unsigned)p->n_req), dim3(kThreads), 0, s, a);
    return e == cudaSuccess ? KVQ_OK : set_last_error(KVQ_ECUDA, "%s: %s", E, cudaGetErrorString(e));
}

}  // extern "C"
