// kvq_kv8.cu — decode attention of one new token a sequence over a paged fp8 K/V cache,
// grouped-query (kvq_kv8_decode).
//
// Bound by the cache's bytes: 2 (head_dim + 4) a row and KV head, against 4 head_dim operations a query
// head.  At eight query heads a KV head and the copy's rate that is 105 TFLOP/s, too much for
// the CUDA cores and little for the tensor cores, so both contractions are mma.sync
// m16n8k16 with register operands (fp16 in, fp32 out): the codes are exact in fp16, and eight query heads are
// the n of one instruction, so nothing is padded at the usual group sizes.
//   score    S[row][head]  = sum_d kcode[row][d] * Q[d][head]       A = K as it lies in memory
//   context  O[d][head]   += sum_row vcode[row][d] * W[row][head]   A = V transposed: bytes of two
//                                                                   rows zipped before they widen
// The k index of a contraction may be permuted freely if both operands are, and so may m: a lane's fragments
// are whole 16-byte pieces of a row (dims 64 c + 16 t .. of K rows g, g + 8; dims 16 g .. of V rows
// 2 t, 2 t + 1, 2 t + 8, 2 t + 9, with g = lane / 4, t = lane % 4).  Each lane loads the pieces that it reads itself
// straight into registers, the next tile's as soon as this one's are used: 8 KB in flight a warp, 12 warps an SM, no
// shared memory and no barrier in the loop.  (A ring in shared memory filled by cp.async cost its reads and
// the queue in front of them: 131072 rows, 8 KV heads x 8, 73 us against 53.)
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>

#include "kvq_internal.cuh"

namespace kvq {

namespace {

namespace cg = cooperative_groups;

constexpr unsigned kFull = 0xffffffffu;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kGroup = 16;               // rows of an instruction's tile
constexpr int kHeads = 8;                // query heads of an n block
constexpr int kIdle = 1;                 // see unit_steps
constexpr int kTeam = 8;                 // CTAs of a short unit at most (what any cluster may have)
constexpr int kTeamSteps = 4;            // places that each takes at most, or where the line's CTAs take nearly as many:
constexpr int kTeamMost = 8, kTeamMore = 5;      // at most, and more than those
constexpr float kSlack = 10.0f;          // log2 by which a weight may pass 1 before the reference moves
constexpr float kNone = -0x1.fffffep127f;        // no reference

struct Kv8Args {
    kvq_kv8_problem p;
    int group, n_hb;                     // query heads a KV head; blocks of heads a KV head
    int line;                            // CTAs of a block of heads: what the line is cut into
    int idle;                            // places of the line that stand for a unit's beginning
    int team, team_rows;                 // short units: CTAs of a unit, rows of each
    float scale;                         // sm_scale log2 e = scale 2^scale_exp, |scale| in [1, 2) or 0
    int scale_exp;
    int4* info;                          // [line * n_hb]: sequence (-1: none), KV head and last CTA of the unit that the
                                         // CTA began and did not end
    float4* part_ml;                     // [line * n_hb][2][heads of a block]: a unit's part's Level: of the one that the CTA
                                         // found begun, of the one that it left
    float* part_o;                       // [line * n_hb][2][heads of a block][D]: sum of weighted rows
    __nv_bfloat16* out;
    float* lse;
    uint32_t* status;
};

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// two e4m3 codes (the low or the high half of w) as f16x2: exact
__device__ __forceinline__ uint32_t wide_lo(uint32_t w)
{
    uint32_t r;
    asm("{.reg .b16 l, h; mov.b32 {l, h}, %1; cvt.rn.f16x2.e4m3x2 %0, l;}" : "=r"(r) : "r"(w));
    return r;
}
__device__ __forceinline__ uint32_t wide_hi(uint32_t w)
{
    uint32_t r;
    asm("{.reg .b16 l, h; mov.b32 {l, h}, %1; cvt.rn.f16x2.e4m3x2 %0, h;}" : "=r"(r) : "r"(w));
    return r;
}

__device__ __forceinline__ uint32_t pack_h2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// the 8 x 8 matrix of 16-bit elements that a warp holds (lane: row lane / 4, columns 2 (lane % 4) ..), transposed
__device__ __forceinline__ uint32_t transpose8(uint32_t x)
{
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float lg2(float x)
{
    float r;
    asm("lg2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float pow2(int k)              // k in [-126, 127]
{
    return __int_as_float((k + 127) << 23);
}

// What a part of a unit's rows leaves beside its weighted rows: x the reference of its sum, y that sum, z the reference of the
// weighted rows above x, in log2, -inf where there is none.  The rows are joined against their own reference, so that V
// rows near the ends of fp32 pass no sum, and come to the sum's with the quotient.  z is kept apart from x, whose rounding,
// where scores are large, would be the outputs'.
using Level = float4;
__device__ __forceinline__ float top_of(float m) { return m == -INFINITY ? 0.0f : m; }
// what a part counts against the reference `base` of sums (a NaN head: no reference, its sum says it)
__device__ __forceinline__ float part_weight(const Level& x, float base) { return x.y != x.y ? x.y : ex2(x.x - base); }
// the reference of a part's weighted rows against that base
__device__ __forceinline__ float rows_level(const Level& x, float base) { return (x.x - base) + x.z; }
// Weighted rows to outputs: 1 / sum, and 2^z, which may pass 2^128 where a reference lags, as two halves.
struct Finish {
    float r, half;
    __device__ __forceinline__ Finish(const Level& x)
        : r(x.y == 0.0f ? 0.0f : 1.0f / x.y), half(ex2(0.5f * x.z))
    {
    }
    __device__ __forceinline__ float operator()(float o) const { return o * r * half * half; }
    __device__ __forceinline__ void store(__nv_bfloat16* out, const float4& o) const
    {
        reinterpret_cast<__nv_bfloat162*>(out)[0] = __floats2bfloat162_rn((*this)(o.x), (*this)(o.y));
        reinterpret_cast<__nv_bfloat162*>(out)[1] = __floats2bfloat162_rn((*this)(o.z), (*this)(o.w));
    }
};
__device__ __forceinline__ float lse_of(const Level& x) { return x.y == 0.0f ? -INFINITY : (top_of(x.x) + log2f(x.y)) * kLn2; }
__device__ __forceinline__ void add_rows(float4& acc, const float4& y, float f)
{
    acc.x = fmaf(y.x, f, acc.x);
    acc.y = fmaf(y.y, f, acc.y);
    acc.z = fmaf(y.z, f, acc.z);
    acc.w = fmaf(y.w, f, acc.w);
}

// bytes of the cache, read once
__device__ __forceinline__ uint4 load16(const uint8_t* p)
{
    uint4 r;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
    return r;
}
template <int BYTES, int N>
__device__ __forceinline__ void load_piece(uint32_t (&w)[N], const uint8_t* p, bool on)
{
    static_assert(BYTES == 4 * N, "a piece is its words");
    if constexpr (N == 4) {
        const uint4 r = on ? load16(p) : make_uint4(0u, 0u, 0u, 0u);
        w[0] = r.x;
        w[1] = r.y;
        w[2] = r.z;
        w[3] = r.w;
    } else {
        uint2 r = make_uint2(0u, 0u);
        if (on) asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p));
        w[0] = r.x;
        w[1] = r.y;
    }
}

// the rows that sequence s sees: [x, y)
__device__ __forceinline__ int2 seen_rows(const kvq_kv8_problem& p, int s)
{
    const int L = min(max(p.seq_len[s], 0), p.max_seq_len);
    return make_int2(p.window > 0 ? max(0, L - p.window) : 0, L);
}

// a unit's rows begin at a multiple of 16: the last at or ahead of the first row that is seen
__host__ __device__ constexpr int first_group(int x) { return x & ~(kGroup - 1); }

// The line.  A unit (a sequence and KV head) takes a place for every STEP rows and, where there are more places than
// CTAs, kIdle places for what it costs to begin one; units follow one another, the KV heads of a sequence side by
// side.  CTA c of n has total / n places, the first total % n one more: the same work for all, whatever the lengths,
// and a partial result only where a cut falls into a unit (64 ragged sequences, 512 to 32768 rows: 198 us with splits
// of one size, which pay for their beginnings, 182 on the line, when it took their place).
template <int STEP>
__device__ __forceinline__ int unit_steps(const int2& seen) { return (seen.y - first_group(seen.x) + STEP - 1) / STEP; }
template <int STEP>
__device__ __forceinline__ int seq_places(const kvq_kv8_problem& p, int s, int idle)
{
    const int n = unit_steps<STEP>(seen_rows(p, s));
    return n > 0 ? (n + idle) * p.cache.n_kv : 0;
}

struct Line {
    int each, more;                      // places of a CTA; CTAs with one more
    __device__ int begin(int c) const { return c * each + min(c, more); }
    __device__ int cta(int place) const
    {
        const int wide = more * (each + 1);
        return place < wide ? place / (each + 1) : more + (place - wide) / each;
    }
};

// What the kernel is built from: D dims, NB blocks of eight heads, R rows a warp's tile, W warps, C CTAs an SM.
template <int D, int NB, int R, int W, int C>
struct Kv8Shape {
    static constexpr int kThreads = 32 * W;
    static constexpr int kKp = D / 64;                      // 16-byte pieces a lane holds of a K row
    static constexpr int kVp = D == 64 ? 1 : D / 128;       // and of a V row (8 bytes at 64 dims)
    static constexpr int kVw = D == 64 ? 2 : 4;             // words of such a piece
    static constexpr int kHb = NB * kHeads;                 // heads of a CTA
    static constexpr int kStep = W * R;                     // rows of a place of the line
    // the merge of the warps: weighted rows, then levels; then the same of the CTA, for its cluster
    static constexpr int kStride = D == 64 ? D : D + 4;     // of a head's weighted rows
    static constexpr int kSmem = (W * (kStride + 4) + D + 4) * kHb * 4;
    // Where dims d, d + 1 of head h are in those: pairs turn within 16 dims by the 16's number, or (64 dims) within 8 by the
    // head's, so that the lanes that write together meet no bank twice (16 sequences of 1024 rows: 13.1 us with the rows as
    // they are, 12.9 so; 7 of 3000 15.2 and 14.9)
    static __device__ __forceinline__ int place(int h, int d)
    {
        return D == 64 ? h * kStride + (d & ~7) + 2 * ((d / 2 + h / 2) & 3) : h * kStride + (d & ~15) + 2 * ((d / 2 + d / 16) & 7);
    }
};

// One CTA: a stretch of the line for one block of up to 8 NB query heads of the KV heads on it.  In each unit its
// warps take the tiles in turn, each with a softmax of its own, and are joined at the end.  TEAM: units are short; each
// one has a cluster of a.team CTAs, which take team_rows of its rows each and join their results through shared
// memory, so that there is no second launch (8 KV heads x 4, 1024 rows: 7.6 us on the line, 5.9 so; 7 sequences of 3000: 18.3
// and 14.9; 16 of 2048: 22.4 and 18.9).  GROUPED: 16 rows from a multiple of 16 are neighbours in the pool (pages of a
// multiple of 16 rows, or no table), so that a group has one address; otherwise every row has its own.
template <int D, int NB, int R, int W, int C, bool GROUPED, bool TEAM>
__global__ void __launch_bounds__(32 * W, C)
kv8_decode_kernel(const Kv8Args a)
{
    using Sh = Kv8Shape<D, NB, R, W, C>;
    constexpr int kP = Sh::kKp, kBlocks = D / 16;           // m blocks of the context, k steps of the score
    constexpr int kGroups = R / kGroup, kStep = Sh::kStep, kScan = 8;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int s_sum[W];
    __shared__ Line s_line;
    __shared__ int4 s_at[W];                                // of a warp: place, end of the stretch, sequence, place in it
    __shared__ float s_rest[W][Sh::kHb];                    // of a warp's heads: the powers of two that their scores still lack
    grid_dependency_wait();
    grid_dependents_launch();
    const kvq_kv8_problem& p = a.p;
    const int c = TEAM ? blockIdx.x / (a.team * a.n_hb) : blockIdx.x / a.n_hb;            // (TEAM: the unit)
    const int hb = TEAM ? blockIdx.x / a.team % a.n_hb : blockIdx.x % a.n_hb;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int heads = min(a.group - hb * Sh::kHb, Sh::kHb);           // query heads at hand

    // ---- this CTA's stretch of the line, and the sequence and place in it where it begins
    if constexpr (!TEAM) {
        int total = 0;
        auto chunk_places = [&](int s0, int (&v)[kScan]) {  // of the sequences from s0 + kScan * threadIdx.x on
            int sum = 0;
#pragma unroll
            for (int u = 0; u < kScan; ++u) {
                const int q = s0 + (int)threadIdx.x * kScan + u;
                v[u] = q < p.n_seq ? seq_places<kStep>(p, q, a.idle) : 0;
                sum += v[u];
            }
            return sum;
        };
        // inclusive prefix sum over the CTA, and the CTA's sum
        auto scan = [&](int v, int& all) {
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(kFull, v, o);
                if (lane >= o) v += u;
            }
            __syncthreads();
            if (lane == 31) s_sum[warp] = v;
            __syncthreads();
            all = 0;
#pragma unroll
            for (int w = 0; w < W; ++w) {
                if (w < warp) v += s_sum[w];
                all += s_sum[w];
            }
            return v;
        };
        constexpr int kChunk = Sh::kThreads * kScan;
        int v[kScan], mine = 0, incl = 0;
        if (p.n_seq == 1) {
            total = seq_places<kStep>(p, 0, a.idle);
        } else {
            for (int s0 = 0; s0 < p.n_seq; s0 += kChunk) {
                int all;
                mine = chunk_places(s0, v);
                incl = scan(mine, all);
                total += all;
            }
        }
        const int n_line = max(1, min(a.line, total));      // (short lengths: fewer stretches, none of them empty)
        const Line line{total / n_line, total % n_line};
        const int at = c < n_line ? line.begin(c) : 0, stop = c < n_line ? line.begin(c + 1) : 0;
        if (p.n_seq == 1) {
            if (threadIdx.x < W) s_at[threadIdx.x] = make_int4(at, stop, 0, at);
        } else if (at < stop) {
            int before = 0;
            for (int s0 = 0; s0 < p.n_seq; s0 += kChunk) {
                int all = total;
                if (p.n_seq > kChunk) {                     // (a single chunk's sums are still at hand)
                    mine = chunk_places(s0, v);
                    incl = scan(mine, all);
                }
                int from = before + incl - mine;
                if (at >= from && at < from + mine) {
#pragma unroll
                    for (int u = 0; u < kScan; ++u) {
                        if (at >= from && at < from + v[u])
#pragma unroll
                            for (int w = 0; w < W; ++w)
                                s_at[w] = make_int4(at, stop, s0 + (int)threadIdx.x * kScan + u, at - from);
                        from += v[u];
                    }
                }
                before += all;
                if (at < before) break;
            }
        } else if (threadIdx.x < W) {
            s_at[threadIdx.x] = make_int4(0, 0, 0, 0);
        }
        if (threadIdx.x == 0) {
            s_line = line;
            if (a.info) a.info[blockIdx.x] = make_int4(-1, 0, 0, 0);
        }
        __syncthreads();
    }

    // ---- the piece of a unit at hand: rows [first, end) of sequence s, KV head kv
    int s = 0, kv = 0, first = 0, end = 0, my_tiles = 0, part = 0;   // part: -1 a whole unit, 0 found begun, 1 begun here
    int2 seen = make_int2(0, 0);
    auto next_piece = [&]() -> bool {
        if constexpr (TEAM) return false;
        int4 q = s_at[warp];                                // place, end of the stretch, sequence, place in it
        bool found = false;
        while (q.x < q.y && !found) {
            seen = seen_rows(p, q.z);
            const int n = unit_steps<kStep>(seen), per = n + a.idle;
            if (n <= 0 || q.w >= per * p.cache.n_kv) {
                q.w = 0;
                // the next sequence that sees anything (there is one: the line goes on)
                for (++q.z;; q.z += 32) {
                    const bool some = q.z + lane >= p.n_seq || seen_rows(p, q.z + lane).y > 0;
                    const unsigned who = __ballot_sync(kFull, some);
                    if (who) {
                        q.z += __ffs(who) - 1;
                        break;
                    }
                }
                continue;
            }
            kv = q.w / per;
            const int inside = q.w - kv * per, take = min(per - inside, q.y - q.x);
            const int g0 = max(inside - a.idle, 0), g1 = max(inside + take - a.idle, 0);
            found = g1 > g0;
            if (found) {
                const int row0 = first_group(seen.x);
                s = q.z;
                first = row0 + g0 * kStep;
                end = g1 == n ? seen.y : row0 + g1 * kStep;
                const int n_tiles = (end - first + R - 1) / R;
                my_tiles = warp < n_tiles ? (n_tiles - warp + W - 1) / W : 0;
                part = g0 > 0 ? 0 : g1 < n ? 1 : -1;
                // (the CTA of the unit's last place)
                if (part == 1 && threadIdx.x == 0) a.info[blockIdx.x] = make_int4(s, kv, s_line.cta(q.x - inside + per - 1), 0);
            }
            q.x += take;
            q.w += take;
        }
        __syncwarp();
        if (lane == 0) s_at[warp] = q;
        __syncwarp();
        return found;
    };

    // Pool row of a position, or of a group's first (a pool holds fewer than 2^31): -2 where there is none
    const int pool = (int)p.cache.n_rows;
    auto pool_row = [&](int pos) -> int {
        if (!p.block_table) {
            const int64_t r = s * p.seq_stride_rows + pos;
            return r < pool ? (int)r : -2;
        }
        const int pg = pos / p.page_size;
        const int id = pg < p.max_pages ? p.block_table[(int64_t)s * p.max_pages + pg] : -1;
        return id >= 0 && ((int64_t)id + 1) * p.page_size <= pool ? id * p.page_size + (pos - pg * p.page_size) : -2;
    };
    // what a lane finds for tile i: GROUPED: the row of group lane % kGroups, else the row of lane % R; -1: none
    auto look_up = [&](int i) -> int {
        if constexpr (GROUPED) {
            const int pos = first + (warp + i * W) * R + (lane % kGroups) * kGroup;
            return pos < end ? pool_row(pos) : -1;
        } else {
            const int pos = first + (warp + i * W) * R + lane % R;
            return pos >= seen.x && pos < end ? pool_row(pos) : -1;
        }
    };
    // The tile at hand, in registers: the lane's pieces of K rows 8 e + g and of V rows 16 (e / 4) + 8 (e / 2 % 2) +
    // 2 t + e % 2, the scales of row lane % R, and the mask of the rows that may be read (zeros stand for the others).
    // Each part is loaded for tile i + 1 as soon as tile i is done with it.
    uint4 kr[2 * kGroups][kP];
    uint32_t vr[4 * kGroups][Sh::kVp][Sh::kVw];
    float k_scale, v_scale;
    uint32_t mask = 0;
    bool bad = false;
    int base[GROUPED ? kGroups : 1];                        // pool rows of the groups (GROUPED: of all lanes alike)
    bool whole = false;
    int64_t head_row = 0;                                   // the KV head's row 0 in the planes
    // where this lane's pieces of a pool row begin
    auto k_at = [&](int row) { return p.cache.k + (head_row + row) * D + 16 * t; };
    auto v_at = [&](int row) { return p.cache.v + (head_row + row) * D + (D == 64 ? 8 : 16) * g; };
    // K and the scales of tile i, found by look_up(i)
    auto load_k = [&](int i, int found) {
        bad |= found == -2;
        int row;
        bool in;
        if constexpr (GROUPED) {
            const int pos0 = first + (warp + i * W) * R;
            whole = pos0 >= seen.x && pos0 + R <= end;
#pragma unroll
            for (int j = 0; j < kGroups; ++j) {
                base[j] = __shfl_sync(kFull, found, j);
                whole = whole && base[j] >= 0 && base[j] <= pool - kGroup;
            }
            row = (lane & (kGroup - 1)) + (kGroups == 2 && lane >= kGroup ? base[kGroups - 1] : base[0]);
            if (whole) {
                mask = ~0u;
                in = true;
#pragma unroll
                for (int e = 0; e < 2 * kGroups; ++e)
#pragma unroll
                    for (int c = 0; c < kP; ++c) kr[e][c] = load16(k_at(base[e / 2] + g) + (e % 2 * 8 * D + 64 * c));
            } else {
                const int lo = seen.x - pos0, hi = end - pos0;
                const int r = lane % R, b = kGroups == 2 && r >= kGroup ? base[kGroups - 1] : base[0];
                in = r >= lo && r < hi && b >= 0 && b + (r & (kGroup - 1)) < pool;
                bad |= r >= lo && r < hi && b >= 0 && b + (r & (kGroup - 1)) >= pool;       // (no table: the pool may end anywhere)
                mask = __ballot_sync(kFull, in);
#pragma unroll
                for (int e = 0; e < 2 * kGroups; ++e) {
                    const bool on = mask >> (8 * e + g) & 1;
#pragma unroll
                    for (int c = 0; c < kP; ++c)
                        kr[e][c] = on ? load16(k_at(base[e / 2] + g) + (e % 2 * 8 * D + 64 * c)) : make_uint4(0u, 0u, 0u, 0u);
                }
            }
        } else {
            base[0] = found;
            row = found;
            in = found >= 0;
            mask = __ballot_sync(kFull, in);
#pragma unroll
            for (int e = 0; e < 2 * kGroups; ++e) {
                const int r = __shfl_sync(kFull, found, 8 * e + g);
#pragma unroll
                for (int c = 0; c < kP; ++c) kr[e][c] = r >= 0 ? load16(k_at(r) + 64 * c) : make_uint4(0u, 0u, 0u, 0u);
            }
        }
        k_scale = in ? __ldg(p.cache.k_scale + head_row + row) : 0.0f;
        v_scale = in ? __ldg(p.cache.v_scale + head_row + row) : 0.0f;
    };
    // V of the tile whose K was loaded last
    auto load_v = [&]() {
#pragma unroll
        for (int e = 0; e < 4 * kGroups; ++e) {
            constexpr int kStep = D == 64 ? 8 : 16;
            const int in_group = 8 * (e / 2 % 2) + e % 2;
            const uint8_t* src;
            bool on = true;
            if constexpr (GROUPED) {
                src = v_at(base[e / 4] + 2 * t) + in_group * D;
                if (!whole) on = mask >> (kGroup * (e / 4) + in_group + 2 * t) & 1;
            } else {
                const int r = __shfl_sync(kFull, base[0], kGroup * (e / 4) + in_group + 2 * t);
                src = v_at(r);
                on = r >= 0;
            }
#pragma unroll
            for (int c = 0; c < Sh::kVp; ++c) load_piece<kStep>(vr[e][c], src + 128 * c, on);
        }
    };
    int next = -1;
    auto begin = [&]() {                                    // the piece's first tile is on its way
        head_row = (int64_t)kv * p.cache.n_rows;
        if (my_tiles > 0) {
            load_k(0, look_up(0));
            load_v();
        }
        next = my_tiles > 1 ? look_up(1) : -1;
    };

    bool more;
    if constexpr (TEAM) {
        s = c / p.cache.n_kv;
        kv = c - s * p.cache.n_kv;
        seen = seen_rows(p, s);
        const int64_t from = first_group(seen.x) + (int64_t)(blockIdx.x % a.team) * a.team_rows;
        first = (int)min(from, (int64_t)seen.y);
        end = (int)min(from + a.team_rows, (int64_t)seen.y);
        const int n_tiles = (end - first + R - 1) / R;
        my_tiles = warp < n_tiles ? (n_tiles - warp + W - 1) / W : 0;
        more = true;
    } else {
        more = next_piece();
    }
    if (more) begin();
    while (more) {
        const int64_t head0 = (int64_t)s * p.n_qh + kv * a.group + hb * Sh::kHb;
        const int this_part = part;
        // Queries as the score's B operand.  bf16 has fp32's range, so a head is scaled by a power of two that puts
        // its largest element into [2^14, 2^15): elements down to 2^-31 of it are exact, the rest within 2^-39 of it.
        uint32_t qf[NB][kBlocks][2];
        float hs[NB][2];                                        // what a score of heads 2 t, 2 t + 1 is multiplied by
        bool wild = false;                                      // whether, for a head of the warp, that and s_rest
        int rest[NB];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            const int h = nb * kHeads + g;
            uint4 w[kP][2];
#pragma unroll
            for (int c = 0; c < kP; ++c) {
                const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) + s * p.ldq +
                                                                  ((int64_t)kv * a.group + hb * Sh::kHb + h) * D + 64 * c + 16 * t);
#pragma unroll
                for (int e = 0; e < 2; ++e) w[c][e] = h < heads ? __ldg(src + e) : make_uint4(0u, 0u, 0u, 0u);
            }
            uint32_t m = 0;                                     // |bfloat16| patterns order like their values
#pragma unroll
            for (int c = 0; c < kP; ++c)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint32_t x[4] = {w[c][e].x, w[c][e].y, w[c][e].z, w[c][e].w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) m = max(m, max(x[j] & 0x7FFFu, (x[j] >> 16) & 0x7FFFu));
                }
            m = max(m, __shfl_xor_sync(kFull, m, 1));
            m = max(m, __shfl_xor_sync(kFull, m, 2));
            // 14 - exponent; 126 is enough for the smallest heads, whose elements, multiples of 2^-133, are exact so
            const int up = min(14 - ((int)(m >> 7) - 127), 126);
            const float f = pow2(up);
#pragma unroll
            for (int c = 0; c < kP; ++c)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint32_t x[4] = {w[c][e].x, w[c][e].y, w[c][e].z, w[c][e].w};
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        qf[nb][4 * c + 2 * e + (j >> 1)][j & 1] =
                            pack_h2(__uint_as_float(x[j] << 16) * f, __uint_as_float(x[j] & 0xFFFF0000u) * f);
                }
            // A score is y scale 2^e kf, |y| < 2^32 the product of query and codes, kf the row's scale, up to 2^120.  Multiplied in
            // this order it does not overflow on the way where e <= 90, and what underflows counts less than 2^-29 in
            // the score where e >= -100; what e has beyond those (queries near the ends of fp32) comes last.
            const int e = m > 0u ? a.scale_exp - up : 0, near = min(max(e, -100), 90);
            rest[nb] = e - near;
            wild |= rest[nb] != 0;
            // (a NaN or an infinity: every score is a NaN, as all of them might be -inf, like those of rows that are not seen)
            const float back = m >= 0x7F80u ? __int_as_float(0x7FFFFFFF) : a.scale * pow2(near);
            hs[nb][0] = __shfl_sync(kFull, back, 8 * t);
            hs[nb][1] = __shfl_sync(kFull, back, 8 * t + 4);
        }
        wild = __any_sync(kFull, wild);
        if (wild) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
                if (t == 0) s_rest[warp][nb * kHeads + g] = pow2(min(max(rest[nb], -126), 127));
            __syncwarp();
        }

        float o[NB][kBlocks][4];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int b = 0; b < kBlocks; ++b)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[nb][b][e] = 0.0f;
        // Two references a head, in log2: ref of the scores, for the sum of exp2(x - ref), and above it wref of (x - ref) +
        // log2(vscale), for the weights that multiply V's codes, so that the largest of those is near 1 whatever the
        // scales, and no rounding of a large score is in a weight.  They move only when something passes them by kSlack;
        // kNone: nothing has yet.
        float ref[NB][2], wref[NB][2], sum[NB][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                ref[nb][e] = wref[nb][e] = kNone;
                sum[nb][e] = 0.0f;
            }

        for (int i = 0; i < my_tiles; ++i) {
            const int after = i + 2 < my_tiles ? look_up(i + 2) : -1;
            // rows 16 j + g (0, 1) and 16 j + g + 8 (2, 3), heads 2 t, 2 t + 1
            float x[kGroups][NB][4];
#pragma unroll
            for (int j = 0; j < kGroups; ++j)
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[j][nb][e] = 0.0f;
#pragma unroll
            for (int c = 0; c < kP; ++c)
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int j = 0; j < kGroups; ++j) {
                        const uint4 &l = kr[2 * j][c], &u = kr[2 * j + 1][c];
                        const uint32_t wl = k == 0 ? l.x : k == 1 ? l.y : k == 2 ? l.z : l.w;
                        const uint32_t wu = k == 0 ? u.x : k == 1 ? u.y : k == 2 ? u.z : u.w;
                        const uint32_t a0 = wide_lo(wl), a1 = wide_lo(wu), a2 = wide_hi(wl), a3 = wide_hi(wu);
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb)
                            mma16816(x[j][nb], a0, a1, a2, a3, qf[nb][4 * c + k][0], qf[nb][4 * c + k][1]);
                    }
            float kf[kGroups][2], lv[kGroups][2];
            const float my_lv = lg2(v_scale);
#pragma unroll
            for (int j = 0; j < kGroups; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    kf[j][e] = __shfl_sync(kFull, k_scale, 16 * j + 8 * e + g);
                    lv[j][e] = __shfl_sync(kFull, my_lv, 16 * j + 8 * e + g);
                }
            const uint32_t now = mask;
            if (i + 1 < my_tiles) load_k(i + 1, next);
            // whether a reference may have to move: the largest score with the largest V scale stands for all rows
            bool over = false;
            float top_lv = -INFINITY;
#pragma unroll
            for (int j = 0; j < kGroups; ++j) top_lv = fmaxf(top_lv, fmaxf(lv[j][0], lv[j][1]));
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float m = -INFINITY;
#pragma unroll
                    for (int j = 0; j < kGroups; ++j)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float& y = x[j][nb][2 * h + e];
                            y = y * hs[nb][e] * kf[j][h];
                            m = fmaxf(m, y);
                        }
                    const float u = m - ref[nb][e];
                    over |= u > kSlack || u + top_lv - wref[nb][e] > kSlack;
                }
            const bool some = now != ~0u;
            if (__any_sync(kFull, over) || some || wild) {      // (rare after the first tile)
                if (wild) {
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float rest = s_rest[warp][nb * kHeads + 2 * t + e];
#pragma unroll
                            for (int j = 0; j < kGroups; ++j) {
                                x[j][nb][e] *= rest;
                                x[j][nb][2 + e] *= rest;
                            }
                        }
                }
                if (some) {
#pragma unroll
                    for (int j = 0; j < kGroups; ++j)
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            if (!(now >> (16 * j + 8 * h + g) & 1)) {
                                lv[j][h] = 0.0f;
#pragma unroll
                                for (int nb = 0; nb < NB; ++nb) x[j][nb][2 * h] = x[j][nb][2 * h + 1] = -INFINITY;
                            }
                }
                // (a head's own scores only: what else brought the warp here must not change the head's bits)
                float m[NB][2];
                auto largest = [&]() {                          // over the warp's rows
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1)
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                            for (int e = 0; e < 2; ++e) m[nb][e] = fmaxf(m[nb][e], __shfl_xor_sync(kFull, m[nb][e], d));
                };
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        m[nb][e] = -INFINITY;
#pragma unroll
                        for (int j = 0; j < kGroups; ++j) m[nb][e] = fmaxf(m[nb][e], fmaxf(x[j][nb][e], x[j][nb][2 + e]));
                    }
                largest();
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float rise = m[nb][e] - ref[nb][e];
                        if (rise > kSlack) {
                            sum[nb][e] *= ex2(-rise);
                            wref[nb][e] = fmaxf(wref[nb][e] - rise, kNone);
                            ref[nb][e] = m[nb][e];
                        }
                        m[nb][e] = -INFINITY;
#pragma unroll
                        for (int j = 0; j < kGroups; ++j)
#pragma unroll
                            for (int h = 0; h < 2; ++h) m[nb][e] = fmaxf(m[nb][e], (x[j][nb][2 * h + e] - ref[nb][e]) + lv[j][h]);
                    }
                largest();
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        if (m[nb][e] - wref[nb][e] > kSlack) {
                            const float f = ex2(wref[nb][e] - m[nb][e]);
#pragma unroll
                            for (int b = 0; b < kBlocks; ++b) {
                                o[nb][b][e] *= f;
                                o[nb][b][e + 2] *= f;
                            }
                            wref[nb][e] = m[nb][e];
                        }
            }
            uint32_t w[kGroups][NB][2];
#pragma unroll
            for (int j = 0; j < kGroups; ++j)
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float u0 = x[j][nb][2 * h] - ref[nb][0], u1 = x[j][nb][2 * h + 1] - ref[nb][1];
                        sum[nb][0] += ex2(u0);
                        sum[nb][1] += ex2(u1);
                        w[j][nb][h] = transpose8(pack_h2(ex2(u0 + lv[j][h] - wref[nb][0]), ex2(u1 + lv[j][h] - wref[nb][1])));
                    }
            // context: block b of a lane is its dims 2 b and 2 b + 1 of the pieces
#pragma unroll
            for (int j = 0; j < kGroups; ++j)
#pragma unroll
                for (int c = 0; c < Sh::kVp; ++c)
#pragma unroll
                    for (int k = 0; k < Sh::kVw; ++k)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t z0 = __byte_perm(vr[4 * j][c][k], vr[4 * j + 1][c][k], h ? 0x7362 : 0x5140);
                            const uint32_t z1 = __byte_perm(vr[4 * j + 2][c][k], vr[4 * j + 3][c][k], h ? 0x7362 : 0x5140);
                            const uint32_t a0 = wide_lo(z0), a1 = wide_hi(z0), a2 = wide_lo(z1), a3 = wide_hi(z1);
#pragma unroll
                            for (int nb = 0; nb < NB; ++nb)
                                mma16816(o[nb][8 * c + 2 * k + h], a0, a1, a2, a3, w[j][nb][0], w[j][nb][1]);
                        }
            if (i + 1 < my_tiles) load_v();
            next = after;
        }
        more = next_piece();
        if (more) begin();

        // ---- the warps are joined: weighted rows, then levels
        __syncthreads();
        float* mo = reinterpret_cast<float*>(smem);             // [warp][head][kStride]
        Level* ml = reinterpret_cast<Level*>(mo + W * Sh::kHb * Sh::kStride);       // [warp][head]
        float* to = reinterpret_cast<float*>(ml + W * Sh::kHb); // [head][D], of the CTA
        Level* tl = reinterpret_cast<Level*>(to + Sh::kHb * D); // [head]
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int h = nb * kHeads + 2 * t + e;
                float l = sum[nb][e];
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l += __shfl_xor_sync(kFull, l, d);
                float* dst = mo + warp * Sh::kHb * Sh::kStride;
#pragma unroll
                for (int b = 0; b < kBlocks; ++b) {
                    const int d = D == 64 ? 8 * g + 2 * b : 128 * (b / 8) + 16 * g + 2 * (b % 8);
                    *reinterpret_cast<float2*>(dst + Sh::place(h, d)) = make_float2(o[nb][b][e], o[nb][b][e + 2]);
                }
                // a head without a row: reference -inf, sum 0; one that holds a NaN keeps it in the sum
                if (g == 0)
                    ml[warp * Sh::kHb + h] = make_float4(ref[nb][e] == kNone ? -INFINITY : ref[nb][e], l,
                                                         wref[nb][e] == kNone ? -INFINITY : wref[nb][e], 0.0f);
            }
        __syncthreads();
        for (int i = threadIdx.x; i < heads * (D / 4); i += Sh::kThreads) {
            const int h = i / (D / 4), d = i % (D / 4) * 4;
            Level all = make_float4(-INFINITY, 0.0f, -INFINITY, 0.0f);
#pragma unroll
            for (int w = 0; w < W; ++w) all.x = fmaxf(all.x, ml[w * Sh::kHb + h].x);
            const float base = top_of(all.x);
#pragma unroll
            for (int w = 0; w < W; ++w) all.z = fmaxf(all.z, rows_level(ml[w * Sh::kHb + h], base));
            const float rows_base = top_of(all.z);
            float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const Level x = ml[w * Sh::kHb + h];
                const float2 y0 = *reinterpret_cast<const float2*>(mo + w * Sh::kHb * Sh::kStride + Sh::place(h, d));
                const float2 y1 = *reinterpret_cast<const float2*>(mo + w * Sh::kHb * Sh::kStride + Sh::place(h, d + 2));
                all.y = fmaf(x.y, part_weight(x, base), all.y);
                add_rows(acc, make_float4(y0.x, y0.y, y1.x, y1.y), ex2(rows_level(x, base) - rows_base));
            }
            const int64_t row = head0 + h;
            if constexpr (TEAM) {
                *reinterpret_cast<float4*>(to + h * D + d) = acc;
                if (d == 0) tl[h] = all;
            } else if (this_part < 0) {
                Finish(all).store(a.out + row * D + d, acc);
                if (d == 0 && a.lse) a.lse[row] = lse_of(all);
            } else {
                const int64_t place = ((int64_t)blockIdx.x * 2 + this_part) * Sh::kHb + h;
                *reinterpret_cast<float4*>(a.part_o + place * D + d) = acc;
                if (d == 0) a.part_ml[place] = all;
            }
        }
    }
    if (__any_sync(kFull, bad) && lane == 0 && a.status) atomicOr(a.status, (unsigned)KVQ_DEV_BAD_PAGE);

    if constexpr (TEAM) {
        // ---- the CTAs are joined, in their order: each one a share of the elements
        const cg::cluster_group team = cg::this_cluster();
        const float* to = reinterpret_cast<const float*>(smem) + W * Sh::kHb * (Sh::kStride + 4);
        const Level* tl = reinterpret_cast<const Level*>(to + Sh::kHb * D);
        const int64_t head0 = (int64_t)s * p.n_qh + kv * a.group + hb * Sh::kHb;
        team.sync();
        for (int i = (int)team.block_rank() * Sh::kThreads + threadIdx.x; i < heads * (D / 4); i += a.team * Sh::kThreads) {
            const int h = i / (D / 4), d = i % (D / 4) * 4;
            Level x[kTeam], all = make_float4(-INFINITY, 0.0f, -INFINITY, 0.0f);
            float4 y[kTeam];
#pragma unroll
            for (int k = 0; k < kTeam; ++k) {
                if (k < a.team) {
                    x[k] = *team.map_shared_rank(tl + h, k);
                    y[k] = *reinterpret_cast<const float4*>(team.map_shared_rank(to, k) + h * D + d);
                    all.x = fmaxf(all.x, x[k].x);
                }
            }
            const float base = top_of(all.x);
#pragma unroll
            for (int k = 0; k < kTeam; ++k)
                if (k < a.team) all.z = fmaxf(all.z, rows_level(x[k], base));
            const float rows_base = top_of(all.z);
            float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int k = 0; k < kTeam; ++k) {
                if (k < a.team) {
                    all.y = fmaf(x[k].y, part_weight(x[k], base), all.y);
                    add_rows(acc, y[k], ex2(rows_level(x[k], base) - rows_base));
                }
            }
            Finish(all).store(a.out + (head0 + h) * D + d, acc);
            if (d == 0 && a.lse) a.lse[head0 + h] = lse_of(all);
        }
        team.sync();                                        // (nobody's shared memory goes before all have read it)
        return;
    }

    // ---- sequences that see nothing
    for (int q = c; q < p.n_seq; q += a.line) {
        if (seen_rows(p, q).y > 0) continue;
        for (int i = threadIdx.x; i < p.cache.n_kv * heads * (D / 2); i += Sh::kThreads) {
            const int h = i / (D / 2);
            const int64_t row = (int64_t)q * p.n_qh + h / heads * a.group + hb * Sh::kHb + h % heads;
            reinterpret_cast<uint32_t*>(a.out)[row * (D / 2) + i % (D / 2)] = 0u;
            if (i % (D / 2) == 0 && a.lse) a.lse[row] = -INFINITY;
        }
    }
}

// The parts of a unit joined, a CTA a query head: groups of D / 4 threads take the parts in turn, four of them in
// flight, with a softmax each, and are joined in their order.  The first part is what CTA c left, the others are
// what the CTAs behind it found begun.  T threads: 512 where units have many parts (131072 rows in 57 parts: the call
// 51.6 us, with 256 threads 51.5, with 128 52.8), 128 where they have few (64 ragged sequences: 182 us, with 512 threads 211).
template <int D, int T>
__global__ void __launch_bounds__(T) kv8_combine_kernel(const Kv8Args a, int n_heads)
{
    constexpr int kJoinThreads = T, kLanes = D / 4, kJoin = kJoinThreads / kLanes, kFlight = 4;
    __shared__ Level s_ml[kJoin];
    __shared__ __align__(16) float s_o[kJoin][D];
    __shared__ int4 s_unit[kJoinThreads];
    __shared__ unsigned s_some[kJoinThreads / 32];
    const kvq_kv8_problem& p = a.p;
    const int hb = blockIdx.x % a.n_hb, h = blockIdx.y;
    const int grp = threadIdx.x / kLanes, d = threadIdx.x % kLanes * 4;
    if (hb * n_heads + h >= a.group) return;
    // the units that one of some neighbouring CTAs of the line began and did not end, a CTA a thread
    const int joins = gridDim.x / a.n_hb, mine = blockIdx.x / a.n_hb;
    const int stop = (int)((mine + 1) * (int64_t)a.line / joins);
    grid_dependency_wait();
    grid_dependents_launch();
    for (int first = (int)(mine * (int64_t)a.line / joins); first < stop; first += kJoinThreads) {
        const int look = first + threadIdx.x;
        const int4 found = look < stop ? a.info[look * a.n_hb + hb] : make_int4(-1, 0, 0, 0);
        const unsigned some = __ballot_sync(kFull, found.x >= 0);
        __syncthreads();                                    // (the last round's units are done with)
        if (found.x >= 0) s_unit[threadIdx.x] = found;
        if ((threadIdx.x & 31) == 0) s_some[threadIdx.x >> 5] = some;
        __syncthreads();
        for (int k = 0; k < kJoinThreads / 32; ++k) {
            for (unsigned left = s_some[k]; left; left &= left - 1) {
                const int at = 32 * k + __ffs(left) - 1;
                const int4 unit = s_unit[at];
                const int c = first + at, n = unit.z - c + 1;
                Level all = make_float4(-INFINITY, 0.0f, -INFINITY, 0.0f);
                float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                for (int i = grp; i < n; i += kJoin * kFlight) {
                    Level x[kFlight];
                    float4 y[kFlight];
                    const Level was = all;
#pragma unroll
                    for (int u = 0; u < kFlight; ++u) {
                        const int q = i + u * kJoin;
                        const int64_t place = (((int64_t)(c + q) * a.n_hb + hb) * 2 + (q == 0)) * n_heads + h;
                        x[u] = q < n ? a.part_ml[place] : make_float4(-INFINITY, 0.0f, -INFINITY, 0.0f);
                        y[u] = q < n ? *reinterpret_cast<const float4*>(a.part_o + place * D + d)
                                     : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    }
#pragma unroll
                    for (int u = 0; u < kFlight; ++u) all.x = fmaxf(all.x, x[u].x);
                    const float base = top_of(all.x);
                    all.z = rows_level(was, base);
#pragma unroll
                    for (int u = 0; u < kFlight; ++u) all.z = fmaxf(all.z, rows_level(x[u], base));
                    const float rows_base = top_of(all.z), f0 = ex2(rows_level(was, base) - rows_base);
                    all.y *= ex2(was.x - base);
                    acc = make_float4(acc.x * f0, acc.y * f0, acc.z * f0, acc.w * f0);
#pragma unroll
                    for (int u = 0; u < kFlight; ++u) {
                        all.y = fmaf(x[u].y, part_weight(x[u], base), all.y);
                        add_rows(acc, y[u], ex2(rows_level(x[u], base) - rows_base));
                    }
                }
                __syncthreads();                            // (the last unit is written)
                *reinterpret_cast<float4*>(&s_o[grp][d]) = acc;
                if (d == 0) s_ml[grp] = all;
                __syncthreads();
                if (grp != 0) continue;
#pragma unroll
                for (int g = 1; g < kJoin; ++g) all.x = fmaxf(all.x, s_ml[g].x);
                const float base = top_of(all.x);
                all.z = -INFINITY;
#pragma unroll
                for (int g = 0; g < kJoin; ++g) all.z = fmaxf(all.z, rows_level(s_ml[g], base));
                const float rows_base = top_of(all.z);
                all.y = 0.0f;
                acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (int g = 0; g < kJoin; ++g) {
                    const Level x = s_ml[g];
                    all.y = fmaf(x.y, part_weight(x, base), all.y);
                    add_rows(acc, *reinterpret_cast<const float4*>(&s_o[g][d]), ex2(rows_level(x, base) - rows_base));
                }
                const int64_t row = (int64_t)unit.x * p.n_qh + unit.y * a.group + hb * n_heads + h;
                Finish(all).store(a.out + row * D + d, acc);
                if (d == 0 && a.lse) a.lse[row] = lse_of(all);
            }
        }
    }
}

// The kernel of a problem: blocks of eight heads a CTA (two share the rows' conversion; at 256 dims their
// accumulators do not fit), rows a tile, warps, CTAs an SM (what the registers allow: at 128 dims 168 a thread, and 16
// bytes spilled by the line's kernel; when that spilled 100, 131072 rows took 0.8 us more).
struct Kv8Plan {
    int n_hb = 1, line = 1;
    bool cuts = false;                   // whether a unit can be cut
    int joins = 1;                       // CTAs of the join, in all blocks of heads
    int idle = 0;
    int team = 0, team_rows = 0;         // short units: CTAs and rows of each; 0: the line
    size_t off_ml = 0, off_o = 0, bytes = 0;
};

template <int D, int NB, int R, int W, int C>
struct Kv8Kind {
    static constexpr int kStep = W * R, kHb = NB * kHeads;
    using Shape = Kv8Shape<D, NB, R, W, C>;
    static void plan(const kvq_kv8_problem& p, Kv8Plan& q)
    {
        const int group = p.n_qh / p.cache.n_kv;
        q.n_hb = (group + kHb - 1) / kHb;
        // places of the longest unit (a window begins a group ahead of its first row at most)
        const int64_t most = p.window > 0 ? std::min<int64_t>((int64_t)p.window + kGroup - 1, p.max_seq_len) : p.max_seq_len;
        const int64_t steps = (most + kStep - 1) / kStep, units = (int64_t)p.n_seq * p.cache.n_kv;
        const int64_t slots = (int64_t)C * sm_count();
        // units that a cluster each can take in a few places, all of them at once (clusters of any size find room for
        // 17 CTAs of 20: 64 clusters of 7 took 29 us where 448 CTAs of the line took 23)
        const int64_t room = slots * 17 / 20;
        q.team = (int)std::min<int64_t>(std::min<int64_t>(kTeam, steps), units > 0 ? room / (units * q.n_hb) : 0);
        const int64_t each = q.team > 0 ? (steps + q.team - 1) / q.team : 0;
        if (q.team > 0 && (each <= kTeamSteps || (each <= kTeamMost && each <= units * q.n_hb * steps / slots + kTeamMore))) {
            q.team = (int)((steps + each - 1) / each);
            q.team_rows = (int)each * kStep;
            return;
        }
        q.team = 0;
        q.cuts = steps > 1;
        q.idle = units * steps > (int64_t)C * sm_count() / q.n_hb ? kIdle : 0;
        q.line = (int)std::max<int64_t>(1, std::min<int64_t>(units * steps, (int64_t)C * sm_count() / q.n_hb));
        q.joins = (int)std::min<int64_t>(units, q.line) * q.n_hb;
        if (!q.cuts) return;
        const size_t ctas = (size_t)q.line * q.n_hb;
        q.off_ml = (ctas * sizeof(int4) + 255) / 256 * 256;
        q.off_o = (q.off_ml + ctas * 2 * kHb * sizeof(Level) + 255) / 256 * 256;
        q.bytes = q.off_o + ctas * 2 * kHb * D * sizeof(float);
    }
    template <bool GROUPED>
    static cudaError_t launch_team(const Kv8Args& a, cudaStream_t s)
    {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)((int64_t)a.p.n_seq * a.p.cache.n_kv * a.n_hb * a.team));
        cfg.blockDim = dim3(32 * W);
        cfg.dynamicSmemBytes = Shape::kSmem;
        cfg.stream = s;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)a.team;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[1].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        return cudaLaunchKernelEx(&cfg, kv8_decode_kernel<D, NB, R, W, C, GROUPED, true>, a);
    }
    template <bool GROUPED>
    static cudaError_t launch_as(const Kv8Args& a, const Kv8Plan& q, cudaStream_t s)
    {
        if (q.team > 0) return launch_team<GROUPED>(a, s);
        const auto kernel = kv8_decode_kernel<D, NB, R, W, C, GROUPED, false>;
        static_assert(Shape::kSmem <= 48 * 1024, "more needs an attribute of the kernel");
        const unsigned ctas = (unsigned)(a.line * a.n_hb);
        cudaError_t e = launch_dependent(kernel, dim3(ctas), dim3(32 * W), Shape::kSmem, s, a);
        if (e == cudaSuccess && q.cuts) {
            const dim3 grid((unsigned)q.joins, (unsigned)std::min(a.group, kHb));
            e = q.line >= 16 * (q.joins / q.n_hb) ? launch_dependent(kv8_combine_kernel<D, 512>, grid, dim3(512), 0, s, a, kHb)
                                                  : launch_dependent(kv8_combine_kernel<D, 128>, grid, dim3(128), 0, s, a, kHb);
        }
        return e;
    }
    static cudaError_t launch(const Kv8Args& a, const Kv8Plan& q, cudaStream_t s)
    {
        const bool grouped = !a.p.block_table || a.p.page_size % kGroup == 0;
        return grouped ? launch_as<true>(a, q, s) : launch_as<false>(a, q, s);
    }
};

// f(kind) for the kind of a problem
template <typename F>
auto of_kind(const kvq_kv8_problem& p, F f)
{
    const bool two = p.n_qh / p.cache.n_kv > kHeads;
    switch (p.cache.head_dim) {
        case 64: return two ? f(Kv8Kind<64, 2, 32, 4, 3>()) : f(Kv8Kind<64, 1, 32, 4, 4>());
        case 128: return two ? f(Kv8Kind<128, 2, 32, 4, 2>()) : f(Kv8Kind<128, 1, 32, 4, 3>());
        default: return f(Kv8Kind<256, 1, 16, 4, 2>());
    }
}

Kv8Plan plan_kv8(const kvq_kv8_problem& p)
{
    Kv8Plan q;
    of_kind(p, [&](auto kind) { kind.plan(p, q); return 0; });
    return q;
}

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

int check_problem(const kvq_kv8_problem* p, const char* E)
{
    if (!p) return set_last_error(KVQ_EINVAL, "%s: NULL problem", E);
    const kvq_kv8_cache& c = p->cache;
    if (c.head_dim != 64 && c.head_dim != 128 && c.head_dim != 256)
        return set_last_error(KVQ_EINVAL, "%s: head_dim %d not 64, 128 or 256", E, c.head_dim);
    if (p->n_seq < 0 || p->n_seq > 65535) return set_last_error(KVQ_EINVAL, "%s: n_seq outside [0, 65535]", E);
    if (c.n_kv < 1 || p->n_qh < 1 || p->n_qh % c.n_kv || p->n_qh > 65536)
        return set_last_error(KVQ_EINVAL, "%s: n_qh must be a multiple of n_kv, at most 65536", E);
    if (p->max_seq_len < 0 || p->max_seq_len > 1 << 30 || p->window < 0)
        return set_last_error(KVQ_EINVAL, "%s: max_seq_len outside [0, 2^30] or window < 0", E);
    if (!std::isfinite(p->sm_scale)) return set_last_error(KVQ_EINVAL, "%s: sm_scale is not finite", E);
    if (p->block_table ? p->max_pages < 1 || p->page_size < 1 : p->seq_stride_rows < 0)
        return set_last_error(KVQ_EINVAL, "%s: bad paging sizes", E);
    if (c.n_rows < 0 || c.n_rows > INT32_MAX) return set_last_error(KVQ_EINVAL, "%s: n_rows outside [0, 2^31)", E);
    if (p->ldq < 0) return set_last_error(KVQ_EINVAL, "%s: ldq < 0", E);
    // (the line counts places of 64 rows or more in 32 bits)
    if ((int64_t)p->n_seq * c.n_kv * (p->max_seq_len / 64 + 2) > INT32_MAX)
        return set_last_error(KVQ_EINVAL, "%s: n_seq * n_kv * max_seq_len beyond 2^37", E);
    if (p->n_seq == 0) return KVQ_OK;
    if (!p->seq_len || !p->q || !c.k || !c.k_scale || !c.v || !c.v_scale)
        return set_last_error(KVQ_EINVAL, "%s: NULL pointer", E);
    if (p->n_seq > 1 && p->ldq < (int64_t)p->n_qh * c.head_dim)
        return set_last_error(KVQ_EINVAL, "%s: ldq smaller than the heads", E);
    if (!aligned(p->q, 16) || p->ldq % 8) return set_last_error(KVQ_EALIGN, "%s: queries not 16-byte aligned", E);
    if (!aligned(c.k, 16) || !aligned(c.v, 16)) return set_last_error(KVQ_EALIGN, "%s: code planes not 16-byte aligned", E);
    if (!aligned(c.k_scale, 4) || !aligned(c.v_scale, 4) || !aligned(p->seq_len, 4) || !aligned(p->block_table, 4))
        return set_last_error(KVQ_EALIGN, "%s: an array is not 4-byte aligned", E);
    return KVQ_OK;
}

}  // namespace

}  // namespace kvq

extern "C" {

size_t kvq_kv8_decode_workspace(const kvq_kv8_problem* p)
{
    using namespace kvq;
    if (check_problem(p, "kvq_kv8_decode_workspace") != KVQ_OK || p->n_seq == 0) return 0;
    return plan_kv8(*p).bytes;
}

int kvq_kv8_decode(const kvq_kv8_problem* p, void* out, float* lse, void* workspace, size_t ws_bytes,
                   uint32_t* dev_status, kvq_stream_t stream)
{
    using namespace kvq;
    const char* E = "kvq_kv8_decode";
    if (int st = fault_injected(E)) return st;
    if (int st = check_problem(p, E)) return st;
    if (p->n_seq == 0) return KVQ_OK;
    if (!out) return set_last_error(KVQ_EINVAL, "%s: NULL out", E);
    if (!aligned(out, 16) || !aligned(lse, 4) || !aligned(dev_status, 4))
        return set_last_error(KVQ_EALIGN, "%s: out, lse or dev_status misaligned", E);
    const Kv8Plan q = plan_kv8(*p);
    if (q.bytes && (!workspace || ws_bytes < q.bytes))
        return set_last_error(KVQ_EWORKSPACE, "%s: workspace of %zu bytes, need %zu", E, workspace ? ws_bytes : (size_t)0, q.bytes);
    if (q.bytes && !aligned(workspace, 256)) return set_last_error(KVQ_EALIGN, "%s: workspace not 256-byte aligned", E);
    int scale_exp = 0;
    const float scale = (float)(2.0 * std::frexp((double)p->sm_scale * 1.4426950408889634, &scale_exp));
    Kv8Args a{*p,      p->n_qh / p->cache.n_kv, q.n_hb, q.line, q.idle, q.team, q.team_rows, scale, scale_exp - 1, nullptr, nullptr,
              nullptr, static_cast<__nv_bfloat16*>(out), lse, dev_status};
    if (q.bytes) {
        uint8_t* ws = static_cast<uint8_t*>(workspace);
        a.info = reinterpret_cast<int4*>(ws);
        a.part_ml = reinterpret_cast<Level*>(ws + q.off_ml);
        a.part_o = reinterpret_cast<float*>(ws + q.off_o);
    }
    const cudaError_t e = of_kind(*p, [&](auto kind) { return kind.launch(a, q, (cudaStream_t)stream); });
    return e == cudaSuccess ? KVQ_OK : set_last_error(KVQ_ECUDA, "%s: %s", E, cudaGetErrorString(e));
}

}  // extern "C"
