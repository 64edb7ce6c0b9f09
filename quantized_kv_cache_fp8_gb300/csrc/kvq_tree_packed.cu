// kvq_tree_packed.cu — attention of drafted trees over the fp8 tier with every (node, head) row
// of a sequence packed into tiles of NR = 64 (or 32) rows that share one pass over the cache
// (tcgen05 kind::f8f6f4; no code is converted).
//
// Per tile of 128 cache rows (M) and NR query rows (N), e4m3 operands but for one digit:
//   S^T[rows x 2 NR] = C_tile[rows x 576] . Qd^T        Qd: two digits of every query row
//   O^T[dims x NR]  += V_tile^T[dims x rows] . Wd^T      Wd: two digits of every weight
// Each 128-dim block of the latent codes is one [128 rows x 128 B] box, 128B-swizzled, read
// K-major by the scores and MN-major by the context, so one copy serves both.  The scales
// of a row stay outside: the softmax applies them to the scores in fp32 and folds the
// latent's into the weights.
//
// Digits of a query.  An e4m3 rounding keeps 4 significant bits, so q = 2^-sigma (Qd_0 + Qd_1 / 16) holds
// the 8 bits of a bfloat16 exactly (down to 2^-21 of the row's largest element).
//
// Digits of a weight.  w is on a scale that keeps the largest weight of a row between 2^kBase and 2^8.
// Wd_0 is its e4m3 rounding, with a remainder of at most 2^-4 w, or 2^-10 where w < 2^-6; Wd_1 is the
// remainder's:
//   NR = 64: in e5m2 (an MMA has a type for each operand), an image of its own summed along K, as tensor
//            memory has no room for more columns;
//   NR = 32: in e4m3, in units of 2^-4, with N columns of its own.
// Either way w is within 2^-8 of itself from 2^-5 on.
// The outputs are rounded to bfloat16 (2^-8), so more digits would not show in a single weight.  Smaller
// ones are small alone, but a long context has many: under one heavy row, the tail's weights of 2^-10 and
// less can be half of the softmax, and if each is rounded to the nearest digit they are off the same
// way together (with e4m3 digits that end at 2^-9, 32768 equal weights of half of the sum were lost whole: an
// error of 0.44 of the output).  So the remainder is rounded up or down by a level that depends on the row's
// position (dither below; NR = 64: where w < 2^-6): off by 2^-13 at most, which is 2^-19 of the largest weight, right on
// the average of any 256 neighbouring rows down to 2^-25, and the same at every call.  Errors of the tail
// then grow with the square root of its rows, 2^-11 of the output for 65536 of them.  Measured against 64
// bits with a heavy row of 0 to 99.9% of the weight before 1000 to 65536 rows that share a mean: 0.0018 to
// 0.0024 of the output's norm, the figures of the per-query form, whose weights keep 16 bits.  What it
// costs: 266.3 -> 270.8 us and 174.1 -> 176.6 us in the first two calls below (kBase 4 and kLazy 4 would take 0.4%
// off, at four times the tail's error).
//
// Softmax: one running maximum m per query row, over u = s + log2(latent scale): the weights are
// 2^(u - m + kBase), the normalizer sums 2^(s - m).  It moves only when a tile exceeds it by more
// than 2^kLazy, and for the sixteen (eight) rows of one part of the warps at a time, so O is
// rescaled rarely.  A latent scale below 2^-kTiny counts as 2^-kTiny in m (so that the normalizer
// stays finite) and its row as zero in the context.
//
// Work: the tiles of every (sequence, row tile) unit laid end to end on one line, cut into
// equal stretches, one per CTA and SM; the cuts come from the lengths on the device, so ragged
// batches are balanced and a captured call follows new lengths.  A unit inside one stretch
// is written out directly; one that a cut crosses leaves partials (m, l, o) that
// tree_combine_kernel joins (at most two per CTA).
//
// Every wait is bounded as in the other tensor-core kernels; a CTA that gives up poisons
// the rows of its stretch.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <atomic>
#include <cfloat>
#include <climits>
#include <cstring>

#include "kvq_internal.cuh"
#include "kvq_sm100.cuh"
#include "kvq_tc_common.cuh"

namespace kvq {

using namespace sm100;

namespace {

using namespace tc;

constexpr int kRT = 128;                     // cache rows per tile
constexpr int kBox = kRT * 128;              // [128 rows x 128 dims] codes
constexpr int kRopeBox = kRT * 64;
constexpr int kStages = 2;
constexpr int kSmx = 16;                     // softmax warps: lane quarter w % 4, query rows NR / 4 (w / 4) ..
constexpr int kWarpLoad = kSmx;            // TMA: the first two latent blocks and the rope key
constexpr int kWarpS = kSmx + 1;             // score MMAs (and tensor memory)
constexpr int kWarpC = kSmx + 2;             // context MMAs
constexpr int kWarpLoad2 = kSmx + 3;         // TMA: the other two
constexpr int kThreads = 32 * (kSmx + 4);
// registers a thread: of the launch's 96 the softmax takes 104 and the rest 64 (with 96 each the
// softmax spills)
constexpr int kRegsSmx = 104, kRegsRest = 64;
constexpr int kRegsNeeded = 32 * kSmx * kRegsSmx + 128 * kRegsRest;
constexpr int kBoxes = 5;                    // four latent blocks and the rope key
constexpr int kPieces = 8;                   // 16-byte pieces of a latent that each quarter of the warps clears
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLazy = 2.0f, kBase = 6.0f;  // kLazy + kBase <= 8: weights stay up to 2^8 < 448
constexpr float kTiny = 96.0f;
constexpr uint64_t kTimeoutNs = kDefaultWaitNs;   // drains
constexpr uint32_t kColO = 256;              // tensor memory: O^T of dims 128 m .. at 256 + 64 m

template <int NR>
struct Cfg {
    static constexpr int kNS = 2 * NR;                       // score columns: digit 0 rows, digit 1 rows
    static constexpr int kGR = NR / 4;                       // query rows per softmax warp
    static constexpr int kWImgs = NR / 32;                   // [128 rows x 64 B] weight images
    static constexpr int kRS = NR == 64 ? 1 : 2;             // rope key stages (64: shared memory is full)
    static constexpr uint32_t kColSL = 0, kColSR = kNS;      // latent and rope scores
    static constexpr int kQBlk = kNS * 128;
    static constexpr int kQRope = 4 * kQBlk;
    static constexpr int kQBytes = kQRope + kNS * 64;
    static constexpr int kOffRope = kStages * 4 * kBox;
    static constexpr int kOffQ = kOffRope + kRS * kRopeBox;
    static constexpr int kOffW = kOffQ + kQBytes;
    static constexpr int kOffRed = kOffW + kWImgs * kRT * 64;   // [4][NR] f32
    // per query row [NR]: gain (sm_scale log2 e 2^-sigma), -m, its last move, 2^move (or the output factor)
    static constexpr int kOffM = kOffRed + 4 * NR * 4;
    static constexpr int kOffBar = kOffM + 4 * NR * 4;
    // full[2][4], empty[2][4], rope full[2], empty[2], s_full, s_empty, p_full, o_done, q_full, drain_s, drain_c
    static constexpr int kNumBars = 2 * kStages * 4 + 2 * 2 + 7;
    static constexpr int kOffMisc = kOffBar + kNumBars * 8;     // tmem base, abort flag, start of the stretch
    static constexpr int kOffRows = kOffMisc + 32;              // [2][2][16] pool rows of a tile's copies
    static constexpr int kSmem = kOffRows + 4 * 16 * 4;
    static_assert(kSmem <= 227 * 1024, "shared memory");
    static_assert(kOffQ % 1024 == 0 && kQBlk % 1024 == 0 && kOffW % 1024 == 0 && kOffBar % 16 == 0, "swizzle atoms");
    static_assert(kColSR + kNS <= kColO, "tensor memory");
};

struct SplitInfo {                           // a unit that starts in a CTA's stretch
    int s, rt;
    int cta;                                 // that CTA; the others follow it
    int slot;                                // its partial; the others' are 2 * cta
    int pieces;                              // CTAs that share it (1: written out directly)
    int pad[3];
};

struct Args {
    CUtensorMap tm_lat, tm_rope;
    kvq_mla_tree_problem p;
    int box_rows;                            // rows a box brings: 128, or what divides the page
    int by_unit;                             // infos are indexed by unit, else by CTA
    int n_rt;                                // row tiles a sequence at most
    int page_shift;                          // log2 of the page size, -1 if it is no power of two
    float* part_ml;                          // [2 CTAs][NR][2]
    float* part_o;                           // [2 CTAs][NR][512]
    SplitInfo* info;
    __nv_bfloat16* out;
    float* lse;
    uint32_t* status;
    uint64_t wait_ns;
};

template <int NR>
struct Shared {
    using C = Cfg<NR>;
    uint8_t* base;
    __device__ uint8_t* box(int st, int b) const { return base + (st * 4 + b) * kBox; }
    __device__ uint8_t* rope(int i) const { return base + C::kOffRope + i * kRopeBox; }
    __device__ uint8_t* q() const { return base + C::kOffQ; }
    __device__ uint8_t* w() const { return base + C::kOffW; }
    __device__ float* red() const { return reinterpret_cast<float*>(base + C::kOffRed); }
    __device__ float* gain() const { return reinterpret_cast<float*>(base + C::kOffM); }
    __device__ float* neg_m() const { return gain() + NR; }
    __device__ float* move() const { return gain() + 2 * NR; }
    __device__ float* factor() const { return gain() + 3 * NR; }
    __device__ uint64_t* bar(int i) const { return reinterpret_cast<uint64_t*>(base + C::kOffBar) + i; }
    __device__ uint64_t* full(int st, int b) const { return b < 4 ? bar(st * 4 + b) : bar(16 + st); }
    __device__ uint64_t* empty(int st, int b) const { return b < 4 ? bar(8 + st * 4 + b) : bar(18 + st); }
    __device__ uint64_t* s_full() const { return bar(20); }
    __device__ uint64_t* s_empty() const { return bar(21); }
    __device__ uint64_t* p_full() const { return bar(22); }
    __device__ uint64_t* o_done() const { return bar(23); }
    __device__ uint64_t* q_full() const { return bar(24); }
    __device__ uint64_t* drain_s() const { return bar(25); }
    __device__ uint64_t* drain_c() const { return bar(26); }
    __device__ uint32_t* tmem_base() const { return reinterpret_cast<uint32_t*>(base + C::kOffMisc); }
    __device__ volatile int* abort_flag() const { return reinterpret_cast<volatile int*>(base + C::kOffMisc + 4); }
    __device__ volatile int64_t* start_off() const { return reinterpret_cast<volatile int64_t*>(base + C::kOffMisc + 8); }
    __device__ volatile int* copy_rows(int i) const { return reinterpret_cast<volatile int*>(base + C::kOffRows) + 16 * i; }
    __device__ volatile int* start_seq() const { return reinterpret_cast<volatile int*>(base + C::kOffMisc + 16); }
};

// Wait for a phase, bounded by %globaltimer.  The one-thread roles poll (kSpin); the 512 softmax
// threads sleep in try_wait, so that their polls stay out of the shared memory pipe (a limit
// below 100 us, set only to exercise the failure path, always polls).
template <bool kSpin, int NR>
__device__ __forceinline__ bool wait_bar(const Shared<NR>& sh, uint64_t* bar, uint32_t parity, const Args& a)
{
    const bool spin = kSpin || a.wait_ns < 100000;
    if (spin ? mbar_test_wait(bar, parity) : mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    for (;;) {
#pragma unroll 1
        for (int k = 0; k < (kSpin ? 32 : 4); ++k)
            if (spin ? mbar_test_wait(bar, parity) : mbar_try_wait(bar, parity)) return true;
        if (*sh.abort_flag()) return false;
        if (globaltimer_ns() - t0 > a.wait_ns) {
            *sh.abort_flag() = 1;
            return false;
        }
    }
}
constexpr bool kSmxSpin = false, kRoleSpin = true;

__device__ __forceinline__ void smx_barrier() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kSmx) : "memory"); }

// barrier `id` of `n` threads; true if `v` holds in any of them
template <int n>
__device__ __forceinline__ bool barrier_any(int id, bool v)
{
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
        "barrier.cta.red.or.pred p, %2, %3, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r) : "r"((uint32_t)v), "r"(id), "n"(n) : "memory");
    return r != 0;
}
// the four warps of part hp (every lane quarter of the same query rows)
__device__ __forceinline__ void part_barrier(int hp) { asm volatile("bar.sync %0, 128;" ::"r"(2 + hp) : "memory"); }

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// two floats in one register pair, and the arithmetic that Blackwell does on them at once
typedef uint64_t f32x2;
__device__ __forceinline__ f32x2 pack2(float lo, float hi)
{
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 unpack2(f32x2 v)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c)
{
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b)
{
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b)
{
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// maximum of three (a NaN is passed over)
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// `shift`: log2 of the page size, -1 if it is no power of two (every softmax thread does this for each of
// its rows, where a division shows: four trees below, pages of 64: 281 us with it, 273 without)
__device__ __forceinline__ int64_t tree_pool_row(const kvq_mla_tree_problem& p, int s, int t, int shift)
{
    if (!p.block_table) return (int64_t)s * p.seq_stride_rows + t;
    const int page = shift >= 0 ? t >> shift : t / p.page_size;
    if (page >= p.max_pages) return -1;
    const int pid = p.block_table[(int64_t)s * p.max_pages + page];
    return pid < 0 ? -1 : (int64_t)pid * p.page_size + (t - page * p.page_size);
}

// ---- the line of tiles --------------------------------------------------------------------
// A unit takes kUnitCost places on the line before its tiles: what a CTA pays to begin another unit
// (epilogue, query image, refill of the pipeline: 25 thousand cycles of a full tile's 4300).  Every
// stretch begins one anyway, so these places even out the stretches with several units.  Full tiles
// with 4, 5, 6, 7 places: 32 ragged trees of 17.1 M pairs of node and row 2182, 2127, 2100, 2084 us, 32 units of 32 tiles 44.4, 44.6,
// 44.4, 46.9; half tiles, two units of 256: 25.0, 24.9, 28.6, 26.8.
template <int NR>
constexpr int kUnitCost = NR == 64 ? 6 : 4;

template <int NR>
__device__ __forceinline__ int64_t seq_places(const kvq_mla_tree_problem& p, int s)
{
    const int2 sh = tree_seq_shape(p, s);
    const int nt = (sh.x + kRT - 1) / kRT;
    return nt == 0 ? 0 : (int64_t)(nt + kUnitCost<NR>) * (((int64_t)sh.y * p.n_heads + NR - 1) / NR);
}

// where the stretch of CTA g of G begins on a line of `total` places
__device__ __forceinline__ int64_t cut(int64_t total, int g, int G) { return total * g / G; }

// the segments of a stretch: row tile rt of sequence s, its tiles [tile, end)
template <int NR>
struct Walk {
    int left;                                // places of the stretch from this unit's first one in it on
    int s, rt, at, tile, end, nt, n_rt, L, n;

    __device__ __forceinline__ void shape(const kvq_mla_tree_problem& p)
    {
        const int2 sh = tree_seq_shape(p, s);
        L = sh.x;
        n = sh.y;
        nt = (L + kRT - 1) / kRT;
        n_rt = (int)(((int64_t)n * p.n_heads + NR - 1) / NR);
    }
    __device__ __forceinline__ int places() const { return min(nt + kUnitCost<NR> - at, left); }
    __device__ __forceinline__ void tiles()
    {
        tile = max(at - kUnitCost<NR>, 0);
        end = max(at + places() - kUnitCost<NR>, 0);
    }
    __device__ __forceinline__ void step(const kvq_mla_tree_problem& p)
    {
        left -= places();
        at = 0;
        if (left <= 0) return;
        if (++rt == n_rt) {
            rt = 0;
            do {
                ++s;
                shape(p);
            } while (nt == 0 || n_rt == 0);               // (there is a place left, so a sequence with tiles)
        }
        tiles();
    }
    __device__ __forceinline__ void next(const kvq_mla_tree_problem& p)
    {
        do step(p); while (left > 0 && tile == end);      // (a stretch may end among a unit's first places)
    }
    __device__ __forceinline__ Walk(const kvq_mla_tree_problem& p, int s0, int64_t off, int64_t count)
        : left((int)count), s(s0), at(0), tile(0), end(0)
    {
        if (left <= 0) return;
        shape(p);
        if (off <= INT32_MAX) {                           // (a 64-bit division takes microseconds)
            rt = (int)off / (nt + kUnitCost<NR>);
            at = (int)off % (nt + kUnitCost<NR>);
        } else {
            rt = (int)(off / (nt + kUnitCost<NR>));
            at = (int)(off % (nt + kUnitCost<NR>));
        }
        tiles();
        if (tile == end) next(p);
    }
    __device__ __forceinline__ bool more() const { return left > 0; }
    // the place behind this unit's last one, of a stretch that ends at `stretch_end`
    __device__ __forceinline__ int64_t unit_end(int64_t stretch_end) const { return stretch_end - left - at + nt + kUnitCost<NR>; }
};

// ---- digits and queries -------------------------------------------------------------------
// Two values of a query -> their two e4m3 digits, the second in units of 1/16.  The value passes through
// binary16 (a query's 8 bits exactly), where the first digit's remainder is exact.
__device__ __forceinline__ void query_digits(float2 v, uint32_t& d0, uint32_t& d1)
{
    const __half2 h = __float22half2_rn(v);
    const __nv_fp8x2_storage_t c = __nv_cvt_halfraw2_to_fp8x2(h, __NV_SATFINITE, __NV_E4M3);
    const __half2 r = __hsub2(h, __half2(__nv_cvt_fp8x2_to_halfraw2(c, __NV_E4M3)));
    d0 = c;
    d1 = __nv_cvt_halfraw2_to_fp8x2(__hmul2(r, __half2half2(__ushort_as_half(0x4C00))), __NV_SATFINITE, __NV_E4M3);   // 16
}

// What a cache row's second digits are rounded with (the same bits in both halves): row t of the
// sequence takes the level 157 t mod 256 of 256 equidistant ones, so that any 256 rows in a row have
// each level once.  NR = 64: the level, added below the digit's last bit; NR = 32: (2 level - 255) 2^-18
// as binary16, from -1/2 to 1/2 of the smallest step of e4m3.
template <int NR>
__device__ __forceinline__ uint32_t dither(int t)
{
    const uint32_t level = (157u * (uint32_t)t) & 255u;
    if (NR == 64) return level * 0x10001u;
    const __half2 d = __half2half2(__float2half_rn((float)(2 * (int)level - 255) * 0x1p-18f));
    uint32_t r;
    memcpy(&r, &d, 4);
    return r;
}

// Four weights -> their two digits, a byte each (0 gives 0).  A weight passes through binary16 (2^-12 of
// it, or 2^-25), where the first digit's remainder r is exact.
template <int NR>
__device__ __forceinline__ void weight_digits(float2 a, float2 b, uint32_t dith, uint32_t& d0, uint32_t& d1)
{
    const __half2 v[2] = {__float22half2_rn(a), __float22half2_rn(b)};
    uint32_t c[2], o[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        c[e] = __nv_cvt_halfraw2_to_fp8x2(v[e], __NV_SATFINITE, __NV_E4M3);
        const __half2 r = __hsub2(v[e], __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)c[e], __NV_E4M3)));
        if constexpr (NR == 64) {
            // e5m2 is the upper byte of binary16: r rounded to the nearest where the weight is 2^-6 or more, else by
            // the row's level (a NaN's pattern, 0x7FFF, carries no further than its own half)
            uint32_t bits;
            memcpy(&bits, &r, 4);
            const uint32_t small = __hlt2_mask(v[e], __half2half2(__ushort_as_half(0x2400)));      // 2^-6
            o[e] = bits + ((small & dith) | (~small & 0x00800080u));
        } else {
            __half2 off;
            memcpy(&off, &dith, 4);
            o[e] = __nv_cvt_halfraw2_to_fp8x2(__hfma2(r, __half2half2(__ushort_as_half(0x4C00)), off), __NV_SATFINITE, __NV_E4M3);   // 16 r
        }
    }
    d0 = c[0] | c[1] << 16;
    d1 = NR == 64 ? prmt(o[0], o[1], 0x7531u) : o[0] | o[1] << 16;
}

// One warp: query rows r0 + i, i = warp, warp + 16, .. (of the sequence's n * H; zero from `rows` on)
// into rows i and NR + i of the Q image.  Lane: 16 latent dims, and (lane < 16) 4 rope dims.  sigma
// puts the row's largest element in [128, 256); a NaN or an infinity in the row makes its gain, and so
// its scores, NaN, and its digits zeros.
template <int NR>
__device__ __forceinline__ void write_queries(const Shared<NR>& sh, const kvq_mla_tree_problem& p, int s, int64_t r0,
                                              int64_t rows, int warp, int lane)
{
    using C = Cfg<NR>;
    constexpr int kRows = NR / kSmx;
    uint32_t w[kRows][10];                       // bf16 pairs, every row's loads in flight at once
#pragma unroll
    for (int n = 0; n < kRows; ++n) {
        const int i = warp + kSmx * n;
        uint4 a = make_uint4(0u, 0u, 0u, 0u), b = a;
        uint2 c = make_uint2(0u, 0u);
        if (i < rows) {
            const int64_t row = (int64_t)s * p.n_q * p.n_heads + r0 + i;
            const uint4* ql = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q_lat) + row * p.ldq_lat) + 2 * lane;
            a = __ldg(ql);
            b = __ldg(ql + 1);
            if (lane < 16) c = __ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.q_rope) + row * p.ldq_rope) + lane);
        }
        w[n][0] = a.x; w[n][1] = a.y; w[n][2] = a.z; w[n][3] = a.w;
        w[n][4] = b.x; w[n][5] = b.y; w[n][6] = b.z; w[n][7] = b.w;
        w[n][8] = c.x; w[n][9] = c.y;
    }
#pragma unroll
    for (int n = 0; n < kRows; ++n) {
        const int i = warp + kSmx * n;
        // the largest exponent: of bf16 patterns without sign, the largest pattern's
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < 10; ++e) m = __vmaxu2(m, w[n][e] & 0x7FFF7FFFu);
        m = max(m & 0xFFFFu, m >> 16);
        m = __reduce_max_sync(kFull, m);
        if (m >= 0x7F80u) {
            // the row's gain says NaN; its digits are zeros, so that the scores of a row tell only of its codes
#pragma unroll
            for (int e = 0; e < 10; ++e) w[n][e] = 0;
        }
        const int sigma = m != 0 ? min(100, max(-120, 7 - ((int)(m >> 7) - 127))) : 0;
        const float scale = __int_as_float((127 + sigma) << 23);
        uint32_t d0[5], d1[5];
#pragma unroll
        for (int e = 0; e < 5; ++e) {
            uint32_t a0, a1, b0, b1;
            const uint32_t x = w[n][2 * e], y = w[n][2 * e + 1];
            query_digits(make_float2(__uint_as_float(x << 16) * scale, __uint_as_float(x & 0xFFFF0000u) * scale), a0, a1);
            query_digits(make_float2(__uint_as_float(y << 16) * scale, __uint_as_float(y & 0xFFFF0000u) * scale), b0, b1);
            d0[e] = a0 | b0 << 16;
            d1[e] = a1 | b1 << 16;
        }
        uint8_t* img = sh.q() + (lane >> 3) * C::kQBlk;
        *reinterpret_cast<uint4*>(img + sw128(i, lane & 7)) = make_uint4(d0[0], d0[1], d0[2], d0[3]);
        *reinterpret_cast<uint4*>(img + sw128(NR + i, lane & 7)) = make_uint4(d1[0], d1[1], d1[2], d1[3]);
        if (lane < 16) {
            uint8_t* rp = sh.q() + C::kQRope;
            const int at = (((lane >> 2) ^ ((i >> 1) & 3)) << 4) + 4 * (lane & 3);      // (NR + i has the same swizzle)
            *reinterpret_cast<uint32_t*>(rp + i * 64 + at) = d0[4];
            *reinterpret_cast<uint32_t*>(rp + (NR + i) * 64 + at) = d1[4];
        }
        if (lane == 0) sh.gain()[i] = m < 0x7F80u ? p.sm_scale * kLog2e * __int_as_float((127 - sigma) << 23) : NAN;
    }
}

// ---- codes that no encoder writes -----------------------------------------------------------
// the 16-byte piece pc of row t: pc < 32 latent block pc / 8, then the rope key's four
template <int NR>
__device__ __forceinline__ uint4* row_piece(const Shared<NR>& sh, int st, int rst, int t, int pc)
{
    return reinterpret_cast<uint4*>(pc < 32 ? sh.box(st, pc >> 3) + t * 128 + (((pc & 7) ^ (t & 7)) << 4)
                                            : sh.rope(rst) + t * 64 + (((pc - 32) ^ ((t >> 1) & 3)) << 4));
}

__device__ __forceinline__ uint32_t clear_unwritten(uint32_t w)
{
    return w & ~prmt((w & 0x7F7F7F7Fu) + 0x01010101u, 0u, 0xBA98u);     // bytes S.1111.111 -> 0
}
__device__ __forceinline__ uint4 clear_unwritten(const uint4& v)
{
    return make_uint4(clear_unwritten(v.x), clear_unwritten(v.y), clear_unwritten(v.z), clear_unwritten(v.w));
}

// the latent's pieces of part hp of row t cleared of the pattern in place, so that the context
// reads it as 0 (whether another part has cleared its pieces yet makes no difference to rescore)
template <int NR>
__device__ __noinline__ void clear_row(const Shared<NR>& sh, int st, int t, int hp)
{
    for (int pc = kPieces * hp; pc < kPieces * hp + kPieces; ++pc) {
        uint4* ptr = row_piece(sh, st, 0, t, pc);
        *ptr = clear_unwritten(*ptr);
    }
}

// q . row from the codes with the pattern read as 0, in fp32, in units of the row's gain
template <int NR>
__device__ __noinline__ float rescore(const Shared<NR>& sh, const kvq_mla_tree_problem& p, int st, int rst, int t,
                                      int64_t row, float gain, float ls, float rs)
{
    const __nv_bfloat16* ql = static_cast<const __nv_bfloat16*>(p.q_lat) + row * p.ldq_lat;
    const __nv_bfloat16* qr = static_cast<const __nv_bfloat16*>(p.q_rope) + row * p.ldq_rope;
    float al = 0.0f, ar = 0.0f;
    for (int pc = 0; pc < 36; ++pc) {
        const uint4 v = clear_unwritten(*row_piece(sh, st, rst, t, pc));
        const uint32_t wd[4] = {v.x, v.y, v.z, v.w};
        const __nv_bfloat16* q = pc < 32 ? ql + 16 * pc : qr + 16 * (pc - 32);
        float acc = 0.0f;
        for (int e = 0; e < 16; ++e) {
            const float c = __half2float(__half(__nv_cvt_fp8_to_halfraw(
                (__nv_fp8_storage_t)((wd[e >> 2] >> (8 * (e & 3))) & 0xFFu), __NV_E4M3)));
            acc = fmaf(__bfloat162float(q[e]), c, acc);
        }
        if (pc < 32) al += acc;
        else ar += acc;
    }
    return gain != 0.0f ? fmaf(ls, al, rs * ar) * (p.sm_scale * kLog2e / gain) : 0.0f;
}

// One stage of a 4 x 4 transposition among four neighbouring lanes, for every group of four values:
// value index bit B and lane bit B change places.
template <int B, int N>
__device__ __forceinline__ void swap_dims(float (&v)[N], int lane)
{
    const bool hi = (lane & B) != 0;
#pragma unroll
    for (int e = 0; e < N; ++e) {
        if ((e & B) == 0) {
            const float got = __shfl_xor_sync(kFull, hi ? v[e] : v[e + B], B);
            if (hi) v[e] = got;
            else v[e + B] = got;
        }
    }
}

// tmem <-> 8 or 16 consecutive columns
__device__ __forceinline__ void tmem_ld_n(uint32_t c, uint32_t (&r)[8]) { tmem_ld_x8(c, r); }
__device__ __forceinline__ void tmem_ld_n(uint32_t c, uint32_t (&r)[16]) { tmem_ld_x16(c, r); }
__device__ __forceinline__ void tmem_st_n(uint32_t c, const uint32_t (&r)[8]) { tmem_st_x8(c, r); }
__device__ __forceinline__ void tmem_st_n(uint32_t c, const uint32_t (&r)[16]) { tmem_st_x16(c, r); }

// ====================================================================================
//  * Warps 0-15: softmax.  Thread = cache row of the tile (lane quarter warp % 4) for the NR / 4
//    query rows of its part warp / 4; query images, epilogue (thread = output dim).
//  * Warps 16 and 19: TMA, five boxes a tile into a two-stage ring (a copy takes its issuing thread
//    about 60 + 1.9 cycles a 128-byte row, so two share them: 16 the first two latent blocks and
//    the rope key, 19 the other two).
//  * Warp 17: tensor memory, score MMAs; warp 18: context MMAs.
// The loaders and the issuers run on into the next unit while the softmax warps finish one.
// The loops of the roles run side by side, so their code shares the instruction cache: loops over the
// boxes, and a status set once at the end, took the calls below from 315, 206 and 2418 us to 282, 186
// and 2213.
//
// A tile of 128 x 64 costs the tensor core 2974 cycles (N = 128 69 cycles, N = 64 54 cycles each MMA
// of K = 32, measured) and the loop takes 4100 to 4500.  What bounds it is a tile's way through a
// ring that shared memory limits to two stages: box free -> copy (about 2000 cycles) -> score MMAs
// (1000 more) -> softmax (2600, 3400 when maxima move) -> context MMAs (2800 beside the next tile's
// scores), which takes two tiles' time.  Tried and slower: the context in two halves of the rows, so
// that the next weights need not wait but the boxes are free later (13%); holding back one of the two
// products while the other runs (9 to 25%); the rope keys' slot freed by the score MMAs and copied
// first (2 to 5%); copies of their own for scores and context (17%).
// Measured, whole calls with the combine: 4 trees of 16 nodes x 64 heads at
// T = 32768 271 us = 1078 TFLOP/s; one of 5 nodes x 128 heads at T = 131072 177 us = 1034; 32 ragged
// ones of up to 32 nodes and 65536 rows 2830 us = 1141 TFLOP/s (23.2 M pairs of node and row, 64 heads).
// ====================================================================================
template <int NR>
__global__ void __launch_bounds__(kThreads, 1) tree_packed_kernel(const __grid_constant__ Args a)
{
    using C = Cfg<NR>;
    constexpr int GR = C::kGR;
    extern __shared__ __align__(1024) uint8_t dsm[];
    const Shared<NR> sh{dsm};
    const kvq_mla_tree_problem& p = a.p;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = blockIdx.x;
    grid_dependents_launch();                    // the combine may start launching

    if (warp == kWarpS) {
        if (lane == 0) {
            for (int st = 0; st < kStages; ++st) {
                for (int b = 0; b < kBoxes; ++b) {
                    mbar_init(sh.full(st, b), 1);
                    mbar_init(sh.empty(st, b), b < 4 ? 1 : kSmx);      // the context; the softmax
                }
            }
            mbar_init(sh.s_full(), 1);
            mbar_init(sh.s_empty(), kSmx);
            mbar_init(sh.p_full(), kSmx);
            mbar_init(sh.o_done(), 1);
            mbar_init(sh.q_full(), kSmx);
            mbar_init(sh.drain_s(), 1);
            mbar_init(sh.drain_c(), 1);
            *sh.abort_flag() = 0;
            fence_mbar_init();
        }
        __syncwarp();
        tmem_alloc(sh.tmem_base(), 512);
        tmem_relinquish();
    }
    // ---- the length of the line, and where this CTA's stretch begins (scratch: the W image) ----
    // One pass over the sequences if they fit the threads; else a first pass for the length.
    int64_t total = 0, t0 = 0, t1 = 0;
    int G = gridDim.x;
    {
        int64_t* s_sum = reinterpret_cast<int64_t*>(sh.w());      // sums of the warps
        constexpr int kW = kThreads / 32;
        const bool one_pass = p.n_seq <= kThreads;
        auto stretch = [&]() {
            G = (int)min((int64_t)G, max(total, (int64_t)1));
            t0 = g < G ? cut(total, g, G) : 0;
            t1 = g < G ? cut(total, g + 1, G) : 0;
        };
        if (!one_pass) {
            int64_t v = 0;
            for (int s = tid; s < p.n_seq; s += kThreads) v += seq_places<NR>(p, s);
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
            if (lane == 0) s_sum[warp] = v;
            __syncthreads();
            for (int w = 0; w < kW; ++w) total += s_sum[w];
            stretch();
            __syncthreads();
        }
        int64_t base = 0;
        for (int c = 0; c < p.n_seq && base <= t0; c += kThreads) {
            const int s = c + tid;
            const int64_t own = s < p.n_seq ? seq_places<NR>(p, s) : 0;
            int64_t incl = own;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t u = __shfl_up_sync(kFull, incl, o);
                if (lane >= o) incl += u;
            }
            if (lane == 31) s_sum[warp] = incl;
            __syncthreads();
            int64_t before = base, all = base;
#pragma unroll
            for (int w = 0; w < kW; ++w) {
                if (w < warp) before += s_sum[w];
                all += s_sum[w];
            }
            if (one_pass) {
                total = all;
                stretch();
            }
            const int64_t lo = before + incl - own;
            if (own > 0 && lo <= t0 && t0 < lo + own) {
                *sh.start_seq() = s;
                *sh.start_off() = t0 - lo;
            }
            base = all;
            if (!one_pass) __syncthreads();
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *sh.tmem_base();
    Walk<NR> k(p, t1 > t0 ? *sh.start_seq() : 0, t1 > t0 ? *sh.start_off() : 0, t1 - t0);

    if (warp < kSmx) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSmx));
        // ================================ softmax ========================================
        // Control flow is the same in all 512 threads (the barriers need every one of them);
        // `ok` only guards work and is kept warp-uniform.
        const int wq = warp & 3, hp = warp >> 2, hb = GR * hp;
        const int t = wq * 32 + lane;                 // row within the tile
        const uint32_t lane_base = (uint32_t)(wq * 32) << 16;
        // the W image: row t is 64 bytes at (t / 8) 512 + (t % 8) 64, 16-byte chunk c at c ^ ((t / 2) % 4).
        // NR = 64: an image a digit, this part's rows are chunk hp; NR = 32: digit d is chunks
        // 2 d, 2 d + 1, this part's rows half a chunk
        constexpr uint32_t kAll = (1u << GR) - 1u;
        const float tiny = ex2(-kTiny);
        const uint32_t w_row = (t >> 3) * 512 + (t & 7) * 64;
        const int wx = (t >> 1) & 3;
        bool ok = true;
        int c = 0;                                    // tiles so far
        bool first_seg = true;
        for (int seg = 0; k.more(); ++seg) {
            const int s = k.s, L = k.L, n = k.n;
            const int64_t r0 = (int64_t)k.rt * NR;    // first query row of the tile, of the sequence's n * H
            const int64_t rows = (int64_t)n * p.n_heads - r0;       // rows there are from r0 on
            const bool whole = k.tile == 0 && k.end == k.nt;
            const int slot = 2 * g + (first_seg ? 0 : 1);
            write_queries(sh, p, s, r0, rows, warp, lane);
            if (tid < NR) sh.neg_m()[tid] = 0.0f;
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(sh.q_full());
            smx_barrier();
            f32x2 l2[GR / 2];                         // this thread's part of the normalizers
#pragma unroll
            for (int e = 0; e < GR / 2; ++e) l2[e] = 0;
            const ulonglong2* gain = reinterpret_cast<const ulonglong2*>(sh.gain() + hb);
            const ulonglong2* neg_m = reinterpret_cast<const ulonglong2*>(sh.neg_m() + hb);
            const ulonglong2* move = reinterpret_cast<const ulonglong2*>(sh.move() + hb);
            bool fresh = true;                        // some row of the part has no maximum yet
            bool mine_fresh = true;                   // lane < GR: row hb + lane has none
            auto pool_row = [&](int tl) -> int64_t {
                if (tl >= L) return -1;
                const int64_t r = tree_pool_row(p, s, tl, a.page_shift);
                if (r < 0 || r >= p.cache.n_rows) {
                    if (hp == 0 && a.status) atomicOr(a.status, (unsigned)KVQ_DEV_BAD_PAGE);
                    return -1;
                }
                return r;
            };
            // the pool row and scales of this thread's row, read one tile ahead
            int64_t row_n = pool_row(k.tile * kRT + t);
            float ls_n = row_n >= 0 ? p.cache.lat_scale[row_n] : 0.0f;
            float rs_n = row_n >= 0 ? p.cache.rope_scale[row_n] : 0.0f;
            for (int i = k.tile; i < k.end; ++i, ++c) {
                const int st = c & 1, rst = C::kRS == 2 ? st : 0;
                const bool have = row_n >= 0;
                const float ls = ls_n, rs = rs_n;
                const float lg = ls >= tiny ? fminf(__log2f(ls), 200.0f) : -kTiny;
                const bool zero_row = !(have && ls >= tiny);
                if (i + 1 < k.end) {
                    row_n = pool_row((i + 1) * kRT + t);
                    ls_n = row_n >= 0 ? p.cache.lat_scale[row_n] : 0.0f;
                    rs_n = row_n >= 0 ? p.cache.rope_scale[row_n] : 0.0f;
                }
                if (ok) ok = wait_bar<kSmxSpin>(sh, sh.s_full(), (uint32_t)c & 1u, a);
                ok = __all_sync(kFull, ok);
                // t: the scores before the row's gain, then score - m; vis: the query rows that see this
                // cache row
                f32x2 t2[GR / 2];
                uint32_t vis = have ? kAll : 0u;
#pragma unroll
                for (int e = 0; e < GR / 2; ++e) t2[e] = 0;
                if (ok) {
                    tc_fence_after();
                    const f32x2 vls = pack2(ls, ls), vrs = pack2(rs, rs);
                    const f32x2 vls16 = pack2(ls * 0.0625f, ls * 0.0625f), vrs16 = pack2(rs * 0.0625f, rs * 0.0625f);
#pragma unroll
                    for (int h = 0; h < GR; h += 8) {
                        uint32_t x0[8], x1[8], y0[8], y1[8];
                        tmem_ld_x8(tmem + lane_base + C::kColSL + hb + h, x0);
                        tmem_ld_x8(tmem + lane_base + C::kColSL + NR + hb + h, x1);
                        tmem_ld_x8(tmem + lane_base + C::kColSR + hb + h, y0);
                        tmem_ld_x8(tmem + lane_base + C::kColSR + NR + hb + h, y1);
                        tmem_ld_wait();
                        auto pair = [](const uint32_t (&r)[8], int e) { return pack2(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1])); };
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            t2[h / 2 + e] = fma2(pair(x0, e), vls, fma2(pair(x1, e), vls16, fma2(pair(y0, e), vrs, mul2(pair(y1, e), vrs16))));
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(sh.s_empty());
                    if (zero_row) {
                        // not a row of the sequence, or a zero row: the context reads it as zeros, whatever
                        // the box brought
                        for (int pc = kPieces * hp; pc < kPieces * hp + kPieces; ++pc)
                            *row_piece(sh, st, rst, t, pc) = make_uint4(0u, 0u, 0u, 0u);
                    }
                    if (have) {
                        // a code that no encoder writes makes the scores of every query row NaN (and a scale that is not
                        // finite may), a query's digits never
                        if (isnan(unpack2(t2[0]).x)) {
                            clear_row(sh, st, t, hp);
#pragma unroll 1
                            for (int e = 0; e < GR; ++e) {
                                const float v = hb + e < rows ? rescore(sh, p, st, rst, t, (int64_t)s * p.n_q * p.n_heads + r0 + hb + e,
                                                                        sh.gain()[hb + e], ls, rs) : 0.0f;
#pragma unroll
                                for (int d = 0; d < GR; d += 2) {
                                    const float2 f = unpack2(t2[d / 2]);
                                    t2[d / 2] = pack2(d == e ? v : f.x, d + 1 == e ? v : f.y);
                                }
                            }
                        }
                        if ((i + 1) * kRT > L - n) {      // the drafted rows: only what the node sees
                            const int kk = i * kRT + t - (L - n);
                            if (kk >= 0) {
                                int node = (int)((r0 + hb) / p.n_heads), head = (int)((r0 + hb) % p.n_heads);
                                uint64_t see = node < n ? tree_visible(p, s, node, n) : 0;
                                vis = 0;
#pragma unroll 1
                                for (int e = 0; e < GR; ++e) {
                                    vis |= (uint32_t)((see >> kk) & 1u) << e;
                                    if (++head == p.n_heads) {
                                        head = 0;
                                        ++node;
                                        see = node < n ? tree_visible(p, s, node, n) : 0;
                                    }
                                }
                            }
                        }
                    }
                }
                // nothing reads this tile's rope keys from here on
                const bool some_hidden = __any_sync(kFull, vis != kAll);
                if (ok && lane == 0) mbar_arrive(sh.empty(rst, 4));
                float top = -INFINITY;
#pragma unroll
                for (int e = 0; e < GR; e += 4) {
                    const ulonglong2 ga = gain[e / 4], nm = neg_m[e / 4];
                    t2[e / 2] = fma2(t2[e / 2], ga.x, nm.x);
                    t2[e / 2 + 1] = fma2(t2[e / 2 + 1], ga.y, nm.y);
                }
                if (some_hidden) {
#pragma unroll
                    for (int e = 0; e < GR; e += 2) {
                        const float2 f = unpack2(t2[e / 2]);
                        t2[e / 2] = pack2((vis >> e) & 1u ? f.x : -INFINITY, (vis >> (e + 1)) & 1u ? f.y : -INFINITY);
                    }
                }
#pragma unroll
                for (int e = 0; e < GR / 2; ++e) {
                    const float2 f = unpack2(t2[e]);
                    top = max3(top, f.x, f.y);
                }
                // the maxima of this part's rows move only if one is exceeded by more than 2^kLazy
                bool moved = false;
                if (barrier_any<128>(2 + hp, fresh || top + lg > kLazy)) {
                    const float old = lane < GR ? sh.neg_m()[hb + lane] : 0.0f;
                    float v[GR];
#pragma unroll
                    for (int e = 0; e < GR; e += 2) {
                        const float2 f = unpack2(t2[e / 2]);
                        v[e] = f.x + lg;
                        v[e + 1] = f.y + lg;
                    }
                    warp_reduce_transpose<true>(v, lane);
                    if (lane < GR) sh.red()[wq * NR + hb + lane] = v[0];
                    part_barrier(hp);
                    // (each of the part's warps computes and stores the same)
                    bool up = false;
                    if (lane < GR) {
                        const float* r = sh.red() + hb + lane;
                        const float by = fmaxf(fmaxf(r[0], r[NR]), fmaxf(r[2 * NR], r[3 * NR]));
                        up = by > kLazy || (mine_fresh && by > -INFINITY);
                        sh.neg_m()[hb + lane] = up ? old - by : old;
                        sh.move()[hb + lane] = up ? -by : 0.0f;
                        sh.factor()[hb + lane] = up && !mine_fresh ? ex2(-by) : 1.0f;
                        mine_fresh = mine_fresh && !up;
                    }
                    __syncwarp();                     // (every lane reads what these lanes stored; a vote orders no memory)
                    moved = __any_sync(kFull, up) && i > k.tile;
                    fresh = __any_sync(kFull, lane < GR && mine_fresh);
#pragma unroll
                    for (int e = 0; e < GR; e += 4) {
                        const ulonglong2 mv = move[e / 4], f = reinterpret_cast<const ulonglong2*>(sh.factor() + hb)[e / 4];
                        t2[e / 2] = add2(t2[e / 2], mv.x);
                        t2[e / 2 + 1] = add2(t2[e / 2 + 1], mv.y);
                        l2[e / 2] = mul2(l2[e / 2], f.x);
                        l2[e / 2 + 1] = mul2(l2[e / 2 + 1], f.y);
                    }
                }
                uint32_t w0[GR / 4], w1[GR / 4];
                const f32x2 up2 = pack2(lg + kBase, lg + kBase);
                const uint32_t dith = dither<NR>(i * kRT + t);
#pragma unroll
                for (int e = 0; e < GR; e += 4) {
                    const float2 va = unpack2(add2(t2[e / 2], up2)), vb = unpack2(add2(t2[e / 2 + 1], up2));
                    weight_digits<NR>(make_float2(ex2(va.x), ex2(va.y)), make_float2(ex2(vb.x), ex2(vb.y)), dith, w0[e / 4], w1[e / 4]);
                }
                // the context of tile c - 1 has read the W image, and O may be rescaled
                if (i > k.tile && ok) ok = wait_bar<kSmxSpin>(sh, sh.o_done(), (uint32_t)(c - 1) & 1u, a);
                ok = __all_sync(kFull, ok);
                if (moved && ok) {
                    tc_fence_after();
                    float f[GR];
#pragma unroll
                    for (int e = 0; e < GR; ++e) f[e] = sh.factor()[hb + e];
#pragma unroll 1
                    for (int m = 0; m < 256 / NR; ++m) {               // (NR = 32: both digits' columns)
                        const uint32_t col = tmem + lane_base + kColO + NR * m + hb;
                        uint32_t x[GR];
                        tmem_ld_n(col, x);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < GR; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * f[e]);
                        tmem_st_n(col, x);
                    }
                    tmem_st_wait();
                }
                if (ok) {
                    if constexpr (NR == 64) {
                        uint8_t* img = sh.w() + w_row + ((hp ^ wx) << 4);
                        *reinterpret_cast<uint4*>(img) = make_uint4(w0[0], w0[1], w0[2], w0[3]);
                        *reinterpret_cast<uint4*>(img + kRT * 64) = make_uint4(w1[0], w1[1], w1[2], w1[3]);
                    } else {
                        uint8_t* img = sh.w() + w_row + 8 * (hp & 1);
                        *reinterpret_cast<uint2*>(img + (((hp >> 1) ^ wx) << 4)) = make_uint2(w0[0], w0[1]);
                        *reinterpret_cast<uint2*>(img + (((2 + (hp >> 1)) ^ wx) << 4)) = make_uint2(w1[0], w1[1]);
                    }
                    tc_fence_before();
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(sh.p_full());
                }
                // the normalizers, while the context runs
#pragma unroll
                for (int e = 0; e < GR / 2; ++e) {
                    const float2 f = unpack2(t2[e]);
                    l2[e] = add2(l2[e], pack2(ex2(f.x), ex2(f.y)));
                }
            }
            // ---- epilogue: l over the 128 rows, then O^T -> out or the partial ---------------
            if (ok) ok = wait_bar<kSmxSpin>(sh, sh.o_done(), (uint32_t)(c - 1) & 1u, a);
            ok = __all_sync(kFull, ok);
            float l[GR];
#pragma unroll
            for (int e = 0; e < GR; e += 2) {
                l[e] = unpack2(l2[e / 2]).x;
                l[e + 1] = unpack2(l2[e / 2]).y;
            }
            warp_reduce_transpose<false>(l, lane);
            if (lane < GR) sh.red()[wq * NR + hb + lane] = l[0];
            const bool aborted = barrier_any<32 * kSmx>(1, !ok);
            const int64_t out_row = (int64_t)s * p.n_q * p.n_heads + r0;
            if (tid < NR) {
                const float* r = sh.red() + tid;
                const float lt = (r[0] + r[NR]) + (r[2 * NR] + r[3 * NR]);
                const float m = -sh.neg_m()[tid], unit = ex2(-kBase);
                if (whole) {
                    sh.factor()[tid] = lt > 0.0f ? unit / lt : lt == 0.0f ? 0.0f : NAN;
                    if (tid < rows && a.lse)
                        a.lse[out_row + tid] = aborted ? NAN : lt == 0.0f ? -INFINITY : (m + log2f(lt)) * kLn2;
                } else {
                    sh.factor()[tid] = unit;
                    reinterpret_cast<float2*>(a.part_ml)[slot * NR + tid] =
                        aborted ? make_float2(INFINITY, INFINITY) : make_float2(lt == 0.0f ? -INFINITY : m, lt);
                }
            }
            smx_barrier();
            tc_fence_after();
            float fac[GR];
#pragma unroll
            for (int e = 0; e < GR; ++e) fac[e] = sh.factor()[hb + e];
#pragma unroll 1
            for (int m = 0; m < 4; ++m) {
                const int dim = 128 * m + 32 * wq + lane;
                float o[GR];
                if (!aborted) {
                    uint32_t x[GR];
                    tmem_ld_n(tmem + lane_base + kColO + 64 * m + hb, x);
                    if constexpr (NR == 32) {
                        uint32_t y[GR];
                        tmem_ld_n(tmem + lane_base + kColO + 64 * m + NR + hb, y);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < GR; ++e) o[e] = fmaf(__uint_as_float(y[e]), 0.0625f, __uint_as_float(x[e])) * fac[e];
                    } else {
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < GR; ++e) o[e] = __uint_as_float(x[e]) * fac[e];
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < GR; ++e) o[e] = NAN;
                }
                // thread = one dim of GR rows -> 4 dims of GR / 4 rows: lane l keeps the rows 4 j + l % 4
                swap_dims<1>(o, lane);
                swap_dims<2>(o, lane);
                const int d0 = dim & ~3, sub = lane & 3;
#pragma unroll
                for (int e = 0; e < GR / 4; ++e) {
                    const int row = hb + 4 * e + sub;
                    const float4 v = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                    if (!whole) {
                        *reinterpret_cast<float4*>(a.part_o + ((int64_t)slot * NR + row) * kDLat + d0) = v;
                    } else if (row < rows) {
                        const __nv_bfloat162 x = __floats2bfloat162_rn(v.x, v.y), y = __floats2bfloat162_rn(v.z, v.w);
                        *reinterpret_cast<uint2*>(a.out + (out_row + row) * kDLat + d0) =
                            make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
                    }
                }
            }
            tc_fence_before();
            smx_barrier();                            // maxima, factors and query scales may change
            first_seg = false;
            k.next(p);
        }
    } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
    if (warp == kWarpLoad || warp == kWarpLoad2) {
        // ================================ TMA loader =====================================
        // The lanes look up a tile's pool rows one tile ahead, one thread issues its copies.
        const bool leader = elect_one();
        const int per = kRT / a.box_rows;             // copies a 128-dim block
        const int who = warp == kWarpLoad ? 0 : 1;
        bool ok = true;
        int c = 0;                                    // tiles so far
        int done[3] = {0, 0, 0};                      // tiles whose box went out: this warp's blocks, the rope key
        for (; k.more() && ok; k.next(p)) {
            auto look_up = [&](int i, int buf) {      // the pool row where copy `lane` of tile i begins
                const int t = i * kRT + lane * a.box_rows;
                if (lane >= per) return;
                const int64_t r = t < k.L ? tree_pool_row(p, k.s, t, a.page_shift) : -1;
                sh.copy_rows(2 * who + buf)[lane] = r < 0 || r >= p.cache.n_rows ? -1 : (int)r;
            };
            // (one tile ahead, from the tile before the first: one copy of the code)
#pragma unroll 1
            for (int i = k.tile - 1; i < k.end && ok; ++i) {
                __syncwarp();                         // (the leader reads the rows that the lanes stored a tile ago)
                if (leader && i >= k.tile) {
                    const int st = c & 1;
                    volatile int* y = sh.copy_rows(2 * who + st);
                    uint32_t n_in = 0;                // rows that come
#pragma unroll 2
                    for (int h = 0; h < per; ++h) n_in += y[h] >= 0 ? a.box_rows : 0;
#pragma unroll
                    for (int b = 0; b < kBoxes; ++b) {
                        if ((b == 2 || b == 3) != (who == 1)) continue;
                        const int slot = b < 4 ? st : C::kRS == 2 ? st : 0;
                        const int use = b < 4 || C::kRS == 2 ? c >> 1 : c;                   // earlier uses of the slot
                        ok = ok && wait_bar<kRoleSpin>(sh, sh.empty(slot, b), ((uint32_t)use & 1u) ^ 1u, a);
                        if (!ok) break;
                        uint64_t* bar = sh.full(slot, b);
                        const int width = b < 4 ? 128 : 64;
                        uint8_t* dst = b < 4 ? sh.box(st, b) : sh.rope(slot);
                        mbar_arrive_expect_tx(bar, n_in * width);
#pragma unroll 2
                        for (int h = 0; h < per; ++h) {
                            const int yh = y[h];
                            if (yh >= 0) {
                                if (b < 4) tma_load_2d(dst + h * a.box_rows * width, &a.tm_lat, 128 * b, yh, bar);
                                else tma_load_2d(dst + h * a.box_rows * width, &a.tm_rope, 0, yh, bar);
                            }
                        }
                        done[b < 4 ? b & 1 : 2] = c + 1;
                    }
                }
                if (i >= k.tile) ++c;
                if (i + 1 < k.end) look_up(i + 1, c & 1);
                ok = __any_sync(kFull, leader && ok);
            }
        }
        // every box issued has landed before the CTA's shared memory is released
        if (leader) {
#pragma unroll
            for (int b = 0; b < kBoxes; ++b) {
                if ((b == 2 || b == 3) != (who == 1)) continue;
                const int n = done[b < 4 ? b & 1 : 2], ns = b < 4 ? kStages : C::kRS;
                for (int i = max(0, n - ns); i < n; ++i) {        // (an earlier use landed before a later one)
                    if (!mbar_wait(sh.full(i % ns, b), (uint32_t)(i / ns) & 1u, kTimeoutNs) && a.status)
                        atomicOr(a.status, (unsigned)KVQ_DEV_TIMEOUT);
                }
            }
        }
        __syncwarp();
    } else if (warp == kWarpS) {
        // ================================ score MMAs ======================================
        const bool leader = elect_one();
        constexpr uint32_t idesc = idesc_e4m3_f32(kRT, C::kNS, false, false);      // C . Qd^T
        const uint32_t q_addr = smem_u32(sh.q());
        bool ok = leader;
        int c = 0;
        for (int seg = 0; k.more() && ok; ++seg, k.next(p)) {
            ok = wait_bar<kRoleSpin>(sh, sh.q_full(), (uint32_t)seg & 1u, a);
            for (int i = k.tile; i < k.end && ok; ++i, ++c) {
                const int st = c & 1, rst = C::kRS == 2 ? st : 0;
                const int ruse = C::kRS == 2 ? c >> 1 : c;
                // S(c) overwrites S(c - 1): the softmax has read it
                if (c > 0) ok = wait_bar<kRoleSpin>(sh, sh.s_empty(), (uint32_t)(c - 1) & 1u, a);
#pragma unroll 1
                for (int b = 0; b < 4; ++b) {
                    ok = ok && wait_bar<kRoleSpin>(sh, sh.full(st, b), (uint32_t)(c >> 1) & 1u, a);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t box = smem_u32(sh.box(st, b)), q_at = q_addr + b * C::kQBlk;
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks) {
                        const uint64_t ad = desc_smem(box + ks * 32, 16, 1024, kSwizzle128);
                        const uint64_t bd = desc_smem(q_at + ks * 32, 16, 1024, kSwizzle128);
                        mma_e4m3_ss(tmem + C::kColSL, ad, bd, idesc, (b | ks) ? 1u : 0u);
                    }
                }
                ok = ok && wait_bar<kRoleSpin>(sh, sh.full(rst, 4), (uint32_t)ruse & 1u, a);
                if (!ok) break;
                tc_fence_after();
                const uint32_t box = smem_u32(sh.rope(rst));
#pragma unroll
                for (int ks = 0; ks < 2; ++ks) {
                    const uint64_t ad = desc_smem(box + ks * 32, 16, 512, kSwizzle64);
                    const uint64_t bd = desc_smem(q_addr + C::kQRope + ks * 32, 16, 512, kSwizzle64);
                    mma_e4m3_ss(tmem + C::kColSR, ad, bd, idesc, ks > 0 ? 1u : 0u);
                }
                mma_commit(sh.s_full());
            }
        }
        if (leader) {
            mma_commit(sh.drain_s());
            if (!mbar_wait(sh.drain_s(), 0, kTimeoutNs) && a.status) atomicOr(a.status, (unsigned)KVQ_DEV_TIMEOUT);
        }
        __syncwarp();
    } else if (warp == kWarpC) {
        // ================================ context MMAs ====================================
        const bool leader = elect_one();
        // V^T . Wd^T, both MN-major; the second image of NR = 64 is e5m2
        constexpr uint32_t idesc = idesc_e4m3_f32(kRT, 64, true, true), idesc1 = idesc_e4m3_f32(kRT, 64, true, true, true);
        // first, the CTA with a unit's first tile tells the combine who shares it (all units of the
        // stretch at once, so that nothing is left out if the CTA gives up)
        if (leader) {
            bool splits = false, first = true;        // the last unit begun goes on in the next CTA
            for (Walk<NR> w = k; w.more(); w.next(p), first = false) {
                if (w.tile != 0) continue;
                int last = g;
                while (cut(total, last + 1, G) < w.unit_end(t1)) ++last;
                SplitInfo* f = a.info + (a.by_unit ? (int64_t)w.s * a.n_rt + w.rt : (int64_t)g);
                f->s = w.s;
                f->rt = w.rt;
                f->cta = g;
                f->slot = 2 * g + (first ? 0 : 1);
                f->pieces = last - g + 1;
                splits = last > g;
            }
            if (!a.by_unit && !splits) a.info[g].pieces = 0;
        }
        const uint32_t wb = smem_u32(sh.w());
        bool ok = leader;
        int c = 0;
        for (; k.more() && ok; k.next(p)) {
            for (int i = k.tile; i < k.end && ok; ++i, ++c) {
                ok = wait_bar<kRoleSpin>(sh, sh.p_full(), (uint32_t)c & 1u, a);
                if (!ok) break;
                tc_fence_after();
                const int st = c & 1;
#pragma unroll 1
                for (int m = 0; m < 4; ++m) {
                    const uint32_t box = smem_u32(sh.box(st, m));
#pragma unroll
                    for (int d = 0; d < C::kWImgs; ++d) {
#pragma unroll
                        for (int ks = 0; ks < kRT / 32; ++ks) {
                            const uint64_t ad = desc_smem(box + ks * 4096, 16, 1024, kSwizzle128);
                            const uint64_t bd = desc_smem(wb + d * kRT * 64 + ks * 2048, 16, 512, kSwizzle64);
                            mma_e4m3_ss(tmem + kColO + 64 * m, ad, bd, d ? idesc1 : idesc, (i == k.tile && d == 0 && ks == 0) ? 0u : 1u);
                        }
                    }
                    mma_commit(sh.empty(st, m));
                }
                mma_commit(sh.o_done());
            }
        }
        if (leader) {
            mma_commit(sh.drain_c());
            if (!mbar_wait(sh.drain_c(), 0, kTimeoutNs) && a.status) atomicOr(a.status, (unsigned)KVQ_DEV_TIMEOUT);
        }
        __syncwarp();
    }
    }

    tc_fence_before();
    __syncthreads();
    if (tid == 0 && *sh.abort_flag() && a.status) atomicOr(a.status, (unsigned)KVQ_DEV_TIMEOUT);
    if (warp == kWarpS) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ------------------------------------------------------------------------------------
// Padding rows (zeros), then the units that several CTAs shared: CTA = (unit or CTA, row of
// the tile, part of the dims); its eight warps take the pieces in turn, lane = 4 V dims.  Few
// rows have their dims split over four CTAs (V = 1), so that the partials of a long sequence
// cut into 152 pieces are read by enough SMs.
// ------------------------------------------------------------------------------------
constexpr int kCombThreads = 256;
constexpr int kCombWarps = kCombThreads / 32;

template <int NR, int V>
__global__ void __launch_bounds__(kCombThreads) tree_combine_kernel(const __grid_constant__ Args a)
{
    constexpr int kDims = 128 * V;
    __shared__ __align__(16) float s_o[kCombWarps][kDims];
    __shared__ float s_l[kCombWarps];
    const kvq_mla_tree_problem& p = a.p;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t H = p.n_heads;
    const int64_t n_cta = (int64_t)gridDim.x * gridDim.y * gridDim.z;
    for (int64_t pr = blockIdx.x + gridDim.x * ((int64_t)blockIdx.y + (int64_t)gridDim.y * blockIdx.z); pr < (int64_t)p.n_seq * p.n_q; pr += n_cta) {
        const int2 sh = tree_seq_shape(p, (int)(pr / p.n_q));
        if (pr % p.n_q < sh.y) continue;              // a node (there is one only if L > 0)
        uint4* o = reinterpret_cast<uint4*>(a.out + pr * H * kDLat);
        for (int64_t i = tid; i < H * kDLat / 8; i += kCombThreads) o[i] = make_uint4(0u, 0u, 0u, 0u);
        for (int64_t i = tid; i < H && a.lse; i += kCombThreads) a.lse[pr * H + i] = -INFINITY;
    }
    grid_dependency_wait();
    if (a.by_unit) {                                  // a unit without tiles has no info
        const int2 sh = tree_seq_shape(p, blockIdx.x / a.n_rt);
        if ((int64_t)(blockIdx.x % a.n_rt) * NR + blockIdx.y >= sh.y * H) return;
    }
    const SplitInfo f = a.info[blockIdx.x];
    if (f.pieces < 2) return;
    const int64_t r = (int64_t)f.rt * NR + blockIdx.y;
    if (r >= tree_seq_shape(p, f.s).y * H) return;
    const float2* ml = reinterpret_cast<const float2*>(a.part_ml);
    auto at = [&](int k) { return (int64_t)(k == 0 ? f.slot : 2 * (f.cta + k)) * NR + blockIdx.y; };
    float M = -FLT_MAX;                               // (finite: a piece that saw nothing has -inf, and so the weight 0)
    bool gave_up = false;
    for (int k = lane; k < f.pieces; k += 32) {
        const float2 x = ml[at(k)];
        gave_up |= x.x == INFINITY;
        M = fmaxf(M, x.x);
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, o));
    gave_up = __any_sync(kFull, gave_up);
    float4 acc[V];
#pragma unroll
    for (int j = 0; j < V; ++j) acc[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float l = 0.0f;
#pragma unroll (8 / V + 2)
    for (int k = warp; k < f.pieces; k += kCombWarps) {
        const int64_t i = at(k);
        const float2 x = ml[i];
        const float w = ex2(x.x - M);
        l = fmaf(x.y, w, l);
        const float4* o = reinterpret_cast<const float4*>(a.part_o + i * kDLat + kDims * blockIdx.z) + lane;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float4 v = o[32 * j];
            acc[j].x = fmaf(v.x, w, acc[j].x);
            acc[j].y = fmaf(v.y, w, acc[j].y);
            acc[j].z = fmaf(v.z, w, acc[j].z);
            acc[j].w = fmaf(v.w, w, acc[j].w);
        }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) reinterpret_cast<float4*>(s_o[warp])[32 * j + lane] = acc[j];
    if (lane == 0) s_l[warp] = l;
    __syncthreads();
    if (tid >= kDims / 2) return;
    float lt = 0.0f;
    float2 o = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int w = 0; w < kCombWarps; ++w) {
        lt += s_l[w];
        const float2 v = reinterpret_cast<const float2*>(s_o[w])[tid];
        o.x += v.x;
        o.y += v.y;
    }
    const float inv = gave_up ? NAN : lt == 0.0f ? 0.0f : 1.0f / lt;
    const int64_t row = (int64_t)f.s * p.n_q * H + r;
    reinterpret_cast<__nv_bfloat162*>(a.out + row * kDLat + kDims * blockIdx.z)[tid] = __floats2bfloat162_rn(o.x * inv, o.y * inv);
    if (tid == 0 && blockIdx.z == 0 && a.lse) a.lse[row] = gave_up ? NAN : lt == 0.0f ? -INFINITY : (M + log2f(lt)) * kLn2;
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// 64 query rows a tile feed the tensor core best.  Up to 32 rows, and problems of few such tiles an
// SM, run in half tiles: more SMs share the work, the softmax, query image and epilogue of each are
// half as long, and so are the partials, which cost the more the fewer units the SMs share (us in
// half and full tiles: one unit of 64 rows, 512 tiles 31.0 / 44.0, 896 42.1 / 48.0, 1280 52.3 / 49.1; two
// units, 512 tiles 28.9 / 32.7, 640 32.9 / 32.2, 1024 42.3 / 40.4; four, 384 28.2 / 27.6, 512 30.1 / 30.1; 16,
// 256 32.4 / 32.9, 512 38.4 / 36.3; 32, 320 32.0 / 33.1, 448 35.6 / 35.4).  The tiles are those of
// max_seq_len, the host's bound: shorter sequences under a generous bound run in full tiles.
int tile_rows(const kvq_mla_tree_problem& p)
{
    const int64_t rows = (int64_t)p.n_q * p.n_heads, tiles = ((int64_t)p.max_seq_len + kRT - 1) / kRT;
    const int64_t units = std::max<int64_t>(1, p.n_seq * ((rows + 63) / 64));
    return rows <= 32 || units * tiles <= 2 * sm_count() * (units + 2) / units ? 32 : 64;
}

int64_t max_units(const kvq_mla_tree_problem& p)
{
    const int nr = tile_rows(p);
    return (int64_t)p.n_seq * (((int64_t)p.n_q * p.n_heads + nr - 1) / nr);
}

struct PackedPlan {
    int ctas;
    int64_t infos;
    size_t off_ml, off_o, off_info, bytes;
};

PackedPlan plan_packed(const kvq_mla_tree_problem& p)
{
    PackedPlan t{};
    t.ctas = sm_count();
    t.infos = std::max<int64_t>(1, std::min<int64_t>(t.ctas, max_units(p)));
    const size_t rows = (size_t)2 * t.ctas * tile_rows(p);
    t.off_ml = 0;
    t.off_o = align256(rows * 2 * sizeof(float));
    t.off_info = t.off_o + align256(rows * kDLat * sizeof(float));
    t.bytes = t.off_info + align256((size_t)t.infos * sizeof(SplitInfo));
    return t;
}

template <int NR>
cudaError_t launch_packed_as(Args& a, const PackedPlan& t, cudaStream_t s)
{
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    static std::atomic<uint64_t> attr_set{0};
    const uint64_t bit = 1ull << (device & 63);
    if (!(attr_set.load() & bit)) {
        // the split above waits for ever if the launch has fewer registers than it hands out
        cudaFuncAttributes fa;
        e = cudaFuncGetAttributes(&fa, tree_packed_kernel<NR>);
        if (e != cudaSuccess) return e;
        if (fa.numRegs * kThreads < kRegsNeeded) return cudaErrorLaunchOutOfResources;
        e = cudaFuncSetAttribute(tree_packed_kernel<NR>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<NR>::kSmem);
        if (e != cudaSuccess) return e;
        attr_set.fetch_or(bit);
    }
    tree_packed_kernel<NR><<<t.ctas, kThreads, Cfg<NR>::kSmem, s>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    if (t.infos * NR <= 1024)
        return launch_dependent(tree_combine_kernel<NR, 1>, dim3((unsigned)t.infos, NR, 4), dim3(kCombThreads), 0, s, a);
    return launch_dependent(tree_combine_kernel<NR, 4>, dim3((unsigned)t.infos, NR), dim3(kCombThreads), 0, s, a);
}

}  // namespace

bool tree_packed_reads(const kvq_mla_tree_problem& p)
{
    // (a stretch of the line counts its places in an int)
    const double places = (double)p.n_seq * ((double)p.n_q * p.n_heads / 32 + 1) * ((double)p.max_seq_len / kRT + 1 + kUnitCost<64>);
    return p.cache.n_rows <= INT32_MAX && (!p.block_table || p.page_size % 8 == 0) && places < 0x1p36;
}

size_t tree_packed_workspace(const kvq_mla_tree_problem& p) { return plan_packed(p).bytes; }

cudaError_t launch_tree_packed(const kvq_mla_tree_problem& p, void* out, float* lse, void* ws,
                               uint32_t* dev_status, cudaStream_t s)
{
    const PackedPlan t = plan_packed(p);
    Args a;
    memset(&a, 0, sizeof(a));
    // boxes of the largest power of two up to 128 rows that divides a page: none crosses a page
    a.box_rows = !p.block_table ? kRT : std::min(kRT, p.page_size & -p.page_size);
    if (p.cache.n_rows > 0 && (!make_code_map(&a.tm_lat, p.cache.lat, p.cache.n_rows, kDLat, 128, a.box_rows) ||
                               !make_code_map(&a.tm_rope, p.cache.rope, p.cache.n_rows, kDRope, 64, a.box_rows)))
        return cudaErrorInvalidValue;
    a.p = p;
    a.page_shift = -1;
    for (int k = 0; k < 31; ++k)
        if (p.block_table && p.page_size == 1 << k) a.page_shift = k;
    char* base = static_cast<char*>(ws);
    a.part_ml = reinterpret_cast<float*>(base + t.off_ml);
    a.part_o = reinterpret_cast<float*>(base + t.off_o);
    a.info = reinterpret_cast<SplitInfo*>(base + t.off_info);
    a.out = static_cast<__nv_bfloat16*>(out);
    a.lse = lse;
    a.status = dev_status;
    a.wait_ns = wait_limit_ns();
    const int nr = tile_rows(p);
    a.n_rt = (int)(((int64_t)p.n_q * p.n_heads + nr - 1) / nr);
    a.by_unit = max_units(p) <= t.ctas ? 1 : 0;
    return nr == 32 ? launch_packed_as<32>(a, t, s) : launch_packed_as<64>(a, t, s);
}

}  // namespace kvq
