// kvq_tree.cu — kvq_mla_tree_decode: its checks, the choice of its form, and the per-query
// form (kvq_mla_decode over the rows before the draft, then the drafted rows joined to it).
//
// The per-query form serves every tier and page size.  With base = L - n rows before the
// draft, the softmax of a node's scores over [0, base) and over the drafted rows it sees are
// two partial softmax states (m, l, o); kvq_mla_decode gives the first as (lse, out), i.e.
// (m, l, o) = (lse, 1, out), and tree_tail_kernel computes the second and adds them:
//     M = max(lse, m),  w0 = e^(lse - M),  w1 = e^(m - M),
//     out = (w0 out + w1 o) / (w0 + w1 l),  lse = M + log(w0 + w1 l).
// Its prefix reads the cache once per query, so where it can read the problem the packed form
// (kvq_tree_packed.cu), which shares one pass among the (node, head) rows, is chosen.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <climits>
#include <cmath>

#include "kvq_internal.cuh"

namespace kvq {

namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kLd = kDLat + kDRope + 4;      // floats of a staged row
constexpr int kStage = 2 * kWarps;           // drafted rows in shared memory at a time

__constant__ float c_cb4[16] = {
    kTq4Centroids[0], kTq4Centroids[1], kTq4Centroids[2], kTq4Centroids[3],
    kTq4Centroids[4], kTq4Centroids[5], kTq4Centroids[6], kTq4Centroids[7],
    kTq4Centroids[8], kTq4Centroids[9], kTq4Centroids[10], kTq4Centroids[11],
    kTq4Centroids[12], kTq4Centroids[13], kTq4Centroids[14], kTq4Centroids[15]};
__constant__ TqCodebook<8> c_cb3 = kTq3;
__constant__ TqCodebook<64> c_cb6 = kTq6;

struct TreeArgs {
    kvq_mla_tree_problem p;
    int32_t* prefix;             // [n_seq] rows before the draft
    float* q_lat;                // [rows][512] fp32 copies of the queries
    float* q_rope;               // [rows][64]
    float* pre_out;              // [rows][512], [rows]: attention over the prefix
    float* pre_lse;
    __nv_bfloat16* out;
    float* lse;
    uint32_t* status;
};

// fp32 copies of the queries (padding reads as 0), which kvq_mla_decode takes, and the prefix lengths:
// a warp a row, 16-byte loads; bound by HBM, 1152 bytes read and 2304 written a row
__global__ void __launch_bounds__(kThreads) tree_prepare_kernel(const TreeArgs a)
{
    const kvq_mla_tree_problem& p = a.p;
    const int64_t rows = (int64_t)p.n_seq * p.n_q * p.n_heads;
    const int lane = threadIdx.x & 31;
    const int64_t warp = (blockIdx.x * (int64_t)blockDim.x + threadIdx.x) >> 5;
    const int64_t n_warps = ((int64_t)gridDim.x * blockDim.x) >> 5;
    for (int64_t s = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; s < p.n_seq; s += (int64_t)gridDim.x * blockDim.x) {
        const int2 sh = tree_seq_shape(p, (int)s);
        a.prefix[s] = sh.x - sh.y;
    }
    for (int64_t r = warp; r < rows; r += n_warps) {
        // (the loads do not wait for the lengths)
        const uint4* ql = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q_lat) + r * p.ldq_lat);
        const uint32_t* qr = reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(p.q_rope) + r * p.ldq_rope);
        const uint4 x[2] = {ql[lane], ql[32 + lane]};
        const uint32_t y = qr[lane];
        const int64_t node = r / p.n_heads;
        const bool live = (int)(node % p.n_q) < tree_seq_shape(p, (int)(node / p.n_q)).y;
        auto wide = [&](uint32_t w) {
            return live ? make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)) : make_float2(0.0f, 0.0f);
        };
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float2 a0 = wide(x[k].x), a1 = wide(x[k].y), a2 = wide(x[k].z), a3 = wide(x[k].w);
            float4* dst = reinterpret_cast<float4*>(a.q_lat + r * kDLat) + 64 * k + 2 * lane;
            dst[0] = make_float4(a0.x, a0.y, a1.x, a1.y);
            dst[1] = make_float4(a2.x, a2.y, a3.x, a3.y);
        }
        reinterpret_cast<float2*>(a.q_rope + r * kDRope)[lane] = wide(y);
    }
}

__device__ __forceinline__ float e4m3_to_float(uint32_t byte)
{
    if ((byte & 0x7Fu) == 0x7Fu) return 0.0f;     // the pattern that no encoder writes
    return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)byte, __NV_E4M3)));
}

// one warp: pool row `row` as numbers in dst[576] (rotated tiers: the rotated row)
__device__ void stage_row(const kvq_mla_tree_problem& p, int64_t row, const float* s_cb, float* dst)
{
    const int lane = threadIdx.x & 31;
    const kvq_mla_cache& C = p.cache;
    if (p.fmt == KVQ_FMT_FP8) {
        const float sc = C.lat_scale[row];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t w = reinterpret_cast<const uint32_t*>(C.lat + row * kDLat)[k * 32 + lane];
            float4 v;
            v.x = e4m3_to_float(w & 0xFFu) * sc;
            v.y = e4m3_to_float((w >> 8) & 0xFFu) * sc;
            v.z = e4m3_to_float((w >> 16) & 0xFFu) * sc;
            v.w = e4m3_to_float(w >> 24) * sc;
            reinterpret_cast<float4*>(dst)[k * 32 + lane] = v;
        }
    } else {
        const int bits = rotated_bits(p.fmt), bytes = kDLat * bits / 8;
        const float sig = C.lat_scale[row] * tq4_inv_sqrt(kDLat);
        const uint8_t* src = C.lat + row * bytes;
#pragma unroll
        for (int k = 0; k < kDLat / 32; ++k) {
            const int b0 = (k * 32 + lane) * bits, at = b0 >> 3;
            const uint32_t w = src[at] | (at + 1 < bytes ? (uint32_t)src[at + 1] << 8 : 0u);
            dst[k * 32 + lane] = s_cb[(w >> (b0 & 7)) & ((1u << bits) - 1u)] * sig;
        }
    }
    const float sr = C.rope_scale[row];
    const uint32_t w = reinterpret_cast<const unsigned short*>(C.rope + row * kDRope)[lane];
    dst[kDLat + 2 * lane] = e4m3_to_float(w & 0xFFu) * sr;
    dst[kDLat + 2 * lane + 1] = e4m3_to_float(w >> 8) * sr;
}

// ------------------------------------------------------------------------------------
// The drafted rows, and the join: CTA = eight (node, head) rows of one sequence, a warp each;
// the drafted rows pass through shared memory sixteen at a time, two dequantised by each warp.
// At most 64 rows a sequence.  Launched to start during the prefix's combine: only the join needs
// its results.  Bound by latency: chains of dependent loads and 64 shuffled dot products a warp, so
// the loads of sixteen rows are in flight together, beside the query's (nine nodes of 20 heads, TQ4,
// two sequences of about 4100 rows: 56.6 us a call, of which the prefix's kvq_mla_decode 44.5; waiting
// for the combine at the start 62.8, eight rows at a time and the queries' copies by 2-byte loads 60.1).
// ------------------------------------------------------------------------------------
__global__ void __launch_bounds__(kThreads) tree_tail_kernel(const TreeArgs a)
{
    __shared__ __align__(16) float s_row[kStage][kLd];
    __shared__ int s_ok[kStage];
    __shared__ float s_cb[64];
    const kvq_mla_tree_problem& p = a.p;
    const int s = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int2 sh = tree_seq_shape(p, s);
    const int L = sh.x, n = sh.y;
    const int64_t in_seq = (int64_t)blockIdx.x * kWarps + warp;          // node * H + head
    const bool there = in_seq < (int64_t)p.n_q * p.n_heads;
    const int node = there ? (int)(in_seq / p.n_heads) : 0;
    const int64_t r = (int64_t)s * p.n_q * p.n_heads + in_seq;
    const bool live = there && node < n;
    const bool rot = rotated_format(p.fmt);
    if (rot && tid < 64) {
        const int bits = rotated_bits(p.fmt);
        s_cb[tid] = bits == 3 ? (tid < 8 ? c_cb3.cb[tid] : 0.0f) : bits == 6 ? c_cb6.cb[tid] : (tid < 16 ? c_cb4[tid] : 0.0f);
    }
    const uint64_t see = live ? tree_visible(p, s, node, n) : 0;
    // the query, element k * 32 + lane in q[k]; rotated tiers: rotated
    float q[16], qr[2] = {0.0f, 0.0f};
    uint32_t neg = 0;
#pragma unroll
    for (int k = 0; k < 16; ++k) q[k] = live ? a.q_lat[r * kDLat + k * 32 + lane] : 0.0f;
    if (live) {
        qr[0] = a.q_rope[r * kDRope + lane];
        qr[1] = a.q_rope[r * kDRope + 32 + lane];
    }
    bool bad = !isfinite(qr[0]) || !isfinite(qr[1]);     // a NaN or an infinity in the query
#pragma unroll
    for (int k = 0; k < 16; ++k) bad |= !isfinite(q[k]);
    bad = __any_sync(kFull, bad);
    bool saw = false;
    if (rot) {
#pragma unroll
        for (int k = 0; k < 16; ++k) neg |= ((p.signs[k] >> lane) & 1u) << k;
#pragma unroll
        for (int k = 0; k < 16; ++k) q[k] = ((neg >> k) & 1u) ? -q[k] : q[k];
        fwht_warp<16>(q, lane);
#pragma unroll
        for (int k = 0; k < 16; ++k) q[k] *= tq4_inv_sqrt(kDLat);
    }
    float m = -INFINITY, l = 0.0f, o[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) o[k] = 0.0f;
    for (int k0 = 0; k0 < n; k0 += kStage) {
        __syncthreads();
        int64_t row[2] = {-1, -1};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int e = k0 + kWarps * i + warp, t = L - n + e;
            if (e >= n) continue;
            if (!p.block_table) {
                row[i] = (int64_t)s * p.seq_stride_rows + t;
            } else {
                const int pg = t / p.page_size;
                const int pid = pg < p.max_pages ? p.block_table[(int64_t)s * p.max_pages + pg] : -1;
                row[i] = pid < 0 ? -1 : (int64_t)pid * p.page_size + t % p.page_size;
            }
            if (row[i] >= p.cache.n_rows) row[i] = -1;
            if (row[i] < 0 && lane == 0 && a.status) atomicOr(a.status, (unsigned)KVQ_DEV_BAD_PAGE);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (row[i] >= 0) stage_row(p, row[i], s_cb, s_row[kWarps * i + warp]);
            if (lane == 0) s_ok[kWarps * i + warp] = row[i] >= 0;
        }
        __syncthreads();
        for (int e = 0; e < kStage && k0 + e < n; ++e) {
            if (!((see >> (k0 + e)) & 1u) || !s_ok[e]) continue;         // (the same in every lane)
            const float* x = s_row[e];
            saw = true;
            float sc = fmaf(qr[0], x[kDLat + lane], qr[1] * x[kDLat + 32 + lane]);
#pragma unroll
            for (int k = 0; k < 16; ++k) sc = fmaf(q[k], x[k * 32 + lane], sc);
#pragma unroll
            for (int w = 16; w >= 1; w >>= 1) sc += __shfl_xor_sync(kFull, sc, w);
            sc *= p.sm_scale;
            const float m2 = fmaxf(m, sc);
            const float keep = m == -INFINITY ? 0.0f : expf(m - m2), w = m2 == -INFINITY ? 0.0f : expf(sc - m2);
            m = m2;
            l = fmaf(l, keep, w);
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = fmaf(o[k], keep, w * x[k * 32 + lane]);
        }
    }
    if (rot) {
        fwht_warp<16>(o, lane);
#pragma unroll
        for (int k = 0; k < 16; ++k) o[k] *= ((neg >> k) & 1u) ? -tq4_inv_sqrt(kDLat) : tq4_inv_sqrt(kDLat);
    }
    grid_dependency_wait();                       // the prefix's combine, launched just before
    if (!there) return;
    float lse0 = live ? a.pre_lse[r] : -INFINITY;
    if (bad && (saw || lse0 != -INFINITY)) lse0 = NAN;
    const float M = fmaxf(lse0, m);
    // (a query with a NaN or an infinity, or a prefix that gave up, has lse0 = NaN: so have w0 and everything after it)
    const float w0 = lse0 == -INFINITY ? 0.0f : expf(lse0 - M), w1 = m == -INFINITY ? 0.0f : expf(m - M);
    const float tot = w0 + w1 * l;
    const float inv = tot == 0.0f ? 0.0f : 1.0f / tot;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        const float pre = w0 == 0.0f ? 0.0f : w0 * a.pre_out[r * kDLat + k * 32 + lane];
        a.out[r * kDLat + k * 32 + lane] = __float2bfloat16_rn(fmaf(w1, o[k], pre) * inv);
    }
    if (lane == 0 && a.lse) a.lse[r] = tot == 0.0f ? -INFINITY : M + logf(tot);
}

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

int validate_tree(const kvq_mla_tree_problem* p, const char* E)
{
    if (!p) return set_last_error(KVQ_EINVAL, "%s: NULL problem", E);
    if (p->d_lat != kDLat || p->d_rope != kDRope) return set_last_error(KVQ_EINVAL, "%s: d_lat/d_rope must be 512/64", E);
    if (p->fmt != KVQ_FMT_FP8 && !rotated_format(p->fmt))
        return set_last_error(KVQ_EFORMAT, "%s: fmt %d is not FP8, TQ3, TQ4 or TQ6", E, p->fmt);
    if (p->n_seq < 0 || p->n_seq > 65535) return set_last_error(KVQ_EINVAL, "%s: n_seq outside [0, 65535]", E);
    if (p->n_q < 1 || p->n_q > 64) return set_last_error(KVQ_EINVAL, "%s: n_q outside [1, 64]", E);
    if (p->n_heads < 1) return set_last_error(KVQ_EINVAL, "%s: n_heads < 1", E);
    if (p->max_seq_len < 0 || p->max_seq_len > 1 << 30) return set_last_error(KVQ_EINVAL, "%s: max_seq_len outside [0, 2^30]", E);
    if ((int64_t)p->n_q * (((int64_t)p->n_heads + 7) / 8) > 65535 || (int64_t)p->n_seq * p->n_q * p->n_heads > INT32_MAX)
        return set_last_error(KVQ_EINVAL, "%s: n_seq * n_q * n_heads too large", E);
    if (p->impl < 0 || p->impl > 2) return set_last_error(KVQ_EINVAL, "%s: impl must be 0..2", E);
    if (!std::isfinite(p->sm_scale)) return set_last_error(KVQ_EINVAL, "%s: sm_scale is not finite", E);
    if (p->ldq_lat < kDLat || p->ldq_rope < kDRope)
        return set_last_error(KVQ_EINVAL, "%s: a query row stride is smaller than its row", E);
    if (p->block_table) {
        if (p->max_pages < 1 || p->page_size < 1) return set_last_error(KVQ_EINVAL, "%s: bad paging sizes", E);
    } else if (p->seq_stride_rows < 0 || (p->n_seq > 1 && p->seq_stride_rows < p->max_seq_len)) {
        return set_last_error(KVQ_EINVAL, "%s: seq_stride_rows smaller than max_seq_len", E);
    }
    if (p->impl == 1 && p->fmt != KVQ_FMT_FP8) return set_last_error(KVQ_EFORMAT, "%s: impl 1 reads FP8 rows only", E);
    if (p->impl == 1 && !tree_packed_reads(*p))
        return set_last_error(KVQ_EINVAL, "%s: impl 1 reads contiguous rows or pages of a multiple of 8 rows (and 2^36 tiles at most)", E);
    if (p->n_seq == 0) return KVQ_OK;
    const kvq_mla_cache& c = p->cache;
    if (!p->seq_len || !p->q_lat || !p->q_rope || !c.lat || !c.lat_scale || !c.rope || !c.rope_scale || c.n_rows < 0 ||
        (rotated_format(p->fmt) && !p->signs))
        return set_last_error(KVQ_EINVAL, "%s: NULL pointer", E);
    if (!aligned(c.lat, 16) || !aligned(c.rope, 16) || !aligned(c.lat_scale, 4) || !aligned(c.rope_scale, 4))
        return set_last_error(KVQ_EALIGN, "%s: cache planes misaligned", E);
    if (!aligned(p->q_lat, 16) || !aligned(p->q_rope, 16) || p->ldq_lat % 8 != 0 || p->ldq_rope % 8 != 0)
        return set_last_error(KVQ_EALIGN, "%s: query rows not 16-byte aligned", E);
    if (!aligned(p->mask, 8)) return set_last_error(KVQ_EALIGN, "%s: mask not 8-byte aligned", E);
    for (const void* q : {(const void*)p->seq_len, (const void*)p->n_node, (const void*)p->block_table,
                          (const void*)(rotated_format(p->fmt) ? p->signs : nullptr)})
        if (!aligned(q, 4)) return set_last_error(KVQ_EALIGN, "%s: an array is not 4-byte aligned", E);
    return KVQ_OK;
}

bool packed_form(const kvq_mla_tree_problem& p)
{
    return p.impl == 1 || (p.impl == 0 && p.fmt == KVQ_FMT_FP8 && tree_packed_reads(p));
}

// the per-query form: its prefix problem, and where its buffers sit in the workspace
struct TreePlan {
    kvq_mla_problem prefix;
    DecodePlan dec;
    size_t off_len, off_ql, off_qr, off_out, off_lse, off_dec, bytes;
};

void plan_tree(const kvq_mla_tree_problem& p, TreePlan& t)
{
    const size_t rows = (size_t)p.n_seq * p.n_q * p.n_heads;
    kvq_mla_problem& d = t.prefix;
    d = kvq_mla_problem{};
    d.n_seq = p.n_seq;
    // every node sees all of the prefix: the (node, head) rows are the heads of one query, so that
    // the kernels' groups of 16 or 32 heads fill up whatever the number of heads
    d.n_q = 1;
    d.n_heads = p.n_q * p.n_heads;
    d.d_lat = kDLat;
    d.d_rope = kDRope;
    d.max_seq_len = p.max_seq_len;
    d.fmt = p.fmt;
    d.block_table = p.block_table;
    d.max_pages = p.max_pages;
    d.page_size = p.page_size;
    d.seq_stride_rows = p.seq_stride_rows;
    (p.fmt == KVQ_FMT_FP8 ? d.fp8 : d.tq4) = p.cache;
    d.tq4_signs = p.signs;
    d.sm_scale = p.sm_scale;
    plan_decode(d, t.dec);
    size_t off = 0;
    auto take = [&](size_t bytes) { const size_t at = off; off += align256(bytes); return at; };
    t.off_len = take((size_t)p.n_seq * sizeof(int32_t));
    t.off_ql = take(rows * kDLat * sizeof(float));
    t.off_qr = take(rows * kDRope * sizeof(float));
    t.off_out = take(rows * kDLat * sizeof(float));
    t.off_lse = take(rows * sizeof(float));
    t.off_dec = take(t.dec.bytes);
    t.bytes = off;
}

cudaError_t launch_per_query(const kvq_mla_tree_problem& p, TreePlan& t, void* out, float* lse, void* ws,
                             uint32_t* dev_status, cudaStream_t s)
{
    char* base = static_cast<char*>(ws);
    TreeArgs a{};
    a.p = p;
    a.prefix = reinterpret_cast<int32_t*>(base + t.off_len);
    a.q_lat = reinterpret_cast<float*>(base + t.off_ql);
    a.q_rope = reinterpret_cast<float*>(base + t.off_qr);
    a.pre_out = reinterpret_cast<float*>(base + t.off_out);
    a.pre_lse = reinterpret_cast<float*>(base + t.off_lse);
    a.out = static_cast<__nv_bfloat16*>(out);
    a.lse = lse;
    a.status = dev_status;
    const int64_t rows = (int64_t)p.n_seq * p.n_q * p.n_heads;
    const int64_t g = std::min<int64_t>((rows + kWarps - 1) / kWarps, (int64_t)sm_count() * 8);
    tree_prepare_kernel<<<(unsigned)g, kThreads, 0, s>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    t.prefix.seq_len = a.prefix;
    t.prefix.q_lat = a.q_lat;
    t.prefix.q_rope = a.q_rope;
    e = launch_mla_decode(t.prefix, t.dec, a.pre_out, a.pre_lse, base + t.off_dec, dev_status, s);
    if (e != cudaSuccess) return e;
    return launch_dependent(tree_tail_kernel, dim3((unsigned)(((int64_t)p.n_q * p.n_heads + kWarps - 1) / kWarps), p.n_seq),
                            dim3(kThreads), 0, s, a);
}

}  // namespace

}  // namespace kvq

extern "C" {

int kvq_mla_tree_decode_kernel(const kvq_mla_tree_problem* p)
{
    if (int st = kvq::validate_tree(p, "kvq_mla_tree_decode_kernel")) return -st;
    return kvq::packed_form(*p) ? 1 : 2;
}

size_t kvq_mla_tree_decode_workspace(const kvq_mla_tree_problem* p)
{
    if (kvq::validate_tree(p, "kvq_mla_tree_decode_workspace") != KVQ_OK) return 0;
    if (kvq::packed_form(*p)) return kvq::tree_packed_workspace(*p);
    kvq::TreePlan t;
    kvq::plan_tree(*p, t);
    return t.bytes;
}

int kvq_mla_tree_decode(const kvq_mla_tree_problem* p, void* out, float* lse, void* workspace,
                        size_t ws_bytes, uint32_t* dev_status, kvq_stream_t stream)
{
    using namespace kvq;
    const char* E = "kvq_mla_tree_decode";
    if (int st = fault_injected(E)) return st;
    if (int st = validate_tree(p, E)) return st;
    if (p->n_seq == 0) return KVQ_OK;
    if (!out) return set_last_error(KVQ_EINVAL, "%s: NULL out", E);
    if (!aligned(out, 16) || !aligned(lse, 4) || !aligned(dev_status, 4))
        return set_last_error(KVQ_EALIGN, "%s: out/lse/dev_status misaligned", E);
    const bool packed = packed_form(*p);
    TreePlan t;
    if (!packed) plan_tree(*p, t);
    const size_t need = packed ? tree_packed_workspace(*p) : t.bytes;
    if (!workspace || ws_bytes < need)
        return set_last_error(KVQ_EWORKSPACE, "%s: workspace %zu bytes, need %zu", E, ws_bytes, need);
    if (!aligned(workspace, 256)) return set_last_error(KVQ_EALIGN, "%s: workspace not 256-byte aligned", E);
    const cudaError_t e = packed ? launch_tree_packed(*p, out, lse, workspace, dev_status, (cudaStream_t)stream)
                                 : launch_per_query(*p, t, out, lse, workspace, dev_status, (cudaStream_t)stream);
    return e == cudaSuccess ? KVQ_OK : set_last_error(KVQ_ECUDA, "%s: %s", E, cudaGetErrorString(e));
}

}  // extern "C"
