// kvq_pages.cu — the bookkeeping of a step over a paged MLA cache: pages and pool rows from
// request lengths (kvq_resize_pages), and the move of an accepted draft path
// (kvq_accept_mla).
#include <algorithm>
#include <climits>

#include "kvq_internal.cuh"

namespace kvq {

namespace {

constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ void flag(uint32_t* status, unsigned bit)
{
    if (status) atomicOr(status, bit);
}

// ------------------------------------------------------------------------------------
// kvq_resize_pages.  The free list is one stack for all sequences, so who gets which page is
// a prefix sum over the sequences: one CTA scans them, then moves the pages with its
// threads spread over the pages (a page finds its sequence by bisection in the prefix
// sums), so that one long prompt among many short requests costs no more than its pages.
// Bound by latency: a handful of dependent global loads and block-wide scans.  A step of few
// tokens writes its slots in the same launch; more tokens than kInlineTokens go to a second
// launch over all SMs.
// ------------------------------------------------------------------------------------
constexpr int kMaxThreads = 1024;
constexpr int kInlineTokens = 4096;
constexpr int kSlotThreads = 256;
constexpr int kSlotRun = 4;                  // consecutive tokens per thread of the second launch
constexpr int kSlotTile = kSlotThreads * kSlotRun;
constexpr int kMoves = 8;                    // page moves of a thread in flight together
constexpr int kMaxPages = 1 << 20;           // pages of a table row: a chunk's moves fit 31 bits
constexpr int kSlotShared = 2048;            // sequence offsets searched in shared memory

struct ResizeArgs {
    kvq_page_plan p;
    uint32_t* status;
    int inline_slots;
};

struct Seq {
    int keep, add, held, need;               // need = held for a sequence refused on sight
    bool fits;
};

__device__ __forceinline__ Seq load_seq(const kvq_page_plan& p, int s)
{
    Seq q;
    q.keep = max(p.keep_len[s], 0);
    q.add = max(p.n_new[s], 0);
    q.held = min(max(p.n_held[s], 0), p.max_pages);
    return q;
}

// the checks that need no other sequence; `tok_end` = the packed end of its tokens
__device__ __forceinline__ void screen_seq(const kvq_page_plan& p, Seq& q, int64_t tok_end, unsigned& bits)
{
    const int64_t len = (int64_t)q.keep + q.add;
    const uint32_t need = ((uint32_t)len + (uint32_t)p.page_size - 1u) / (uint32_t)p.page_size;   // (if len fits)
    q.fits = false;
    q.need = q.held;
    if (len > INT32_MAX || (q.add > 0 && tok_end > p.max_tokens)) {
        bits |= KVQ_DEV_BAD_INDEX;
    } else if (q.keep > (int64_t)q.held * p.page_size) {
        bits |= KVQ_DEV_BAD_PAGE;
    } else if (need > (uint32_t)p.max_pages) {
        bits |= KVQ_DEV_NO_PAGE;
    } else {
        q.fits = true;
        q.need = (int)need;
    }
}

// a packed end as tok_start holds it: INT32_MAX stands for that or more, past any max_tokens
__device__ __forceinline__ int64_t packed_end(int64_t end) { return end >= INT32_MAX ? (int64_t)INT32_MAX + 1 : end; }

// Inclusive prefix sum over the CTA; *total = the CTA's sum.  s_warp: 32 entries that no thread may
// still be reading from an earlier call (one barrier a call: callers alternate buffers).
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* s_warp, int64_t* total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(kFull, v, o);
        if (lane >= o) v += u;
    }
    if (lane == 31) s_warp[warp] = v;
    __syncthreads();
    int64_t w = lane < nw ? s_warp[lane] : 0;            // every warp scans the warps' sums itself
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(kFull, w, o);
        if (lane >= o) w += u;
    }
    *total = __shfl_sync(kFull, w, 31);
    const int64_t before = __shfl_sync(kFull, w, (warp + 31) & 31);
    return warp > 0 ? v + before : v;
}

// the largest i in [lo, hi] with a[i] <= x (a ascending, a[lo] <= x)
template <typename T>
__device__ __forceinline__ int last_not_above(const T* a, int lo, int hi, T x)
{
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a[mid] <= x) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// slot and position of packed token i of sequence s (whose tokens start at `start`)
__device__ __forceinline__ void write_slot(const kvq_page_plan& p, int i, int s, int start, bool inside, uint32_t* status)
{
    int slot = -1, pos = -1;
    if (inside) {
        const int keep = max(p.keep_len[s], 0), add = max(p.n_new[s], 0);
        if ((int64_t)p.seq_len[s] == (int64_t)keep + add) {            // served
            const int t = keep + (i - start);
            const int page = p.block_table[(int64_t)s * p.max_pages + t / p.page_size];
            if (page < 0 || page >= p.n_pages) {
                flag(status, KVQ_DEV_BAD_PAGE);
            } else {
                slot = page * p.page_size + t % p.page_size;
                pos = t;
            }
        }
    }
    p.slot_map[i] = slot;
    if (p.tok_pos) p.tok_pos[i] = pos;
}

// The moves of a chunk of sequences: sequence c + k moves the pages of its table entries s_first[k] ..,
// s_pre[k + 1] - s_pre[k] of them; its first one's place in the list is s_base[k], descending.
// kBack: table -> list (the entries become -1), else list -> table (s_base -1: none).  Returns whether
// a page found no place in the list.
template <bool kBack>
__device__ __forceinline__ bool move_pages(const kvq_page_plan& p, int c, int sum, const int* s_pre, const int* s_first, const int64_t* s_base)
{
    const int T = blockDim.x, lane = threadIdx.x & 31;
    bool lost = false;
    // a warp takes 32 kMoves moves in a row, neighbouring lanes neighbouring entries
    for (int i0 = (threadIdx.x & ~31) * kMoves + lane; i0 < sum; i0 += T * kMoves) {
        int32_t* e[kMoves];
        int64_t at[kMoves];
        int32_t page[kMoves];
        int k = last_not_above(s_pre, 0, T - 1, i0);
#pragma unroll
        for (int u = 0; u < kMoves; ++u) {
            const int i = i0 + 32 * u;
            e[u] = nullptr;
            if (i >= sum) continue;
            while (s_pre[k + 1] <= i) ++k;
            const int64_t b = s_base[k];
            if (!kBack && b < 0) continue;
            const int d = i - s_pre[k];
            e[u] = p.block_table + (int64_t)(c + k) * p.max_pages + s_first[k] + d;
            at[u] = b - d;
            page[u] = kBack ? *e[u] : p.free_list[at[u]];
        }
#pragma unroll
        for (int u = 0; u < kMoves; ++u) {
            if (!e[u]) continue;
            if (!kBack) {
                *e[u] = page[u];
            } else {
                if (at[u] < p.n_pages) p.free_list[at[u]] = page[u];
                else lost = true;
                *e[u] = -1;
            }
        }
    }
    return lost;
}

__global__ void __launch_bounds__(kMaxThreads) resize_pages_kernel(const ResizeArgs a)
{
    __shared__ int64_t s_warp[4][32];                    // scan buffers, in turn
    __shared__ int s_pre[kMaxThreads + 1];               // exclusive prefix of the chunk's page moves, then all
    __shared__ int s_first[kMaxThreads];                 // first table entry of the sequence that moves
    __shared__ int64_t s_base[kMaxThreads];              // list place of that entry's page (-1: refused)
    __shared__ int s_used;
    const kvq_page_plan& p = a.p;
    const int tid = threadIdx.x, T = blockDim.x;
    grid_dependents_launch();                            // the slot launch may get ready
    unsigned bits = 0;
    const int n_free0 = p.n_free[0];
    const int n_free = min(max(n_free0, 0), p.n_pages);
    if (n_free0 != n_free && tid == 0) bits |= KVQ_DEV_BAD_INDEX;
    if (tid == 0) s_used = 0;
    const bool one = p.n_seq <= T;                       // a single chunk stays in registers throughout

    // ---- tokens' packed order, and the pages given back in all.  Pages given and taken share
    // one scan: a chunk's counts fit 31 bits each, given in the upper half
    int64_t tok = 0, both = 0, sum = 0;
    int64_t give_all = 0;
    Seq q{};
    for (int c = 0; c < p.n_seq; c += T) {
        const int s = c + tid;
        const bool live = s < p.n_seq;
        if (live) {
            q = load_seq(p, s);
            if (p.keep_len[s] < 0 || p.n_new[s] < 0 || p.n_held[s] != q.held) bits |= KVQ_DEV_BAD_INDEX;
        }
        const int buf = (c / T & 1) * 2;
        const int64_t end = tok + block_scan(live ? q.add : 0, s_warp[buf], &sum);
        tok += sum;
        int64_t v = 0;
        if (live) {
            screen_seq(p, q, packed_end(end), bits);
            p.tok_start[s + 1] = (int)min(end, (int64_t)INT32_MAX);
            v = ((int64_t)max(q.held - q.need, 0) << 32) + max(q.need - q.held, 0);
        }
        both = block_scan(v, s_warp[buf + 1], &sum);
        give_all += sum >> 32;
    }
    if (tid == 0) p.tok_start[0] = 0;
    const int have = (int)min((int64_t)n_free + give_all, (int64_t)p.n_pages);

    // a chunk's sequences and scan again: same-thread reads of what this thread wrote, or of
    // inputs that have not changed yet
    auto reload = [&](int c, int s) {
        if (one) return;
        unsigned ignore = 0;
        int64_t v = 0;
        if (s < p.n_seq) {
            q = load_seq(p, s);
            screen_seq(p, q, packed_end(p.tok_start[s + 1]), ignore);
            v = ((int64_t)max(q.held - q.need, 0) << 32) + max(q.need - q.held, 0);
        }
        both = block_scan(v, s_warp[c / T & 3], &sum);
    };

    // ---- pages go back: sequence s's page e (from its last) to n_free + (given by later ones) + e
    if (give_all > 0) {
        int64_t carry = 0;
        for (int c = 0; c < p.n_seq; c += T) {
            __syncthreads();                             // the last chunk's moves are made
            reload(c, c + tid);
            const int give = c + tid < p.n_seq ? max(q.held - q.need, 0) : 0, incl = (int)(both >> 32);
            s_pre[tid] = incl - give;
            s_first[tid] = q.need;
            s_base[tid] = n_free + (give_all - carry - incl) + give - 1;   // of entry q.need
            if (tid == 0) s_pre[T] = (int)(sum >> 32);
            __syncthreads();
            if (move_pages<true>(p, c, (int)(sum >> 32), s_pre, s_first, s_base)) bits |= KVQ_DEV_BAD_PAGE;
            carry += sum >> 32;
        }
    }

    // ---- pages are taken: the d-th page wanted is the d-th from the top
    int64_t carry = 0;
    for (int c = 0; c < p.n_seq; c += T) {
        __syncthreads();
        const int s = c + tid;
        const bool live = s < p.n_seq;
        reload(c, s);
        const int take = live ? max(q.need - q.held, 0) : 0, incl = (int)(both & 0x7FFFFFFF);
        const int64_t end = carry + incl;
        const bool served = live && q.fits && (take == 0 || end <= have);
        if (live && q.fits && !served) bits |= KVQ_DEV_NO_PAGE;
        s_pre[tid] = incl - take;
        s_first[tid] = q.held;
        s_base[tid] = served ? have - 1 - (int)(end - take) : -1;
        if (tid == 0) s_pre[T] = (int)(sum & 0x7FFFFFFF);
        if (served && take > 0) atomicMax(&s_used, (int)end);
        __syncthreads();
        (void)move_pages<false>(p, c, (int)(sum & 0x7FFFFFFF), s_pre, s_first, s_base);
        if (live) {
            p.seq_len[s] = served ? q.keep + q.add : (int)min((int64_t)q.keep, (int64_t)q.held * p.page_size);
            if (served) p.n_held[s] = q.need;
        }
        carry += sum & 0x7FFFFFFF;
    }
    __syncthreads();
    if (tid == 0) p.n_free[0] = have - s_used;
    if (bits) flag(a.status, bits);

    if (a.inline_slots) {
        const int n_tok = p.tok_start[p.n_seq];
        for (int i = tid; i < p.max_tokens; i += T) {
            const bool inside = i < n_tok;
            const int s = inside ? last_not_above(p.tok_start, 0, p.n_seq - 1, i) : 0;
            write_slot(p, i, s, inside ? p.tok_start[s] : 0, inside, a.status);
        }
    }
}

// Thread = kSlotRun consecutive tokens: one search for the first one's sequence, then the
// sequences, and the pages, in passing; 16-byte stores.
__global__ void __launch_bounds__(kSlotThreads) slot_map_kernel(const ResizeArgs a)
{
    __shared__ int s_start[kSlotShared + 1];
    const kvq_page_plan& p = a.p;
    grid_dependency_wait();
    const bool shared = p.n_seq <= kSlotShared;
    if (shared)
        for (int s = threadIdx.x; s <= p.n_seq; s += kSlotThreads) s_start[s] = p.tok_start[s];
    __syncthreads();
    const int* start = shared ? s_start : p.tok_start;
    const int n_tok = start[p.n_seq];
    const int64_t first = (int64_t)blockIdx.x * kSlotTile + threadIdx.x * kSlotRun;
    if (first >= p.max_tokens) return;
    int slot[kSlotRun], pos[kSlotRun];
    int s = -1, begin = 0, end = 0;                      // the sequence at hand and its tokens
    int base = 0, page_at = -1, page = -1;               // its first new position; the page last looked up
    bool served = false;
#pragma unroll
    for (int u = 0; u < kSlotRun; ++u) {
        const int64_t i = first + u;
        slot[u] = pos[u] = -1;
        if (i >= n_tok) continue;
        if (i >= end) {
            s = s < 0 ? last_not_above(start, 0, p.n_seq - 1, (int)i) : s + 1;
            while (start[s + 1] <= i) ++s;               // (sequences without tokens)
            begin = start[s];
            end = start[s + 1];
            const int keep = max(p.keep_len[s], 0), add = max(p.n_new[s], 0);
            served = (int64_t)p.seq_len[s] == (int64_t)keep + add;
            base = keep;
            page_at = -1;
        }
        if (!served) continue;
        const int t = base + (int)(i - begin), at = t / p.page_size;
        if (at != page_at) {
            page_at = at;
            page = p.block_table[(int64_t)s * p.max_pages + at];
        }
        if (page < 0 || page >= p.n_pages) {
            flag(a.status, KVQ_DEV_BAD_PAGE);
        } else {
            slot[u] = page * p.page_size + (t - at * p.page_size);
            pos[u] = t;
        }
    }
    const bool whole = first + kSlotRun <= p.max_tokens;
    auto store = [&](int32_t* dst, const int (&v)[kSlotRun]) {
        if (whole && ((uintptr_t)(dst + first) & 15) == 0) {
            *reinterpret_cast<int4*>(dst + first) = make_int4(v[0], v[1], v[2], v[3]);
        } else {
#pragma unroll
            for (int u = 0; u < kSlotRun; ++u)
                if (first + u < p.max_tokens) dst[first + u] = v[u];
        }
    };
    store(p.slot_map, slot);
    if (p.tok_pos) store(p.tok_pos, pos);
}

// ------------------------------------------------------------------------------------
// kvq_accept_mla: one CTA a sequence.  A path ascends, so its k-th node is at row k or behind
// it, but a row may be both a source and a destination: every piece is read into registers
// before the first is written.  At most 64 rows of 37 pieces (16 bytes of codes, or the two
// scales) = 5 pieces a thread.
// ------------------------------------------------------------------------------------
constexpr int kAccThreads = 512;
constexpr int kAccNodes = 64;

struct AcceptArgs {
    kvq_mla_accept_desc d;
    uint32_t* status;
    int row_bytes;                           // latent bytes of a row
};

__global__ void __launch_bounds__(kAccThreads) accept_mla_kernel(const AcceptArgs a)
{
    __shared__ int64_t s_src[kAccNodes], s_dst[kAccNodes];
    __shared__ int s_n;
    const kvq_mla_accept_desc& d = a.d;
    const int s = blockIdx.x, tid = threadIdx.x;
    const int L = max(d.seq_len[s], 0);
    const int n = min(max(d.n_node ? d.n_node[s] : d.n_q, 0), min(d.n_q, L));
    const int want = min(max(d.n_acc[s], 0), n);
    const int base = L - n;                                   // row of node 0
    if (tid == 0) s_n = want;
    __syncthreads();
    if (tid < want) {
        const int32_t* path = d.path + (int64_t)s * d.n_q;
        const int k = path[tid], before = tid > 0 ? path[tid - 1] : -1;
        if (k <= before || k < 0 || k >= n) {
            atomicMin(&s_n, tid);                             // the path ends before the first such entry
            flag(a.status, KVQ_DEV_BAD_INDEX);
        }
        int64_t row[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int t = base + (e ? tid : min(max(k, 0), n - 1));
            row[e] = -1;
            if (!d.block_table) {
                row[e] = (int64_t)s * d.seq_stride_rows + t;
            } else {
                const int pg = t / d.page_size;
                const int pid = pg < d.max_pages ? d.block_table[(int64_t)s * d.max_pages + pg] : -1;
                if (pid >= 0) row[e] = (int64_t)pid * d.page_size + t % d.page_size;
            }
            if (row[e] >= d.cache.n_rows) row[e] = -1;
        }
        s_src[tid] = row[0];
        s_dst[tid] = row[1];
    }
    __syncthreads();
    const int m = s_n;
    if (tid < m && (s_src[tid] < 0 || s_dst[tid] < 0)) flag(a.status, KVQ_DEV_BAD_PAGE);
    if (tid == 0) d.new_len[s] = base + m;

    uint8_t* lat = const_cast<uint8_t*>(d.cache.lat);
    uint8_t* rope = const_cast<uint8_t*>(d.cache.rope);
    float* ls = const_cast<float*>(d.cache.lat_scale);
    float* rs = const_cast<float*>(d.cache.rope_scale);
    const int lp = a.row_bytes / 16, per = lp + kDRope / 16 + 1;   // pieces of a row
    constexpr int kPer = (kAccNodes * (kDLat / 16 + kDRope / 16 + 1) + kAccThreads - 1) / kAccThreads;
    uint4 v[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int it = tid + i * kAccThreads;
        if (it < m * per) {
            const int k = it / per, e = it % per;
            const int64_t src = s_src[k];
            if (src >= 0 && s_dst[k] >= 0) {
                if (e < lp) v[i] = reinterpret_cast<const uint4*>(lat + src * a.row_bytes)[e];
                else if (e < per - 1) v[i] = reinterpret_cast<const uint4*>(rope + src * kDRope)[e - lp];
                else v[i] = make_uint4(__float_as_uint(ls[src]), __float_as_uint(rs[src]), 0u, 0u);
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int it = tid + i * kAccThreads;
        if (it < m * per) {
            const int k = it / per, e = it % per;
            const int64_t dst = s_dst[k];
            if (s_src[k] >= 0 && dst >= 0 && s_src[k] != dst) {
                if (e < lp) {
                    reinterpret_cast<uint4*>(lat + dst * a.row_bytes)[e] = v[i];
                } else if (e < per - 1) {
                    reinterpret_cast<uint4*>(rope + dst * kDRope)[e - lp] = v[i];
                } else {
                    ls[dst] = __uint_as_float(v[i].x);
                    rs[dst] = __uint_as_float(v[i].y);
                }
            }
        }
    }
}

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

int cuda_status(cudaError_t e, const char* entry)
{
    return e == cudaSuccess ? KVQ_OK : set_last_error(KVQ_ECUDA, "%s: %s", entry, cudaGetErrorString(e));
}

}  // namespace

}  // namespace kvq

extern "C" {

int kvq_resize_pages(const kvq_page_plan* p, uint32_t* dev_status, kvq_stream_t stream)
{
    using namespace kvq;
    const char* E = "kvq_resize_pages";
    if (int st = fault_injected(E)) return st;
    if (!p) return set_last_error(KVQ_EINVAL, "%s: NULL plan", E);
    if (p->n_seq < 0 || p->n_seq > 65535) return set_last_error(KVQ_EINVAL, "%s: n_seq outside [0, 65535]", E);
    if (p->max_pages < 1 || p->max_pages > kMaxPages || p->page_size < 1 || p->n_pages < 0 || p->max_tokens < 0)
        return set_last_error(KVQ_EINVAL, "%s: bad sizes", E);
    if ((int64_t)p->n_pages * p->page_size > INT32_MAX)
        return set_last_error(KVQ_EINVAL, "%s: a pool of more than INT32_MAX rows", E);
    if (!p->n_free || !p->tok_start || (p->n_pages > 0 && !p->free_list) || (p->max_tokens > 0 && !p->slot_map) ||
        (p->n_seq > 0 && (!p->keep_len || !p->n_new || !p->block_table || !p->n_held || !p->seq_len)))
        return set_last_error(KVQ_EINVAL, "%s: NULL pointer", E);
    if (p->n_seq > 0 && (p->seq_len == p->keep_len || p->seq_len == p->n_new))
        return set_last_error(KVQ_EINVAL, "%s: seq_len must not be keep_len or n_new", E);
    const void* ptrs[] = {p->keep_len, p->n_new, p->block_table, p->n_held, p->free_list, p->n_free,
                          p->seq_len, p->tok_start, p->slot_map, p->tok_pos, dev_status};
    for (const void* q : ptrs)
        if (!aligned(q, 4)) return set_last_error(KVQ_EALIGN, "%s: an array is not 4-byte aligned", E);
    ResizeArgs a{*p, dev_status, p->max_tokens <= kInlineTokens ? 1 : 0};
    const int threads = p->n_seq <= 256 && p->max_tokens <= 1024 ? 256 : kMaxThreads;
    resize_pages_kernel<<<1, threads, 0, (cudaStream_t)stream>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess && !a.inline_slots)
        e = launch_dependent(slot_map_kernel, dim3((unsigned)((p->max_tokens + (int64_t)kSlotTile - 1) / kSlotTile)),
                             dim3(kSlotThreads), 0, (cudaStream_t)stream, a);
    return cuda_status(e, E);
}

int kvq_accept_mla(const kvq_mla_accept_desc* d, uint32_t* dev_status, kvq_stream_t stream)
{
    using namespace kvq;
    const char* E = "kvq_accept_mla";
    if (int st = fault_injected(E)) return st;
    if (!d) return set_last_error(KVQ_EINVAL, "%s: NULL descriptor", E);
    if (d->fmt != KVQ_FMT_FP8 && !rotated_format(d->fmt)) return set_last_error(KVQ_EFORMAT, "%s: fmt %d", E, d->fmt);
    if (d->n_seq < 0) return set_last_error(KVQ_EINVAL, "%s: n_seq < 0", E);
    if (d->n_q < 1 || d->n_q > kAccNodes) return set_last_error(KVQ_EINVAL, "%s: n_q outside [1, 64]", E);
    if (d->block_table ? d->max_pages < 1 || d->page_size < 1 : d->seq_stride_rows < (d->n_seq > 1 ? 1 : 0))
        return set_last_error(KVQ_EINVAL, "%s: bad paging sizes", E);
    if (d->n_seq == 0) return KVQ_OK;
    const kvq_mla_cache& c = d->cache;
    if (!d->seq_len || !d->path || !d->n_acc || !d->new_len || !c.lat || !c.lat_scale || !c.rope || !c.rope_scale ||
        c.n_rows < 0)
        return set_last_error(KVQ_EINVAL, "%s: NULL pointer", E);
    if (!aligned(c.lat, 16) || !aligned(c.rope, 16) || !aligned(c.lat_scale, 4) || !aligned(c.rope_scale, 4))
        return set_last_error(KVQ_EALIGN, "%s: cache planes misaligned", E);
    for (const void* q : {(const void*)d->seq_len, (const void*)d->n_node, (const void*)d->path, (const void*)d->n_acc,
                          (const void*)d->new_len, (const void*)d->block_table, (const void*)dev_status})
        if (!aligned(q, 4)) return set_last_error(KVQ_EALIGN, "%s: an array is not 4-byte aligned", E);
    AcceptArgs a{*d, dev_status, d->fmt == KVQ_FMT_FP8 ? kDLat : kDLat * rotated_bits(d->fmt) / 8};
    accept_mla_kernel<<<d->n_seq, kAccThreads, 0, (cudaStream_t)stream>>>(a);
    return cuda_status(cudaGetLastError(), E);
}

}  // extern "C"
