// kvq_fork.cu — pages of a pool that several sequences share: block tables after a fork, a
// reordering or a release (kvq_fork_pages), compaction (kvq_compact_pages), and the page copies that they
// ask for (kvq_copy_pages).
#include <cooperative_groups.h>

#include <algorithm>
#include <climits>

#include "kvq_internal.cuh"

namespace kvq {

namespace {

namespace cg = cooperative_groups;

constexpr unsigned kFull = 0xffffffffu;
constexpr int kMaxPages = 1 << 20;       // of a sequence
// pages of a pool: what a list holds and what is pushed to it, one after the other, is counted in 32 bits; entries of a copy list
constexpr int kMaxPool = 1 << 29, kMaxCopies = 1 << 30;
constexpr int kCluster = 8;              // CTAs of a planning kernel where one is not enough
constexpr int kThreads = 1024;           // of each; of a single one:
constexpr int kThreadsOne = 512;
constexpr int kSeqShared = 512;          // sequences of a CTA whose lengths are kept in shared memory
constexpr int kRowsShared = 8192;        // table entries of a single CTA that are
constexpr int kPagesOne = 8192;          // pages that a single CTA goes over (5 bytes of shared memory each)
constexpr size_t kPlainSmem = 39 * 1024; // dynamic shared memory that needs no attribute, beside the kernels' own
constexpr int kPagesShared = 65536;      // pages whose marks fit the CTAs' shared memory
// the most that a single CTA and one of a cluster ask for (2 bytes of marks a page, 4 of keepers an own page, a single
// one's table rows); always this much is allowed, so that calls of several threads do not lower each other's limit
constexpr int kMostSmemOne = 6 * kPagesOne + 4 * kRowsShared, kMostSmem = 200 * 1024;
static_assert(2 * kPagesShared + 4 * kPagesShared / kCluster <= kMostSmem, "marks and keepers fit");

__device__ __forceinline__ void flag(uint32_t* status, unsigned bit)
{
    if (status) atomicOr(status, bit);
}

// pages of n rows (n + page - 1 may pass 2^31)
__device__ __forceinline__ int pages_of(int n, int page) { return n / page + (n % page != 0); }

// Inclusive prefix sum over the CTA; *total = the CTA's sum.  s_warp: 32 entries.
__device__ __forceinline__ int block_scan(int v, int* s_warp, int* total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(kFull, v, o);
        if (lane >= o) v += u;
    }
    __syncthreads();                                     // an earlier call's readers are done
    if (lane == 31) s_warp[warp] = v;
    __syncthreads();
    int w = lane < nw ? s_warp[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(kFull, w, o);
        if (lane >= o) w += u;
    }
    *total = __shfl_sync(kFull, w, 31);
    const int before = __shfl_sync(kFull, w, (warp + 31) & 31);
    return warp > 0 ? v + before : v;
}

// ------------------------------------------------------------------------------------
// The planning kernels.  Small problems run as one CTA, larger ones as a cluster of kCluster; either way one launch,
// whose phases are parted by the CTA's or the cluster's barrier.  A CTA goes over the table rows of its share of the
// sequences and leaves marks, a byte a page, in its own set; each CTA then owns a range of the pages, and reads that
// range of all the sets.  Marks are plain stores of one value, so that no order changes them; lists of pages come from
// prefix sums over the marks, in the order of the ids.  The sets are in shared memory, read across the cluster, up to
// kPagesShared pages, else in the workspace.  Bound by latency: a handful of dependent accesses between barriers
// (4 beams: 12.5 us with the marks in global memory and a barrier of a cluster, 6.7 as one CTA; 512 beams of 70 pages, as
// a cluster: 22.6 with the marks in global memory, 13.2).
// ------------------------------------------------------------------------------------
template <bool ONE, bool SHARED>
struct Team {
    uint8_t* shared;                     // this CTA's dynamic shared memory
    uint8_t* global;                     // the workspace that stands for it, `stride` bytes a CTA
    size_t stride;
    int cta;
    static constexpr int n_cta = ONE ? 1 : kCluster;

    __device__ Team(uint8_t* sh, uint8_t* gl, size_t st) : shared(sh), global(gl), stride(st), cta(0)
    {
        if constexpr (!ONE) cta = (int)cg::this_cluster().block_rank();
    }
    __device__ void sync() const
    {
        if constexpr (ONE) __syncthreads();
        else cg::this_cluster().sync();
    }
    // CTA c's part of the storage, from byte `at` on
    template <typename T>
    __device__ T* part(int c, size_t at) const
    {
        if constexpr (!SHARED) return reinterpret_cast<T*>(global + c * stride + at);
        else if constexpr (ONE) return reinterpret_cast<T*>(shared + at);
        else return reinterpret_cast<T*>(cg::this_cluster().map_shared_rank(shared, c) + at);
    }
    template <typename T>
    __device__ T* mine(size_t at) const
    {
        if constexpr (!SHARED) return reinterpret_cast<T*>(global + cta * stride + at);
        else return reinterpret_cast<T*>(shared + at);
    }
    // a static shared variable of CTA c
    template <typename T>
    __device__ T* of(int c, T* v) const
    {
        if constexpr (ONE) return v;
        else return cg::this_cluster().map_shared_rank(v, c);
    }
};

// Marks come in words of four pages; the words' ranges of the CTAs, and where a page's owner has what it keeps of it
struct Words {
    int n, each;
    __host__ __device__ Words(int n_pages, int n_cta) : n((n_pages + 3) / 4), each(((n_pages + 3) / 4 + n_cta - 1) / n_cta) {}
    __host__ __device__ size_t bytes() const { return ((size_t)n * 4 + 15) / 16 * 16; }       // of a set of marks
};

__device__ __forceinline__ void clear(uint8_t* p, size_t bytes)
{
    for (size_t i = threadIdx.x; i < bytes / 16; i += blockDim.x) reinterpret_cast<uint4*>(p)[i] = make_uint4(0u, 0u, 0u, 0u);
}

// use(r, e, v) for the entries e < r.n of the rows r = row(s), s = s0 .. s1 - 1, with v = load(r, e): warps take rows,
// several a row where there are few, and lanes entries, four of a lane loaded together
template <typename R, typename G, typename F>
__device__ __forceinline__ void over_rows(int s0, int s1, R row, G load, F use)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n_warps = blockDim.x >> 5;
    const int per_row = max(1, n_warps / max(1, s1 - s0)), rows = n_warps / per_row;
    if (warp >= rows * per_row) return;
    for (int s = s0 + warp / per_row; s < s1; s += rows) {
        const auto r = row(s);
        for (int e0 = warp % per_row * 128 + lane; e0 < r.n; e0 += per_row * 128) {
            decltype(load(r, e0)) v[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (e0 + 32 * u < r.n) v[u] = load(r, e0 + 32 * u);
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (e0 + 32 * u < r.n) use(r, e0 + 32 * u, v[u]);
        }
    }
}

// ------------------------------------------------------------------------------------
// kvq_fork_pages.  Two sets of marks, the pages that the tables held (was) and those that the new ones hold (stays), and
// for a page that is some sequence's last, in part, the lowest such sequence (keeper, with the page's owner).
// ------------------------------------------------------------------------------------
struct ForkArgs {
    kvq_fork_plan p;
    uint32_t* status;
    uint8_t* store;                      // the CTAs' marks and keepers, where they are not in shared memory
    size_t stride;
    int32_t* row;                        // [n_seq][max_pages]: the new tables
    int4* seq;                           // [n_seq], see below
    int rows_shared;                     // whether the new tables are in shared memory, a CTA's in its own
};

template <bool ONE, bool SHARED>
__global__ void __launch_bounds__(ONE ? kThreadsOne : kThreads) fork_pages_kernel(const ForkArgs a)
{
    extern __shared__ __align__(16) uint8_t s_store[];
    __shared__ int s_warp[32];
    __shared__ int4 s_seq[kSeqShared];
    __shared__ int s_copies, s_given;
    const kvq_fork_plan& p = a.p;
    const Team<ONE, SHARED> team(s_store, a.store, a.stride);
    const Words words(p.n_pages, team.n_cta);
    const size_t set = words.bytes();
    grid_dependency_wait();
    grid_dependents_launch();
    const int tid = threadIdx.x, T = blockDim.x, ps = p.page_size;
    uint8_t *was = team.template mine<uint8_t>(0), *stays = team.template mine<uint8_t>(set);
    auto keeper = [&](int page) {
        const int owner = page / 4 / words.each;
        return team.template part<int32_t>(owner, 2 * set) + (page - owner * words.each * 4);
    };
    const int seqs = (p.n_seq + team.n_cta - 1) / team.n_cta;
    const int s0 = min(team.cta * seqs, p.n_seq), s1 = min(s0 + seqs, p.n_seq);
    // of a sequence: parent (-1: none), later its number among the copies (-1: none); rows; last page if held in
    // part (-1: none); pages held before
    int4* const seq = seqs <= kSeqShared ? s_seq - s0 : a.seq;
    int32_t* const row = SHARED && a.rows_shared
                             ? reinterpret_cast<int32_t*>(s_store + 2 * set + (size_t)words.each * 16) - (int64_t)s0 * p.max_pages
                             : a.row;
    unsigned bits = 0;
    const int n_free0 = p.n_free[0], n_free = min(max(n_free0, 0), p.n_pages);
    if (n_free != n_free0) bits |= KVQ_DEV_BAD_INDEX;

    // ---- marks cleared; every sequence's parent, rows and last page
    const int par0 = s0 + tid < s1 ? p.parent[s0 + tid] : -1;           // (on its way while the marks are cleared)
    clear(was, set);
    clear(stays, set);
    for (int i = tid; i < words.each * 4; i += T) team.template mine<int32_t>(2 * set)[i] = INT_MAX;
    for (int s = s0 + tid; s < s1; s += T) {
        int par = s == s0 + tid ? par0 : p.parent[s];
        const int held = p.n_held[s], own = min(max(held, 0), p.max_pages);
        if (par < -1 || par >= p.n_seq) {
            bits |= KVQ_DEV_BAD_INDEX;
            par = -1;
        }
        if (held != own) bits |= KVQ_DEV_BAD_INDEX;
        int len = 0, last = -1;
        if (par >= 0) {
            const int have = min(max(p.n_held[par], 0), p.max_pages);
            len = p.seq_len[par];
            if (len < 0) {
                bits |= KVQ_DEV_BAD_INDEX;
                len = 0;
            }
            if (len > (int64_t)have * ps) {
                bits |= KVQ_DEV_BAD_PAGE;
                len = have * ps;                            // (below len, so it fits)
            }
            if (p.keep_len) len = min(len, max(p.keep_len[s], 0));
            if (len % ps) {
                const int page = p.block_table[(int64_t)par * p.max_pages + len / ps];
                if (page >= 0 && page < p.n_pages) last = page;
            }
        }
        seq[s] = make_int4(par, len, last, own);
    }
    team.sync();

    // ---- the pages that the tables held, those that the new ones hold whole, and the new rows
    for (int s = s0 + tid; s < s1; s += T) {
        const int last = seq[s].z;
        if (last >= 0) atomicMin(keeper(last), s);
    }
    struct Row {
        int n, own, need, whole;                            // entries in all, before, after, after and whole
        int64_t at, parent;                                 // where the row begins, and its parent's
    };
    over_rows(
        s0, s1,
        [&](int s) {
            const int4 q = seq[s];
            const int need = pages_of(q.y, ps);
            return Row{max(q.w, need), q.w, need, q.y / ps, (int64_t)s * p.max_pages, (int64_t)q.x * p.max_pages};
        },
        [&](const Row& r, int e) {                          // its entry before, its parent's
            return make_int2(e < r.own ? p.block_table[r.at + e] : -1, e < r.need ? p.block_table[r.parent + e] : -1);
        },
        [&](const Row& r, int e, int2 v) {
            if (e < r.own) {
                if (v.x >= 0 && v.x < p.n_pages) was[v.x] = 1;
                else bits |= KVQ_DEV_BAD_PAGE;
            }
            if (e < r.need) {
                int page = v.y;
                if (page < 0 || page >= p.n_pages) {
                    bits |= KVQ_DEV_BAD_PAGE;
                    page = -1;
                } else if (e < r.whole) {
                    stays[page] = 1;
                }
                row[r.at + e] = page;
            }
        });
    team.sync();

    // ---- who copies, in the order of the sequences; who keeps its last page
    int copies = 0;
    for (int c = s0; c < s1; c += T) {
        const int s = c + tid;
        bool copy = false;
        int last = -1;
        if (s < s1) {
            last = seq[s].z;
            // (a mark that another thread sets here is for a keeper that is not s: s copies either way)
            copy = last >= 0 && *keeper(last) != s;
            if (last >= 0 && !copy)
#pragma unroll
                for (int k = 0; k < team.n_cta; ++k) copy |= team.template part<uint8_t>(k, set)[last] != 0;
            if (last >= 0 && !copy) stays[last] = 1;
        }
        int sum;
        const int r = block_scan(copy ? 1 : 0, s_warp, &sum);
        if (s < s1) seq[s].x = copy ? copies + r - 1 : -1;
        copies += sum;
    }
    if (tid == 0) s_copies = copies;
    team.sync();

    // ---- pages given back, in this CTA's range: its own marks become theirs
    const int w0 = min(team.cta * words.each, words.n), w1 = min(w0 + words.each, words.n);
    uint32_t* const given = reinterpret_cast<uint32_t*>(was);
    int mine = 0, here;
    for (int i = w0 + tid; i < w1; i += T) {
        uint32_t held = 0, kept = 0;
#pragma unroll
        for (int k = 0; k < team.n_cta; ++k) {
            held |= team.template part<uint32_t>(k, 0)[i];
            kept |= team.template part<uint32_t>(k, set)[i];
        }
        given[i] = held & ~kept;
        mine += __popc(held & ~kept);
    }
    const int mine_to = block_scan(mine, s_warp, &here);
    int above = 0, total = here, want = s_copies, copies0 = 0;
    if constexpr (!ONE) {
        if (tid == 0) s_given = here;
        team.sync();
        total = want = 0;
#pragma unroll
        for (int k = 0; k < team.n_cta; ++k) {
            const int v = *team.of(k, &s_given), w = *team.of(k, &s_copies);
            total += v;
            want += w;
            if (k > team.cta) above += v;
            if (k < team.cta) copies0 += w;
        }
    }
    // the highest id first
    auto push = [&](int i, uint32_t g, int at) {
#pragma unroll
        for (int b = 3; b >= 0; --b)
            if (g >> (8 * b) & 1) {
                if (at < p.n_pages) p.free_list[at] = i * 4 + b;
                else bits |= KVQ_DEV_BAD_PAGE;
                ++at;
            }
    };
    if (w1 - w0 <= T) {                                     // (a word a thread: the scan is done)
        if (mine > 0) push(w0 + tid, given[w0 + tid], n_free + above + here - mine_to);
    } else {
        for (int top = w1; here > 0 && top > w0; top -= T) {
            const int i = top - 1 - tid;
            const uint32_t g = i >= w0 ? given[i] : 0;
            int sum;
            push(i, g, n_free + above + block_scan(__popc(g), s_warp, &sum) - __popc(g));
            above += sum;
        }
    }
    team.sync();

    // ---- pages for the copies, and the tables
    const int have = min(n_free + total, p.n_pages), used = min(want, have);
    for (int s = s0 + tid; s < s1; s += T) {
        const int4 q = seq[s];
        int len = q.y;
        if (q.x >= 0) {
            const int r = copies0 + q.x;
            int page = -1;
            if (r < have) {
                page = p.free_list[have - 1 - r];
                p.copy_src[r] = q.z;
                p.copy_dst[r] = page;
                p.copy_rows[r] = len % ps;
            } else {
                bits |= KVQ_DEV_NO_PAGE;
                len -= len % ps;
            }
            p.block_table[(int64_t)s * p.max_pages + q.y / ps] = page;
        }
        if (s >= used) p.copy_src[s] = p.copy_dst[s] = p.copy_rows[s] = -1;
        p.seq_len[s] = len;
        p.n_held[s] = pages_of(len, ps);
    }
    if (team.cta == 0 && tid == 0) {
        p.n_free[0] = have - used;
        p.n_copy[0] = used;
    }
    over_rows(
        s0, s1,
        [&](int s) {
            const int4 q = seq[s];
            const int need = pages_of(q.y, ps);
            // (whole: a copy's last page is written above)
            return Row{max(q.w, need), q.w, need, q.x >= 0 ? q.y / ps : -1, (int64_t)s * p.max_pages, 0};
        },
        [&](const Row& r, int e) { return e < r.need ? row[r.at + e] : -1; },
        [&](const Row& r, int e, int page) {
            if (e != r.whole) p.block_table[r.at + e] = page;
        });
    if (bits) flag(a.status, bits);
}

// ------------------------------------------------------------------------------------
// kvq_compact_pages: a mark a held page; the number of the held pages is U, and the i-th held page of id U or more
// goes to the i-th page below U without a mark.
// ------------------------------------------------------------------------------------
struct CompactArgs {
    kvq_compact_plan p;
    uint32_t* status;
    uint8_t* store;                      // as in ForkArgs
    size_t stride;
    int32_t* rank;                       // [n_pages]: number of a page among those that move
};

template <bool ONE, bool SHARED>
__global__ void __launch_bounds__(ONE ? kThreadsOne : kThreads) compact_pages_kernel(const CompactArgs a)
{
    extern __shared__ __align__(16) uint8_t s_store[];
    __shared__ int s_warp[32];
    __shared__ int s_used, s_holes, s_moves;
    const kvq_compact_plan& p = a.p;
    const Team<ONE, SHARED> team(s_store, a.store, a.stride);
    const Words words(p.n_pages, team.n_cta);
    grid_dependency_wait();
    grid_dependents_launch();
    const int tid = threadIdx.x, T = blockDim.x, all = team.n_cta * T, me = team.cta * T + tid;
    uint8_t* const used = team.template mine<uint8_t>(0);
    const int seqs = (p.n_seq + team.n_cta - 1) / team.n_cta;
    const int s0 = min(team.cta * seqs, p.n_seq), s1 = min(s0 + seqs, p.n_seq);
    unsigned bits = 0;

    clear(used, words.bytes());
    __syncthreads();
    struct Row {
        int n, held;                                        // entries in all, held
        int64_t at;                                         // where the row begins
    };
    over_rows(
        s0, s1,
        [&](int s) {
            const int held = p.n_held[s], n = min(max(held, 0), p.max_pages);
            if (held != n) bits |= KVQ_DEV_BAD_INDEX;
            return Row{n, n, (int64_t)s * p.max_pages};
        },
        [&](const Row& r, int e) { return p.block_table[r.at + e]; },
        [&](const Row&, int, int page) {
            if (page >= 0 && page < p.n_pages) used[page] = 1;
            else bits |= KVQ_DEV_BAD_PAGE;
        });
    team.sync();

    // ---- held pages of this CTA's range: its own marks become all CTAs'
    const int w0 = min(team.cta * words.each, words.n), w1 = min(w0 + words.each, words.n);
    uint32_t* const marks = reinterpret_cast<uint32_t*>(used);
    int mine = 0, sum;
    for (int i = w0 + tid; i < w1; i += T) {
        uint32_t held = 0;
#pragma unroll
        for (int k = 0; k < team.n_cta; ++k) held |= team.template part<uint32_t>(k, 0)[i];
        marks[i] = held;
        mine += __popc(held);
    }
    (void)block_scan(mine, s_warp, &sum);
    int n_used = sum;
    if constexpr (!ONE) {
        if (tid == 0) s_used = sum;
        team.sync();
        n_used = 0;
        for (int k = 0; k < team.n_cta; ++k) n_used += *team.of(k, &s_used);
    }
    // pages that are moved to (not held, below U) and that move (held, from U on), a byte of 1 each
    auto below = [&](int i) {
        const int n = min(max(n_used - 4 * i, 0), 4);
        return n == 4 ? 0x01010101u : 0x01010101u & ((1u << 8 * n) - 1u);
    };
    auto holes_of = [&](int i) { return ~marks[i] & below(i); };
    auto moves_of = [&](int i) { return marks[i] & ~below(i); };
    int hole_at = 0, move_at = 0, total, my_hole, my_move;
    {
        int holes = 0, moves = 0, sum_h, sum_m;
        for (int i = w0 + tid; i < w1; i += T) {
            holes += __popc(holes_of(i));
            moves += __popc(moves_of(i));
        }
        my_hole = block_scan(holes, s_warp, &sum_h) - holes;
        my_move = block_scan(moves, s_warp, &sum_m) - moves;
        total = sum_m;
        if constexpr (!ONE) {
            if (tid == 0) {
                s_holes = sum_h;
                s_moves = sum_m;
            }
            team.sync();
            total = 0;
            for (int k = 0; k < team.n_cta; ++k) {
                const int m = *team.of(k, &s_moves);
                total += m;
                if (k < team.cta) {
                    hole_at += *team.of(k, &s_holes);
                    move_at += m;
                }
            }
        }
    }
    auto list = [&](int i, uint32_t hole, uint32_t move, int h, int m) {
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            if (hole >> (8 * b) & 1) p.copy_dst[h++] = i * 4 + b;
            if (move >> (8 * b) & 1) {
                p.copy_src[m] = i * 4 + b;
                a.rank[i * 4 + b] = m++;
            }
        }
    };
    if (w1 - w0 <= T) {                                     // (a word a thread: the scans are done)
        if (w0 + tid < w1) list(w0 + tid, holes_of(w0 + tid), moves_of(w0 + tid), hole_at + my_hole, move_at + my_move);
    } else {
        for (int low = w0; low < w1; low += T) {
            const int i = low + tid;
            const uint32_t hole = i < w1 ? holes_of(i) : 0, move = i < w1 ? moves_of(i) : 0;
            int sum_h, sum_m;
            const int h = hole_at + block_scan(__popc(hole), s_warp, &sum_h) - __popc(hole);
            list(i, hole, move, h, move_at + block_scan(__popc(move), s_warp, &sum_m) - __popc(move));
            hole_at += sum_h;
            move_at += sum_m;
        }
    }
    for (int i = me; i < p.max_copy; i += all) {
        p.copy_rows[i] = i < total ? p.page_size : -1;
        if (i >= total) p.copy_src[i] = p.copy_dst[i] = -1;
    }
    for (int i = me; i < p.n_pages; i += all) p.free_list[i] = i < p.n_pages - n_used ? p.n_pages - 1 - i : -1;
    if (me == 0) {
        p.n_free[0] = p.n_pages - n_used;
        p.n_used[0] = n_used;
        p.n_copy[0] = total;
    }
    team.sync();

    over_rows(
        s0, s1, [&](int s) { return Row{p.max_pages, p.n_held[s], (int64_t)s * p.max_pages}; },
        [&](const Row& r, int e) {
            const int page = e < r.held ? p.block_table[r.at + e] : -1;
            if (page < 0 || page >= p.n_pages) return -1;
            return page < n_used ? page : p.copy_dst[a.rank[page]];
        },
        [&](const Row& r, int e, int page) { p.new_table[r.at + e] = page; });
    if (bits) flag(a.status, bits);
}

// ------------------------------------------------------------------------------------
// kvq_copy_pages: pieces of 4 KiB (a warp each, its loads before its stores) of every outer array of every
// plane, for every entry of the list; as many warps as the machine holds go over them.  Bound by the
// bytes, read and written once (3900 pages of 68 KB: 83 us, 6.4 TB/s of reads and writes).
// ------------------------------------------------------------------------------------
constexpr int kMaxPlanes = 64, kFewPlanes = 4;
constexpr int kCopyThreads = 256;
constexpr int kPiece = 4096;

struct CopyPlane {
    uint8_t* base;
    int64_t row_bytes, n_rows, outer_stride;
    int32_t piece_end;                   // pieces of an entry in this plane and the ones before it
    int32_t per_outer;                   // pieces of a page in one outer array
    int32_t width;                       // bytes at a time: 16, 4 or 1
};

template <int N>                         // planes at most (the arguments travel with every launch)
struct CopyArgs {
    int32_t n_planes, page_size, max_copy;
    const int32_t *src, *dst, *rows, *n_copy;
    uint32_t* status;
    CopyPlane plane[N];
};

template <typename T>
__device__ __forceinline__ void copy_piece(uint8_t* dst, const uint8_t* src, int bytes, int lane)
{
    const int n = bytes / (int)sizeof(T);
    T* d = reinterpret_cast<T*>(dst);
    const T* s = reinterpret_cast<const T*>(src);
    constexpr int kU = 8;
    for (int i = lane; i < n; i += 32 * kU) {
        T v[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u)
            if (i + 32 * u < n) v[u] = __ldcs(s + i + 32 * u);
#pragma unroll
        for (int u = 0; u < kU; ++u)
            if (i + 32 * u < n) d[i + 32 * u] = v[u];
    }
}

template <int N>
__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const __grid_constant__ CopyArgs<N> a)
{
    const int lane = threadIdx.x & 31;
    grid_dependency_wait();                                 // (of the plan, as a rule)
    grid_dependents_launch();
    const int n_copy = min(max(a.n_copy[0], 0), a.max_copy);
    const int per = a.plane[a.n_planes - 1].piece_end;
    const int64_t n = (int64_t)n_copy * per;
    const int64_t n_warps = ((int64_t)gridDim.x * kCopyThreads) >> 5;
    for (int64_t i = (blockIdx.x * (int64_t)kCopyThreads + threadIdx.x) >> 5; i < n; i += n_warps) {
        const int c = (int)(i / per);
        int e = (int)(i - (int64_t)c * per), k = 0;
        while (a.plane[k].piece_end <= e) ++k;
        const CopyPlane& pl = a.plane[k];
        if (k > 0) e -= a.plane[k - 1].piece_end;
        const int outer = e / pl.per_outer, piece = e - outer * pl.per_outer;
        const int src = a.src[c], dst = a.dst[c], rows = min(max(a.rows[c], 0), a.page_size);
        if (src < 0 || dst < 0 || src == dst || rows == 0) continue;
        const int64_t sr = (int64_t)src * a.page_size, dr = (int64_t)dst * a.page_size;
        if (sr + a.page_size > pl.n_rows || dr + a.page_size > pl.n_rows) {
            if (lane == 0) flag(a.status, KVQ_DEV_BAD_PAGE);
            continue;
        }
        const int64_t first = (int64_t)piece * kPiece;
        const int bytes = (int)min((int64_t)kPiece, rows * pl.row_bytes - first);
        if (bytes <= 0) continue;
        uint8_t* base = pl.base + outer * pl.outer_stride + first;
        uint8_t* d = base + dr * pl.row_bytes;
        const uint8_t* s = base + sr * pl.row_bytes;
        if (pl.width == 16) {
            const int whole = bytes & ~15;                  // the rest, of rows narrower than 16 bytes, below
            copy_piece<uint4>(d, s, whole, lane);
            if (lane < bytes - whole) d[whole + lane] = s[whole + lane];
        } else if (pl.width == 4) {
            copy_piece<uint32_t>(d, s, bytes, lane);
        } else {
            copy_piece<uint8_t>(d, s, bytes, lane);
        }
    }
}

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

int cuda_status(cudaError_t e, const char* entry)
{
    return e == cudaSuccess ? KVQ_OK : set_last_error(KVQ_ECUDA, "%s: %s", entry, cudaGetErrorString(e));
}

size_t up(size_t n) { return (n + 255) / 256 * 256; }

// How a planning kernel runs: one CTA where that is enough, else a cluster; its marks in shared memory where they fit
struct TeamPlan {
    bool one = false, shared = false;
    size_t bytes = 0;                    // of a CTA's marks and keepers
    size_t rows = 0;                     // of its sequences' new tables, where they are in shared memory
};

TeamPlan plan_team(int n_seq, int max_pages, int n_pages, int sets, bool keepers)
{
    TeamPlan t;
    t.one = n_pages <= kPagesOne && n_seq <= kSeqShared && (int64_t)n_seq * max_pages <= kRowsShared;
    t.shared = n_pages <= kPagesShared;
    const Words w(n_pages, t.one ? 1 : kCluster);
    t.bytes = sets * w.bytes() + (keepers ? (size_t)w.each * 16 : 0);
    t.bytes = (t.bytes + 15) / 16 * 16;
    if (keepers && t.shared) {
        const size_t rows = (size_t)(t.one ? n_seq : (n_seq + kCluster - 1) / kCluster) * max_pages * 4;
        t.rows = t.one || t.bytes + rows <= (size_t)kMostSmem ? rows : 0;
    }
    return t;
}

template <typename Args>
cudaError_t launch_team(void (*one)(Args), void (*shared)(Args), void (*global)(Args), const TeamPlan& t, const Args& a,
                        cudaStream_t s)
{
    const size_t smem = t.shared ? t.bytes + t.rows : 0;
    if (t.one) {
        if (smem > kPlainSmem) {
            cudaError_t e = cudaFuncSetAttribute(one, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmemOne);
            if (e != cudaSuccess) return e;
        }
        return launch_dependent(one, dim3(1), dim3(kThreadsOne), smem, s, a);
    }
    const auto kernel = t.shared ? shared : global;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kCluster);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    if (smem > kPlainSmem) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kCluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

int check_pool(const char* E, int n_seq, int max_pages, int page_size, int n_pages)
{
    if (n_seq < 0 || n_seq > 65535) return set_last_error(KVQ_EINVAL, "%s: n_seq outside [0, 65535]", E);
    if (max_pages < 1 || max_pages > kMaxPages || page_size < 1 || n_pages < 0)
        return set_last_error(KVQ_EINVAL, "%s: bad sizes", E);
    if (n_pages > kMaxPool) return set_last_error(KVQ_EINVAL, "%s: a pool of more than 2^29 pages", E);
    if ((int64_t)n_pages * page_size > INT32_MAX)
        return set_last_error(KVQ_EINVAL, "%s: a pool of more than INT32_MAX rows", E);
    return KVQ_OK;
}

int check_fork(const kvq_fork_plan* p, const char* E)
{
    if (!p) return set_last_error(KVQ_EINVAL, "%s: NULL plan", E);
    if (int st = check_pool(E, p->n_seq, p->max_pages, p->page_size, p->n_pages)) return st;
    if (p->n_seq == 0) return KVQ_OK;
    if (!p->parent || !p->block_table || !p->n_held || !p->n_free || !p->seq_len || !p->copy_src || !p->copy_dst ||
        !p->copy_rows || !p->n_copy || (p->n_pages > 0 && !p->free_list))
        return set_last_error(KVQ_EINVAL, "%s: NULL pointer", E);
    if (p->keep_len == p->seq_len || p->parent == p->seq_len || p->parent == p->n_held)
        return set_last_error(KVQ_EINVAL, "%s: parent and keep_len must not be seq_len or n_held", E);
    for (const void* q : {(const void*)p->parent, (const void*)p->keep_len, (const void*)p->block_table,
                          (const void*)p->n_held, (const void*)p->free_list, (const void*)p->n_free,
                          (const void*)p->seq_len, (const void*)p->copy_src, (const void*)p->copy_dst,
                          (const void*)p->copy_rows, (const void*)p->n_copy})
        if (!aligned(q, 4)) return set_last_error(KVQ_EALIGN, "%s: an array is not 4-byte aligned", E);
    return KVQ_OK;
}

int check_compact(const kvq_compact_plan* p, const char* E)
{
    if (!p) return set_last_error(KVQ_EINVAL, "%s: NULL plan", E);
    if (int st = check_pool(E, p->n_seq, p->max_pages, p->page_size, p->n_pages)) return st;
    if (p->max_copy < p->n_pages / 2 || p->max_copy > kMaxCopies)
        return set_last_error(KVQ_EINVAL, "%s: max_copy outside [n_pages / 2, 2^30]", E);
    if (!p->n_free || !p->n_used || !p->n_copy || (p->n_pages > 0 && !p->free_list) ||
        (p->max_copy > 0 && (!p->copy_src || !p->copy_dst || !p->copy_rows)) ||
        (p->n_seq > 0 && (!p->block_table || !p->n_held || !p->new_table)))
        return set_last_error(KVQ_EINVAL, "%s: NULL pointer", E);
    for (const void* q : {(const void*)p->block_table, (const void*)p->n_held, (const void*)p->new_table,
                          (const void*)p->free_list, (const void*)p->n_free, (const void*)p->n_used,
                          (const void*)p->copy_src, (const void*)p->copy_dst, (const void*)p->copy_rows,
                          (const void*)p->n_copy})
        if (!aligned(q, 4)) return set_last_error(KVQ_EALIGN, "%s: an array is not 4-byte aligned", E);
    return KVQ_OK;
}

// the workspace of a plan: offsets as they are handed out
struct Layout {
    size_t bytes = 0;
    size_t take(size_t n)
    {
        const size_t at = bytes;
        bytes += up(n);
        return at;
    }
};

int check_workspace(const char* E, const void* workspace, size_t ws_bytes, size_t need)
{
    if (!workspace || ws_bytes < need)
        return set_last_error(KVQ_EWORKSPACE, "%s: workspace of %zu bytes, need %zu", E, workspace ? ws_bytes : (size_t)0, need);
    if (!aligned(workspace, 256)) return set_last_error(KVQ_EALIGN, "%s: workspace not 256-byte aligned", E);
    return KVQ_OK;
}

TeamPlan plan_team(const kvq_fork_plan& p) { return plan_team(p.n_seq, p.max_pages, p.n_pages, 2, true); }
TeamPlan plan_team(const kvq_compact_plan& p) { return plan_team(p.n_seq, p.max_pages, p.n_pages, 1, false); }

size_t lay_out(const kvq_fork_plan& p, uint8_t* ws, ForkArgs* a)
{
    Layout l;
    const TeamPlan t = plan_team(p);
    const size_t n = (size_t)p.n_seq;
    const size_t row = l.take(t.rows ? 16 : n * p.max_pages * 4), seq = l.take(t.one ? 16 : n * 16);
    const size_t store = l.take(t.shared ? 0 : t.bytes * kCluster);
    if (a) {
        a->row = reinterpret_cast<int32_t*>(ws + row);
        a->seq = reinterpret_cast<int4*>(ws + seq);
        a->store = ws + store;
        a->stride = t.bytes;
        a->rows_shared = t.rows > 0;
    }
    return l.bytes;
}

size_t lay_out(const kvq_compact_plan& p, uint8_t* ws, CompactArgs* a)
{
    Layout l;
    const TeamPlan t = plan_team(p);
    const size_t rank = l.take((size_t)p.n_pages * 4 + 16), store = l.take(t.shared ? 0 : t.bytes * kCluster);
    if (a) {
        a->rank = reinterpret_cast<int32_t*>(ws + rank);
        a->store = ws + store;
        a->stride = t.bytes;
    }
    return l.bytes;
}

}  // namespace

}  // namespace kvq

extern "C" {

size_t kvq_fork_pages_workspace(const kvq_fork_plan* p)
{
    using namespace kvq;
    return check_fork(p, "kvq_fork_pages_workspace") != KVQ_OK || p->n_seq == 0 ? 0 : lay_out(*p, nullptr, nullptr);
}

int kvq_fork_pages(const kvq_fork_plan* p, void* workspace, size_t ws_bytes, uint32_t* dev_status, kvq_stream_t stream)
{
    using namespace kvq;
    const char* E = "kvq_fork_pages";
    if (int st = fault_injected(E)) return st;
    if (int st = check_fork(p, E)) return st;
    if (!aligned(dev_status, 4)) return set_last_error(KVQ_EALIGN, "%s: dev_status misaligned", E);
    if (p->n_seq == 0) return KVQ_OK;
    if (int st = check_workspace(E, workspace, ws_bytes, lay_out(*p, nullptr, nullptr))) return st;
    ForkArgs a{};
    a.p = *p;
    a.status = dev_status;
    lay_out(*p, static_cast<uint8_t*>(workspace), &a);
    return cuda_status(launch_team(fork_pages_kernel<true, true>, fork_pages_kernel<false, true>, fork_pages_kernel<false, false>,
                                   plan_team(*p), a, (cudaStream_t)stream), E);
}

size_t kvq_compact_pages_workspace(const kvq_compact_plan* p)
{
    using namespace kvq;
    return check_compact(p, "kvq_compact_pages_workspace") != KVQ_OK ? 0 : lay_out(*p, nullptr, nullptr);
}

int kvq_compact_pages(const kvq_compact_plan* p, void* workspace, size_t ws_bytes, uint32_t* dev_status,
                      kvq_stream_t stream)
{
    using namespace kvq;
    const char* E = "kvq_compact_pages";
    if (int st = fault_injected(E)) return st;
    if (int st = check_compact(p, E)) return st;
    if (!aligned(dev_status, 4)) return set_last_error(KVQ_EALIGN, "%s: dev_status misaligned", E);
    if (int st = check_workspace(E, workspace, ws_bytes, lay_out(*p, nullptr, nullptr))) return st;
    CompactArgs a{};
    a.p = *p;
    a.status = dev_status;
    lay_out(*p, static_cast<uint8_t*>(workspace), &a);
    return cuda_status(launch_team(compact_pages_kernel<true, true>, compact_pages_kernel<false, true>,
                                   compact_pages_kernel<false, false>, plan_team(*p), a, (cudaStream_t)stream), E);
}

int kvq_copy_pages(const kvq_page_copy* d, uint32_t* dev_status, kvq_stream_t stream)
{
    using namespace kvq;
    const char* E = "kvq_copy_pages";
    if (int st = fault_injected(E)) return st;
    if (!d) return set_last_error(KVQ_EINVAL, "%s: NULL descriptor", E);
    if (d->n_planes < 1 || d->n_planes > kMaxPlanes || !d->planes)
        return set_last_error(KVQ_EINVAL, "%s: n_planes outside [1, 64] or NULL planes", E);
    if (d->page_size < 1 || d->max_copy < 0) return set_last_error(KVQ_EINVAL, "%s: bad sizes", E);
    CopyArgs<kMaxPlanes> a;
    a.n_planes = d->n_planes;
    a.page_size = d->page_size;
    a.max_copy = d->max_copy;
    int64_t end = 0;
    for (int i = 0; i < d->n_planes; ++i) {
        const kvq_plane& s = d->planes[i];
        CopyPlane& t = a.plane[i];
        if (!s.base || s.row_bytes < 1 || s.n_rows < 0 || s.n_outer < 1 ||
            (s.n_outer > 1 && (s.outer_stride < 0 || s.outer_stride / s.row_bytes < s.n_rows)))
            return set_last_error(KVQ_EINVAL, "%s: plane %d: a NULL base or bad sizes", E, i);
        if (s.row_bytes > INT64_MAX / d->page_size) return set_last_error(KVQ_EINVAL, "%s: plane %d: a page too large", E, i);
        const int64_t page = s.row_bytes * d->page_size, per = (page + kPiece - 1) / kPiece;
        if (per > INT32_MAX || s.n_outer > INT32_MAX || end + per * s.n_outer > INT32_MAX)
            return set_last_error(KVQ_EINVAL, "%s: plane %d: a page too large", E, i);
        end += per * s.n_outer;
        t.base = static_cast<uint8_t*>(s.base);
        t.row_bytes = s.row_bytes;
        t.n_rows = s.n_rows;
        t.outer_stride = s.n_outer > 1 ? s.outer_stride : 0;
        t.piece_end = (int32_t)end;
        t.per_outer = (int32_t)per;
        // pages begin at multiples of `page`, pieces at multiples of kPiece of them
        const int64_t all = page | t.outer_stride | (int64_t)(uintptr_t)s.base;
        t.width = all % 16 == 0 ? 16 : all % 4 == 0 && s.row_bytes % 4 == 0 ? 4 : 1;
    }
    if (d->max_copy == 0) return KVQ_OK;
    if (!d->copy_src || !d->copy_dst || !d->copy_rows || !d->n_copy) return set_last_error(KVQ_EINVAL, "%s: NULL pointer", E);
    for (const void* q : {(const void*)d->copy_src, (const void*)d->copy_dst, (const void*)d->copy_rows,
                          (const void*)d->n_copy, (const void*)dev_status})
        if (!aligned(q, 4)) return set_last_error(KVQ_EALIGN, "%s: an array is not 4-byte aligned", E);
    a.src = d->copy_src;
    a.dst = d->copy_dst;
    a.rows = d->copy_rows;
    a.n_copy = d->n_copy;
    a.status = dev_status;
    const int64_t warps = (int64_t)d->max_copy * end;
    const int64_t grid = std::min<int64_t>((warps - 1) / (kCopyThreads / 32) + 1, (int64_t)sm_count() * 8);
    if (d->n_planes > kFewPlanes)
        return cuda_status(launch_dependent(copy_pages_kernel<kMaxPlanes>, dim3((unsigned)grid), dim3(kCopyThreads), 0,
                                            (cudaStream_t)stream, a), E);
    CopyArgs<kFewPlanes> few{a.n_planes, a.page_size, a.max_copy, a.src, a.dst, a.rows, a.n_copy, a.status, {}};
    std::copy(a.plane, a.plane + d->n_planes, few.plane);
    return cuda_status(launch_dependent(copy_pages_kernel<kFewPlanes>, dim3((unsigned)grid), dim3(kCopyThreads), 0,
                                        (cudaStream_t)stream, few), E);
}

}  // extern "C"
