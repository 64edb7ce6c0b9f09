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
constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kMaxPages = 1 << 20;
constexpr int kCluster = 8;              // CTAs of the planning kernels where there is work for them
constexpr int kRun = 16;                 // page marks a thread scans at once (one 16-byte load)

__device__ __forceinline__ void flag(uint32_t* status, unsigned bit)
{
    if (status) atomicOr(status, bit);
}

// Inclusive prefix sum over the CTA; *total = the CTA's sum.  s_warp: kWarps entries.
__device__ __forceinline__ int block_scan(int v, int* s_warp, int* total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(kFull, v, o);
        if (lane >= o) v += u;
    }
    __syncthreads();                                     // an earlier call's readers are done
    if (lane == 31) s_warp[warp] = v;
    __syncthreads();
    int w = s_warp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(kFull, w, o);
        if (lane >= o) w += u;
    }
    *total = __shfl_sync(kFull, w, 31);
    const int before = __shfl_sync(kFull, w, (warp + 31) & 31);
    return warp > 0 ? v + before : v;
}

// The planning kernels are one cluster of CTAs, whose barrier orders their accesses to the workspace and to
// the tables: a launch for what would be five.  Loads of what another CTA of the cluster wrote go past the L1.
template <typename T>
__device__ __forceinline__ T fresh(const T* p) { return __ldcg(p); }

// ------------------------------------------------------------------------------------
// kvq_fork_pages.  Which pages stay held, and who keeps a shared last page, are marks a page: a byte where a
// sequence holds it as a whole page or keeps it (stays), one where the old tables hold it (was), and the
// lowest sequence that has it as a last page (keeper).  Marks are set by plain stores of one value or by a
// minimum, so that no order changes them; free pages come from a scan of the marks in the order of the ids.
// Latency bound: a handful of dependent accesses between cluster barriers.
// ------------------------------------------------------------------------------------
struct ForkArgs {
    kvq_fork_plan p;
    uint32_t* status;
    uint8_t* was;                        // [n_pages, padded to kRun]
    uint8_t* stays;                      // [n_pages, padded]
    int32_t* keeper;                     // [n_pages], set where some sequence's last page is
    int32_t* row;                        // [n_seq][max_pages]: the new tables
    int4* seq;                           // [n_seq]: parent (-1: none), len, last page (-1: none), old n_held
    int32_t* rank;                       // [n_seq]: number among the copies, -1: none
    int32_t* count;                      // [kCluster]: pages given back by a CTA's range; [kCluster]: copies wanted
};

__global__ void __launch_bounds__(kThreads) fork_pages_kernel(const ForkArgs a)
{
    __shared__ int s_warp[kWarps];
    const cg::cluster_group cluster = cg::this_cluster();
    const kvq_fork_plan& p = a.p;
    const int tid = threadIdx.x, lane = tid & 31;
    const int n_cta = (int)cluster.num_blocks(), cta = (int)cluster.block_rank();
    const int all = n_cta * kThreads, me = cta * kThreads + tid;
    const int ps = p.page_size;
    unsigned bits = 0;

    const int n_free0 = p.n_free[0], n_free = min(max(n_free0, 0), p.n_pages);
    if (n_free != n_free0) bits |= KVQ_DEV_BAD_INDEX;

    // ---- marks cleared; every sequence's parent, rows and last page
    const int n_marks = (p.n_pages + kRun - 1) / kRun;      // 16-byte words of marks
    for (int i = me; i < n_marks; i += all) {
        reinterpret_cast<uint4*>(a.was)[i] = make_uint4(0u, 0u, 0u, 0u);
        reinterpret_cast<uint4*>(a.stays)[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    for (int s = me; s < p.n_seq; s += all) {
        int par = p.parent[s];
        if (par < -1 || par >= p.n_seq) {
            bits |= KVQ_DEV_BAD_INDEX;
            par = -1;
        }
        const int held = p.n_held[s], own = min(max(held, 0), p.max_pages);
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
                if (page >= 0 && page < p.n_pages) {
                    last = page;
                    a.keeper[page] = INT_MAX;
                }
            }
        }
        a.seq[s] = make_int4(par, len, last, own);
    }
    cluster.sync();

    // ---- the pages that the tables held, and that the new ones hold whole.  A warp takes 128 entries.
    const int warp = me >> 5, n_warps = all >> 5;
    const int per_row = (p.max_pages + 127) / 128;
    for (int64_t i = warp; i < (int64_t)p.n_seq * per_row; i += n_warps) {
        const int s = (int)(i / per_row), e0 = (int)(i - (int64_t)s * per_row) * 128;
        const int4 q = fresh(a.seq + s);
        const int32_t* mine = p.block_table + (int64_t)s * p.max_pages;
        const int32_t* from = p.block_table + (int64_t)q.x * p.max_pages;
        int32_t* to = a.row + (int64_t)s * p.max_pages;
        const int whole = q.y / ps, need = (q.y + ps - 1) / ps;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int e = e0 + 32 * u + lane;
            if (e < q.w) {
                const int page = mine[e];
                if (page >= 0 && page < p.n_pages) a.was[page] = 1;
                else bits |= KVQ_DEV_BAD_PAGE;
            }
            if (e < need) {
                int page = from[e];
                if (page < 0 || page >= p.n_pages) {
                    bits |= KVQ_DEV_BAD_PAGE;
                    page = -1;
                } else if (e < whole) {
                    a.stays[page] = 1;
                }
                to[e] = page;
            }
        }
        if (e0 == 0 && lane == 0 && q.z >= 0) atomicMin(a.keeper + q.z, s);
    }
    cluster.sync();

    // ---- who copies, in the order of the sequences (one CTA); who keeps its last page
    if (cta == 0) {
        int carry = 0;
        for (int c = 0; c < p.n_seq; c += kThreads) {
            const int s = c + tid;
            bool copy = false;
            int last = -1;
            if (s < p.n_seq) {
                last = fresh(a.seq + s).z;
                // (a mark that another thread sets here is for a keeper that is not s: s copies either way)
                copy = last >= 0 && (fresh(a.keeper + last) != s || fresh(a.stays + last) != 0);
            }
            int sum;
            const int r = block_scan(copy ? 1 : 0, s_warp, &sum);
            if (s < p.n_seq) {
                a.rank[s] = copy ? carry + r - 1 : -1;
                if (last >= 0 && !copy) a.stays[last] = 1;
            }
            carry += sum;
        }
        if (tid == 0) a.count[kCluster] = carry;
    }
    cluster.sync();

    // ---- pages given back: each CTA a range of ids
    const int per_cta = (n_marks + n_cta - 1) / n_cta;
    const int m0 = min(cta * per_cta, n_marks), m1 = min(m0 + per_cta, n_marks);
    auto given = [&](int i) {                               // a byte of 1 for each page of word i that goes back
        const uint4 w = fresh(reinterpret_cast<const uint4*>(a.was) + i), st = fresh(reinterpret_cast<const uint4*>(a.stays) + i);
        return make_uint4(w.x & ~st.x, w.y & ~st.y, w.z & ~st.z, w.w & ~st.w);
    };
    auto ones = [](uint4 g) { return __popc(g.x) + __popc(g.y) + __popc(g.z) + __popc(g.w); };
    int mine = 0;
    for (int i = m0 + tid; i < m1; i += kThreads) mine += ones(given(i));
    int sum;
    (void)block_scan(mine, s_warp, &sum);
    if (tid == 0) a.count[cta] = sum;
    cluster.sync();

    int above = 0, total = 0;                               // given back by ranges of higher ids; by all
    for (int c = 0; c < n_cta; ++c) {
        const int v = fresh(a.count + c);
        total += v;
        if (c > cta) above += v;
    }
    // the highest id first: chunks of words from the top
    for (int top = m1; sum > 0 && top > m0; top -= kThreads) {
        const int i = top - 1 - tid;
        const uint4 g = i >= m0 ? given(i) : make_uint4(0u, 0u, 0u, 0u);
        const int n = ones(g);
        int in_chunk;
        int at = n_free + above + block_scan(n, s_warp, &in_chunk) - n;
        const uint32_t w[4] = {g.x, g.y, g.z, g.w};
        if (n > 0) {
#pragma unroll
            for (int b = kRun - 1; b >= 0; --b)
                if (w[b / 4] >> (8 * (b % 4)) & 1) {
                    if (at < p.n_pages) p.free_list[at] = i * kRun + b;
                    else bits |= KVQ_DEV_BAD_PAGE;
                    ++at;
                }
        }
        above += in_chunk;
    }
    cluster.sync();

    // ---- pages for the copies, and the tables
    const int have = min(n_free + total, p.n_pages);
    const int want = fresh(a.count + kCluster), used = min(want, have);
    for (int s = me; s < p.n_seq; s += all) {
        const int4 q = fresh(a.seq + s);
        const int r = fresh(a.rank + s);
        int len = q.y;
        if (r >= 0) {
            if (r < have) {
                const int page = fresh(p.free_list + have - 1 - r);
                a.row[(int64_t)s * p.max_pages + len / ps] = page;
                p.copy_src[r] = q.z;
                p.copy_dst[r] = page;
                p.copy_rows[r] = len % ps;
            } else {
                bits |= KVQ_DEV_NO_PAGE;
                len -= len % ps;
                a.row[(int64_t)s * p.max_pages + len / ps] = -1;
            }
        }
        if (s >= used) p.copy_src[s] = p.copy_dst[s] = p.copy_rows[s] = -1;
        p.seq_len[s] = len;
        p.n_held[s] = (len + ps - 1) / ps;
    }
    if (me == 0) {
        p.n_free[0] = have - used;
        p.n_copy[0] = used;
    }
    cluster.sync();
    for (int64_t i = warp; i < (int64_t)p.n_seq * per_row; i += n_warps) {
        const int s = (int)(i / per_row), e0 = (int)(i - (int64_t)s * per_row) * 128;
        const int4 q = fresh(a.seq + s);
        const int need = (q.y + ps - 1) / ps;               // (a refused last page is -1 in the row)
        int32_t* to = p.block_table + (int64_t)s * p.max_pages;
        const int32_t* from = a.row + (int64_t)s * p.max_pages;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int e = e0 + 32 * u + lane;
            if (e < need) to[e] = fresh(from + e);
            else if (e < q.w) to[e] = -1;
        }
    }
    if (bits) flag(a.status, bits);
}

// ------------------------------------------------------------------------------------
// kvq_compact_pages: a mark a held page; the number of the held pages is U, and the i-th held page of id U or more
// goes to the i-th page below U without a mark.
// ------------------------------------------------------------------------------------
struct CompactArgs {
    kvq_compact_plan p;
    uint32_t* status;
    uint8_t* used;                       // [n_pages, padded to kRun]
    int32_t* rank;                       // [n_pages]: number of a page among those that move
    int32_t* count;                      // [kCluster] held pages of a CTA's range, [kCluster] unheld ones below U,
                                         // [kCluster] held ones from U on
};

__global__ void __launch_bounds__(kThreads) compact_pages_kernel(const CompactArgs a)
{
    __shared__ int s_warp[kWarps];
    const cg::cluster_group cluster = cg::this_cluster();
    const kvq_compact_plan& p = a.p;
    const int tid = threadIdx.x, lane = tid & 31;
    const int n_cta = (int)cluster.num_blocks(), cta = (int)cluster.block_rank();
    const int all = n_cta * kThreads, me = cta * kThreads + tid;
    unsigned bits = 0;

    const int n_marks = (p.n_pages + kRun - 1) / kRun;
    for (int i = me; i < n_marks; i += all) reinterpret_cast<uint4*>(a.used)[i] = make_uint4(0u, 0u, 0u, 0u);
    cluster.sync();

    const int warp = me >> 5, n_warps = all >> 5;
    const int per_row = (p.max_pages + 127) / 128;
    for (int64_t i = warp; i < (int64_t)p.n_seq * per_row; i += n_warps) {
        const int s = (int)(i / per_row), e0 = (int)(i - (int64_t)s * per_row) * 128;
        const int held0 = p.n_held[s], held = min(max(held0, 0), p.max_pages);
        if (held != held0) bits |= KVQ_DEV_BAD_INDEX;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int e = e0 + 32 * u + lane;
            if (e >= held) continue;
            const int page = p.block_table[(int64_t)s * p.max_pages + e];
            if (page >= 0 && page < p.n_pages) a.used[page] = 1;
            else bits |= KVQ_DEV_BAD_PAGE;
        }
    }
    cluster.sync();

    const int per_cta = (n_marks + n_cta - 1) / n_cta;
    const int m0 = min(cta * per_cta, n_marks), m1 = min(m0 + per_cta, n_marks);
    auto marks = [&](int i) { return fresh(reinterpret_cast<const uint4*>(a.used) + i); };
    auto ones = [](uint4 g) { return __popc(g.x) + __popc(g.y) + __popc(g.z) + __popc(g.w); };
    int mine = 0, sum;
    for (int i = m0 + tid; i < m1; i += kThreads) mine += ones(marks(i));
    (void)block_scan(mine, s_warp, &sum);
    if (tid == 0) a.count[cta] = sum;
    cluster.sync();
    int n_used = 0;
    for (int c = 0; c < n_cta; ++c) n_used += fresh(a.count + c);

    // pages that move (held, from U on) or are moved to (not held, below U): a bit each of the run
    auto places = [&](int i) {
        const uint4 g = marks(i);
        const uint32_t w[4] = {g.x, g.y, g.z, g.w};
        unsigned hole = 0, move = 0;
#pragma unroll
        for (int b = 0; b < kRun; ++b) {
            const int page = i * kRun + b;
            const bool on = w[b / 4] >> (8 * (b % 4)) & 1;
            if (page < n_used && !on) hole |= 1u << b;
            if (page >= n_used && on) move |= 1u << b;
        }
        return make_uint2(hole, move);
    };
    int holes = 0, moves = 0;
    for (int i = m0 + tid; i < m1; i += kThreads) {
        const uint2 q = places(i);
        holes += __popc(q.x);
        moves += __popc(q.y);
    }
    (void)block_scan(holes, s_warp, &sum);
    if (tid == 0) a.count[kCluster + cta] = sum;
    (void)block_scan(moves, s_warp, &sum);
    if (tid == 0) a.count[2 * kCluster + cta] = sum;
    cluster.sync();
    int hole_at = 0, move_at = 0, total = 0;
    for (int c = 0; c < n_cta; ++c) {
        const int h = fresh(a.count + kCluster + c), m = fresh(a.count + 2 * kCluster + c);
        total += m;
        if (c < cta) {
            hole_at += h;
            move_at += m;
        }
    }
    for (int low = m0; low < m1; low += kThreads) {
        const int i = low + tid;
        const uint2 q = i < m1 ? places(i) : make_uint2(0u, 0u);
        int sum_h, sum_m;
        int h = hole_at + block_scan(__popc(q.x), s_warp, &sum_h) - __popc(q.x);
        int m = move_at + block_scan(__popc(q.y), s_warp, &sum_m) - __popc(q.y);
#pragma unroll
        for (int b = 0; b < kRun; ++b) {
            if (q.x >> b & 1) p.copy_dst[h++] = i * kRun + b;
            if (q.y >> b & 1) {
                p.copy_src[m] = i * kRun + b;
                a.rank[i * kRun + b] = m++;
            }
        }
        hole_at += sum_h;
        move_at += sum_m;
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
    cluster.sync();

    for (int64_t i = warp; i < (int64_t)p.n_seq * per_row; i += n_warps) {
        const int s = (int)(i / per_row), e0 = (int)(i - (int64_t)s * per_row) * 128;
        const int held = min(max(p.n_held[s], 0), p.max_pages);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int e = e0 + 32 * u + lane;
            if (e >= p.max_pages) continue;
            const int64_t at = (int64_t)s * p.max_pages + e;
            int page = -1;
            if (e < held) {
                page = p.block_table[at];
                if (page < 0 || page >= p.n_pages) page = -1;
                else if (page >= n_used) page = fresh(p.copy_dst + fresh(a.rank + page));
            }
            p.new_table[at] = page;
        }
    }
    if (bits) flag(a.status, bits);
}

// ------------------------------------------------------------------------------------
// kvq_copy_pages: pieces of 4 KiB (a warp each, its loads before its stores) of every outer array of every
// plane, for every entry of the list; as many warps as the machine holds go over them.  Bound by the
// bytes, read and written once.
// ------------------------------------------------------------------------------------
constexpr int kMaxPlanes = 64;
constexpr int kCopyThreads = 256;
constexpr int kPiece = 4096;

struct CopyPlane {
    uint8_t* base;
    int64_t row_bytes, n_rows, outer_stride;
    int32_t piece_end;                   // pieces of an entry in this plane and the ones before it
    int32_t per_outer;                   // pieces of a page in one outer array
    int32_t width;                       // bytes at a time: 16, 4 or 1
};

struct CopyArgs {
    int32_t n_planes, page_size, max_copy;
    const int32_t *src, *dst, *rows, *n_copy;
    uint32_t* status;
    CopyPlane plane[kMaxPlanes];
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

__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const __grid_constant__ CopyArgs a)
{
    const int lane = threadIdx.x & 31;
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

// one CTA where its threads can go over the tables and the marks in a few rounds, else a cluster
template <typename Args>
cudaError_t launch_plan(void (*kernel)(Args), const Args& a, int64_t entries, int64_t pages, cudaStream_t s)
{
    const int n_cta = entries <= 8 * kThreads && pages <= 8 * kThreads * kRun ? 1 : kCluster;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)n_cta);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)n_cta;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

int check_pool(const char* E, int n_seq, int max_pages, int page_size, int n_pages)
{
    if (n_seq < 0 || n_seq > 65535) return set_last_error(KVQ_EINVAL, "%s: n_seq outside [0, 65535]", E);
    if (max_pages < 1 || max_pages > kMaxPages || page_size < 1 || n_pages < 0)
        return set_last_error(KVQ_EINVAL, "%s: bad sizes", E);
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
    if (p->max_copy < p->n_pages / 2) return set_last_error(KVQ_EINVAL, "%s: max_copy below n_pages / 2", E);
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

size_t lay_out(const kvq_fork_plan& p, uint8_t* ws, ForkArgs* a)
{
    Layout l;
    const size_t marks = ((size_t)p.n_pages + kRun - 1) / kRun * kRun, n = (size_t)p.n_seq;
    const size_t was = l.take(marks), stays = l.take(marks), keeper = l.take((size_t)p.n_pages * 4);
    const size_t row = l.take(n * p.max_pages * 4), seq = l.take(n * 16), rank = l.take(n * 4);
    const size_t count = l.take((kCluster + 1) * 4);
    if (a) {
        a->was = ws + was;
        a->stays = ws + stays;
        a->keeper = reinterpret_cast<int32_t*>(ws + keeper);
        a->row = reinterpret_cast<int32_t*>(ws + row);
        a->seq = reinterpret_cast<int4*>(ws + seq);
        a->rank = reinterpret_cast<int32_t*>(ws + rank);
        a->count = reinterpret_cast<int32_t*>(ws + count);
    }
    return l.bytes;
}

size_t lay_out(const kvq_compact_plan& p, uint8_t* ws, CompactArgs* a)
{
    Layout l;
    const size_t used = l.take(((size_t)p.n_pages + kRun - 1) / kRun * kRun), rank = l.take((size_t)p.n_pages * 4);
    const size_t count = l.take(3 * kCluster * 4);
    if (a) {
        a->used = ws + used;
        a->rank = reinterpret_cast<int32_t*>(ws + rank);
        a->count = reinterpret_cast<int32_t*>(ws + count);
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
    return cuda_status(launch_plan(fork_pages_kernel, a, (int64_t)p->n_seq * p->max_pages, p->n_pages, (cudaStream_t)stream), E);
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
    return cuda_status(launch_plan(compact_pages_kernel, a, (int64_t)p->n_seq * p->max_pages, p->n_pages, (cudaStream_t)stream), E);
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
    CopyArgs a{};
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
    const int64_t grid = std::min<int64_t>((warps * 32 + kCopyThreads - 1) / kCopyThreads, (int64_t)sm_count() * 8);
    copy_pages_kernel<<<(unsigned)grid, kCopyThreads, 0, (cudaStream_t)stream>>>(a);
    return cuda_status(cudaGetLastError(), E);
}

}  // extern "C"
