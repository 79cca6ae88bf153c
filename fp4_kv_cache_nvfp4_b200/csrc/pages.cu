// The pages' own operations on a paged cache: copy, fork, free, compact.
//
// State that the caller keeps on the device: the page table, one reference
// count per physical page (how many page-table entries hold it; 0: free) and
// the sequences' lengths.  The counts are the allocator: a page is free when
// its count is 0, and new pages are the free ones with the lowest numbers, so
// the same state and request give the same pages on every run.
//
// What it costs: 4 bytes per page to find free or live pages, 4 bytes per
// page-table entry, and page_size * 288 bytes read and written for a page that
// is copied (codes 128, scales 16, indexer K 128 and pooled indexer K 16 bytes
// per entry).
// Small requests are bound by their two or three launches (about 10 us in a graph,
// each waiting for the one before it), large ones by the copies' latency: a CTA moves a
// whole page, loads before stores, and of compact's CTAs four fit on an SM (63 registers).
// Measured in a graph: 256 forks in 3 caches 19 us, compacting 12,000 pages 31 us
// (99 MB, 3.2 TB/s); a call from Python takes 41 and 39 us, the host's share included.
#include <algorithm>

#include "checks.h"
#include "common.cuh"
#include "kernels.h"

namespace csa2 {

constexpr int kMaxCaches = 16;          // caches (layers) that share a page table
constexpr int kMaxForks = 1024;         // forks of one call
constexpr int kMaxPages = 1 << 22;      // physical pages of a cache
constexpr int PG_CHUNK = 4096;          // reference counts per CTA
constexpr int PG_SCAN_THREADS = 1024;   // four counts per thread
constexpr int PG_COPY_THREADS = 256;
// Up to this many chunks every CTA counts the chunks before its own (and, to
// compact, all) itself from L2; above, a kernel counts each chunk once first.
// Measured, compact with little to move, counting itself / by a kernel: 255
// pages 10.6 / 11.9 us, 12,000 pages 12.6 / 13.4, 60,000 pages 14.7 / 12.9,
// 240,000 pages 27.5 / 13.3.
constexpr int PG_SELF_COUNT = 6;

struct PageCaches {
    uint8_t* codes[kMaxCaches];
    uint8_t* scales[kMaxCaches];
    uint16_t* idx[kMaxCaches];
    uint16_t* pooled[kMaxCaches];
    int n, page_size;
};

// Copies a physical page in every array of cache c.  Its 16-byte pieces (18 per
// entry: codes 8, indexer K 8, scales 1, pooled indexer K 1) are one index space,
// so that a page of 64 entries is one round of five loads in flight per thread, not
// one latency per array.
__device__ __forceinline__ void copy_page(const PageCaches& p, int c, int32_t src, int32_t dst) {
    const int ps = p.page_size, n = ps * (p.idx[c] ? (p.pooled[c] ? 18 : 17) : 9);
    auto piece = [&](int i, int32_t page) -> uint4* {
        uint8_t* base = p.codes[c];
        int per = 8 * ps;
        if (i >= per) {
            i -= per;
            if (i < ps) base = p.scales[c], per = ps;
            else if ((i -= ps) < per) base = reinterpret_cast<uint8_t*>(p.idx[c]);
            else i -= per, base = reinterpret_cast<uint8_t*>(p.pooled[c]), per = ps;
        }
        return reinterpret_cast<uint4*>(base) + (int64_t)per * page + i;
    };
    constexpr int U = 5;
    for (int i0 = threadIdx.x; i0 < n; i0 += U * PG_COPY_THREADS) {
        uint4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i0 + u * PG_COPY_THREADS < n) v[u] = *piece(i0 + u * PG_COPY_THREADS, src);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i0 + u * PG_COPY_THREADS < n) *piece(i0 + u * PG_COPY_THREADS, dst) = v[u];
    }
}

// ---- copy: pairs of pages -----------------------------------------------------
__global__ void __launch_bounds__(PG_COPY_THREADS) pages_copy_kernel(PageCaches p, const int32_t* src,
                                                                     const int32_t* dst, int n, int32_t n_pages,
                                                                     int32_t* err) {
    pdl_wait();
    pdl_trigger();
    for (int i = blockIdx.x; i < n * p.n; i += gridDim.x) {
        const int pair = i / p.n;
        const int32_t s = src[pair], d = dst[pair];
        if (s == -1 || d == -1) continue;
        if (s < 0 || s >= n_pages || d < 0 || d >= n_pages) {
            if (threadIdx.x == 0) dev_error(err, CSA2_DEV_PAGE);
            continue;
        }
        if (s != d) copy_page(p, i % p.n, s, d);
    }
}

// ---- finding pages ------------------------------------------------------------------
// Four counts from a multiple of four on.
__device__ __forceinline__ int4 load_refs(const int32_t* refs, int32_t n_pages, int32_t at) {
    if (at + 4 <= n_pages) return *reinterpret_cast<const int4*>(refs + at);
    int4 v = make_int4(1, 1, 1, 1);  // behind the last page: never free
    if (at < n_pages) v.x = refs[at];
    if (at + 1 < n_pages) v.y = refs[at + 1];
    if (at + 2 < n_pages) v.z = refs[at + 2];
    return v;
}

struct ForkPlan {
    int32_t child;   // row to fill, -1: nothing to do
    int32_t parent;
    int32_t len;
    int32_t rank;    // rank of the new page among the free ones, -1: no partial page
};

struct ForkArgs {
    PageCaches p;
    int32_t* table;
    int32_t* refs;
    int32_t* lens;
    const int32_t* parents;
    const int32_t* children;
    int32_t* chunk_free;  // [chunks]
    int32_t* free_list;   // [n]: free pages, ascending
    int32_t* n_free;      // [1]
    ForkPlan* plan;       // [n]
    int32_t* err;
    int32_t n, n_seqs, max_pages, n_pages, page_shift;
};

__device__ __forceinline__ uint32_t free_of(const int4& v) {
    return (uint32_t)(v.x == 0) + (v.y == 0) + (v.z == 0) + (v.w == 0);
}

// Free pages of each chunk.
__global__ void __launch_bounds__(PG_SCAN_THREADS) fork_count_kernel(ForkArgs a) {
    __shared__ uint32_t tmp[64];
    pdl_wait();
    pdl_trigger();
    uint32_t total;
    block_excl_scan(free_of(load_refs(a.refs, a.n_pages, (int)blockIdx.x * PG_CHUNK + 4 * (int)threadIdx.x)), tmp, &total);
    if (threadIdx.x == 0) a.chunk_free[blockIdx.x] = (int)total;
}

// CTAs 0 .. chunks-1 list the first n free pages, ascending; the last CTA checks
// the requests and ranks those that need a page.
__global__ void __launch_bounds__(PG_SCAN_THREADS) fork_list_kernel(ForkArgs a) {
    __shared__ uint32_t tmp[64];
    __shared__ __align__(16) int32_t s_child[kMaxForks], s_parent[kMaxForks];
    const int tid = threadIdx.x, chunks = (int)gridDim.x - 1;
    pdl_wait();
    pdl_trigger();
    if ((int)blockIdx.x < chunks) {
        uint32_t mine = 0;
        if (chunks <= PG_SELF_COUNT) {
            for (int c = 0; c < (int)blockIdx.x; ++c) mine += free_of(load_refs(a.refs, a.n_pages, c * PG_CHUNK + 4 * tid));
        } else {
            for (int c = tid; c < (int)blockIdx.x; c += PG_SCAN_THREADS) mine += (uint32_t)a.chunk_free[c];
        }
        uint32_t before, total;
        block_excl_scan(mine, tmp, &before);  // the scan's total
        const int at = (int)blockIdx.x * PG_CHUNK + 4 * tid;
        const int4 v = load_refs(a.refs, a.n_pages, at);
        const int f[4] = {v.x == 0, v.y == 0, v.z == 0, v.w == 0};
        uint32_t r = before + block_excl_scan((uint32_t)(f[0] + f[1] + f[2] + f[3]), tmp, &total);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (f[e]) {
                if (r < (uint32_t)a.n) a.free_list[r] = at + e;
                ++r;
            }
        if ((int)blockIdx.x + 1 == chunks && tid == 0) *a.n_free = (int)(before + total);
        return;
    }
    if (tid < kMaxForks) {
        s_child[tid] = tid < a.n ? a.children[tid] : -1;
        s_parent[tid] = tid < a.n ? a.parents[tid] : -1;
    }
    __syncthreads();
    ForkPlan pl{-1, -1, 0, -1};
    bool part = false;
    if (tid < a.n) {
        const int32_t c = s_child[tid], f = s_parent[tid];
        if (c == -1 && f == -1) {
            // padding
        } else if (c < 0 || c >= a.n_seqs || f < 0 || f >= a.n_seqs) {
            dev_error(a.err, CSA2_DEV_SLOT);
        } else {
            bool taken = a.lens[c] != 0;  // the row is in use
            for (int j = 0; j < a.n; j += 4) {  // (behind the last request both are -1)
                const int4 x = *reinterpret_cast<const int4*>(s_child + j), y = *reinterpret_cast<const int4*>(s_parent + j);
                taken |= (x.x == c && j < tid) || (x.y == c && j + 1 < tid) || (x.z == c && j + 2 < tid) ||
                         (x.w == c && j + 3 < tid) || y.x == c || y.y == c || y.z == c || y.w == c;
            }
            const int32_t len = a.lens[f];
            if (taken) {
                dev_error(a.err, CSA2_DEV_SLOT);
            } else if (len < 0 || ((int64_t)len + (1 << a.page_shift) - 1) >> a.page_shift > a.max_pages) {
                dev_error(a.err, CSA2_DEV_LEN);
            } else {
                const int32_t full = len >> a.page_shift;
                part = (len & ((1 << a.page_shift) - 1)) != 0;
                if (part) {
                    const int32_t pg = a.table[(int64_t)f * a.max_pages + full];
                    if (pg < 0 || pg >= a.n_pages) {
                        dev_error(a.err, CSA2_DEV_PAGE);
                        part = false;
                    } else {
                        pl = ForkPlan{c, f, len, 0};
                    }
                } else {
                    pl = ForkPlan{c, f, len, -1};
                }
            }
        }
    }
    uint32_t total;
    const uint32_t rank = block_excl_scan(part ? 1u : 0u, tmp, &total);
    if (part) pl.rank = (int)rank;
    if (tid < a.n) a.plan[tid] = pl;
}

// CTA (i, 0) fills child i's row and counts its pages; CTA (i, 1 + c) copies
// the partly filled last page of cache c.
__global__ void __launch_bounds__(PG_COPY_THREADS) fork_apply_kernel(ForkArgs a) {
    pdl_wait();
    pdl_trigger();
    const ForkPlan pl = a.plan[blockIdx.x];
    if (pl.child < 0) return;
    const int tid = threadIdx.x;
    if (pl.rank >= 0 && pl.rank >= *a.n_free) {  // no page left: the child stays free
        if (blockIdx.y == 0 && tid == 0) dev_error(a.err, CSA2_DEV_POOL);
        return;
    }
    const int32_t full = pl.len >> a.page_shift;
    const int32_t* from = a.table + (int64_t)pl.parent * a.max_pages;
    const int32_t page = pl.rank >= 0 ? a.free_list[pl.rank] : -1;
    if (blockIdx.y > 0) {
        if (page >= 0) copy_page(a.p, (int)blockIdx.y - 1, from[full], page);
        return;
    }
    int32_t* to = a.table + (int64_t)pl.child * a.max_pages;
    for (int j = tid; j < a.max_pages; j += PG_COPY_THREADS) {
        int32_t v = j < full ? from[j] : -1;
        if (j < full) {
            if (v >= 0 && v < a.n_pages) {
                atomicAdd(a.refs + v, 1);
            } else {
                dev_error(a.err, CSA2_DEV_PAGE);
                v = -1;
            }
        } else if (j == full && page >= 0) {
            v = page;
            a.refs[page] = 1;
        }
        to[j] = v;
    }
    if (tid == 0) a.lens[pl.child] = pl.len;
}

// ---- free ------------------------------------------------------------------------------
// One CTA per sequence of the list.  The exchange takes each entry once, so a
// sequence listed twice is freed once.
__global__ void __launch_bounds__(PG_COPY_THREADS) pages_free_kernel(int32_t* table, int32_t* refs, int32_t* lens,
                                                                     const int32_t* seqs, int32_t n_seqs,
                                                                     int32_t max_pages, int32_t n_pages,
                                                                     int32_t* err) {
    pdl_wait();
    pdl_trigger();
    const int32_t b = seqs[blockIdx.x];
    if (b == -1) return;
    if (b < 0 || b >= n_seqs) {
        if (threadIdx.x == 0) dev_error(err, CSA2_DEV_SLOT);
        return;
    }
    int32_t* row = table + (int64_t)b * max_pages;
    for (int j = threadIdx.x; j < max_pages; j += PG_COPY_THREADS) {
        if (row[j] == -1) continue;
        const int32_t pg = atomicExch(row + j, -1);
        if (pg == -1) continue;
        if (pg < 0 || pg >= n_pages) {
            dev_error(err, CSA2_DEV_PAGE);
        } else if (atomicSub(refs + pg, 1) <= 0) {  // held more often than counted
            atomicAdd(refs + pg, 1);
            dev_error(err, CSA2_DEV_PAGE);
        }
    }
    if (threadIdx.x == 0) lens[b] = 0;
}

// ---- compact -----------------------------------------------------------------------------
// With n live pages, the live ones numbered n and above move into the free
// numbers below n, the k-th lowest into the k-th lowest: as few moves as there
// can be, and no page is both read and written, so all move at once.
struct CompactArgs {
    PageCaches p;
    int32_t* table;
    int32_t* refs;
    int32_t* page_map;    // [n_pages] out
    int32_t* n_live_out;  // [1]
    int32_t* chunk_live;  // [chunks]
    int32_t* holes;       // [n_pages]: free pages below n_live, ascending
    int32_t* high;        // [n_pages]: live pages from n_live on, ascending
    int32_t* where;       // [n_pages]: p itself (stays), -1 (free), -2 - k (the k-th high page)
    int32_t* n_move;      // [1]
    int32_t* err;
    int64_t table_size;
    int32_t n_pages;
};

// Live pages (count > 0) of each chunk of PG_CHUNK.
__device__ __forceinline__ uint32_t live_in(const int32_t* refs, int n_pages, int at, int below) {
    const int4 v = load_refs(refs, n_pages, at);
    const int end = min(n_pages, below);
    return (uint32_t)(v.x > 0 && at < end) + (v.y > 0 && at + 1 < end) + (v.z > 0 && at + 2 < end) +
           (v.w > 0 && at + 3 < end);
}
__global__ void __launch_bounds__(PG_SCAN_THREADS) compact_count_kernel(CompactArgs a) {
    __shared__ uint32_t tmp[64];
    pdl_wait();
    pdl_trigger();
    uint32_t total;
    block_excl_scan(live_in(a.refs, a.n_pages, (int)blockIdx.x * PG_CHUNK + 4 * (int)threadIdx.x, a.n_pages), tmp, &total);
    if (threadIdx.x == 0) a.chunk_live[blockIdx.x] = (int)total;
}

// Every CTA sums the live pages of all chunks, of those before its own and of
// those below n_live, then ranks its pages.
__global__ void __launch_bounds__(PG_SCAN_THREADS) compact_list_kernel(CompactArgs a) {
    __shared__ uint32_t tmp[64];
    const int tid = threadIdx.x, chunks = (int)gridDim.x, at = (int)blockIdx.x * PG_CHUNK + 4 * tid;
    const bool self = chunks <= PG_SELF_COUNT;
    pdl_wait();
    pdl_trigger();
    uint32_t mine = 0, all = 0;
    if (self) {
        for (int c = 0; c < chunks; ++c) {
            const uint32_t x = live_in(a.refs, a.n_pages, c * PG_CHUNK + 4 * tid, a.n_pages);
            all += x;
            if (c < (int)blockIdx.x) mine += x;
        }
    } else {
        for (int c = tid; c < chunks; c += PG_SCAN_THREADS) {
            const uint32_t x = (uint32_t)a.chunk_live[c];
            all += x;
            if (c < (int)blockIdx.x) mine += x;
        }
    }
    uint32_t before, n_live, low;
    block_excl_scan(mine, tmp, &before);
    block_excl_scan(all, tmp, &n_live);
    // live pages below n_live: whole chunks, and the part of the chunk it falls into
    const int cut = (int)(n_live / PG_CHUNK);
    uint32_t l = 0;
    if (self)
        for (int c = 0; c < cut; ++c) l += live_in(a.refs, a.n_pages, c * PG_CHUNK + 4 * tid, a.n_pages);
    else
        for (int c = tid; c < cut; c += PG_SCAN_THREADS) l += (uint32_t)a.chunk_live[c];
    l += live_in(a.refs, a.n_pages, cut * PG_CHUNK + 4 * tid, (int)n_live);
    block_excl_scan(l, tmp, &low);
    const int4 v = load_refs(a.refs, a.n_pages, at);
    const int r[4] = {v.x, v.y, v.z, v.w};
    uint32_t live[4], c = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        live[e] = at + e < a.n_pages && r[e] > 0;
        c += live[e];
    }
    uint32_t total;
    uint32_t rank = before + block_excl_scan(c, tmp, &total);  // live pages before this one
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int p = at + e;
        if (p >= a.n_pages) break;
        int w = -1;
        if (live[e]) {
            w = p;
            if (p >= (int)n_live) {
                const int k = (int)(rank - low);
                a.high[k] = p;
                w = -2 - k;
            }
        } else if (p < (int)n_live) {
            a.holes[p - (int)rank] = p;
        }
        a.where[p] = w;
        rank += live[e];
    }
    if (blockIdx.x == 0 && tid == 0) {
        *a.n_move = (int)(n_live - low);
        *a.n_live_out = (int)n_live;
    }
}

__global__ void __launch_bounds__(PG_COPY_THREADS) compact_move_kernel(CompactArgs a) {
    pdl_wait();
    pdl_trigger();
    const int n_move = *a.n_move;
    auto moved = [&](int32_t w) { return w <= -2 ? a.holes[-2 - w] : w; };
    const int64_t stride = (int64_t)gridDim.x * PG_COPY_THREADS, first = (int64_t)blockIdx.x * PG_COPY_THREADS + threadIdx.x;
    for (int64_t i = first; i < a.table_size; i += stride) {
        const int32_t pg = a.table[i];
        if (pg == -1) continue;
        int32_t to = -1;
        if (pg >= 0 && pg < a.n_pages) to = moved(a.where[pg]);
        if (to < 0) dev_error(a.err, CSA2_DEV_PAGE);  // not a live page
        if (to != pg) a.table[i] = to;
    }
    for (int64_t i = first; i < a.n_pages; i += stride) a.page_map[i] = moved(a.where[i]);
    for (int64_t i = first; i < n_move; i += stride) {
        const int32_t s = a.high[i], d = a.holes[i];
        a.refs[d] = a.refs[s];
        a.refs[s] = 0;
    }
    for (int64_t i = blockIdx.x; i < (int64_t)n_move * a.p.n; i += gridDim.x) {
        const int k = (int)(i / a.p.n);
        copy_page(a.p, (int)(i % a.p.n), a.high[k], a.holes[k]);
    }
}

struct PagesWs {
    size_t chunks, count, list_a, list_b, list_c, plan, total;
};
static PagesWs pages_ws_layout(int64_t n_pages, int32_t n) {
    PagesWs w{};
    size_t o = 0;
    auto take = [&](size_t bytes) {
        const size_t at = o;
        o += (bytes + 255) & ~size_t(255);
        return at;
    };
    w.chunks = take(((size_t)n_pages + PG_CHUNK - 1) / PG_CHUNK * 4);
    w.count = take(4);
    w.list_a = take((size_t)std::max<int64_t>(n_pages, n) * 4);
    w.list_b = take((size_t)n_pages * 4);
    w.list_c = take((size_t)n_pages * 4);
    w.plan = take((size_t)n * sizeof(ForkPlan));
    w.total = o;
    return w;
}

template <typename K, typename... A>
static cudaError_t go(K kernel, dim3 grid, int threads, cudaStream_t stream, A... args) {
    LaunchCfg c(grid, dim3((unsigned)threads), 0, stream);
    return cudaLaunchKernelEx(&c.cfg, kernel, args...);
}

}  // namespace csa2

using namespace csa2;

namespace {

csa2_status page_caches(int32_t n, const csa2_kv_cache* caches, PageCaches& p) {
    if (n < 1 || !caches) return CSA2_ERR_INVALID_ARG;
    if (n > kMaxCaches) return CSA2_ERR_UNSUPPORTED;
    p = PageCaches{};
    p.n = n;
    p.page_size = caches[0].page_size;
    for (int i = 0; i < n; ++i) {
        const csa2_kv_cache& c = caches[i];
        const csa2_status s = check_cache(&c, false, false);
        if (s != CSA2_OK) return s;
        if (c.idx_k ? !aligned(c.idx_k, 16) : c.idx_k_pooled != nullptr) return CSA2_ERR_INVALID_ARG;
        if (c.page_size != p.page_size || c.n_phys_pages != caches[0].n_phys_pages ||
            c.max_pages_per_seq != caches[0].max_pages_per_seq)
            return CSA2_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (caches[j].codes == c.codes) return CSA2_ERR_INVALID_ARG;  // the same cache twice
        p.codes[i] = c.codes;
        p.scales[i] = c.scales;
        p.idx[i] = c.idx_k;
        p.pooled[i] = c.idx_k_pooled;
    }
    if (caches[0].n_phys_pages > kMaxPages) return CSA2_ERR_UNSUPPORTED;
    return CSA2_OK;
}

bool al4(const void* p) { return p && aligned(p, 4); }
bool err_ok(const int32_t* e) { return !e || aligned(e, 4); }

}  // namespace

extern "C" {

size_t csa2_kv_pages_workspace_bytes(int64_t n_phys_pages, int32_t n) {
    if (n_phys_pages < 1 || n_phys_pages > kMaxPages || n < 0 || n > kMaxForks) return 0;
    return pages_ws_layout(n_phys_pages, n).total;
}

csa2_status csa2_kv_pages_copy(int32_t n_caches, const csa2_kv_cache* caches, const int32_t* src, const int32_t* dst,
                               int32_t n, int32_t* err_word, void* stream) {
    PageCaches p;
    const csa2_status s = page_caches(n_caches, caches, p);
    if (s != CSA2_OK) return s;
    if (n < 0 || n > kMaxPages || !err_ok(err_word)) return CSA2_ERR_INVALID_ARG;
    if (n == 0) return CSA2_OK;
    if (!al4(src) || !al4(dst)) return CSA2_ERR_INVALID_ARG;
    const int64_t jobs = (int64_t)n * n_caches;
    return from_cuda(go(pages_copy_kernel, dim3((unsigned)std::min<int64_t>(jobs, 148 * 8)), PG_COPY_THREADS,
                        (cudaStream_t)stream, p, src, dst, n, (int32_t)caches[0].n_phys_pages, err_word));
}

csa2_status csa2_kv_pages_fork(int32_t n_caches, const csa2_kv_cache* caches, int32_t* page_table, int32_t n_seqs,
                               int32_t* refs, int32_t* seq_lens, const int32_t* parents, const int32_t* children,
                               int32_t n, void* workspace, size_t ws_bytes, int32_t* err_word, void* stream) {
    ForkArgs a{};
    csa2_status s = page_caches(n_caches, caches, a.p);
    if (s != CSA2_OK) return s;
    if (n < 0 || n_seqs < 1 || !err_ok(err_word)) return CSA2_ERR_INVALID_ARG;
    if (n > kMaxForks) return CSA2_ERR_UNSUPPORTED;
    if (n == 0) return CSA2_OK;
    if (!al4(page_table) || !refs || !aligned(refs, 16) || !al4(seq_lens) || !al4(parents) || !al4(children))
        return CSA2_ERR_INVALID_ARG;
    const int64_t n_pages = caches[0].n_phys_pages;
    const PagesWs w = pages_ws_layout(n_pages, n);
    if (!workspace || !aligned(workspace, 256) || ws_bytes < w.total) return CSA2_ERR_WORKSPACE;
    char* ws = static_cast<char*>(workspace);
    a.table = page_table;
    a.refs = refs;
    a.lens = seq_lens;
    a.parents = parents;
    a.children = children;
    a.chunk_free = reinterpret_cast<int32_t*>(ws + w.chunks);
    a.n_free = reinterpret_cast<int32_t*>(ws + w.count);
    a.free_list = reinterpret_cast<int32_t*>(ws + w.list_a);
    a.plan = reinterpret_cast<ForkPlan*>(ws + w.plan);
    a.err = err_word;
    a.n = n;
    a.n_seqs = n_seqs;
    a.max_pages = caches[0].max_pages_per_seq;
    a.n_pages = (int32_t)n_pages;
    a.page_shift = page_shift_of(caches[0]);
    const unsigned chunks = (unsigned)((n_pages + PG_CHUNK - 1) / PG_CHUNK);
    cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e = cudaSuccess;
    if (chunks > PG_SELF_COUNT) e = go(fork_count_kernel, dim3(chunks), PG_SCAN_THREADS, st, a);
    if (e == cudaSuccess) e = go(fork_list_kernel, dim3(chunks + 1), PG_SCAN_THREADS, st, a);
    if (e == cudaSuccess)
        e = go(fork_apply_kernel, dim3((unsigned)n, 1u + (unsigned)n_caches), PG_COPY_THREADS, st, a);
    return from_cuda(e);
}

csa2_status csa2_kv_pages_free(const csa2_kv_cache* cache, int32_t* page_table, int32_t n_seqs, int32_t* refs,
                               int32_t* seq_lens, const int32_t* seqs, int32_t n, int32_t* err_word, void* stream) {
    const csa2_status s = check_cache(cache, false, false);
    if (s != CSA2_OK) return s;
    if (n < 0 || n_seqs < 1 || !err_ok(err_word)) return CSA2_ERR_INVALID_ARG;
    if (cache->n_phys_pages > kMaxPages) return CSA2_ERR_UNSUPPORTED;
    if (n == 0) return CSA2_OK;
    if (!al4(page_table) || !al4(refs) || !al4(seq_lens) || !al4(seqs)) return CSA2_ERR_INVALID_ARG;
    return from_cuda(go(pages_free_kernel, dim3((unsigned)n), PG_COPY_THREADS, (cudaStream_t)stream, page_table, refs,
                        seq_lens, seqs, n_seqs, cache->max_pages_per_seq, (int32_t)cache->n_phys_pages, err_word));
}

csa2_status csa2_kv_pages_compact(int32_t n_caches, const csa2_kv_cache* caches, int32_t* page_table, int32_t n_seqs,
                                  int32_t* refs, int32_t* page_map, int32_t* n_live, void* workspace, size_t ws_bytes,
                                  int32_t* err_word, void* stream) {
    CompactArgs a{};
    csa2_status s = page_caches(n_caches, caches, a.p);
    if (s != CSA2_OK) return s;
    if (n_seqs < 1 || !err_ok(err_word)) return CSA2_ERR_INVALID_ARG;
    if (!al4(page_table) || !refs || !aligned(refs, 16) || !al4(page_map) || !al4(n_live)) return CSA2_ERR_INVALID_ARG;
    const int64_t n_pages = caches[0].n_phys_pages;
    const PagesWs w = pages_ws_layout(n_pages, 0);
    if (!workspace || !aligned(workspace, 256) || ws_bytes < w.total) return CSA2_ERR_WORKSPACE;
    char* ws = static_cast<char*>(workspace);
    a.table = page_table;
    a.refs = refs;
    a.page_map = page_map;
    a.n_live_out = n_live;
    a.chunk_live = reinterpret_cast<int32_t*>(ws + w.chunks);
    a.n_move = reinterpret_cast<int32_t*>(ws + w.count);
    a.holes = reinterpret_cast<int32_t*>(ws + w.list_a);
    a.high = reinterpret_cast<int32_t*>(ws + w.list_b);
    a.where = reinterpret_cast<int32_t*>(ws + w.list_c);
    a.err = err_word;
    a.table_size = (int64_t)n_seqs * caches[0].max_pages_per_seq;
    a.n_pages = (int32_t)n_pages;
    const unsigned chunks = (unsigned)((n_pages + PG_CHUNK - 1) / PG_CHUNK);
    cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e = cudaSuccess;
    if (chunks > PG_SELF_COUNT) e = go(compact_count_kernel, dim3(chunks), PG_SCAN_THREADS, st, a);
    if (e == cudaSuccess) e = go(compact_list_kernel, dim3(chunks), PG_SCAN_THREADS, st, a);
    const int64_t jobs = std::max<int64_t>(n_pages / 2 * n_caches, (a.table_size + 1023) / 1024);
    if (e == cudaSuccess)
        e = go(compact_move_kernel, dim3((unsigned)std::max<int64_t>(1, std::min<int64_t>(jobs, 148 * 8))),
               PG_COPY_THREADS, st, a);
    return from_cuda(e);
}

}  // extern "C"
