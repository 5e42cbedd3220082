// pages.cu -- the pool of a paged cache's pages: reserving, forking and releasing them, and the
// copies that a fork asks for.
//
// The pool lives on the device, so that sequences whose lengths only the device knows grow, fork
// and shrink without the host: a count of holders for each page and a stack of free pages.
// The bookkeeping is a few bytes a page -- latency bounds it -- and has to give the same tables in
// every run.  So it is one cluster of 8 blocks: its warps take equal runs of (row, 64 entries)
// in order, a scan over the warps (through the blocks' shared memory) ranks what is
// taken or given back, and only counts, whose order does not matter, are atomic.
#include "pages.cuh"

namespace up {

namespace {

using namespace books;

constexpr int kRun = 64;  // entries of a row that a warp takes at once, two a lane

// The runs of a table [rows][max_pages], in order, cut into equal shares.
struct Runs {
    int per_row;
    int64_t from, to;
    __device__ Runs(int rows, int max_pages) {
        per_row = (max_pages + kRun - 1) / kRun;
        const int64_t n = (int64_t)rows * per_row, w = cluster_warp();
        from = n * w / kAllWarps;
        to = n * (w + 1) / kAllWarps;
    }
};

// The pages [x, y) of a row that begin in its tokens [first, end); empty where the end cannot be
// (UP_DEVERR_BAD_KV_LENS).
__device__ __forceinline__ int2 pages_in(const PageTable &t, int first, int end, unsigned int *err) {
    if (end > (int64_t)t.max_pages * t.page_size) {
        atomicOr(err, kErrKvLens);
        return make_int2(0, 0);
    }
    const int x = first <= 0 ? 0 : (first - 1) / t.page_size + 1;
    const int y = end <= 0 ? 0 : (end - 1) / t.page_size + 1;
    return make_int2(x, max(x, y));
}

// Free pages of the pool; -1 (UP_DEVERR_BAD_REFS set) where their number cannot be: the call then
// takes and gives back none, since nothing tells which entries of the stack are free pages.
__device__ __forceinline__ int free_of(const PagePool &p) {
    const int n = *p.num_free;
    if (n >= 0 && n <= p.num_pages) return n;
    atomicOr(p.err, kErrRefs);
    return -1;
}
// The page `rank` places below the stack's top (0 <= rank < top), held by its taker from now on; -1
// when the stack holds no page there.
__device__ __forceinline__ int take(const PagePool &p, int top, int rank) {
    const int pg = p.free[top - 1 - rank];
    if (pg < 0 || pg >= p.num_pages) {
        atomicOr(p.err, kErrRefs);
        return -1;
    }
    p.refs[pg] = 1;
    return pg;
}

// ---------------------------------------------------------------- reserve

__global__ void __cluster_dims__(kBlocks) __launch_bounds__(kThreads, 1)
    reserve_kernel(const PagePool pool, const PageTable t, const int32_t *have, const int32_t *want) {
    const int lane = threadIdx.x & 31;
    pdl_wait();
    const int top = free_of(pool);
    const Runs runs(t.num_seqs, t.max_pages);
    // does entry i of row s want a page?
    auto wants = [&](int s, int i, int2 r) {
        return top >= 0 && i >= r.x && i < r.y && t.entries[(int64_t)s * t.max_pages + i] < 0;
    };
    int mine = 0;
    for (int64_t k = runs.from; k < runs.to; ++k) {
        const int s = (int)(k / runs.per_row), i = (int)(k % runs.per_row) * kRun + lane;
        const int2 r = pages_in(t, have[s], want[s], pool.err);
        mine += __popc(__ballot_sync(0xffffffffu, wants(s, i, r)));
        mine += __popc(__ballot_sync(0xffffffffu, wants(s, i + 32, r)));
    }
    int total, rank = before_warp(mine, &total);
    arrive();
    for (int64_t k = runs.from; k < runs.to; ++k) {
        const int s = (int)(k / runs.per_row), i0 = (int)(k % runs.per_row) * kRun + lane;
        const int2 r = pages_in(t, have[s], want[s], pool.err);
        for (int i = i0; i < i0 + kRun; i += 32) {
            const bool w = wants(s, i, r);
            const unsigned m = __ballot_sync(0xffffffffu, w);
            const int at = rank + __popc(m & ((1u << lane) - 1u));
            if (w && at < top) t.entries[(int64_t)s * t.max_pages + i] = take(pool, top, at);
            rank += __popc(m);
        }
    }
    await_all();
    // (all blocks have read the count: they met in the scan)
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        if (total > max(top, 0)) atomicOr(pool.err, kErrNoPages);
        if (total) *pool.num_free = max(top - total, 0);
    }
}

// ---------------------------------------------------------------- release

__global__ void __cluster_dims__(kBlocks) __launch_bounds__(kThreads, 1)
    release_kernel(const PagePool pool, const PageTable t, const int32_t *first, const int32_t *end) {
    __shared__ int s_over;  // in the cluster some entry has found its page without a holder
    const int lane = threadIdx.x & 31;
    if (threadIdx.x == 0) s_over = 0;
    pdl_wait();
    const int top = free_of(pool);
    __syncwarp();
    arrive();
    const Runs runs(t.num_seqs, t.max_pages);
    const int num = t.num_seqs * t.max_pages;
    auto each = [&](auto &&f) {
        for (int64_t k = runs.from; k < runs.to; ++k) {
            const int s = (int)(k / runs.per_row), i0 = (int)(k % runs.per_row) * kRun + lane;
            const int2 r = top < 0 ? make_int2(0, 0) : pages_in(t, first ? first[s] : 0, end[s], pool.err);
            if (i0 - lane >= r.y || i0 - lane + kRun <= r.x) continue;
            for (int i = i0; i < i0 + kRun; i += 32) {
                const int at = s * t.max_pages + i;
                f(at, i >= r.x && i < r.y ? t.entries[at] : -1);
            }
        }
    };
    // One holder less for each entry.  Where more entries name a page than hold it, which of them find no holder is
    // chance; they stay in the table as kOver + page, so that the page still goes back with the first of all.
    constexpr int kOver = INT32_MIN;
    bool over = false;
    each([&](int at, int pg) {
        if (pg < 0) return;
        if (pg >= pool.num_pages) {
            atomicOr(pool.err, kErrPage);
            t.entries[at] = -1;
        } else if (atomicSub(pool.refs + pg, 1) <= 0) {
            atomicAdd(pool.refs + pg, 1);
            atomicOr(pool.err, kErrRefs);
            t.entries[at] = kOver + pg;
            over = true;
        }
    });
    __syncwarp();
    await_all();  // every block's s_over has its 0
    if (over)
        for (int b = 0; b < kBlocks; ++b) write_other(&s_over, b, 1);
    __syncwarp();
    meet();
    const bool some_over = s_over;
    // the page of an entry that has found no holder, -1 for any other
    auto page_over = [&](int pg) { return some_over && pg < -1 && pg - kOver < pool.num_pages ? pg - kOver : -1; };
    if (some_over) {  // (two more passes, after an error)
        // a count below zero is one that cannot be, and its page does not go back
        each([&](int at, int pg) {
            const int o = page_over(pg);
            if (o >= 0 && __ldcg(pool.refs + o) < 0) t.entries[at] = -1;
        });
        meet();
    }
    // a page without a holder goes back with the first entry that let it go: its count becomes that
    // entry's number, less the number of all
    each([&](int at, int pg) {
        if (pg >= 0 && __ldcg(pool.refs + pg) <= 0) atomicMin(pool.refs + pg, at - num);
    });
    meet();
    if (some_over) {
        each([&](int at, int pg) {
            const int o = page_over(pg);
            if (o >= 0 && __ldcg(pool.refs + o) < 0) atomicMin(pool.refs + o, at - num);
        });
        meet();
    }
    auto goes_back = [&](int at, int pg) { return pg >= 0 && __ldcg(pool.refs + pg) == at - num; };
    int mine = 0;
    each([&](int at, int pg) { mine += __popc(__ballot_sync(0xffffffffu, goes_back(at, max(pg, page_over(pg))))); });
    int total, rank = before_warp(mine, &total);
    arrive();
    // the first entry's page on top: reserving the same entries again gives the same pages
    each([&](int at, int entry) {
        const int pg = max(entry, page_over(entry));
        const bool back = goes_back(at, pg);
        const unsigned m = __ballot_sync(0xffffffffu, back);
        if (back) {
            const int to = top + total - 1 - rank - __popc(m & ((1u << lane) - 1u));
            if (to < pool.num_pages) pool.free[to] = pg;
            else atomicOr(pool.err, kErrRefs);
            pool.refs[pg] = 0;
        }
        if (pg >= 0) t.entries[at] = -1;
        rank += __popc(m);
    });
    await_all();
    if (blockIdx.x == 0 && threadIdx.x == 0 && total) *pool.num_free = min(top + total, pool.num_pages);
}

// ---------------------------------------------------------------- fork

// What child i takes over from its parent: full pages shared, and the rows of a last one that is copied.  Nothing
// where the pool cannot be (top < 0).
struct Child {
    int parent, len, full, rows;
};
__device__ __forceinline__ Child child_of(const ForkArgs &a, int i, int top) {
    Child c{a.parents[i], 0, 0, 0};
    if (top < 0) return c;
    if (c.parent < 0 || c.parent >= a.from.num_seqs) {
        atomicOr(a.pool.err, kErrTree);
        return c;
    }
    c.len = a.kv_lens[c.parent];
    if (c.len < 0 || c.len > (int64_t)a.from.max_pages * a.from.page_size) {
        atomicOr(a.pool.err, kErrKvLens);
        c.len = 0;
    }
    c.full = c.len / a.from.page_size;
    c.rows = c.len - c.full * a.from.page_size;
    return c;
}
// The parent's page `i`, -1 for none or (with an error) one outside the pool.
__device__ __forceinline__ int entry_of(const ForkArgs &a, int parent, int i) {
    const int pg = a.from.entries[(int64_t)parent * a.from.max_pages + i];
    if (pg >= a.pool.num_pages) atomicOr(a.pool.err, kErrPage);
    return pg < 0 || pg >= a.pool.num_pages ? -1 : pg;
}

__global__ void __cluster_dims__(kBlocks) __launch_bounds__(kThreads, 1) fork_kernel(const ForkArgs a) {
    const int lane = threadIdx.x & 31, n = a.children;
    pdl_wait();
    const int top = free_of(a.pool);
    // the children in equal runs over the warps: who needs a page of its own?
    const int w = cluster_warp(), from = (int)((int64_t)n * w / kAllWarps), to = (int)((int64_t)n * (w + 1) / kAllWarps);
    int mine = 0;
    for (int i0 = from; i0 < to; i0 += 32) {
        const int i = i0 + lane;
        bool need = false;
        if (i < to) {
            const Child c = child_of(a, i, top);
            need = c.rows && entry_of(a, c.parent, c.full) >= 0;
        }
        mine += __popc(__ballot_sync(0xffffffffu, need));
    }
    int total, rank = before_warp(mine, &total);
    for (int i0 = from; i0 < to; i0 += 32) {
        const int i = i0 + lane;
        Child c{-1, 0, 0, 0};
        int src = -1, dst = -1;
        if (i < to) {
            c = child_of(a, i, top);
            if (c.rows) src = entry_of(a, c.parent, c.full);
        }
        const unsigned m = __ballot_sync(0xffffffffu, src >= 0);
        const int at = rank + __popc(m & ((1u << lane) - 1u));
        rank += __popc(m);
        if (src >= 0 && at < top) dst = take(a.pool, top, at);
        if (src >= 0 && dst < 0) c.len = c.rows = 0, src = -1;  // no page: the child is empty
        if (i < to) {
            a.lens[i] = c.len;
            a.copies[i] = src;
            a.copies[n + i] = dst;
            a.copies[2 * n + i] = c.rows;
        }
    }
    meet();
    const Runs runs(n, a.from.max_pages);
    for (int64_t k = runs.from; k < runs.to; ++k) {
        const int i = (int)(k / runs.per_row), j0 = (int)(k % runs.per_row) * kRun + lane;
        const int parent = a.parents[i], len = __ldcg(a.lens + i), own = __ldcg(a.copies + n + i);
        const int full = len / a.from.page_size;
        for (int j = j0; j < j0 + kRun && j < a.from.max_pages; j += 32) {
            int pg = -1;
            if (j < full) {
                pg = entry_of(a, parent, j);
                if (pg >= 0) atomicAdd(a.pool.refs + pg, 1);
            } else if (j == full) {
                pg = own;
            }
            a.table[(int64_t)i * a.from.max_pages + j] = pg;
        }
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        if (total > max(top, 0)) atomicOr(a.pool.err, kErrNoPages);
        if (total) *a.pool.num_free = max(top - total, 0);  // (none is asked for where top < 0)
    }
}

// ---------------------------------------------------------------- copies

// A block takes rows of one head of the keys or values of one copy, up to kCopyBytes of them.
constexpr int kCopyThreads = 256;
constexpr int kCopyBytes = kCopyThreads * 4 * 16;
int copy_segments(const PagedKv &kv) {
    return (int)(((int64_t)kv.page_size * kv.d * 2 + kCopyBytes - 1) / kCopyBytes);
}

__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const PagedKv kv, const int32_t *copies, int n, int segments) {
    const int parts = 2 * kv.Hk * segments, x = blockIdx.x / parts, y = blockIdx.x % parts;
    const int seg = y % segments, part = y / segments, j = part >> 1, tid = threadIdx.x;
    pdl_wait();
    const int src = copies[x], dst = copies[n + x], rows = copies[2 * n + x];
    if (src < 0 || dst < 0 || rows == 0) return;
    if (src >= kv.num_pages || dst >= kv.num_pages || rows < 0 || rows > kv.page_size) {
        if (tid == 0 && y == 0) atomicOr(kv.err, kErrPage);
        return;
    }
    const int64_t head = (int64_t)kv.page_size * kv.d * 2;  // bytes
    const int64_t bytes = (int64_t)rows * kv.d * 2;
    char *base = static_cast<char *>(part & 1 ? kv.v : kv.k);
    const uint4 *from = reinterpret_cast<const uint4 *>(base + ((int64_t)src * kv.Hk + j) * head);
    uint4 *to = reinterpret_cast<uint4 *>(base + ((int64_t)dst * kv.Hk + j) * head);
    uint4 v[4];
    const int64_t at = (int64_t)seg * (kCopyBytes / 16) + tid;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if ((at + k * kCopyThreads) * 16 < bytes) v[k] = from[at + k * kCopyThreads];
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if ((at + k * kCopyThreads) * 16 < bytes) to[at + k * kCopyThreads] = v[k];
    if (kv.pos && y == 0)
        for (int r = tid; r < rows; r += kCopyThreads)
            kv.pos[(int64_t)dst * kv.page_size + r] = kv.pos[(int64_t)src * kv.page_size + r];
}

}  // namespace

cudaError_t launch_reserve(const PagePool &pool, const PageTable &t, const int32_t *have, const int32_t *want,
                           cudaStream_t st) {
    return launch_pdl(reserve_kernel, dim3(kBlocks), dim3(kThreads), 0, st, pool, t, have, want);
}

cudaError_t launch_release(const PagePool &pool, const PageTable &t, const int32_t *first, const int32_t *end,
                           cudaStream_t st) {
    return launch_pdl(release_kernel, dim3(kBlocks), dim3(kThreads), 0, st, pool, t, first, end);
}

cudaError_t launch_fork(const ForkArgs &a, cudaStream_t st) {
    return launch_pdl(fork_kernel, dim3(kBlocks), dim3(kThreads), 0, st, a);
}

int64_t copy_blocks(const PagedKv &kv, int n) { return (int64_t)2 * kv.Hk * copy_segments(kv) * n; }

cudaError_t launch_copy_pages(const PagedKv &kv, const int32_t *copies, int n, cudaStream_t st) {
    const int segments = copy_segments(kv);
    return launch_pdl(copy_pages_kernel, dim3((unsigned)(2 * kv.Hk * segments) * (unsigned)n), dim3(kCopyThreads), 0, st,
                      kv, copies, n, segments);
}

}  // namespace up
