// compact_kv.cu -- compaction of a paged cache in place: of the last n_s cached tokens of every
// sequence those with a flag move together, in order, behind the tokens before them.
//
// A kept token's rows are read once and written once, (2 * Hk * d * 2 + 4) bytes each way; what
// lies before the first dropped token stays.  So memory bounds a long prompt's compaction,
// latency that of a few accepted tokens.
//
// In place a row's new slot may be another row's old one.  A kept token never moves
// up: the token of rank r comes from a slot >= r.  So a tile of rows with ranks [a, b) writes
// slots that only tiles up to itself read, and a tile that has its rows in registers
// needs to know of those -- few, and long gone where many tokens are dropped -- that
// they have read theirs.  Blocks take tiles in that order from a counter: whoever waits, waits
// for tiles that running blocks hold and that are read without any wait, so the waits end whatever
// the number of blocks on the GPU.
//
// Two launches: a plan (one cluster of blocks: the scan of the flags, which lists the kept slots and
// ranks the tiles' edges) and the move.  131072 tokens of 8 heads of 128 that keep a quarter of their blocks of
// 64: 57 us in a graph, of it 46 the move of 134 MB each way at 5.8 TB/s together, where a plain copy would
// take 40 (what is left is the beginning -- a ticket, its description, its rows' pages, one after another -- and the
// last tickets' end: with a ring of three tiles in shared memory, loaded two ahead, it took 50).  Where the
// sequences have few flagged tokens one launch does both.
#include "pages.cuh"

namespace up {

namespace {

using namespace books;

constexpr int kMoveThreads = 128, kMovePerSm = 8;
constexpr int kInFlight = 8;  // 16-byte pieces a thread holds of a tile
constexpr int kTileBytes = kMoveThreads * kInFlight * 16;

__host__ __device__ constexpr int tile_rows(int d) { return kTileBytes / (2 * d); }

struct Head {
    int ticket;   // tickets handed out
    int abort;
    int tickets;  // of the call
    int pad;
};
// One sequence: the slot of its first flagged token (-1: left out), the list's place of its first
// kept one, its kept tokens, those before the first dropped one (they stay), its first ticket and
// the tickets of a tile.
struct alignas(32) Moved {
    int base, at, kept, stay, ticket0, groups, pad[2];
};

struct Layout {
    size_t head, seqs, list, edges, flags, total;
};
Layout layout_of(int64_t T, int num_seqs, int Hk, int d) {
    Layout L{};
    size_t off = 0;
    auto take = [&](size_t n) { const size_t at = off; off = (off + n + 255) & ~size_t(255); return at; };
    const int64_t tiles = T / tile_rows(d) + num_seqs;  // of one head
    L.head = take(sizeof(Head));
    L.seqs = take(sizeof(Moved) * (size_t)num_seqs);
    L.list = take(sizeof(int32_t) * (size_t)T);
    L.edges = take(sizeof(int32_t) * (size_t)tiles);
    L.flags = take(sizeof(int32_t) * (size_t)tiles * 2 * (size_t)Hk);
    L.total = off;
    return L;
}

struct Params {
    KvCompactArgs a;
    int r_log2, g_log2, p_log2;  // of R, G and the page size (-1: no power of two)
    Head *head;
    Moved *seqs;
    int32_t *list;   // the kept tokens' numbers among their sequence's flagged ones
    int32_t *edges;  // for every R-th flagged token of a sequence, the kept ones before it
    int32_t *flags;  // a tile's rows have been read
    int R;
};

// where the edges of sequence s begin: every sequence before it may have a partial one
__device__ __forceinline__ int64_t edges_of(const Params &p, int s) { return (p.a.cu_seqlens[s] >> p.r_log2) + (int64_t)s; }

// The slot before sequence s's flagged tokens, where its flags begin, and whether they can be.
struct Region {
    int base, flags, end;  // base: -1 for a sequence that is left out; end: of its tokens
};
__device__ __forceinline__ Region region_of(const KvCompactArgs &a, int s, bool tell) {
    const int c0 = a.cu_seqlens[s], c1 = a.cu_seqlens[s + 1], n = c1 - c0, nb = n ? (n - 1) / a.G + 1 : 0;
    const int b0 = a.cu_blocks[s], b1 = a.cu_blocks[s + 1], kv = a.kv.kv_lens[s];
    Region r{kv - n, b0, c1};
    if (tell) kv_len_of(a.kv, s, n);  // (its error bit)
    if (kv < n || kv > INT32_MAX - 65536 || kv > (int64_t)a.kv.max_pages * a.kv.page_size) {
        r.base = -1;
    } else if (b0 < 0 || b1 < b0 || b1 - b0 < nb || b1 > a.num_flags) {
        if (tell) atomicOr(a.kv.err, 0x10u);  // UP_DEVERR_BAD_CU_BLOCKS
        r.base = -1;
    }
    return r;
}

// Tickets of a sequence that moves m rows: tiles of R rows of one chain each; where all rows
// are fewer, as many chains (a power of two) as fill a tile share a ticket.
__host__ __device__ __forceinline__ int chains_of(int m, int R) {
    int c = 1;
    while (c < 64 && 2 * c * m <= R) c *= 2;
    return c;
}

// The last of the numbers 0 .. n - 1 for which f holds, which it does up to it (for 0 at least); by a
// warp, 32 at a time.
template <typename F>
__device__ __forceinline__ int last_of(int n, F &&f) {
    const int lane = threadIdx.x & 31;
    int lo = 0;
    while (n > 1) {
        const int step = (n + 31) / 32;
        const unsigned m = __ballot_sync(0xffffffffu, lane * step < n && f(lo + lane * step));
        const int hit = 31 - __clz(m | 1u);
        lo += hit * step;
        n = min(step, n - hit * step);
    }
    return lo;
}

// The scan: 8 blocks, 256 warps, equal runs of the flagged tokens.  A lane looks at up to
// kAhead tokens at once -- the loads of a step hang on one another, so latency is what it costs (131072
// tokens: 35 us one at a time).
constexpr int kAhead = 16;

__global__ void __cluster_dims__(kBlocks) __launch_bounds__(kThreads, 1) kv_plan_kernel(const Params p) {
    __shared__ int s_bad;
    const KvCompactArgs &a = p.a;
    const int B = a.kv.num_seqs, tid = threadIdx.x, lane = tid & 31;
    const int me = blockIdx.x * kThreads + tid;
    if (tid == 0) s_bad = 0;
    pdl_wait();
    __syncthreads();
    // every block checks all of cu_seqlens: nothing below reads past it
    for (int s = tid; s < B; s += kThreads) {
        const int c0 = a.cu_seqlens[s], c1 = a.cu_seqlens[s + 1];
        if (c0 < 0 || c1 < c0 || c1 > a.T || (s == 0 && c0 != 0)) s_bad = 1;
    }
    __syncthreads();
    if (me == 0) *p.head = Head{0, 0, 0, 0};
    if (s_bad) {
        if (me == 0) atomicOr(a.kv.err, kErrCuSeqlens);
        for (int s = me; s < B; s += kBlocks * kThreads) a.lens_out[s] = a.kv.kv_lens[s];
        return;  // all blocks do
    }
    const int T = a.cu_seqlens[B];
    for (int s = me; s < B; s += kBlocks * kThreads) {
        const Region r = region_of(a, s, true);
        p.seqs[s] = Moved{r.base, 0, 0, r.end - a.cu_seqlens[s], 0, 0, {0, 0}};
    }
    const int64_t flags = ((int64_t)T / p.R + B) * 2 * a.kv.Hk;
    for (int64_t i = me; i < flags; i += kBlocks * kThreads) p.flags[i] = 0;
    // this warp's run of tokens, in groups of kAhead * 32
    const int w = cluster_warp();
    const int from = (int)((int64_t)T * w / kAllWarps), to = (int)((int64_t)T * (w + 1) / kAllWarps);
    const int s_first = last_of(B, [&](int s) { return a.cu_seqlens[s] <= from; });  // of token `from`
    // The warp's tokens in groups: kept, a bit of 32 tokens for each step of a group, one(s, r, g0, kept) for a
    // group of one sequence's, some(t, s, r, kept) for the 32 of any.
    auto block_of = [&](int i) { return p.g_log2 >= 0 ? i >> p.g_log2 : i / a.G; };
    auto each = [&](auto &&one, auto &&some) {
        int s = s_first;
        Region r = from < to ? region_of(a, s, false) : Region{-1, 0, 0};
        for (int g0 = from; g0 < to; g0 += 32 * kAhead) {
            if (min(g0 + 32 * kAhead, to) <= r.end) {
                const int c0 = a.cu_seqlens[s];
                uint32_t kept = 0;
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {  // the loads do not wait for one another
                    const int t = g0 + 32 * k + lane;
                    if (t < to && r.base >= 0 && a.keep[r.flags + block_of(t - c0)]) kept |= 1u << k;
                }
                one(s, c0, r.end, g0, kept);
                continue;
            }
#pragma unroll 1
            for (int t0 = g0; t0 < min(to, g0 + 32 * kAhead); t0 += 32) {
                const int t = t0 + lane;
                bool kept = false;
                if (t < to) {
                    if (t >= r.end) {
                        while (a.cu_seqlens[s + 1] <= t) ++s;
                        r = region_of(a, s, false);
                    }
                    kept = r.base >= 0 && a.keep[r.flags + block_of(t - a.cu_seqlens[s])];
                }
                some(t, s, r.end, kept);
            }
            // the lanes go on from the last one's sequence
            s = __reduce_max_sync(0xffffffffu, s);
            r = region_of(a, s, false);
        }
    };
    int mine = 0;
    each([&](int, int, int, int, uint32_t kept) { mine += __reduce_add_sync(0xffffffffu, __popc(kept)); },
         [&](int, int, int, bool kept) { mine += __popc(__ballot_sync(0xffffffffu, kept)); });
    int total, rank = before_warp(mine, &total);
    int told = -1;  // the sequence whose first dropped token this warp has told of
    each(
        [&](int s, int c0, int end, int g0, uint32_t kept) {
            const int n = min(32 * kAhead, to - g0), e0 = (c0 >> p.r_log2) + s;  // (see edges_of)
            const uint32_t there = lane < n ? (2u << ((n - 1 - lane) >> 5)) - 1u : 0u, gone = there & ~kept;
            // (a lane each, and 8192 of them on one address, took 15 us of 131072 tokens' 27)
            const int first = __reduce_min_sync(0xffffffffu, gone ? 32 * (__ffs(gone) - 1) + lane : INT32_MAX);
            if (first != INT32_MAX && told != s) {
                if (lane == 0) atomicMin(&p.seqs[s].stay, g0 + first - c0);
                told = s;
            }
            if (lane == 0 && g0 == c0) p.seqs[s].at = rank;
#pragma unroll 4
            for (int k = 0; k < kAhead; ++k) {
                if (32 * k >= n) break;
                const bool keep = kept >> k & 1u;
                const unsigned m = __ballot_sync(0xffffffffu, keep);
                const int r = rank + __popc(m & ((1u << lane) - 1u)), i = g0 + 32 * k + lane - c0;
                if (keep) p.list[r] = i;
                // of all kept tokens; the sequence's share comes off later
                if ((i & (p.R - 1)) == 0 && there >> k & 1u) p.edges[e0 + (i >> p.r_log2)] = r;
                rank += __popc(m);
            }
            if (lane == 0 && g0 + n == end) p.seqs[s].kept = rank;  // `at` comes off below
        },
        [&](int t, int s, int end, bool kept) {
            const unsigned m = __ballot_sync(0xffffffffu, kept);
            // sequences rise over the lanes: of each, the first dropped token
            const unsigned gone = __ballot_sync(0xffffffffu, t < to && !kept), below = gone & ((1u << lane) - 1u);
            const int before = __shfl_sync(0xffffffffu, s, below ? 31 - __clz(below) : 0);
            if (t < to) {
                const int r = rank + __popc(m & ((1u << lane) - 1u)), c0 = a.cu_seqlens[s], i = t - c0;
                if (!kept && s != (below ? before : told)) atomicMin(&p.seqs[s].stay, i);
                if (i == 0) p.seqs[s].at = r;
                if (t + 1 == end) p.seqs[s].kept = r + kept;
                if ((i & (p.R - 1)) == 0) p.edges[(c0 >> p.r_log2) + s + (i >> p.r_log2)] = r;
                if (kept) p.list[r] = i;
            }
            if (gone) told = __shfl_sync(0xffffffffu, s, 31 - __clz(gone));
            rank += __popc(m);
        });
    meet();
    if (blockIdx.x) return;
    // kept tokens of every sequence, and the tickets' numbers (many sequences in rounds)
    __shared__ int s_sum[kWarps];
    int tickets = 0;
    for (int s0 = 0; s0 < B; s0 += kThreads) {
        const int s = s0 + tid;
        int n = 0;
        Moved q{};
        if (s < B) {
            q = Moved{__ldcg(&p.seqs[s].base), __ldcg(&p.seqs[s].at), 0, __ldcg(&p.seqs[s].stay), 0, 0, {0, 0}};
            q.kept = q.base >= 0 ? __ldcg(&p.seqs[s].kept) - q.at : 0;
            a.lens_out[s] = q.base < 0 ? a.kv.kv_lens[s] : q.base + q.kept;
            const int m = max(q.kept - q.stay, 0);
            q.groups = (2 * a.kv.Hk - 1) / chains_of(max(m, 1), p.R) + 1;
            n = (m + p.R - 1) / p.R * q.groups;
        }
        int inc = n;
#pragma unroll
        for (int k = 1; k < 32; k <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, inc, k);
            if (lane >= k) inc += y;
        }
        if (lane == 31) s_sum[tid >> 5] = inc;
        __syncthreads();
        int sum = s_sum[lane];
#pragma unroll
        for (int k = 1; k < 32; k <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, sum, k);
            if (lane >= k) sum += y;
        }
        const int before = (tid >> 5) ? __shfl_sync(0xffffffffu, sum, (tid >> 5) - 1) : 0;
        const int all = __shfl_sync(0xffffffffu, sum, 31);
        if (s < B) {
            q.ticket0 = tickets + before + inc - n;
            p.seqs[s] = q;
        }
        tickets += all;
        __syncthreads();
    }
    if (tid == 0) p.head->tickets = tickets;
}

__device__ __forceinline__ int load_acquire(const int *at) {
    int v;
    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(at) : "memory");
    return v;
}
__device__ __forceinline__ void store_release(int *at, int v) {
    asm volatile("st.release.gpu.global.s32 [%0], %1;" ::"l"(at), "r"(v) : "memory");
}

// What a ticket stands for: rows [r0, r0 + rows) of a sequence, of the chains (keys and values of the
// heads in turn) [chain, chain + chains), and the tickets [w0, w1) by `step` whose rows must have been read.
struct Ticket {
    int number, rows, chain, chains, base, r0, places, w0, w1, step;
};

// By one warp; number = -1 where there is none.
__device__ Ticket describe(const Params &p, int number, int all, int *list_at, int *seq) {
    const KvCompactArgs &a = p.a;
    Ticket k{};
    k.number = number < all ? number : -1;
    if (k.number < 0) return k;
    const int lo = last_of(a.kv.num_seqs, [&](int s) { return __ldg(&p.seqs[s].ticket0) <= number; });
    Moved q;
    reinterpret_cast<int4 *>(&q)[0] = __ldg(reinterpret_cast<const int4 *>(p.seqs + lo));
    reinterpret_cast<int4 *>(&q)[1] = __ldg(reinterpret_cast<const int4 *>(p.seqs + lo) + 1);
    const int per = q.groups, i = (number - q.ticket0) / per, group = (number - q.ticket0) % per;
    const int moved = q.kept - q.stay;
    k.chains = chains_of(moved, p.R);
    k.chain = group * k.chains;
    k.chains = min(k.chains, 2 * a.kv.Hk - k.chain);
    k.base = q.base;
    k.r0 = q.stay + i * p.R;
    k.rows = min(p.R, q.kept - k.r0);
    k.places = a.kv.pos && group == 0;
    // The tiles that read what this one is about to write over: those of the kept tokens in slots
    // [r0, r0 + rows), by the ranks at the edges around them.
    const int64_t e = edges_of(p, lo);
    const int len = a.cu_seqlens[lo + 1] - a.cu_seqlens[lo], next = ((k.r0 + k.rows - 1) >> p.r_log2) + 1;
    const int ea = __ldg(p.edges + e + (k.r0 >> p.r_log2)) - q.at;
    const int eb = next < (len + p.R - 1) >> p.r_log2 ? __ldg(p.edges + e + next) - q.at : q.kept;
    const int t0 = max(ea - q.stay, 0) >> p.r_log2, t1 = min((max(eb - q.stay, 0) + p.R - 1) >> p.r_log2, i);
    k.w0 = q.ticket0 + t0 * per + group;
    k.w1 = q.ticket0 + t1 * per + group;
    k.step = per;
    *list_at = q.at + k.r0;
    *seq = lo;
    return k;
}

// A block reads a tile's rows into registers, and while they come one warp describes the ticket after
// next and all look up the next one's rows (each a chain of loads as long as the rows' own; with one ticket
// looked up whole at a time 131072 tokens took 62 us).  It tells that its rows are there, waits for whoever still
// has to read the slots that they go to, and writes them.  (Eight blocks of 128 threads an SM took 51 us where
// four of 256 took 54, before the addresses were cut down: 47.)
template <int D>
__global__ void __launch_bounds__(kMoveThreads, kMovePerSm) kv_move_kernel(const Params p) {
    constexpr int kMaxRows = tile_rows(D), kRowPieces = D / 8;  // of 16 bytes
    static_assert(kMaxRows <= kMoveThreads && kMoveThreads % kRowPieces == 0, "a thread a row, whole rows at a time");
    __shared__ int64_t s_src[3][kMaxRows], s_dst[3][kMaxRows];  // bytes behind the head's first row
    __shared__ Ticket s_ticket[3];
    __shared__ int s_list[3], s_seq[3], s_stop, s_first, s_both;
    const KvCompactArgs &a = p.a;
    const int tid = threadIdx.x, Hk = a.kv.Hk, ps = a.kv.page_size;
    pdl_wait();
    const int all = p.head->tickets;
    if (all == 0) return;
    // The block's chains of loads run side by side: rows are looked up by the first warps, flags
    // asked for by those behind them, tickets described by the last (all in the first: 54 us of 131072
    // tokens, a third of it at the barrier).
    constexpr int kLast = kMoveThreads - 32;
    int number = 0;  // the last warp's first thread: the next ticket
    auto next_ticket = [&](int slot) {  // by the last warp
        int at = 0, seq = 0;
        const Ticket k = describe(p, __shfl_sync(0xffffffffu, number, 0), all, &at, &seq);
        if (tid == kLast) {
            s_ticket[slot] = k;
            s_list[slot] = at;
            s_seq[slot] = seq;
            if (k.number >= 0) number = atomicAdd(&p.head->ticket, 1);
        }
    };
    auto look_up = [&](int slot) {
        if (s_ticket[slot].number >= 0 && tid < s_ticket[slot].rows) {
            const int base = s_ticket[slot].base;
            const int src = base + __ldg(p.list + s_list[slot] + tid), dst = base + s_ticket[slot].r0 + tid;
            const int32_t *table = a.kv.block_table + (int64_t)s_seq[slot] * a.kv.max_pages;
            const int i = p.p_log2 >= 0 ? src >> p.p_log2 : src / ps, j = p.p_log2 >= 0 ? dst >> p.p_log2 : dst / ps;
            const int from = table[i], to = table[j];
            const bool ok = from >= 0 && from < a.kv.num_pages && to >= 0 && to < a.kv.num_pages;
            if (!ok) atomicOr(a.kv.err, kErrPage);
            s_src[slot][tid] = ok ? ((int64_t)from * Hk * ps + src - i * ps) * (2 * D) : -1;
            s_dst[slot][tid] = ((int64_t)to * Hk * ps + dst - j * ps) * (2 * D);
        }
    };
    if (tid == kLast) {
        // two at once where there are enough for all, a describing warp each (1 us of a long move's beginning)
        const int both = all >= 2 * (int)gridDim.x;
        number = atomicAdd(&p.head->ticket, 1 + both);
        s_first = number;
        s_both = both;
        s_stop = 0;
    }
    __syncthreads();
    if (tid >= kLast) {
        next_ticket(0);
        if (!s_both) next_ticket(1);
    } else if (s_both && tid >= kLast - 32) {
        int at = 0, seq = 0;
        const Ticket k = describe(p, s_first + 1, all, &at, &seq);
        if (tid == kLast - 32) {
            s_ticket[1] = k;
            s_list[1] = at;
            s_seq[1] = seq;
        }
    }
    __syncthreads();
    look_up(0);
    __syncthreads();
    for (int b = 0;; b = b == 2 ? 0 : b + 1) {
        const Ticket k = s_ticket[b];
        if (k.number < 0) return;
        // The tile's pieces, kMoveThreads at a time: of one chain's rows, where each thread keeps its place in a
        // row (addresses worked out from x alone took half of the block's time), or of several chains'.
        const int per = k.rows * kRowPieces;  // pieces of a chain
        const int col = tid % kRowPieces * 16, row0 = tid / kRowPieces;
        auto head_of = [&](int c) {
            return static_cast<char *>(c & 1 ? a.kv.v : a.kv.k) + (int64_t)(c >> 1) * ps * (2 * D) + col;
        };
        char *const head = head_of(k.chain);
        auto at = [&](int i, const int64_t *rows, char *&p16) {
            int r = row0 + i * (kMoveThreads / kRowPieces);
            char *h = head;
            if (k.chains > 1) {
                const int x = tid + i * kMoveThreads, c = x / per;
                if (c >= k.chains) return false;
                r -= c * k.rows;
                h = head_of(k.chain + c);
            } else if (r >= k.rows) {
                return false;
            }
            p16 = h + rows[r];
            return s_src[b][r] >= 0;
        };
        uint4 v[kInFlight];
#pragma unroll
        for (int i = 0; i < kInFlight; ++i) {
            char *src;
            v[i] = make_uint4(0, 0, 0, 0);
            if (at(i, s_src[b], src)) v[i] = *reinterpret_cast<const uint4 *>(src);
        }
        // the first chains' ticket moves the positions too: row (page * Hk) * ps + slot, less the heads
        auto pos_at = [&](int64_t bytes) {
            const int64_t row = bytes / (2 * D);
            return row / ((int64_t)Hk * ps) * ps + row % ((int64_t)Hk * ps);
        };
        const bool places = k.places && tid < k.rows && s_src[b][tid] >= 0;
        int pos = 0;
        if (places) pos = a.kv.pos[pos_at(s_src[b][tid])];
        // most of those that this one has to wait for have long read their rows
        int64_t t = k.w0 + (int64_t)((tid + kMoveThreads / 2) % kMoveThreads) * k.step;
        while (t < k.w1 && load_acquire(p.flags + t)) t += kMoveThreads * k.step;
        if (tid >= kLast) next_ticket(b == 0 ? 2 : b - 1);
        look_up(b == 2 ? 0 : b + 1);
        // All rows of the block have come: the barrier and the release order the reads before whatever
        // a waiter writes, and the sum makes every thread hold its values before it arrives.  (A fence
        // of every thread waits for the stores of the ticket before, too.)
        uint32_t sum = 0;
#pragma unroll
        for (int j = 0; j < kInFlight; ++j) sum ^= v[j].x ^ v[j].y ^ v[j].z ^ v[j].w;
        const bool some = __syncthreads_or((t < k.w1) | (sum == 0x9e3779b9u) | (pos == INT32_MIN));
        if (tid == kLast - 32) store_release(p.flags + k.number, 1);
        if (some) {
            const long long began = clock64();
            while (t < k.w1) {
                if (load_acquire(p.flags + t)) {
                    t += kMoveThreads * k.step;
                } else if (*(volatile int *)&p.head->abort || clock64() - began > a.wait_limit) {
                    *(volatile int *)&p.head->abort = 1;
                    s_stop = 1;
                    break;
                }
            }
            __syncthreads();
            if (s_stop) {
                if (tid == 0) atomicOr(a.kv.err, kErrTimeout);
                return;
            }
        }
#pragma unroll
        for (int i = 0; i < kInFlight; ++i) {
            char *dst;
            if (at(i, s_dst[b], dst)) *reinterpret_cast<uint4 *>(dst) = v[i];
        }
        if (places) a.kv.pos[pos_at(s_dst[b][tid])] = pos;
        // (of the three slots the next pass writes the one that no thread reads any more)
    }
}

// ---------------------------------------------------------------- few tokens a sequence

// Block (j, s): the keys and values of head j of sequence s, in one launch.  It scans the sequence's flags
// kRun at a time and moves what they keep itself, a tile of rows read into registers before it is
// written; so nothing waits for another block.  In a graph, 8 heads of 128 of which 10 to 97 % stay: 64 sequences
// of 64 tokens 6-8 us (by tickets 16-17), 256 of 16 13-15 (17), one of 256 5-10 (13-15).  But a sequence that has most of
// the tokens is one block's work for each head: 1024 take 11-34 us (14-16 by tickets), 4096 39-127 (18-24), 16384
// 150-513 (23-47); and every block checks all of cu_seqlens: 1024 sequences of 4 tokens take 36-46 (18), 16384 of
// one 1050-1160 (56).  The host knows how many tokens and sequences there are, not whose they are; so this is for 4096
// tokens and 256 sequences at most, and for no more tokens than 1024 times the root of the sequences.
constexpr int kFewThreads = 256, kRun = kFewThreads;  // a thread a flag
bool few_tokens(int64_t T, int64_t num_seqs) { return T <= 4096 && num_seqs <= 256 && T * T <= num_seqs << 20; }

__global__ void __launch_bounds__(kFewThreads) kv_few_kernel(const Params p) {
    __shared__ int64_t s_src[kRun], s_dst[kRun];
    __shared__ int s_warp[kFewThreads / 32], s_bad;
    const KvCompactArgs &a = p.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int j = blockIdx.x % a.kv.Hk, s = blockIdx.x / a.kv.Hk, Hk = a.kv.Hk, ps = a.kv.page_size, d2 = a.kv.d * 2;
    const int shift = a.kv.d == 64 ? 3 : a.kv.d == 128 ? 4 : 5;
    if (tid == 0) s_bad = 0;
    pdl_wait();
    __syncthreads();
    // a malformed cu_seqlens is one for all sequences
    for (int x = tid; x < a.kv.num_seqs; x += kFewThreads) {
        const int c0 = a.cu_seqlens[x], c1 = a.cu_seqlens[x + 1];
        if (c0 < 0 || c1 < c0 || c1 > a.T || (x == 0 && c0 != 0)) s_bad = 1;
    }
    __syncthreads();
    Region r{-1, 0, 0};
    if (s_bad) {
        if (blockIdx.x == 0 && tid == 0) atomicOr(a.kv.err, kErrCuSeqlens);
    } else {
        r = region_of(a, s, j == 0 && tid == 0);
    }
    if (r.base < 0) {
        if (j == 0 && tid == 0) a.lens_out[s] = a.kv.kv_lens[s];
        return;
    }
    const int n = r.end - a.cu_seqlens[s];
    int kept = 0;  // of the runs before
    for (int i0 = 0; i0 < n; i0 += kRun) {
        const int i = i0 + tid;
        const bool keep = i < n && a.keep[r.flags + (p.g_log2 >= 0 ? i >> p.g_log2 : i / a.G)];
        const unsigned m = __ballot_sync(0xffffffffu, keep);
        if (lane == 0) s_warp[warp] = __popc(m);
        __syncthreads();
        int before = 0, rows = 0;
#pragma unroll
        for (int w = 0; w < kFewThreads / 32; ++w) {
            if (w == warp) before = rows;
            rows += s_warp[w];
        }
        before += __popc(m & ((1u << lane) - 1u));
        if (keep) {
            const int src = r.base + i, dst = r.base + kept + before;
            // (one that stays where it is, like the others whose pages are none, does not move)
            const int from = src == dst ? -1 : page_of(a.kv, s, src), to = from < 0 ? -1 : page_of(a.kv, s, dst);
            s_src[before] = to < 0 ? -1 : ((int64_t)from * Hk + j) * ps + src % ps;
            s_dst[before] = ((int64_t)to * Hk + j) * ps + dst % ps;
        }
        __syncthreads();
        const int pieces = rows << shift;  // of the keys; the values' follow
        // kept tokens of this run go to slots of this run and of those before: read in order, they can be
        // written in order
        for (int x0 = 0; x0 < 2 * pieces; x0 += kInFlight * kFewThreads) {
            uint4 v[kInFlight];
            auto at = [&](int x, const int64_t *row) {
                const bool value = x >= pieces;
                const int y = value ? x - pieces : x;
                return static_cast<char *>(value ? a.kv.v : a.kv.k) + row[y >> shift] * d2 + (y & ((1 << shift) - 1)) * 16;
            };
            auto moves = [&](int x) { return x < 2 * pieces && s_src[(x >= pieces ? x - pieces : x) >> shift] >= 0; };
#pragma unroll
            for (int k = 0; k < kInFlight; ++k) {
                const int x = x0 + tid + k * kFewThreads;
                if (moves(x)) v[k] = *reinterpret_cast<const uint4 *>(at(x, s_src));
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < kInFlight; ++k) {
                const int x = x0 + tid + k * kFewThreads;
                if (moves(x)) *reinterpret_cast<uint4 *>(at(x, s_dst)) = v[k];
            }
            __syncthreads();
        }
        if (j == 0 && a.kv.pos) {
            auto place = [&](int64_t row) { return row / ((int64_t)Hk * ps) * ps + row % ps; };
            const bool moves = tid < rows && s_src[tid] >= 0;
            const int pos = moves ? a.kv.pos[place(s_src[tid])] : 0;
            __syncthreads();
            if (moves) a.kv.pos[place(s_dst[tid])] = pos;
        }
        kept += rows;
        __syncthreads();
    }
    if (j == 0 && tid == 0) a.lens_out[s] = r.base + kept;
}

}  // namespace

size_t kv_compact_workspace(int64_t T, int num_seqs, int Hk, int d) { return layout_of(T, num_seqs, Hk, d).total; }

cudaError_t launch_kv_compact(const KvCompactArgs &a, int num_sms, cudaStream_t st) {
    Params p{};
    p.a = a;
    p.R = tile_rows(a.kv.d);
    while (1 << p.r_log2 < p.R) ++p.r_log2;
    while (p.g_log2 < 30 && 1 << p.g_log2 < a.G) ++p.g_log2;
    if (1 << p.g_log2 != a.G) p.g_log2 = -1;
    while (p.p_log2 < 30 && 1 << p.p_log2 < a.kv.page_size) ++p.p_log2;
    if (1 << p.p_log2 != a.kv.page_size) p.p_log2 = -1;
    const Layout L = layout_of(a.T, a.kv.num_seqs, a.kv.Hk, a.kv.d);
    char *ws = static_cast<char *>(a.workspace);
    p.head = reinterpret_cast<Head *>(ws + L.head);
    p.seqs = reinterpret_cast<Moved *>(ws + L.seqs);
    p.list = reinterpret_cast<int32_t *>(ws + L.list);
    p.edges = reinterpret_cast<int32_t *>(ws + L.edges);
    p.flags = reinterpret_cast<int32_t *>(ws + L.flags);
    // Few tokens a sequence: one launch, unless it would write lengths that its other blocks still read.
    const int32_t *lens = a.kv.kv_lens;
    const bool apart = a.lens_out + a.kv.num_seqs <= lens || lens + a.kv.num_seqs <= a.lens_out;
    if (apart && few_tokens(a.T, a.kv.num_seqs) && (int64_t)a.kv.num_seqs * a.kv.Hk <= INT32_MAX)
        return launch_pdl(kv_few_kernel, dim3((unsigned)a.kv.num_seqs * (unsigned)a.kv.Hk), dim3(kFewThreads), 0, st, p);
    cudaError_t e = launch_pdl(kv_plan_kernel, dim3(kBlocks), dim3(kThreads), 0, st, p);
    if (e != cudaSuccess) return e;
    const int64_t most = ((int64_t)a.T / p.R + a.kv.num_seqs) * 2 * a.kv.Hk;
    const int64_t grid = most < (int64_t)num_sms * kMovePerSm ? most : (int64_t)num_sms * kMovePerSm;
    auto move = a.kv.d == 64 ? kv_move_kernel<64> : a.kv.d == 128 ? kv_move_kernel<128> : kv_move_kernel<256>;
    return launch_pdl(move, dim3((unsigned)grid), dim3(kMoveThreads), 0, st, p);
}

}  // namespace up
