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
// ranks the tiles' edges) and the move.
#include "pages.cuh"

namespace up {

namespace {

using namespace books;

constexpr int kMoveThreads = 256;
constexpr int kInFlight = 8;  // 16-byte pieces a thread holds of a tile
constexpr int kTileBytes = kMoveThreads * kInFlight * 16;

__host__ __device__ constexpr int tile_rows(int d) { return kTileBytes / (2 * d); }

struct Head {
    int ticket;   // tiles handed out
    int abort;
    int tiles;    // of the call
    int pad;
};
// One sequence: the slot of its first flagged token, the list's place of its first kept one, its kept
// tokens, those before the first dropped one (they stay), its first tile.
struct Moved {
    int base, at, kept, stay, tile0, pad[3];
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
    Head *head;
    Moved *seqs;
    int32_t *list;   // the kept tokens' numbers among their sequence's flagged ones
    int32_t *edges;  // for every R-th flagged token of a sequence, the kept ones before it
    int32_t *flags;  // a tile's rows have been read
    int R;
};

// where the edges of sequence s begin: every sequence before it may have a partial one
__device__ __forceinline__ int64_t edges_of(const Params &p, int s) { return p.a.cu_seqlens[s] / p.R + (int64_t)s; }

__global__ void __cluster_dims__(kBlocks) __launch_bounds__(kThreads) kv_plan_kernel(const Params p) {
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
    // base: -1 for a sequence that is left out
    for (int s = me; s < B; s += kBlocks * kThreads) {
        const int n = a.cu_seqlens[s + 1] - a.cu_seqlens[s], nb = (n + a.G - 1) / a.G;
        const int kv = kv_len_of(a.kv, s, n);
        const int b0 = a.cu_blocks[s], b1 = a.cu_blocks[s + 1];
        int base = kv - n;
        if (kv < 0) {
            base = -1;
        } else if (b0 < 0 || b1 < b0 || b1 - b0 < nb || b1 > a.num_flags) {
            atomicOr(a.kv.err, 0x10u);  // UP_DEVERR_BAD_CU_BLOCKS
            base = -1;
        }
        p.seqs[s] = Moved{base, 0, 0, n, 0, {0, 0, 0}};
    }
    meet();
    // the tokens in equal runs over the warps
    const int w = cluster_warp();
    const int64_t T = a.cu_seqlens[B];
    const int from = (int)(T * w / kAllWarps), to = (int)(T * (w + 1) / kAllWarps);
    int s_first = 0;  // the sequence of token `from`
    {
        int lo = 0, hi = B - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (a.cu_seqlens[mid] <= from) lo = mid; else hi = mid - 1;
        }
        s_first = lo;
    }
    auto each = [&](auto &&f) {
        int s = s_first;
        for (int t0 = from; t0 < to; t0 += 32) {
            const int t = t0 + lane;
            bool kept = false, there = t < to;
            int i = 0;
            if (there) {
                while (a.cu_seqlens[s + 1] <= t) ++s;
                i = t - a.cu_seqlens[s];
                kept = __ldcg(&p.seqs[s].base) >= 0 && a.keep[a.cu_blocks[s] + i / a.G];
            }
            f(t, s, i, there, kept, __ballot_sync(0xffffffffu, kept));
        }
    };
    int mine = 0;
    each([&](int, int, int, bool, bool, unsigned m) { mine += __popc(m); });
    int total, rank = before_warp(mine, &total);
    int last_s = -1;
    each([&](int t, int s, int i, bool there, bool kept, unsigned m) {
        const int r = rank + __popc(m & ((1u << lane) - 1u));
        if (there) {
            if (i == 0) p.seqs[s].at = r;
            if (t + 1 == a.cu_seqlens[s + 1]) p.seqs[s].kept = r + kept;  // `at` comes off below
            if (i % p.R == 0) p.edges[edges_of(p, s) + i / p.R] = r;  // of all; the sequence's share comes off later
            if (kept) p.list[r] = i;
            else if (s != last_s) atomicMin(&p.seqs[s].stay, i);  // (later ones of the run are larger)
            if (!kept) last_s = s;
        }
        rank += __popc(m);
    });
    meet();
    // kept tokens of every sequence, and the tiles' numbers (block 0; many sequences in rounds)
    if (blockIdx.x == 0) {
        __shared__ int s_sum[kWarps];
        int tiles = 0;
        for (int s0 = 0; s0 < B; s0 += kThreads) {
            const int s = s0 + tid;
            int n = 0, kept = 0;
            Moved q{};
            if (s < B) {
                q = Moved{__ldcg(&p.seqs[s].base), __ldcg(&p.seqs[s].at), 0, __ldcg(&p.seqs[s].stay), 0, {0, 0, 0}};
                kept = q.base >= 0 ? __ldcg(&p.seqs[s].kept) - q.at : 0;
                a.lens_out[s] = q.base < 0 ? a.kv.kv_lens[s] : q.base + kept;
                n = (max(kept - q.stay, 0) + p.R - 1) / p.R;
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
                q.kept = kept;
                q.tile0 = tiles + before + inc - n;
                p.seqs[s] = q;
            }
            tiles += all;
            __syncthreads();
        }
        if (tid == 0) p.head->tiles = tiles;
    }
    meet();
    const int64_t flags = (int64_t)__ldcg(&p.head->tiles) * 2 * a.kv.Hk;
    for (int64_t i = me; i < flags; i += kBlocks * kThreads) p.flags[i] = 0;
}

__device__ __forceinline__ int load_acquire(const int *at) {
    int v;
    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(at) : "memory");
    return v;
}
__device__ __forceinline__ void store_release(int *at, int v) {
    asm volatile("st.release.gpu.global.s32 [%0], %1;" ::"l"(at), "r"(v) : "memory");
}

__global__ void __launch_bounds__(kMoveThreads) kv_move_kernel(const Params p) {
    __shared__ int64_t s_src[tile_rows(64)], s_dst[tile_rows(64)];
    __shared__ int s_ticket, s_stop;
    const KvCompactArgs &a = p.a;
    const int tid = threadIdx.x, Hk = a.kv.Hk, ps = a.kv.page_size;
    const int pieces = a.kv.d / 8;  // of a row
    pdl_wait();
    const int64_t all = (int64_t)p.head->tiles * 2 * Hk;
    for (;;) {
        if (tid == 0) {
            s_ticket = atomicAdd(&p.head->ticket, 1);
            s_stop = 0;
        }
        __syncthreads();
        const int64_t ticket = s_ticket;
        if (ticket >= all) return;
        const int tile = (int)(ticket / (2 * Hk)), chain = (int)(ticket % (2 * Hk));
        int lo = 0, hi = a.kv.num_seqs - 1;  // the last sequence whose first tile is <= tile
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (p.seqs[mid].tile0 <= tile) lo = mid; else hi = mid - 1;
        }
        const int s = lo;
        const Moved q = p.seqs[s];
        const int i = tile - q.tile0;                      // tile of the sequence
        const int r0 = q.stay + i * p.R, rows = min(p.R, q.kept - r0);
        const int j = chain >> 1;
        for (int r = tid; r < rows; r += kMoveThreads) {
            const int src = q.base + p.list[q.at + r0 + r], dst = q.base + r0 + r;
            const int ps_ = page_of(a.kv, s, src), pd = page_of(a.kv, s, dst);
            s_src[r] = ps_ < 0 || pd < 0 ? -1 : (int64_t)ps_ * Hk * ps + src % ps;
            s_dst[r] = (int64_t)pd * Hk * ps + dst % ps;
        }
        __syncthreads();
        char *base = static_cast<char *>(chain & 1 ? a.kv.v : a.kv.k) + (int64_t)j * ps * a.kv.d * 2;
        uint4 v[kInFlight];
        int pos = 0;
#pragma unroll
        for (int k = 0; k < kInFlight; ++k) {
            const int x = tid + k * kMoveThreads, r = x / pieces;
            if (r < rows && s_src[r] >= 0)
                v[k] = *reinterpret_cast<const uint4 *>(base + s_src[r] * (a.kv.d * 2) + (x % pieces) * 16);
        }
        // the first chain moves the positions too: row (page * Hk) * ps + slot, less the heads
        auto pos_at = [&](int64_t row) { return row / ((int64_t)Hk * ps) * ps + row % ((int64_t)Hk * ps); };
        const bool places = a.kv.pos && chain == 0 && tid < rows && s_src[tid] >= 0;
        if (places) pos = a.kv.pos[pos_at(s_src[tid])];
        // read: nothing that this tile wrote over later can reach these rows any more
        __threadfence();
        __syncthreads();
        if (tid == 0) store_release(p.flags + ticket, 1);
        // the tiles that read what this one is about to write over
        const int64_t e = edges_of(p, s);
        const int n = a.cu_seqlens[s + 1] - a.cu_seqlens[s];
        const int ea = p.edges[e + r0 / p.R] - q.at;
        const int eb = (r0 + rows - 1) / p.R + 1 < (n + p.R - 1) / p.R ? p.edges[e + (r0 + rows - 1) / p.R + 1] - q.at : q.kept;
        const int t0 = max(ea - q.stay, 0) / p.R, t1 = min((max(eb - q.stay, 0) + p.R - 1) / p.R, i);
        for (int t = t0 + tid; t < t1; t += kMoveThreads) {
            const int *flag = p.flags + (int64_t)(q.tile0 + t) * 2 * Hk + chain;
            const long long began = clock64();
            while (!load_acquire(flag)) {
                if (*(volatile int *)&p.head->abort || clock64() - began > a.wait_limit) {
                    *(volatile int *)&p.head->abort = 1;
                    s_stop = 1;
                    break;
                }
            }
        }
        __syncthreads();
        if (s_stop) {
            if (tid == 0) atomicOr(a.kv.err, kErrTimeout);
            return;
        }
#pragma unroll
        for (int k = 0; k < kInFlight; ++k) {
            const int x = tid + k * kMoveThreads, r = x / pieces;
            if (r < rows && s_src[r] >= 0)
                *reinterpret_cast<uint4 *>(base + s_dst[r] * (a.kv.d * 2) + (x % pieces) * 16) = v[k];
        }
        if (places) a.kv.pos[pos_at(s_dst[tid])] = pos;
        __syncthreads();  // s_src, s_dst and the ticket are free
    }
}

}  // namespace

size_t kv_compact_workspace(int64_t T, int num_seqs, int Hk, int d) { return layout_of(T, num_seqs, Hk, d).total; }

cudaError_t launch_kv_compact(const KvCompactArgs &a, int num_sms, cudaStream_t st) {
    Params p{};
    p.a = a;
    p.R = tile_rows(a.kv.d);
    const Layout L = layout_of(a.T, a.kv.num_seqs, a.kv.Hk, a.kv.d);
    char *ws = static_cast<char *>(a.workspace);
    p.head = reinterpret_cast<Head *>(ws + L.head);
    p.seqs = reinterpret_cast<Moved *>(ws + L.seqs);
    p.list = reinterpret_cast<int32_t *>(ws + L.list);
    p.edges = reinterpret_cast<int32_t *>(ws + L.edges);
    p.flags = reinterpret_cast<int32_t *>(ws + L.flags);
    cudaError_t e = launch_pdl(kv_plan_kernel, dim3(kBlocks), dim3(kThreads), 0, st, p);
    if (e != cudaSuccess) return e;
    const int64_t most = ((int64_t)a.T / p.R + a.kv.num_seqs) * 2 * a.kv.Hk;
    const int64_t grid = most < (int64_t)num_sms * 4 ? most : (int64_t)num_sms * 4;
    return launch_pdl(kv_move_kernel, dim3((unsigned)grid), dim3(kMoveThreads), 0, st, p);
}

}  // namespace up
