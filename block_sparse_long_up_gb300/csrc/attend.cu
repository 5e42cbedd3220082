// attend.cu -- attention of new tokens over the paged cache on the sm_103a tensor
// cores (tcgen05 + TMEM + TMA).
//
// out = softmax(logits) V with 4*d flops for every visible (query head, query, slot):
// the tensor cores bound a chunk or a prompt, the cache's bandwidth or latency a few
// tokens.  One pass over the keys with a running maximum and sum, the logits and
// weights never leave the SM.
//
// The g query heads of a KV head and 128/g consecutive tokens are the 128 rows of a
// tile (row = token * g + head), so a key tile in shared memory serves the whole
// group.  A unit is two tiles (256 rows) of one sequence and KV head, one tile at
// head_dim 256, against the key tiles of 128 slots that any of its rows sees.  A
// plan kernel lists the units with their key tiles; all key tiles of all units and
// KV heads are laid end to end and block c of the grid (one per SM) takes the c-th
// equal share, so causal, windowed, ragged and few-row batches load every SM alike
// without the host knowing a length.  2048 tokens over 65536 of 32/8 heads of 128 take
// 1.68-1.71 ms a call among others (1.28 PFLOP/s, 0.66 of the measured burst rate; the
// power limit holds then) and 1.44-1.54 ms in a graph of ten: products are
// issued one every ~92 cycles instead of 64 (one chain into each accumulator; whether
// shared memory's rate has a part in it was not separated).  A unit cut by a share's end
// leaves its running maximum, sum and unnormalised output in the workspace for the join
// kernel (fixed order: results are reproducible); a whole unit is written by its block.
//
// The weights are rounded once to the cache's type before their product with the
// values: the tensor cores take no wider operand, and a low part beside them would double that
// product.  Against 64 bits outputs are off by 2.1-2.3e-3 in the 2-norm in bf16, where one
// rounding of the result leaves 1.6-1.7e-3; the sum counts the weights unrounded.
//
// Roles of a block:
//   warp 0      keys and values, TMA into a ring (boxes of the largest power of two
//               up to 128 that divides the page size, so pages may end inside a tile);
//   warp 2      queries, TMA, one 3-D box per tile and 64 dims;
//   warps 1, 3  MMA issuers.  Two tiles: each issues its tile's products, S = Q K^T
//               then O += P V with P read from TMEM.  One tile: warp 1 the
//               former, warp 3 the latter, with two S buffers.  Two instruction
//               streams alternate accumulators, which is what the tensor pipe needs
//               for its full rate;
//   warps 4-11  two softmax warpgroups, one per tile (at head_dim 256 one per 64 keys of
//               the only tile).  Thread = row.  It holds the row's logits in registers,
//               writes the weights over them in TMEM, and rescales its output row
//               there only when the maximum has grown by more than 2^8 (see kSlack), which
//               after the first tiles is rare.
#include "attend.cuh"
#include "tma_host.cuh"

namespace up {

namespace {

using namespace sm100;

constexpr int kRows = 128;        // rows of a tile, keys of a step
constexpr int kMinTiles = 4;      // shares are not cut finer than this: more parts cost
                                  // more to join than a step (128 tokens over 4K: 29.8,
                                  // 23.6, 22.4 and 26.5 us with 1, 2, 4 and 8)
constexpr int kPanel = 128 * 128; // 128 rows x 64 elements
// Tiles' worth of time that a unit costs beside its tiles: without it a share of short
// units takes far longer than one of long ones (three ragged sequences, 16/2 heads of
// 256, capped and biased: 380 us with 0, 305 with 2, 287 with 3, 292 with 5; since rows'
// references are exact and only logits that count choose the cap's form 319 with 3)
constexpr int kUnitCost = 3;

template <int D>
struct Cfg {
    static constexpr int kTiles = D == 256 ? 1 : 2;
    static constexpr int kThreads = 384;
    static constexpr int kStageDims = D < 128 ? D : 128;          // dims of one ring stage
    static constexpr int kStagePanels = kStageDims / 64;
    static constexpr int kStageBytes = kStagePanels * kPanel;
    static constexpr int kParts = D / kStageDims;                 // stages of a key (value) tile
    static constexpr int kQTile = D / 64 * kPanel;
    static constexpr int kQBytes = kTiles * kQTile;
    static constexpr int kStages = D == 64 ? 8 : D == 128 ? 4 : 5;
    static constexpr int kOutBytes = D == 256 ? 0 : 8 * 4096;      // the warps' output rows on their way
    static constexpr int kPosBytes = kTiles * 2 * 128 * 4;        // two steps' key positions
    static constexpr int kXchBytes = kTiles == 1 ? 1024 : 0;      // what the threads of a row tell one another
    static constexpr int kTail = kQBytes + kStages * kStageBytes; // where these begin
    static constexpr int kPad = 512;  // dynamic shared memory begins at a multiple of 1024 (checked)
    static constexpr int kSmem = kTail + kOutBytes + kPosBytes + kXchBytes + 512 + kPad;
    static constexpr int kOutCol = 256;                           // S: columns 0..255
    static constexpr int kUnitRows = kTiles * kRows;
    static_assert(kSmem <= 227 * 1024, "shared memory");
    static_assert(kOutCol + kTiles * D <= 512, "tensor memory");
};

struct Unit {
    int s, tok0, ntok;  // sequence, first token (of the batch), tokens
    int kt0, tiles;     // first key tile and how many
    int hi0;            // causal end of the first token's slots
    int kv;             // cached tokens of the sequence
    // Slots outside [first, end) no row of the unit sees, and those outside [seen0, seen1)
    // may hold anything.  All four lie in the unit's first and last key
    // tile; a byte each: first, end - 1, seen0, seen1 - 1 in its tile (a unit is read
    // ahead by every role, so its size counts in registers).  The first byte's high bit: there
    // may be slots between first and end that no row of the unit sees.
    uint32_t edges;
    int64_t prefix;     // width of the units before this one

    __device__ __forceinline__ int last_tile() const { return (kt0 + tiles - 1) * kRows; }
    __device__ __forceinline__ int first() const { return kt0 * kRows + (int)(edges & 127u); }
    __device__ __forceinline__ bool gaps() const { return edges & 128u; }
    __device__ __forceinline__ int end() const { return last_tile() + (int)(edges >> 8 & 255u) + 1; }
    __device__ __forceinline__ int seen0() const { return kt0 * kRows + (int)(edges >> 16 & 255u); }
    __device__ __forceinline__ int seen1() const { return last_tile() + (int)(edges >> 24) + 1; }
    __device__ __forceinline__ void set_seen(int lo, int hi) {
        const uint32_t a = (uint32_t)max(lo - kt0 * kRows, 0), b = (uint32_t)(min(hi - last_tile(), kRows) - 1);
        edges = (edges & 0xffffu) | a << 16 | b << 24;
    }
    __device__ __forceinline__ void set_range(int lo, int hi) {
        kt0 = lo / kRows;
        tiles = (hi + kRows - 1) / kRows - kt0;
        edges = (uint32_t)(lo - kt0 * kRows) | (uint32_t)(hi - last_tile() - 1) << 8;
    }
};
struct Plan {
    int64_t W;  // width of one KV head's units
    int units;
    int16_t bad;   // cu_seqlens is malformed: no unit, every row is that of an empty mask
    int16_t gaps;  // some sequence has slots between those its tokens see that none of them sees
};

// What a block's share leaves unfinished at its end: a unit that begins in it.
struct Cut {
    int parted, j, unit, pad;
};

struct Layout {
    size_t seq_off, seen, units, cuts, parts, total;
    int64_t max_units;
};
Layout layout_of(int64_t T, int num_seqs, int Hq, int Hk, int d) {
    Layout L{};
    const int g = Hq / Hk, tiles = d == 256 ? 1 : 2, tpu = tiles * (kRows / g);
    L.max_units = T / tpu + num_seqs;
    size_t off = 256;
    auto take = [&](size_t n) { const size_t at = off; off = (off + n + 255) & ~size_t(255); return at; };
    L.seq_off = take(sizeof(int32_t) * (size_t)(num_seqs + 1));
    L.seen = take(sizeof(int4) * (size_t)(num_seqs + 1));
    L.units = take(sizeof(Unit) * (size_t)(L.max_units > 0 ? L.max_units : 1));
    L.cuts = take(sizeof(Cut) * kMaxSms);
    L.parts = take((size_t)2 * kMaxSms * tiles * kRows * (size_t)(d + 4) * sizeof(float));
    L.total = off;
    return L;
}

struct Params {
    AttendArgs a;
    Plan *plan;
    int32_t *seq_off;
    int4 *seen;    // the slots that a sequence's tokens see lie in [x, y); z: with gaps
    Unit *units;
    Cut *cuts;
    float *parts;
    int64_t max_units;
    int tpt;       // tokens of a tile
    int box;       // rows of a key box
    int grid;
};

// ---------------------------------------------------------------- the plan

// [lo, hi) of a token from its entry in `visible`, cut to the cached slots.
__device__ __forceinline__ int2 cut_range(int2 v, int kv) {
    const int lo = max(v.x, 0), hi = min(v.y, kv);
    return lo < hi ? make_int2(lo, hi) : make_int2(INT32_MAX, 0);
}

// [lo, hi) of the token tl tokens behind the unit's first one.
__device__ __forceinline__ int2 sees(const AttendArgs &a, const Unit &u, int tl) {
    if (!a.visible) return make_int2(0, u.hi0 + tl);
    return cut_range(reinterpret_cast<const int2 *>(a.visible)[u.tok0 + tl], u.kv);
}

// A unit's width in the work laid end to end: its key tiles, and in front of them what
// beginning and ending it costs (queries, first logits, output).
__host__ __device__ __forceinline__ int width_of(const Unit &u) { return u.tiles ? u.tiles + kUnitCost : 0; }

constexpr int kPlanThreads = 1024;

// Exclusive scan of one value a thread over the block; *total gets the sum.
__device__ int64_t block_scan(int64_t v, int64_t *total, int64_t *sh) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    int64_t inc = v;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, inc, k);
        if (lane >= k) inc += y;
    }
    if (lane == 31) sh[w] = inc;
    __syncthreads();
    if (w == 0) {
        int64_t x = lane < (int)(blockDim.x >> 5) ? sh[lane] : 0;
#pragma unroll
        for (int k = 1; k < 32; k <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, x, k);
            if (lane >= k) x += y;
        }
        sh[lane] = x;
    }
    __syncthreads();
    const int64_t before = (w ? sh[w - 1] : 0) + inc - v;
    *total = sh[(blockDim.x >> 5) - 1];
    __syncthreads();
    return before;
}

// The range of the last token with one before this lane's: among the round's (one a lane)
// or, where there is none, `last`, which is then moved behind the round.  Empty ranges have y = 0.
__device__ __forceinline__ int2 range_before(int2 r, int2 &last) {
    const int lane = threadIdx.x & 31;
    const unsigned some = __ballot_sync(0xffffffffu, r.y > 0), below = some & ((1u << lane) - 1u);
    const int from = below ? 31 - __clz(below) : 0, to = some ? 31 - __clz(some) : 0;
    int2 b = make_int2(__shfl_sync(0xffffffffu, r.x, from), __shfl_sync(0xffffffffu, r.y, from));
    if (!below) b = last;
    const int2 end = make_int2(__shfl_sync(0xffffffffu, r.x, to), __shfl_sync(0xffffffffu, r.y, to));
    if (some) last = end;
    return b;
}
// Neither empty, and slots between them that are in neither.
__device__ __forceinline__ bool apart(int2 a, int2 b) {
    return a.y > 0 && b.y > 0 && max(a.x, b.x) > min(a.y, b.y);
}

// Bits [lo, hi) of a word, as far as it has them.
__device__ __forceinline__ uint32_t span_bits(int lo, int hi) {
    lo = max(lo, 0), hi = min(hi, 32);
    return lo < hi ? (0xffffffffu >> (32 - hi)) & (0xffffffffu << lo) : 0u;
}

// Which of the 32 slots at key0 some row of the unit sees, a bit each; by the whole warp,
// which shares the unit's tokens among its lanes.  (A word at a time: the roles that ask have
// few registers.)
__device__ __forceinline__ uint32_t seen_word(const AttendArgs &a, const Unit &u, int key0) {
    uint32_t m = 0;
#pragma unroll 1
    for (int tl = threadIdx.x & 31; tl < u.ntok; tl += 32) {
        const int2 r = sees(a, u, tl);
        m |= span_bits(r.x - key0, r.y - key0);
    }
    return __reduce_or_sync(0xffffffffu, m);
}

// Marks the units in which some range lies apart from that of the token with one before
// it, and the sequences that have such a place and whose ranges together do not
// cover one range either (where a few sweeps do not settle it, it is taken for a gap: that
// costs time only).
__device__ __forceinline__ void mark_gaps(const Params &p, int64_t units) {
    const int tid = threadIdx.x, lane = tid & 31;
    for (int64_t i = tid >> 5; i < units; i += kPlanThreads / 32) {
        const Unit u = p.units[i];
        bool gaps = false;
        int2 last = make_int2(INT32_MAX, 0);
        for (int t0 = 0; t0 < u.ntok; t0 += 32) {
            const int2 r = t0 + lane < u.ntok && u.kv >= 0 ? sees(p.a, u, t0 + lane) : make_int2(INT32_MAX, 0);
            gaps |= apart(r, range_before(r, last));
        }
        if (__any_sync(0xffffffffu, gaps) && lane == 0) {
            p.units[i].edges |= 128u;
            atomicOr(&p.seen[u.s].z, 1);
        }
    }
    __syncthreads();
    for (int64_t i = tid; i < units; i += kPlanThreads) {  // between a sequence's units
        const Unit u = p.units[i];
        if (!u.tiles) continue;
        int64_t b = i - 1;
        while (b >= 0 && p.units[b].s == u.s && !p.units[b].tiles) --b;
        if (b < 0 || p.units[b].s != u.s) continue;
        if (max(u.first(), p.units[b].first()) > min(u.end(), p.units[b].end())) atomicOr(&p.seen[u.s].z, 1);
    }
    __syncthreads();
    // a warp a sequence: what is covered from the first seen slot on
    for (int s = tid >> 5; s < p.a.kv.num_seqs; s += kPlanThreads / 32) {
        const int4 all = __ldcg(p.seen + s);
        if (!all.z) continue;
        const int c0 = p.a.cu_seqlens[s], c1 = p.a.cu_seqlens[s + 1], kv = p.a.kv.kv_lens[s];
        int upto = all.x;
        for (int sweep = 0; sweep < 8 && upto < all.y; ++sweep) {
            const int before = upto;
            for (int t0 = c0; t0 < c1 && upto < all.y; t0 += 128) {
                int2 r[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int t = t0 + 32 * k + lane;
                    r[k] = t < c1 ? cut_range(reinterpret_cast<const int2 *>(p.a.visible)[t], kv) : make_int2(INT32_MAX, 0);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) upto = max(upto, __reduce_max_sync(0xffffffffu, r[k].x <= upto ? r[k].y : 0));
            }
            if (upto == before) break;
        }
        __syncwarp();
        if (upto >= all.y && lane == 0) p.seen[s].z = 0;
    }
}

// Lists the units (one block): sequences' unit counts and their scan, then every
// unit's key tiles and their scan.  Calls without `visible` have a shorter kernel of their own
// (128 tokens over 4K: 23 us instead of 24).
template <bool kVisible>
__global__ void __launch_bounds__(kPlanThreads) attend_plan_kernel(const Params p, int tpu) {
    __shared__ int64_t sh[32];
    __shared__ int bad, torn, gaps;
    const AttendArgs &a = p.a;
    const int B = a.kv.num_seqs, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) bad = torn = 0;
    pdl_wait();
    pdl_trigger();  // what came before is complete: the main kernel's set-up may overlap
    __syncthreads();
    int64_t units = 0;
    for (int s0 = 0; s0 < B; s0 += kPlanThreads) {
        const int s = s0 + tid;
        int64_t n = 0;
        if (s < B) {
            const int c0 = a.cu_seqlens[s], c1 = a.cu_seqlens[s + 1];
            if (c0 < 0 || c1 < c0 || c1 > a.T || (s == 0 && c0 != 0) || (s == B - 1 && c1 != a.T)) bad = 1;
            else n = (c1 - c0 + tpu - 1) / tpu;
        }
        int64_t total;
        const int64_t at = units + block_scan(n, &total, sh);
        if (s < B) {
            p.seq_off[s] = (int)(at < p.max_units ? at : p.max_units);
            p.seen[s] = make_int4(INT32_MAX, 0, 0, 0);
        }
        units += total;
    }
    __syncthreads();
    if (bad || units > p.max_units) {
        if (tid == 0) {
            atomicOr(a.kv.err, kErrCuSeqlens);
            *p.plan = Plan{0, 0, 1, 0};
        }
        return;
    }
    for (int64_t i = tid; i < units; i += kPlanThreads) {
        int lo = 0, hi = B - 1;  // the last sequence with seq_off <= i
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (p.seq_off[mid] <= i) lo = mid; else hi = mid - 1;
        }
        const int c0 = a.cu_seqlens[lo], c1 = a.cu_seqlens[lo + 1];
        Unit u{};
        u.s = lo;
        u.tok0 = c0 + (int)(i - p.seq_off[lo]) * tpu;
        u.ntok = min(tpu, c1 - u.tok0);
        u.kv = kv_len_of(a.kv, lo, c1 - c0);
        u.hi0 = u.kv - (c1 - u.tok0) + 1;
        u.prefix = u.tok0 > c0;  // until the scan: a token of the sequence comes before
        if (u.kv >= 0 && !kVisible) {
            u.set_range(0, u.hi0 + u.ntok - 1);
            u.set_seen(0, u.kv);
        }
        p.units[i] = u;
    }
    if constexpr (kVisible) {
        __syncthreads();
        // A warp looks at its units' ranges, lane by token, kSame units at once.  Where every range
        // overlaps or touches that of the token before it (one empty token between is enough
        // not to know), what the sequence sees is one range without gaps.
        constexpr int kSame = 4;
        for (int64_t i0 = warp * kSame; i0 < units; i0 += kPlanThreads / 32 * kSame) {
            int first[kSame], end[kSame];
            Unit u[kSame];
            bool gaps = false;
#pragma unroll
            for (int k = 0; k < kSame; ++k) {
                u[k] = p.units[min(i0 + k, units - 1)];
                first[k] = INT32_MAX;
                end[k] = 0;
            }
            for (int t = lane; t < tpu; t += 32) {
                int2 r[kSame], b[kSame];
#pragma unroll
                for (int k = 0; k < kSame; ++k) {
                    const bool some = u[k].kv >= 0 && t < u[k].ntok;
                    r[k] = some ? sees(a, u[k], t) : make_int2(INT32_MAX, 0);
                    b[k] = some && (t || u[k].prefix) ? sees(a, u[k], t - 1) : r[k];
                }
#pragma unroll
                for (int k = 0; k < kSame; ++k) {
                    first[k] = min(first[k], r[k].x);
                    end[k] = max(end[k], r[k].y);
                    gaps |= r[k].y > 0 && max(b[k].x, r[k].x) > min(b[k].y, r[k].y);
                }
            }
            if (gaps) torn = 1;
#pragma unroll
            for (int k = 0; k < kSame; ++k) {
                const int lo = __reduce_min_sync(0xffffffffu, first[k]), hi = __reduce_max_sync(0xffffffffu, end[k]);
                if (lane == k && i0 + k < units && lo < hi) {
                    p.units[i0 + k].set_range(lo, hi);
                    atomicMin(&p.seen[u[k].s].x, lo);
                    atomicMax(&p.seen[u[k].s].y, hi);
                }
            }
        }
        __syncthreads();
        if (torn) mark_gaps(p, units);  // seldom, so it may take longer
    }
    if (tid == 0) gaps = 0;
    __syncthreads();
    int64_t W = 0;
    for (int64_t u0 = 0; u0 < units; u0 += kPlanThreads) {
        const int64_t i = u0 + tid;
        int64_t total;
        const int64_t at = block_scan(i < units ? width_of(p.units[i]) : 0, &total, sh);
        if (i < units) {
            p.units[i].prefix = W + at;
            if (kVisible && p.units[i].tiles) {
                // Where the atomics left it.  In a sequence with gaps only what a unit's own rows
                // see is known to be seen.
                const int4 r = __ldcg(p.seen + p.units[i].s);
                if (r.z) gaps = 1;
                p.units[i].set_seen(r.z ? p.units[i].first() : r.x, r.z ? p.units[i].end() : r.y);
            }
        }
        W += total;
    }
    __syncthreads();
    if (tid == 0) *p.plan = Plan{W, (int)units, 0, (int16_t)gaps};
}

// The unit at x (0 <= x < W) of a KV head's work.
__device__ __forceinline__ int find_unit(const Unit *units, int n, int64_t x) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (units[mid].prefix <= x) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// A block's share, piece by piece: the part of a (KV head, unit) that lies in it.
struct Pieces {
    const Params &p;
    Shares sh;
    int64_t W1, at, end;
    int j, ui, n;        // KV head, unit index, units
    int64_t base;        // width of the KV heads before j
    Unit u, behind;
    int after = -1;      // the index of `behind`
    int ta, tb;          // tiles [ta, tb) of the unit
    int64_t index = -1;  // pieces so far, less one

    __device__ explicit Pieces(const Params &pp) : p(pp) {
        const Plan pl = *pp.plan;
        W1 = pl.W;
        n = pl.units;
        at = end = 0;
        if (W1 == 0) return;
        sh = shares_of(W1 * pp.a.kv.Hk, pp.grid, kMinTiles);
        if ((int)blockIdx.x >= sh.n) return;
        at = share_begin(sh, blockIdx.x);
        end = share_begin(sh, blockIdx.x + 1);
        j = (int)(at / W1);
        base = (int64_t)j * W1;
        ui = find_unit(pp.units, n, at - base);
        u = pp.units[ui];
    }
    __device__ bool next() {
        while (at < end) {
            while (at - base >= u.prefix + width_of(u)) {  // units without tiles, or the last one done
                if (++ui == n) {
                    ui = 0;
                    ++j;
                    base += W1;
                }
                u = ui == after ? behind : p.units[ui];
            }
            const int64_t first = base + u.prefix + kUnitCost;  // of the unit's tiles
            ta = (int)max(at - first, (int64_t)0);
            tb = (int)min((int64_t)u.tiles, end - first);
            at = min(end, first + u.tiles);
            if (ta >= tb) continue;  // the share ends before the unit's first tile
            ++index;
            // the next unit's description, on its way while this one is worked on
            after = ui + 1 < n ? ui + 1 : 0;
            behind = p.units[after];
            return true;
        }
        return false;
    }
    __device__ int steps() const { return tb - ta; }
    __device__ int tiles_used() const { return u.ntok > p.tpt ? 2 : 1; }  // row tiles with tokens
    // First slot of step t.  A distance bias makes the logits grow towards the query, so
    // with one the steps go from the last key tile to the first: the maximum is then
    // found at once, instead of growing past the slack at every step.
    __device__ int key0(int t) const {
        return (u.kt0 + (p.a.slopes ? u.tiles - 1 - ta - t : ta + t)) * kRows;
    }
};

// ---------------------------------------------------------------- shared state

constexpr int kMaxStages = 8;
struct Shared {
    uint64_t full[kMaxStages], empty[kMaxStages];  // the ring
    uint64_t qfull, qempty;
    uint64_t pieces;        // a piece's products are complete
    // S buffers: one set of barriers for pieces of one row tile, one for those of two
    uint64_t sfull[2][2];   // the buffer holds logits
    uint64_t pfull[2][2][2];  // the buffer holds the weights of the first, the second 64 keys
    uint64_t pdone[2][2];   // the weights have been multiplied into O
    uint64_t turn[2];    // an issuer may issue its step's products
    uint64_t xch[4];     // the two warps of 32 rows have met (one row tile)
    uint64_t pos[2];     // a warpgroup's key positions are in shared memory
    uint64_t fin[2];
    uint32_t tmem;
    int abort;
};

// Uses of the S buffers by all pieces so far: every role walks the same pieces and
// counts them alike, so barrier parities need no talk.  A parity tells a phase from
// its neighbours only: whoever waits for a use must know that the one before it is
// over.  So the second softmax warpgroup, which has no part in pieces of one row
// tile, shares no barrier with them.  Pieces of one tile take the buffers in turn,
// across pieces too.
struct Uses {
    uint32_t two = 0, one = 0;
    __device__ void add(int steps, int tiles_used) { (tiles_used == 2 ? two : one) += steps; }
    // buffer and parity of its use by step t of row tile e
    __device__ int buf(int t, int e, int tiles_used) const { return tiles_used == 2 ? e : (int)((one + t) & 1u); }
    __device__ uint32_t par(int t, int tiles_used) const {
        return (tiles_used == 2 ? two + t : (one + t) >> 1) & 1u;
    }
};

__device__ __forceinline__ void drain(uint32_t bar, uint32_t parity) {
    const long long t0 = clock64();
    while (!mbar_try_wait(bar, parity))
        if (clock64() - t0 > 4000000000LL) break;
}

__device__ __forceinline__ uint64_t desc_mn_sw128(uint32_t saddr) {
    // MN-major operand (rows of 64 elements along N, one row per k): 8-row groups
    // 1024 bytes apart, the next 64 elements of N one panel on
    uint64_t d = 0;
    d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
    d |= (uint64_t)((uint32_t)kPanel >> 4) << 16;
    d |= (uint64_t)(1024u >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

__host__ __device__ constexpr uint32_t idesc_f32(bool fp16, int M, int N, bool b_mn_major) {
    return (1u << 4) | ((fp16 ? 0u : 1u) << 7) | ((fp16 ? 0u : 1u) << 10) | ((b_mn_major ? 1u : 0u) << 16) |
           ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// D[tmem] (+)= A[tmem] * B[smem], issued by one thread.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b),
        "r"(idesc), "r"(acc)
        : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t t, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
        "%13, %14, %15, %16};" ::"r"(t), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]),
        "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]),
        "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// ---------------------------------------------------------------- roles

// One key or value tile into ring stages it, it+1, ... (kParts of them), by the whole
// warp: lane l loads the l-th box of 128 / box, from page pg (-1, nothing that a row of
// the unit sees or a bad page: a box outside the pool, which reads as zeros).
template <int D>
__device__ bool load_tile(const CUtensorMap *map, const Params &p, Shared &sh, uint32_t ring, uint32_t &it,
                          const Pieces &w, int key0, int pg) {
    using C = Cfg<D>;
    const AttendArgs &a = p.a;
    const int r = (threadIdx.x & 31) * p.box;
    const int z = pg < 0 ? (int)(a.kv.num_pages * a.kv.Hk) : pg * a.kv.Hk + w.j;
    const int y = pg < 0 ? 0 : (key0 + r) % a.kv.page_size;
#pragma unroll 1
    for (int part = 0; part < C::kParts; ++part, ++it) {
        const int st = it % C::kStages;
        if (!mbar_wait_warp(smem_u32(&sh.empty[st]), ((it / C::kStages) & 1) ^ 1, &sh.abort, a.wait_limit))
            return false;
        const uint32_t bar = smem_u32(&sh.full[st]);
        if ((threadIdx.x & 31) == 0) mbar_arrive_expect_tx(bar, C::kStageBytes);
        __syncwarp();
        if (r < kRows) {
#pragma unroll
            for (int pn = 0; pn < C::kStagePanels; ++pn)
                tma_load_3d(ring + st * C::kStageBytes + pn * kPanel + r * 128, map,
                            part * C::kStageDims + pn * 64, y, z, bar);
        }
        __syncwarp();
    }
    return true;
}

template <int D, bool kGaps>
__device__ void role_kv(const CUtensorMap *km, const CUtensorMap *vm, const Params &p, Shared &sh, uint32_t ring) {
    using C = Cfg<D>;
    uint32_t it = 0;
    bool ok = true;
    Pieces w(p);
    const int r = (threadIdx.x & 31) * p.box;
    while (ok && w.next()) {
        const int n = w.steps();
        // the page of this lane's box, looked up two steps ahead
        const int from = w.u.first() - p.box, end = w.u.end();
        auto page = [&](int t) {
            const int key = w.key0(t) + r;
            bool some = t < n && r < kRows && key < end && key > from;
            if constexpr (kGaps) {
                if (w.u.gaps() && t < n) {  // boxes in a gap are not looked up
                    uint32_t box = 0;
#pragma unroll 1
                    for (int k = 0; k < kRows; k += 32)
                        box |= seen_word(p.a, w.u, w.key0(t) + k) & span_bits(r - k, r + p.box - k);
                    some = some && box;
                }
            }
            return some ? page_of(p.a.kv, w.u.s, key) : -1;
        };
        int p0 = page(0), p1 = page(1), p2 = page(2);
        // the order in which the products need them: one tile runs a step ahead with its keys
        const int ahead = C::kTiles == 1 || w.tiles_used() == 1;
        ok = load_tile<D>(km, p, sh, ring, it, w, w.key0(0), p0);
        for (int t = 0; ok && t < n; ++t) {
            if (ahead && t + 1 < n) ok = load_tile<D>(km, p, sh, ring, it, w, w.key0(t + 1), p1);
            if (ok) ok = load_tile<D>(vm, p, sh, ring, it, w, w.key0(t), p0);
            if (ok && !ahead && t + 1 < n) ok = load_tile<D>(km, p, sh, ring, it, w, w.key0(t + 1), p1);
            p0 = p1;
            p1 = p2;
            p2 = page(t + 3);
        }
    }
    if (ok && !*(volatile int *)&sh.abort) return;
    // nobody consumes what is in flight after an abort: let it land
    for (uint32_t k = 0; k < (uint32_t)C::kStages && k < it; ++k) {
        const uint32_t i = it - 1 - k;
        drain(smem_u32(&sh.full[i % C::kStages]), (i / C::kStages) & 1);
    }
}

template <int D>
__device__ void role_q(const CUtensorMap *qm, const Params &p, Shared &sh, uint32_t q) {
    using C = Cfg<D>;
    uint32_t n = 0;
    bool ok = true;
    Pieces w(p);
    Cut cut{0, 0, 0, 0};
    while (w.next()) {
        cut = Cut{w.ta == 0 && w.tb < w.u.tiles, w.j, w.ui, 0};
        ok = mbar_wait(smem_u32(&sh.qempty), (n & 1) ^ 1, &sh.abort, p.a.wait_limit);
        if (!ok) break;
        const int used = C::kTiles == 1 ? 1 : w.tiles_used();
        const uint32_t bar = smem_u32(&sh.qfull);
        mbar_arrive_expect_tx(bar, (uint32_t)(used * (D / 64) * 128 * p.a.g * p.tpt));
        for (int e = 0; e < used; ++e)
            for (int pn = 0; pn < D / 64; ++pn)
                tma_load_3d(q + e * C::kQTile + pn * kPanel, qm, pn * 64, w.j * p.a.g, w.u.tok0 + e * p.tpt, bar);
        ++n;
    }
    p.cuts[blockIdx.x] = cut;  // of the last piece
    if (*(volatile int *)&sh.abort && n) drain(smem_u32(&sh.qfull), (n - 1) & 1);
}

// Zeros the rows of a value tile in shared memory outside [from, to): slots that no new
// token sees (they may hold anything, and zero weights would multiply it).  Slots that
// only this unit's rows do not see hold finite values, by the call's contract: clearing
// those too cost 3-10 % on ragged prompts, so it is done only where the sequence's ranges
// leave gaps.
template <int D>
__device__ __forceinline__ void clear_unseen(uint32_t stage, int from, int to) {
    using C = Cfg<D>;
    const int lane = threadIdx.x & 31;
    auto zero = [&](uint32_t at) {
        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(at), "r"(0) : "memory");
    };
    for (int pn = 0; pn < C::kStagePanels; ++pn) {
        for (int i = lane; i < min(from, kRows) * 8; i += 32) zero(stage + pn * kPanel + i * 16);
        for (int i = max(to, 0) * 8 + lane; i < kRows * 8; i += 32) zero(stage + pn * kPanel + i * 16);
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
}

// The same for those of the 32 rows from `from` on whose bit in m is clear.
template <int D>
__device__ __forceinline__ void clear_gaps(uint32_t stage, int from, uint32_t m) {
#pragma unroll 1
    for (int i = threadIdx.x & 31; i < 32 * 8 * Cfg<D>::kStagePanels; i += 32)
        if (!(m >> (i >> 3 & 31) & 1u))
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(stage + (i >> 8) * kPanel + from * 128 + (i & 255) * 16),
                         "r"(0)
                         : "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
}

// MMA issuer x (0: warp 1, 1: warp 3).  The whole warp walks the loop and one elected
// lane issues.  With two row tiles both issuers read every stage and each releases
// it; with one, the keys' issuer and the values' issuer each wait for their own stages and
// release them twice.  A parity tells a phase from the one before only to whoever knows
// that one to be over, and a stage's last use may have been the other issuer's: so each
// waits first for what tells it.  (Without, at head_dim 256 a value stage whose last keys
// were still on their way passed for full.)
template <bool kFp16, int D, bool kGaps>
__device__ void role_mma(const Params &p, Shared &sh, uint32_t q, uint32_t ring, uint32_t tmem, int x) {
    using C = Cfg<D>;
    constexpr uint32_t id_s = idesc_f32(kFp16, kRows, kRows, false);
    constexpr uint32_t id_o = idesc_f32(kFp16, kRows, C::kStageDims, true);
    const long long lim = p.a.wait_limit;
    int *ab = &sh.abort;
    const bool leader = elect_one();
    uint32_t it = 0, nq = 0, turns = 0;
    Uses use;
    Pieces w(p);
    auto wait_stage = [&](uint32_t i) {
        return mbar_wait_warp(smem_u32(&sh.full[i % C::kStages]), (i / C::kStages) & 1, ab, lim);
    };
    auto release = [&](uint32_t i, int times) {
        if (leader)
            for (int k = 0; k < times; ++k) mma_commit(smem_u32(&sh.empty[i % C::kStages]));
        __syncwarp();
    };
    // S[buf] = Q[e] K^T with the keys in stages i .. i + kParts - 1, seen full
    auto qk = [&](int e, int buf, uint32_t i, int set) {
        tc_fence_after();
#pragma unroll 1
        for (int part = 0; part < C::kParts; ++part) {
            const uint32_t kb = ring + ((i + part) % C::kStages) * C::kStageBytes;
            const uint32_t qb = q + e * C::kQTile + part * C::kStageBytes;
            if (leader) {
#pragma unroll
                for (int pn = 0; pn < C::kStagePanels; ++pn)
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        mma_bf16(tmem + buf * kRows, smem_desc_sw128(qb + pn * kPanel) + 2 * ks,
                                 smem_desc_sw128(kb + pn * kPanel) + 2 * ks, id_s, (part | pn | ks) != 0);
            }
            __syncwarp();
        }
        if (leader) mma_commit(smem_u32(&sh.sfull[set][buf]));
        __syncwarp();
    };
    // O[e] += P[buf] V
    auto pv = [&](int e, int buf, uint32_t i, bool first, int set, uint32_t parity) {
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
            if (!mbar_wait_warp(smem_u32(&sh.pfull[set][buf][half]), parity, ab, lim)) return false;
            tc_fence_after();
#pragma unroll 1
            for (int part = 0; part < C::kParts; ++part) {
                const uint64_t vd = desc_mn_sw128(ring + ((i + part) % C::kStages) * C::kStageBytes);
                if (leader) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {  // 16 keys: 8 columns of P, two 8-row groups of V
                        const int ks = 4 * half + k;
                        mma_ts(tmem + C::kOutCol + e * D + part * C::kStageDims, tmem + buf * kRows + 8 * ks,
                               vd + 128 * ks, id_o, !first || ks != 0);
                    }
                }
                __syncwarp();
            }
        }
        if (leader) mma_commit(smem_u32(&sh.pdone[set][buf]));
        __syncwarp();
        return true;
    };
    int edge0 = -1, edge1 = -1;  // first slots of this piece's tiles with something to clear
    auto ready_v = [&](uint32_t i, int t) {  // the value tile of step t, what nobody sees cleared
        for (int part = 0; part < C::kParts; ++part)
            if (!wait_stage(i + part)) return false;
        const int key0 = w.key0(t);
        if constexpr (kGaps) {
            // all that the unit's own rows do not see
            if (!w.u.gaps() && key0 != w.u.kt0 * kRows && key0 != w.u.last_tile()) return true;
#pragma unroll 1
            for (int k = 0; k < kRows; k += 32) {
                const uint32_t m = seen_word(p.a, w.u, key0 + k);
                if (m == 0xffffffffu) continue;
#pragma unroll 1
                for (int part = 0; part < C::kParts; ++part)
                    clear_gaps<D>(ring + ((i + part) % C::kStages) * C::kStageBytes, k, m);
            }
            return true;
        }
        if (key0 == edge0 || key0 == edge1) {
            const int from = w.u.seen0() - key0, to = w.u.seen1() - key0;
            for (int part = 0; part < C::kParts; ++part)
                clear_unseen<D>(ring + ((i + part) % C::kStages) * C::kStageBytes, from, to);
        }
        return true;
    };
    int before = 0;  // row tiles of the piece before
    while (w.next()) {
        const int n = w.steps(), used = C::kTiles == 1 ? 1 : w.tiles_used();
        edge0 = (w.u.edges >> 16 & 255u) ? w.u.kt0 * kRows : -1;
        edge1 = (w.u.edges >> 24) != kRows - 1 ? w.u.last_tile() : -1;
        if (!mbar_wait_warp(smem_u32(&sh.qfull), nq & 1, ab, lim)) goto out;
        // Between two pieces of two tiles each issuer's own order keeps its S buffer
        // safe, between two of one tile the buffers' turns do; where the kind
        // changes, the first issuer's logits would overwrite weights that the other one
        // still multiplies.  (The queries came after both had finished the piece
        // before the last, so that piece's phase cannot be mistaken for this one.)
        if (x == 0 && before && before != used &&
            !mbar_wait_warp(smem_u32(&sh.pieces), (nq - 1) & 1, ab, lim))
            goto out;
        before = used;
        ++nq;
        if (used == 2) {
            // stages: K0, V0, K1, V1, ...
            if (!wait_stage(it)) goto out;
            qk(x, x, it, 1);
            release(it, 1);
            if (n == 1 && leader) mma_commit(smem_u32(&sh.qempty));
            for (int t = 0; t < n; ++t) {
                const uint32_t iv = it + 1 + 2 * t, ik = iv + 1;
                if (!ready_v(iv, t)) goto out;
                // The issuers take turns, a step's products each: one tile's softmax then
                // runs while the other's products do.  Left alone the tiles fall into step
                // and the tensor cores idle while both wait for the same units; turns
                // of the softmax warpgroups do less (2048 tokens over 16K: 471 us
                // with neither, 400 with those, 381 with these).
                if (!(turns == 0 && x == 0) &&
                    !mbar_wait_warp(smem_u32(&sh.turn[x]), (turns + (x ^ 1)) & 1, ab, lim))
                    goto out;
                ++turns;
                if (!pv(x, x, iv, t == 0, 1, use.par(t, 2))) goto out;
                release(iv, 1);
                if (t + 1 == n && leader) mbar_arrive(smem_u32(&sh.turn[x ^ 1]));
                if (t + 1 < n) {
                    if (!wait_stage(ik)) goto out;
                    qk(x, x, ik, 1);
                    if (leader) mbar_arrive(smem_u32(&sh.turn[x ^ 1]));
                    release(ik, 1);
                    // after the last logits the queries' place is free
                    if (t + 2 == n && leader) mma_commit(smem_u32(&sh.qempty));
                }
            }
            it += 2 * n;
        } else {
            // stages: K0, K1, V0, K2, V1, ..., V(n-1): kParts each
            constexpr int P = C::kParts;
            auto at_k = [&](int t) { return it + P * (t < 2 ? t : 2 * t - 1); };
            auto at_v = [&](int t) { return it + P * (t + 1 < n ? 2 * t + 2 : 2 * t + 1); };
            if (x == 1 && leader) mma_commit(smem_u32(&sh.qempty));  // it reads no queries
            for (int t = 0; t < n; ++t) {
                const int buf = use.buf(t, 0, 1);
                if (x == 0) {
                    const uint32_t i = at_k(t);
                    // The buffer's weights of two steps ago have been multiplied; so their values
                    // had come, which these stages or later ones held.
                    if (use.one + t >= 2 && !mbar_wait_warp(smem_u32(&sh.pdone[0][buf]), use.par(t - 2, 1), ab, lim))
                        goto out;
                    for (int part = 0; part < P; ++part)
                        if (!wait_stage(i + part)) goto out;
                    qk(0, buf, i, 0);
                    for (int part = 0; part < P; ++part) release(i + part, 2);
                } else {
                    const uint32_t i = at_v(t);
                    // The step's logits: its keys had come, which one of these stages may have held.
                    // (Where a tile is one stage, the ring's order puts only older keys there.)
                    if (P > 1 && !mbar_wait_warp(smem_u32(&sh.sfull[0][buf]), use.par(t, 1), ab, lim)) goto out;
                    if (!ready_v(i, t)) goto out;
                    if (!pv(0, buf, i, t == 0, 0, use.par(t, 1))) goto out;
                    for (int part = 0; part < P; ++part) release(i + part, 2);
                }
            }
            it += 2 * n * P;
            if (x == 0 && leader) mma_commit(smem_u32(&sh.qempty));
        }
        if (leader) mma_commit(smem_u32(&sh.pieces));
        __syncwarp();
        use.add(n, used);
    }
out:
    if (leader) mma_commit(smem_u32(&sh.fin[x]));
    __syncwarp();
    drain(smem_u32(&sh.fin[x]), 0);
}

template <bool kFp16>
__device__ __forceinline__ uint32_t pack_pair(float x, float y) {
    if constexpr (kFp16) {
        const __half2 h = __floats2half2_rn(x, y);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}

template <bool kFp16, int D, bool kMore>
__device__ void role_softmax(const Params &p, Shared &sh, uint8_t *s_out, float *s_pos, uint8_t *s_xch, uint32_t tmem,
                             int e) {
    using C = Cfg<D>;
    constexpr bool kSplit = C::kTiles == 1;      // the warpgroups share a row tile, 64 columns each
    constexpr int kCh = kSplit ? 2 : 4;          // chunks of 32 columns of a thread
    const int et = kSplit ? 0 : e;               // row tile
    const int ch0 = kSplit ? 2 * e : 0;          // first chunk
    const AttendArgs &a = p.a;
    const int tid = threadIdx.x & 127, lane = tid & 31, quarter = (threadIdx.x >> 5) & 3;
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    const int tl = tid / a.g, h = tid - tl * a.g;  // token and head of this row
    const float sc = a.scale * kLog2e;
    Cap cap;
    if constexpr (kMore) cap.set(a.scale, a.softcap > 0.f ? a.softcap : 1.f);
    const uint32_t ocol = tmem + lane_base + C::kOutCol + et * D;
    uint32_t pos_steps = 0, swaps = 0;
    int ahead_tok = -1;  // the token whose range `ahead` is
    int2 ahead = make_int2(0, 0);
    // the two threads of a row meet (the pair of warps does): false after an abort
    auto meet = [&]() {
        const uint32_t bar = smem_u32(&sh.xch[quarter]);
        mbar_arrive(bar);
        const bool ok = mbar_wait(bar, swaps & 1, &sh.abort, a.wait_limit);
        __syncwarp();
        ++swaps;
        return (bool)__all_sync(0xffffffffu, ok);
    };
    Uses use;
    Pieces w(p);
    while (w.next()) {
        const int n = w.steps(), used = kSplit ? 1 : w.tiles_used();
        if (et >= used) {
            use.add(n, used);
            continue;
        }
        const int tok = et * p.tpt + tl;  // of the unit
        const bool valid = tl < p.tpt && tok < w.u.ntok;
        int2 vis = make_int2(INT32_MIN, INT32_MAX);  // a row nobody reads needs no mask
        if (valid) {
            if (a.visible && w.u.tok0 + tok == ahead_tok) vis = cut_range(ahead, w.u.kv);
            else vis = sees(a, w.u, tok);
        }
        if (a.visible) {
            // the same row of the unit behind this one: read now, used if that one is next
            const int64_t nt = (int64_t)w.u.tok0 + w.u.ntok + tok;
            ahead_tok = nt < a.T ? (int)nt : -1;
            if (ahead_tok >= 0) ahead = reinterpret_cast<const int2 *>(a.visible)[nt];
        }
        const int head = w.j * a.g + h;
        float slope = 0.f;
        int qp = 0;
        if constexpr (kMore) {
            if (a.slopes && valid) {
                slope = a.slopes[head] * kLog2e;
                qp = a.q_pos[w.u.tok0 + tok];
            }
        }
        float m = -INFINITY, l = 0.f;
        int kp = 0, kp0 = 0;  // positions of this thread's key of the next step and of its first seen one
        const int first = w.u.first(), end = w.u.end();
        auto position = [&](int key) {
            // (bad pages are reported where their keys are loaded; one in a gap is none)
            const int pg = key >= first && key < end ? find_page(a.kv, w.u.s, key) : -1;
            return pg < 0 ? 0 : a.kv.pos[(int64_t)pg * a.kv.page_size + key % a.kv.page_size];
        };
        auto fetch_pos = [&](int t) {
            if constexpr (kMore) {
                if (a.slopes && t < n) {
                    if (!kSplit || e == 0) kp = position(w.key0(t) + tid);
                    kp0 = position(max(w.key0(t), first));
                }
            }
        };
        fetch_pos(0);
        for (int t = 0; t < n; ++t) {
            const int buf = use.buf(t, et, used), k0 = w.key0(t);
            float at = 0.f;  // this row's position relative to the step's first seen key
            const float *sp = s_pos + (2 * et + (pos_steps & 1)) * 128;
            if constexpr (kMore) {
                if (a.slopes) {
                    // positions relative to the step's first seen one: exact in fp32, and so are
                    // their distances, up to 2^24.  Two buffers: a thread writes one again
                    // only when all have come past the step between.
                    at = (float)(qp - kp0);
                    if (!kSplit || e == 0) {
                        const_cast<float *>(sp)[tid] = (float)(kp - kp0);
                        mbar_arrive(smem_u32(&sh.pos[et]));
                    }
                    const bool ok = mbar_wait(smem_u32(&sh.pos[et]), pos_steps & 1, &sh.abort, a.wait_limit);
                    __syncwarp();
                    if (!__all_sync(0xffffffffu, ok)) return;
                    ++pos_steps;
                    fetch_pos(t + 1);
                }
            }
            {
                const bool ok = mbar_wait(smem_u32(&sh.sfull[used - 1][buf]), use.par(t, used), &sh.abort, a.wait_limit);
                __syncwarp();
                if (!__all_sync(0xffffffffu, ok)) return;
            }
            tc_fence_after();
            const uint32_t sb = tmem + lane_base + buf * kRows;
            float v[kCh][32];
#pragma unroll
            for (int c = 0; c < kCh; ++c) tmem_ld32(sb + 32 * (ch0 + c), v[c]);
#pragma unroll
            for (int c = 0; c < kCh; ++c) tmem_wait_ld_dep(v[c]);
            if constexpr (kMore) {
                if (a.softcap > 0.f) {
                    // Only logits that count choose the form, so that the others' cannot change
                    // a bit: unseen ones are zeros for it, and rows nobody reads have no say.
                    if (!__all_sync(0xffffffffu, vis.x <= k0 && vis.y >= k0 + kRows)) {
#pragma unroll
                        for (int c = 0; c < kCh; ++c) {
                            const int from = max(vis.x, k0) - k0 - 32 * (ch0 + c);
                            const int to = min(vis.y, k0 + kRows) - k0 - 32 * (ch0 + c);
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (i < from || i >= to) v[c][i] = 0.f;
                        }
                    }
#pragma unroll
                    for (int c = 0; c < kCh; ++c) {
                        float up = fmaxf(v[c][0], v[c][1]), dn = fminf(v[c][0], v[c][1]);
#pragma unroll
                        for (int i = 2; i < 32; i += 2) {
                            up = max3(up, v[c][i], v[c][i + 1]);
                            dn = min3(dn, v[c][i], v[c][i + 1]);
                        }
                        const float most = valid ? fmaxf(up, -dn) * cap.reach : 0.f;
                        if (__all_sync(0xffffffffu, most < 0.2f)) {
#pragma unroll
                            for (int i = 0; i < 32; i += 2) cap.small<4>(v[c][i], v[c][i + 1]);
                        } else if (__all_sync(0xffffffffu, most < 0.5f)) {
#pragma unroll
                            for (int i = 0; i < 32; i += 2) cap.small<8>(v[c][i], v[c][i + 1]);
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[c][i] = cap.any(v[c][i]);
                        }
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < kCh; ++c)
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[c][i] *= sc;
                }
                if (a.slopes) {
#pragma unroll
                    for (int c = 0; c < kCh; ++c)
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float4 k4 = reinterpret_cast<const float4 *>(sp)[8 * (ch0 + c) + i];
                            v[c][4 * i] = fmaf(-slope, fabsf(at - k4.x), v[c][4 * i]);
                            v[c][4 * i + 1] = fmaf(-slope, fabsf(at - k4.y), v[c][4 * i + 1]);
                            v[c][4 * i + 2] = fmaf(-slope, fabsf(at - k4.z), v[c][4 * i + 2]);
                            v[c][4 * i + 3] = fmaf(-slope, fabsf(at - k4.w), v[c][4 * i + 3]);
                        }
                }
            }
            if (!__all_sync(0xffffffffu, vis.x <= k0 && vis.y >= k0 + kRows)) {
                // the rows of a warp are a few tokens', so their ranges begin and end close
                // together, and most of its chunks are seen by all of them
                const int lo = vis.x <= k0 ? 0 : vis.x >= k0 + kRows ? kRows : vis.x - k0;
                const int hi = vis.y >= k0 + kRows ? kRows : vis.y <= k0 ? 0 : vis.y - k0;
#pragma unroll
                for (int c = 0; c < kCh; ++c) {
                    const int from = lo - 32 * (ch0 + c), to = hi - 32 * (ch0 + c);
                    if (!__all_sync(0xffffffffu, from <= 0 && to >= 32)) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (i < from || i >= to) v[c][i] = -INFINITY;
                    }
                }
            }
            float mt = -INFINITY;
            {
                float mx[kCh];
#pragma unroll
                for (int c = 0; c < kCh; ++c) {
                    mx[c] = fmaxf(v[c][0], v[c][1]);
#pragma unroll
                    for (int i = 2; i < 32; i += 2) mx[c] = max3(mx[c], v[c][i], v[c][i + 1]);
                    mt = fmaxf(mt, mx[c]);
                }
            }
            if constexpr (!kMore) mt *= sc;
            if constexpr (kSplit) {
                // Both threads of the row need one reference: the larger of their maxima, in all its
                // bits (a maximum rounded to 16 bits is off by a part of itself, and weights
                // by 2^that: beyond both types for the far keys of a distance bias).  One
                // buffer of 32 bits is what shared memory leaves, hence two meetings: 13 us of
                // the capped case's 311, 1 of 344 for 2048 plain tokens over 16K.
                float *x = reinterpret_cast<float *>(s_xch);
                x[e * 128 + tid] = mt;
                if (!meet()) return;
                mt = fmaxf(x[tid], x[128 + tid]);
                if (!meet()) return;  // read before the place is written again
            }
            const bool grew = mt > m + (kSlack + kLift<kFp16>);
            if (__any_sync(0xffffffffu, grew)) {
                const float f = grew ? exp2f(m - (mt - kLift<kFp16>)) : 1.f;
                if (grew) m = mt - kLift<kFp16>;
                l *= f;
                if (t > 0) {
                    const bool ok = mbar_wait(smem_u32(&sh.pdone[used - 1][use.buf(t - 1, et, used)]), use.par(t - 1, used),
                                              &sh.abort, a.wait_limit);
                    __syncwarp();
                    if (!__all_sync(0xffffffffu, ok)) return;
                    tc_fence_after();
                    constexpr int kScaled = kSplit ? D / 2 : D;
                    const uint32_t from = ocol + (kSplit ? e * kScaled : 0);
#pragma unroll 1
                    for (int c = 0; c < kScaled; c += 16) {
                        uint32_t r[16];
                        asm volatile(
                            "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
                            "%11, %12, %13, %14, %15}, [%16];\n\ttcgen05.wait::ld.sync.aligned;"
                            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
                              "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
                              "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                            : "r"(from + c)
                            : "memory");
#pragma unroll
                        for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * f);
                        tmem_st16(from + c, r);
                    }
                    if constexpr (kSplit) {
                        // the first half's product adds to all of the row: both halves of it
                        // are rescaled before either warpgroup hands over its weights
                        tmem_wait_st();
                        tc_fence_before();
                        if (!meet()) return;
                        tc_fence_after();
                    }
                }
            }
            const float ref = m == -INFINITY ? 0.f : m;
            const uint64_t sc2 = pack2(kMore ? 1.f : sc, kMore ? 1.f : sc), ref2 = pack2(-ref, -ref);
            uint64_t sum[2] = {0, 0};
#pragma unroll
            for (int c = 0; c < kCh; ++c) {
                uint32_t pk[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    float z0, z1;
                    unpack2(fma2(pack2(v[c][2 * i], v[c][2 * i + 1]), sc2, ref2), z0, z1);
                    z0 = ex2_approx(z0);
                    z1 = ex2_approx(z1);
                    sum[i & 1] = add2(sum[i & 1], pack2(z0, z1));
                    pk[i] = pack_pair<kFp16>(z0, z1);
                }
                tmem_st16(sb + 16 * (ch0 + c), pk);
                if (c & 1) {  // the first half's products start while the second is computed
                    tmem_wait_st();
                    tc_fence_before();
                    mbar_arrive(smem_u32(&sh.pfull[used - 1][buf][(ch0 + c) >> 1]));
                }
            }
            float x, y;
            unpack2(add2(sum[0], sum[1]), x, y);
            l += x + y;
        }
        {
            const bool ok = mbar_wait(smem_u32(&sh.pdone[used - 1][use.buf(n - 1, et, used)]), use.par(n - 1, used),
                                      &sh.abort, a.wait_limit);
            __syncwarp();
            if (!__all_sync(0xffffffffu, ok)) return;
        }
        tc_fence_after();
        if constexpr (kSplit) {  // the row's sum is both threads'
            float *x = reinterpret_cast<float *>(s_xch);
            x[e * 128 + tid] = l;
            if (!meet()) return;
            l = x[tid] + x[128 + tid];
            if (!meet()) return;  // read before the place is written again
        }
        const bool whole = w.ta == 0 && w.tb == w.u.tiles;
        const int64_t orow = (int64_t)(w.u.tok0 + tok) * a.Hq + head;
        float *part = p.parts + (int64_t)(2 * blockIdx.x + (w.index ? 1 : 0)) * C::kUnitRows * (D + 4);
        const int prow = et * kRows + tid;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        if (valid && (!kSplit || e == 0)) {
            if (!whole) {
                part[prow] = m;
                part[C::kUnitRows + prow] = l;
            } else if (a.lse) {
                a.lse[orow] = ((m == -INFINITY ? 0.f : m) + log2f(l)) * kLn2;
            }
        }
        const int row_at = valid ? (int)orow : -1;
        constexpr int kCols = kSplit ? D / 2 : D;
#pragma unroll 1
        for (int c0 = 0; c0 < kCols; c0 += 64) {
            const int c = c0 + (kSplit ? e * kCols : 0);
            float o[2][32];
            tmem_ld32(ocol + c, o[0]);
            tmem_ld32(ocol + c + 32, o[1]);
            tmem_wait_ld_dep(o[0]);
            tmem_wait_ld_dep(o[1]);
            if (whole) {
                uint4 pc[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    uint32_t *r = reinterpret_cast<uint32_t *>(&pc[k]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float *src = &o[k >> 2][(k & 3) * 8 + 2 * i];
                        r[i] = l == 0.f ? 0u : pack_pair<kFp16>(src[0] * inv, src[1] * inv);
                    }
                }
                // 16-byte pieces change lanes, so that 8 lanes store 128 adjacent bytes of
                // a row: a store of 16 bytes to each of 32 rows takes the load-store
                // unit 8 times as long, and everybody's loads with it (4000 cycles a
                // piece, against a step's 3000)
                if constexpr (C::kOutBytes > 0) {
                    uint8_t *st = s_out + ((threadIdx.x >> 5) - 4) * 4096;  // 32 rows x 128 bytes
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        *reinterpret_cast<uint4 *>(st + lane * 128 + ((k ^ (lane & 7)) << 4)) = pc[k];
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const int r = (lane >> 3) + 4 * k;
                        const int at = __shfl_sync(0xffffffffu, row_at, r);
                        const uint4 x = *reinterpret_cast<const uint4 *>(st + r * 128 + (((lane & 7) ^ (r & 7)) << 4));
                        if (at >= 0)
                            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + (int64_t)at * D + c +
                                                       8 * (lane & 7)) = x;
                    }
                    __syncwarp();
                } else {
#pragma unroll
                    for (int x = 1; x < 8; x <<= 1)
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            if (k & x) continue;
                            const bool up = lane & x;
                            uint32_t *lo = reinterpret_cast<uint32_t *>(&pc[k]);
                            uint32_t *hi = reinterpret_cast<uint32_t *>(&pc[k | x]);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const uint32_t y = __shfl_xor_sync(0xffffffffu, up ? lo[i] : hi[i], x);
                                if (up) lo[i] = y; else hi[i] = y;
                            }
                        }
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const int at = __shfl_sync(0xffffffffu, row_at, (lane & 24) + k);
                        if (at >= 0)
                            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + (int64_t)at * D + c +
                                                       8 * (lane & 7)) = pc[k];
                    }
                }
            } else if (valid) {
                // in fours of columns, rows adjacent
                float4 *dst = reinterpret_cast<float4 *>(part + 4 * C::kUnitRows) + (c / 4) * C::kUnitRows + prow;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float *src = &o[i >> 3][(i & 7) * 4];
                    dst[i * C::kUnitRows] = make_float4(src[0], src[1], src[2], src[3]);
                }
            }
        }
        tc_fence_before();  // the reads end before the next piece's first product is let in
        use.add(n, used);
    }
}

// kGaps: the kernel of calls whose ranges leave gaps.  Of the two that a call with ranges launches
// the plan lets one work.  In the ordinary kernel the other's code, even as roles of its
// own that are not run, cost a capped call 7 % and documents 2 %; a launch that returns costs
// 4 us of 347.
template <bool kFp16, int D, bool kMore, bool kGaps>
__global__ void __launch_bounds__(Cfg<D>::kThreads, 1)
    attend_kernel(const __grid_constant__ CUtensorMap qm, const __grid_constant__ CUtensorMap km,
                  const __grid_constant__ CUtensorMap vm, const Params p) {
    using C = Cfg<D>;
    extern __shared__ uint8_t raw[];
    const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
    uint8_t *mem = raw + (base - smem_u32(raw));
    const uint32_t q = base, ring = base + C::kQBytes;
    uint8_t *s_out = mem + C::kTail, *s_xch = s_out + C::kOutBytes + C::kPosBytes;
    float *s_pos = reinterpret_cast<float *>(s_out + C::kOutBytes);
    Shared &sh = *reinterpret_cast<Shared *>(s_xch + C::kXchBytes);
    static_assert(sizeof(Shared) <= 512, "Shared");
    if (base - smem_u32(raw) > C::kPad) {  // cannot be; nothing has been touched yet
        if (threadIdx.x == 0) atomicOr(p.a.kv.err, kErrTimeout);
        return;
    }
    if constexpr (kGaps) {
        pdl_wait();
        if (!p.plan->gaps) return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(smem_u32(&sh.full[i]), 1);
            mbar_init(smem_u32(&sh.empty[i]), 2);
        }
        mbar_init(smem_u32(&sh.qfull), 1);
        mbar_init(smem_u32(&sh.qempty), 2);
        mbar_init(smem_u32(&sh.pieces), 2);
        for (int i = 0; i < 4; ++i) mbar_init(smem_u32(&sh.xch[i]), 64);
        for (int i = 0; i < 2; ++i) {
            for (int b = 0; b < 2; ++b) {
                mbar_init(smem_u32(&sh.sfull[i][b]), 1);
                mbar_init(smem_u32(&sh.pfull[i][b][0]), 128);
                mbar_init(smem_u32(&sh.pfull[i][b][1]), 128);
                mbar_init(smem_u32(&sh.pdone[i][b]), 1);
            }
            mbar_init(smem_u32(&sh.turn[i]), 1);
            mbar_init(smem_u32(&sh.pos[i]), 128);
            mbar_init(smem_u32(&sh.fin[i]), 1);
        }
        sh.abort = 0;
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(smem_u32(&sh.tmem), 512);
        tmem_relinquish();
    }
    if (threadIdx.x == 64) {
        tma_prefetch_desc(&qm);
        tma_prefetch_desc(&km);
        tma_prefetch_desc(&vm);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    if constexpr (!kGaps) pdl_wait();
    if (!kGaps && p.plan->gaps) {
        // the other kernel's call
    } else if (warp < 4) {
        // 128 * 88 + 256 * 208 and 128 * 112 + 256 * 192 are at most 384 * 168
        if constexpr (D == 256) asm volatile("setmaxnreg.dec.sync.aligned.u32 112;");
        else asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        if (warp == 0) {
            role_kv<D, kGaps>(&km, &vm, p, sh, ring);
        } else if (warp == 2) {
            if (lane == 0) role_q<D>(&qm, p, sh, q);
        } else {
            role_mma<kFp16, D, kGaps>(p, sh, q, ring, tmem, warp == 1 ? 0 : 1);
        }
        __syncwarp();
    } else {
        if constexpr (D == 256) asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
        else asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        role_softmax<kFp16, D, kMore>(p, sh, s_out, s_pos, s_xch, tmem, (warp - 4) >> 2);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tmem, 512);
    if (threadIdx.x == 0 && sh.abort) atomicOr(p.a.kv.err, kErrTimeout);
}

// ---------------------------------------------------------------- the join

constexpr int kJoinThreads = 256, kJoinRows = 32;

// Block (c, y): the unit that the end of share c cuts, if c is the first to cut it,
// rows [32y, 32y + 32): a lane takes a row, a warp every eighth four of its columns, the
// parts in the order of their slots.  All
// blocks together also write the rows of the units without a visible slot, or of all tokens
// when the batch is malformed.
template <bool kFp16, int D>
__global__ void __launch_bounds__(kJoinThreads) attend_join_kernel(const Params p) {
    using C = Cfg<D>;
    const AttendArgs &a = p.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();
    const Plan pl = *p.plan;
    const int nb = gridDim.x * gridDim.y, me = blockIdx.y * gridDim.x + blockIdx.x;
    for (int i = me; i < (pl.bad ? a.T : pl.units); i += nb) {
        int64_t r0 = (int64_t)i * a.Hq, nr = a.Hq;
        if (!pl.bad) {
            const Unit u = p.units[i];
            if (u.tiles) continue;
            r0 = (int64_t)u.tok0 * a.Hq, nr = (int64_t)u.ntok * a.Hq;
        }
        for (int64_t k = tid; k < nr * D / 8; k += kJoinThreads)
            reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + r0 * D)[k] = make_uint4(0, 0, 0, 0);
        if (a.lse)
            for (int64_t k = tid; k < nr; k += kJoinThreads) a.lse[r0 + k] = -INFINITY;
    }
    if (pl.W == 0) return;
    const Shares sh = shares_of(pl.W * a.kv.Hk, p.grid, kMinTiles);
    const int c0 = blockIdx.x;
    if (c0 + 1 >= sh.n) return;
    const Cut cut = p.cuts[c0];
    if (!cut.parted) return;
    const Unit u = p.units[cut.unit];
    const int j = cut.j;
    const int64_t ub = (int64_t)j * pl.W + u.prefix, ue = ub + width_of(u);
    const int n = share_of(sh, ue - 1) - c0 + 1;
    // a block's first piece is in its slot 0, a later one (this unit's first) in slot 1
    const int slot0 = 2 * c0 + (share_begin(sh, c0) < ub);
    auto part = [&](int i) { return p.parts + (int64_t)(i == 0 ? slot0 : 2 * (c0 + i)) * C::kUnitRows * (D + 4); };
    constexpr int kC = D / 32;  // fours of columns of a warp
    __shared__ __align__(16) uint32_t s_out[kJoinRows][D / 2 + 4];
    __shared__ int s_row[kJoinRows];
    const int r = blockIdx.y * kJoinRows + lane, e = r / kRows, rr = r % kRows;
    const int tl = rr / a.g, tok = e * p.tpt + tl;
    const bool valid = tl < p.tpt && tok < u.ntok;
    float M = -INFINITY, L = 0.f;
    float4 O[kC];
#pragma unroll
    for (int k = 0; k < kC; ++k) O[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (valid) {
#pragma unroll 4
        for (int i = 0; i < n; ++i) M = fmaxf(M, part(i)[r]);
        const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll 4
        for (int i = 0; i < n; ++i) {
            const float *src = part(i);
            const float w = exp2f(src[r] - ref);
            L = fmaf(w, src[C::kUnitRows + r], L);
            const float4 *o = reinterpret_cast<const float4 *>(src + 4 * C::kUnitRows) + r;
#pragma unroll
            for (int k = 0; k < kC; ++k) {
                const float4 v = o[(warp + 8 * k) * C::kUnitRows];
                O[k].x = fmaf(w, v.x, O[k].x); O[k].y = fmaf(w, v.y, O[k].y);
                O[k].z = fmaf(w, v.z, O[k].z); O[k].w = fmaf(w, v.w, O[k].w);
            }
        }
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
    for (int k = 0; k < kC; ++k) {
        uint32_t *dst = &s_out[lane][2 * (warp + 8 * k)];
        dst[0] = L == 0.f ? 0u : pack_pair<kFp16>(O[k].x * inv, O[k].y * inv);
        dst[1] = L == 0.f ? 0u : pack_pair<kFp16>(O[k].z * inv, O[k].w * inv);
    }
    if (warp == 0) {
        const int orow = (u.tok0 + tok) * a.Hq + j * a.g + rr - tl * a.g;
        s_row[lane] = valid ? orow : -1;
        if (valid && a.lse) a.lse[orow] = ((M == -INFINITY ? 0.f : M) + log2f(L)) * kLn2;
    }
    __syncthreads();
    for (int i = tid; i < kJoinRows * D / 8; i += kJoinThreads) {
        const int k = i / (D / 8), c = i - k * (D / 8);
        if (s_row[k] >= 0)
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + (int64_t)s_row[k] * D + 8 * c) =
                *reinterpret_cast<const uint4 *>(&s_out[k][4 * c]);
    }
}

// ---------------------------------------------------------------- host

bool encode_maps(const AttendArgs &a, int tpt, int box, CUtensorMap *qm, CUtensorMap *km, CUtensorMap *vm) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    const CUtensorMapDataType dt = a.kv.fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const cuuint32_t estr[3] = {1, 1, 1};
    const cuuint64_t D = (cuuint64_t)a.kv.d;
    {
        const cuuint64_t dims[3] = {D, (cuuint64_t)a.Hq, (cuuint64_t)a.T};
        const cuuint64_t strides[2] = {D * 2, D * 2 * (cuuint64_t)a.Hq};
        const cuuint32_t bx[3] = {64, (cuuint32_t)a.g, (cuuint32_t)tpt};
        if (enc(qm, dt, 3, const_cast<void *>(a.q), dims, strides, bx, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return false;
    }
    const cuuint64_t dims[3] = {D, (cuuint64_t)a.kv.page_size, (cuuint64_t)(a.kv.num_pages * a.kv.Hk)};
    const cuuint64_t strides[2] = {D * 2, D * 2 * (cuuint64_t)a.kv.page_size};
    const cuuint32_t bx[3] = {64, (cuuint32_t)box, 1};
    for (int i = 0; i < 2; ++i)
        if (enc(i ? vm : km, dt, 3, i ? a.kv.v : a.kv.k, dims, strides, bx, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return false;
    return true;
}

template <bool kFp16, int D>
cudaError_t launch_type(const AttendArgs &a, int num_sms, cudaStream_t st) {
    using C = Cfg<D>;
    Params p{};
    p.a = a;
    p.tpt = kRows / a.g;
    p.box = 128;
    while (a.kv.page_size % p.box) p.box >>= 1;  // 16 at least: page_size is a multiple of it
    p.grid = num_sms < kMaxSms ? num_sms : kMaxSms;
    const Layout L = layout_of(a.T, a.kv.num_seqs, a.Hq, a.kv.Hk, D);
    char *ws = static_cast<char *>(a.workspace);
    p.plan = reinterpret_cast<Plan *>(ws);
    p.seq_off = reinterpret_cast<int32_t *>(ws + L.seq_off);
    p.seen = reinterpret_cast<int4 *>(ws + L.seen);
    p.units = reinterpret_cast<Unit *>(ws + L.units);
    p.cuts = reinterpret_cast<Cut *>(ws + L.cuts);
    p.parts = reinterpret_cast<float *>(ws + L.parts);
    p.max_units = L.max_units;
    CUtensorMap qm, km, vm;
    if (!encode_maps(a, p.tpt, p.box, &qm, &km, &vm)) return cudaErrorInvalidValue;
    // a scale that is not positive turns the maximum around: the general path
    // scales before it compares
    const bool more = a.softcap > 0.f || a.slopes || !(a.scale > 0.f);
    auto kernel = more ? attend_kernel<kFp16, D, true, false> : attend_kernel<kFp16, D, false, false>;
    cudaError_t e = more ? allow_smem<attend_kernel<kFp16, D, true, false>>(C::kSmem)
                         : allow_smem<attend_kernel<kFp16, D, false, false>>(C::kSmem);
    if (e == cudaSuccess && a.visible) e = allow_smem<attend_kernel<kFp16, D, true, true>>(C::kSmem);
    if (e != cudaSuccess) return e;
    e = launch_pdl(a.visible ? attend_plan_kernel<true> : attend_plan_kernel<false>, dim3(1), dim3(kPlanThreads), 0, st, p, C::kTiles * p.tpt);
    if (e != cudaSuccess) return e;
    e = launch_pdl(kernel, dim3((unsigned)p.grid), dim3(C::kThreads), C::kSmem, st, qm, km, vm, p);
    if (e == cudaSuccess && a.visible)
        e = launch_pdl(attend_kernel<kFp16, D, true, true>, dim3((unsigned)p.grid), dim3(C::kThreads), C::kSmem, st, qm,
                       km, vm, p);
    if (e != cudaSuccess) return e;
    return launch_pdl(attend_join_kernel<kFp16, D>, dim3((unsigned)p.grid, C::kUnitRows / kJoinRows),
                      dim3(kJoinThreads), 0, st, p);
}

}  // namespace

size_t attend_workspace(int64_t T, int num_seqs, int Hq, int Hk, int d) {
    return layout_of(T, num_seqs, Hq, Hk, d).total;
}

cudaError_t launch_attend(const AttendArgs &a, int num_sms, cudaStream_t st) {
    switch (a.kv.d) {
        case 64: return a.kv.fp16 ? launch_type<true, 64>(a, num_sms, st) : launch_type<false, 64>(a, num_sms, st);
        case 128: return a.kv.fp16 ? launch_type<true, 128>(a, num_sms, st) : launch_type<false, 128>(a, num_sms, st);
        default: return a.kv.fp16 ? launch_type<true, 256>(a, num_sms, st) : launch_type<false, 256>(a, num_sms, st);
    }
}

}  // namespace up
