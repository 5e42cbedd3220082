// decode.cu -- attention of one new token per sequence over the paged cache.
//
// Every cached key and value is read once, 4*d bytes a slot and KV head, and
// serves the g query heads of its group: 4*g*d flops for 4*d bytes, so the cache's
// bandwidth bounds the call (a step of short caches is bounded by latency): 24 sequences
// of up to 128K, 32/8 heads of 128, take 642 us at 6.8 TB/s, one of 128K 89 us at
// 6.0 TB/s; of one of 4096 with 8/2 heads of 64 the kernels take 8 us in a graph, a call
// 28 us, the host's.
//
// The visible slots of every (sequence, KV head) are cut into tiles of 64 and all
// tiles are laid end to end; block c of the grid takes the c-th equal share of
// them, wherever it begins and ends.  So one long sequence and a ragged batch
// load every SM alike.  A share that holds only a part of a (sequence, KV head)
// leaves its running maximum, sum and unnormalised output in the workspace and
// a second kernel joins the parts in a fixed order; a (sequence, KV head) that lies in
// one share is finished by its block.
//
// Four warps split a tile, 16 slots each, and never wait for one another inside
// a share: each has its own ring of stages filled by 16-byte asynchronous copies
// (rows that the query does not see are filled with zeros, whatever is stored
// there) and its own softmax state; the four are joined in shared memory
// at the end.  The products run on mma m16n8k16 with the group's query heads as
// the 16 rows: at g = 16 they need 109 TFLOP/s at the full memory rate, far
// below what that instruction reaches, so the wider tensor-core path with its
// 128 rows has nothing to give here.  The weights are split into a high and a low
// part of the cache's type, two products each, so rounding them costs nothing (up
// to 8 heads: the low parts are the fragment's other 8 rows, in the same product).
#include "attend.cuh"

namespace up {

namespace {

using namespace sm100;

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kGroup = 16;               // slots of a warp's step
constexpr int kTile = kGroup * kWarps;   // slots of a block's step
constexpr int kMaxPerSm = 3;
constexpr int kMinTiles = 2;             // shares are not cut finer than this

template <int D>
struct Cfg {
    // 128 KB or more in flight on an SM, with one stage being read
    static constexpr int kStages = D == 64 ? 4 : 3;
    static constexpr int kPerSm = D == 64 ? 3 : D == 128 ? 2 : 1;
    static constexpr int kRowBytes = 2 * D;
    static constexpr int kHalfBytes = kGroup * kRowBytes;          // a warp's keys of a stage
    static constexpr int kStageBytes = 2 * kHalfBytes + 64;        // keys, values, positions
    static constexpr int kWarpBytes = (kStages * kStageBytes + 127) / 128 * 128;
    static constexpr int kSmem = kWarps * kWarpBytes;
    // the join of the four warps reuses the rings: 16 rows of D + 2 floats each
    static_assert(kWarps * 16 * (D + 2) * 4 <= kSmem, "join fits");
};

// Tiles' worth of time that a (sequence, KV head) costs beside its tiles (queries, first
// loads, the warps' join): it lies in front of its tiles where all are laid end to end
// (48 windowed sequences at head_dim 256: 81.4 us with 0, 74.8 with 1, 73.6 with 2,
// 75.7 with 4; long sequences do not feel it).
constexpr int kUnitCost = 2;

// First slot and end of what sequence s's query sees, and the tiles they take
// (tiles begin at a multiple of 16 slots, so 16 slots never straddle a page).  First tokens
// that stay visible apart from the window, the slots below sinks < lo, take stiles tiles of their
// own in front.
struct Span {
    int lo, hi, first, tiles, sinks, stiles;
    __device__ __forceinline__ int width() const { return tiles ? tiles + kUnitCost : 0; }
};

__device__ __forceinline__ Span span_of(const AttendArgs &a, int s) {
    Span r;
    r.hi = max(kv_len_of(a.kv, s, 0), 0);
    r.lo = a.kv_start ? max(a.kv_start[s], 0) : 0;
    r.sinks = min(a.sinks, r.hi);
    if (r.lo >= r.hi) {
        r.hi = r.sinks;
        r.lo = r.sinks = 0;
    } else if (r.lo <= r.sinks) {
        r.lo = a.sinks ? 0 : r.lo;
        r.sinks = 0;
    }
    r.first = r.lo & ~(kGroup - 1);
    r.stiles = (r.sinks + kTile - 1) / kTile;
    r.tiles = (r.hi - r.first + kTile - 1) / kTile + r.stiles;
    return r;
}

// Width of one KV head of the sequences before `upto`, summed by the whole block;
// every thread gets the sum.
template <int NT>
__device__ int64_t total_tiles(const AttendArgs &a, int upto, long long *scratch) {
    long long sum = 0;
    for (int s = threadIdx.x; s < upto; s += NT) sum += span_of(a, s).width();
#pragma unroll
    for (int k = 16; k; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = sum;
    __syncthreads();
    sum = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) sum += scratch[w];
    return sum;
}

// The sequence at x (a sequence's Hk heads lie together), and where it begins: every
// warp for itself, 32 sequences at a time.
__device__ void find_sequence(const AttendArgs &a, int64_t x, int &s_out, int64_t &begin) {
    const int lane = threadIdx.x & 31;
    int64_t before = 0;
    for (int s0 = 0; s0 < a.kv.num_seqs; s0 += 32) {
        const int s = s0 + lane;
        int64_t own = s < a.kv.num_seqs ? (int64_t)span_of(a, s).width() * a.kv.Hk : 0, inc = own;
#pragma unroll
        for (int k = 1; k < 32; k <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, inc, k);
            if (lane >= k) inc += y;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, before + inc > x && own > 0);
        if (hit) {
            const int l = __ffs(hit) - 1;
            s_out = s0 + l;
            begin = before + __shfl_sync(0xffffffffu, inc - own, l);
            return;
        }
        before += __shfl_sync(0xffffffffu, inc, 31);
    }
    s_out = a.kv.num_seqs;
    begin = before;
}

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
template <bool kFp16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (kFp16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two weights as a pair of the cache's type (high) and what that rounding left (low).
template <bool kFp16>
__device__ __forceinline__ void split2(float x, float y, uint32_t &hi, uint32_t &lo) {
    if constexpr (kFp16) {
        const __half2 h = __floats2half2_rn(x, y);
        const float2 b = __half22float2(h);
        const __half2 l = __floats2half2_rn(x - b.x, y - b.y);
        hi = *reinterpret_cast<const uint32_t *>(&h);
        lo = *reinterpret_cast<const uint32_t *>(&l);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        const float2 b = __bfloat1622float2(h);
        const __nv_bfloat162 l = __floats2bfloat162_rn(x - b.x, y - b.y);
        hi = *reinterpret_cast<const uint32_t *>(&h);
        lo = *reinterpret_cast<const uint32_t *>(&l);
    }
}

// A part in the workspace: g rows of (maximum in log2 units, sum, D outputs); the
// outputs begin on a 16-byte boundary behind all rows' statistics.
__device__ __forceinline__ float *part_of(const AttendArgs &a, int D, int slot) {
    return static_cast<float *>(a.workspace) + (int64_t)slot * a.g * (D + 4);
}

template <bool kFp16, int D, bool kFew, bool kMore, bool kSinks>
__global__ void __launch_bounds__(kThreads, Cfg<D>::kPerSm) decode_kernel(const AttendArgs a) {
    using C = Cfg<D>;
    constexpr int kCpr = D / 8;          // 16-byte chunks of a row
    constexpr int kRpi = 32 / kCpr > 0 ? 32 / kCpr : 1;  // rows a warp copies at once
    constexpr int kR = kFew ? 1 : 2;     // fragment rows in use: lane/4 and lane/4 + 8
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ long long s_scan[kWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int row = lane >> 2, col = 2 * (lane & 3);
    pdl_wait();
    // every kernel before this one is complete, so the join may read the lengths
    pdl_trigger();
    const int Hk = a.kv.Hk, g = a.g;
    const int64_t W = total_tiles<kThreads>(a, a.kv.num_seqs, s_scan) * Hk;
    if (W == 0) return;
    const Shares sh = shares_of(W, gridDim.x, kMinTiles);
    if ((int)blockIdx.x >= sh.n) return;
    int64_t at = share_begin(sh, blockIdx.x);
    const int64_t end = share_begin(sh, blockIdx.x + 1);
    int s;
    int64_t begin;  // where sequence s begins
    find_sequence(a, at, s, begin);
    if (s >= a.kv.num_seqs) return;
    const uint32_t ring = smem_u32(smem) + warp * C::kWarpBytes;
    const float scale2 = a.scale * kLog2e;
    Cap cap;
    if constexpr (kMore) cap.set(a.scale, a.softcap > 0.f ? a.softcap : 1.f);
    bool first_part = true;
    Span sp = span_of(a, s);
    while (at < end) {
        while (sp.tiles == 0 || at >= begin + (int64_t)sp.width() * Hk) {
            begin += (int64_t)sp.width() * Hk;
            if (++s >= a.kv.num_seqs) return;
            sp = span_of(a, s);
        }
        const int j = (int)((at - begin) / sp.width());
        const int64_t unit = begin + (int64_t)j * sp.width() + kUnitCost;  // its first tile
        const int ta = (int)max(at - unit, (int64_t)0), tb = (int)min((int64_t)sp.tiles, end - unit);
        at = min(end, unit + sp.tiles);
        if (ta >= tb) break;  // the share ends before the first tile
        // the group's queries as fragments (rows past g are zeros)
        uint32_t q[D / 16][4];
        {
            const uint16_t *qb = static_cast<const uint16_t *>(a.q) + ((int64_t)s * a.Hq + (int64_t)j * g) * D;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = row + (i & 1) * 8;
                    q[kk][i] = (r < g && !(kFew && (i & 1)))
                                   ? *reinterpret_cast<const uint32_t *>(qb + r * D + 16 * kk + col + (i >> 1) * 8)
                                   : 0u;
                }
        }
        float slope[kR];
        int qp = 0;
        if constexpr (kMore) {
#pragma unroll
            for (int r = 0; r < kR; ++r)
                slope[r] = a.slopes && row + 8 * r < g ? a.slopes[j * g + row + 8 * r] * kLog2e : 0.f;
            if (a.slopes) qp = a.q_pos[s];
        }
        float m[kR], l[kR], o[D / 8][4];
#pragma unroll
        for (int r = 0; r < kR; ++r) m[r] = -INFINITY, l[r] = 0.f;
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[n][i] = 0.f;

        const int steps = tb - ta;
        // this warp's first slot of a step, and the slots that it may see
        const int key_a = sp.first + (ta - (kSinks ? sp.stiles : 0)) * kTile + warp * kGroup;
        const int apart = kSinks ? sp.stiles - ta : 0;  // steps of the first tokens
        auto key_of = [&](int step) {
            return kSinks && step < apart ? (ta + step) * kTile + warp * kGroup : key_a + step * kTile;
        };
        auto lo_of = [&](int step) { return kSinks && step < apart ? 0 : sp.lo; };
        auto hi_of = [&](int step) { return kSinks && step < apart ? sp.sinks : sp.hi; };
        auto page_at = [&](int step) -> int {
            const int key = key_of(step);
            return step < steps && key < hi_of(step) ? page_of(a.kv, s, key) : -1;
        };
        int pg = page_at(0);  // page of the next step to load, looked up a step ahead
        auto load = [&](int step) {
            if (step < steps) {
                const int key = key_of(step), in_page = key % a.kv.page_size;
                const int lo = lo_of(step), hi = hi_of(step);
                const uint32_t st = ring + (step % C::kStages) * C::kStageBytes;
                const int64_t rb = pg < 0 ? 0 : ((int64_t)pg * Hk + j) * a.kv.page_size + in_page;
                const int r0 = lane / kCpr, c = lane % kCpr;
                const uint8_t *ks = static_cast<const uint8_t *>(a.kv.k) + rb * C::kRowBytes;
                const uint8_t *vs = static_cast<const uint8_t *>(a.kv.v) + rb * C::kRowBytes;
#pragma unroll
                for (int i = 0; i < kGroup / kRpi; ++i) {
                    const int r = r0 + i * kRpi;
                    const bool ok = pg >= 0 && key + r >= lo && key + r < hi;
                    const int off = ok ? r * C::kRowBytes + c * 16 : 0;
                    const uint32_t dst = st + r * C::kRowBytes + ((c ^ (r & 7)) << 4);
                    cp16(dst, ks + off, ok);
                    cp16(dst + C::kHalfBytes, vs + off, ok);
                }
                if constexpr (kMore) {
                    if (a.slopes && lane < 4) {
                        const int32_t *ps = a.kv.pos + (pg < 0 ? 0 : (int64_t)pg * a.kv.page_size + in_page + 4 * lane);
                        cp16(st + 2 * C::kHalfBytes + 16 * lane, ps, pg >= 0);
                    }
                }
                pg = page_at(step + 1);
            }
            cp_commit();
        };
#pragma unroll
        for (int i = 0; i < C::kStages - 1; ++i) load(i);
        for (int step = 0; step < steps; ++step) {
            cp_wait<C::kStages - 2>();
            __syncwarp();
            load(step + C::kStages - 1);
            const uint32_t st = ring + (step % C::kStages) * C::kStageBytes;
            float x[2][4] = {}, x2[2][4] = {};  // two chains of products each
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                uint32_t b[4];
                const int r = ((lane >> 4) << 3) + (lane & 7), c = 2 * kk + ((lane >> 3) & 1);
                ldsm4(st + r * C::kRowBytes + ((c ^ (r & 7)) << 4), b);
                mma16816<kFp16>((kk & 1) ? x2[0] : x[0], q[kk], b[0], b[1]);
                mma16816<kFp16>((kk & 1) ? x2[1] : x[1], q[kk], b[2], b[3]);
            }
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int i = 0; i < 2 * kR; ++i) x[n][i] += x2[n][i];
            const int key = key_of(step), from = lo_of(step), to = hi_of(step);
            // logits in log2 units
            if constexpr (kMore) {
                if (a.softcap > 0.f) {
                    float most = 0.f;
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int i = 0; i < 2 * kR; ++i) most = fmaxf(most, fabsf(x[n][i]));
                    const bool small = __all_sync(0xffffffffu, most * cap.reach < 0.5f);
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int i = 0; i < 2 * kR; i += 2) {
                            if (small) {
                                cap.small<8>(x[n][i], x[n][i + 1]);
                            } else {
                                x[n][i] = cap.any(x[n][i]);
                                x[n][i + 1] = cap.any(x[n][i + 1]);
                            }
                        }
                }
            }
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int i = 0; i < 2 * kR; ++i) {
                    if (!kMore || !(a.softcap > 0.f)) x[n][i] *= scale2;
                    if constexpr (kMore) {
                        if (a.slopes) {
                            int kp;
                            asm volatile("ld.shared.b32 %0, [%1];" : "=r"(kp)
                                         : "r"(st + 2 * C::kHalfBytes + 4 * (8 * n + col + (i & 1))) : "memory");
                            x[n][i] -= slope[i >> 1] * fabsf((float)(qp - kp));
                        }
                    }
                }
            if (key < from || key + kGroup > to) {
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int i = 0; i < 2 * kR; ++i) {
                        const int k = key + 8 * n + col + (i & 1);
                        if (k < from || k >= to) x[n][i] = -INFINITY;
                    }
            }
            bool moved = false;
            float c[kR], ref[kR];
#pragma unroll
            for (int r = 0; r < kR; ++r) {
                float mx = fmaxf(fmaxf(x[0][2 * r], x[0][2 * r + 1]), fmaxf(x[1][2 * r], x[1][2 * r + 1]));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                const bool grew = mx > m[r] + (kSlack + kLift<kFp16>);
                c[r] = grew ? exp2f(m[r] - (mx - kLift<kFp16>)) : 1.f;
                m[r] = grew ? mx - kLift<kFp16> : m[r];
                ref[r] = m[r] == -INFINITY ? 0.f : m[r];
                moved |= grew;
            }
            if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                for (int r = 0; r < kR; ++r) l[r] *= c[r];
#pragma unroll
                for (int n = 0; n < D / 8; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[n][i] *= c[kFew ? 0 : i >> 1];
            }
            uint32_t hi[4] = {}, lo[4] = {};
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int r = 0; r < kR; ++r) {
                    const float p0 = ex2_approx(x[n][2 * r] - ref[r]), p1 = ex2_approx(x[n][2 * r + 1] - ref[r]);
                    l[r] += p0 + p1;
                    split2<kFp16>(p0, p1, hi[2 * n + r], lo[2 * n + r]);
                }
#pragma unroll
            for (int n = 0; n < D / 16; ++n) {
                uint32_t b[4];
                const int r = (((lane >> 3) & 1) << 3) + (lane & 7), c8 = 2 * n + (lane >> 4);
                ldsm4t(st + C::kHalfBytes + r * C::kRowBytes + ((c8 ^ (r & 7)) << 4), b);
                if constexpr (kFew) {
                    const uint32_t both[4] = {hi[0], lo[0], hi[2], lo[2]};
                    mma16816<kFp16>(o[2 * n], both, b[0], b[1]);
                    mma16816<kFp16>(o[2 * n + 1], both, b[2], b[3]);
                } else {
                    mma16816<kFp16>(o[2 * n], hi, b[0], b[1]);
                    mma16816<kFp16>(o[2 * n + 1], hi, b[2], b[3]);
                    mma16816<kFp16>(o[2 * n], lo, b[0], b[1]);
                    mma16816<kFp16>(o[2 * n + 1], lo, b[2], b[3]);
                }
            }
            __syncwarp();
        }
        // join the four warps: rows of (m, l) first, then their outputs
        cp_wait<0>();
        __syncthreads();
        float *st_f = reinterpret_cast<float *>(smem);              // [kWarps][16][2]
        float *o_f = st_f + kWarps * 16 * 2;                        // [kWarps][16][D]
#pragma unroll
        for (int r = 0; r < kR; ++r) {
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
            if ((lane & 3) == 0) {
                st_f[(warp * 16 + row + 8 * r) * 2] = m[r];
                st_f[(warp * 16 + row + 8 * r) * 2 + 1] = l[r];
            }
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
                *reinterpret_cast<float2 *>(o_f + (warp * 16 + row + 8 * r) * D + 8 * n + col) =
                    kFew ? make_float2(o[n][0] + o[n][2], o[n][1] + o[n][3])
                         : make_float2(o[n][2 * r], o[n][2 * r + 1]);
        }
        __syncthreads();
        const bool whole = ta == 0 && tb == sp.tiles;
        float *part = part_of(a, D, 2 * blockIdx.x + (first_part ? 0 : 1));
        for (int i = tid; i < g * (D / 4); i += kThreads) {
            const int r = i / (D / 4), c4 = i - r * (D / 4);
            float M = -INFINITY, L = 0.f;
            float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, st_f[(w * 16 + r) * 2]);
            const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float e = exp2f(st_f[(w * 16 + r) * 2] - ref);
                const float4 v = *reinterpret_cast<const float4 *>(o_f + (w * 16 + r) * D + 4 * c4);
                L = fmaf(e, st_f[(w * 16 + r) * 2 + 1], L);
                O.x = fmaf(e, v.x, O.x); O.y = fmaf(e, v.y, O.y);
                O.z = fmaf(e, v.z, O.z); O.w = fmaf(e, v.w, O.w);
            }
            if (whole) {
                const float inv = L == 0.f ? 0.f : 1.f / L;
                const int64_t orow = (int64_t)s * a.Hq + (int64_t)j * g + r;
                store_row4<kFp16>(a.out, orow * D + 4 * c4,
                                  make_float4(O.x * inv, O.y * inv, O.z * inv, O.w * inv));
                if (a.lse && c4 == 0) a.lse[orow] = (ref + log2f(L)) * kLn2;
            } else {
                *reinterpret_cast<float4 *>(part + 4 * g + r * D + 4 * c4) = O;
                if (c4 == 0) {
                    part[2 * r] = M;
                    part[2 * r + 1] = L;
                }
            }
        }
        __syncthreads();
        first_part = false;
    }
}

// Joins the parts of one (sequence, query head) in the order of its slots, and
// writes the rows that see nothing.
constexpr int kJoinThreads = 128;

template <bool kFp16, int D>
__global__ void __launch_bounds__(kJoinThreads) decode_join_kernel(const AttendArgs a, int grid) {
    __shared__ long long s_scan[kJoinThreads / 32];
    __shared__ float s_w[kMaxSms * kMaxPerSm];
    __shared__ float4 s_o[kJoinThreads * 4 / D][D / 4];
    const int h = blockIdx.x % a.Hq, s = blockIdx.x / a.Hq;
    const int j = h / a.g, r = h - j * a.g;
    // the lengths are the caller's, older than the kernel before; only the parts are not
    const int64_t W = total_tiles<kJoinThreads>(a, a.kv.num_seqs, s_scan) * a.kv.Hk;
    const int64_t before = total_tiles<kJoinThreads>(a, s, s_scan) * a.kv.Hk;
    const Span sp = span_of(a, s);
    const int64_t orow = (int64_t)s * a.Hq + h;
    const int tid = threadIdx.x;
    pdl_wait();
    if (sp.tiles == 0) {
        for (int c = tid; c < D / 4; c += kJoinThreads)
            store_row4<kFp16>(a.out, orow * D + 4 * c, make_float4(0.f, 0.f, 0.f, 0.f));
        if (a.lse && tid == 0) a.lse[orow] = -INFINITY;
        return;
    }
    const Shares sh = shares_of(W, grid, kMinTiles);
    const int64_t unit = before + (int64_t)j * sp.width();
    const int c0 = share_of(sh, unit + kUnitCost), c1 = share_of(sh, unit + sp.width() - 1);
    if (c0 == c1) return;  // finished by its block
    const int n = c1 - c0 + 1;
    // a block's first part is in its slot 0, a later one (this unit's first) in slot 1
    const int slot0 = 2 * c0 + (share_begin(sh, c0) < unit);
    auto part = [&](int i) { return part_of(a, D, i == 0 ? slot0 : 2 * (c0 + i)); };
    const int lane = tid & 31;
    float M = -INFINITY, L = 0.f;
    for (int i = lane; i < n; i += 32) M = fmaxf(M, part(i)[2 * r]);
#pragma unroll
    for (int k = 16; k; k >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, k));
    const float ref = M == -INFINITY ? 0.f : M;
    for (int i = lane; i < n; i += 32) {
        const float2 ml = *reinterpret_cast<const float2 *>(part(i) + 2 * r);
        const float e = exp2f(ml.x - ref);
        if (tid < 32) s_w[i] = e;
        L = fmaf(e, ml.y, L);
    }
#pragma unroll
    for (int k = 16; k; k >>= 1) L += __shfl_xor_sync(0xffffffffu, L, k);
    __syncthreads();
    // kRows rows of threads take every kRows-th part each, D/4 threads a row
    constexpr int kCols = D / 4, kRows = kJoinThreads / kCols;
    const int c = tid % kCols, i0 = tid / kCols;
    float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i = i0; i < n; i += kRows) {
        const float4 v = *reinterpret_cast<const float4 *>(part(i) + 4 * a.g + r * D + 4 * c);
        const float e = s_w[i];
        O.x = fmaf(e, v.x, O.x); O.y = fmaf(e, v.y, O.y);
        O.z = fmaf(e, v.z, O.z); O.w = fmaf(e, v.w, O.w);
    }
    if (i0) s_o[i0 - 1][c] = O;
    __syncthreads();
    if (i0) return;
#pragma unroll
    for (int k = 1; k < kRows; ++k) {
        const float4 v = s_o[k - 1][c];
        O.x += v.x; O.y += v.y; O.z += v.z; O.w += v.w;
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    store_row4<kFp16>(a.out, orow * D + 4 * c, make_float4(O.x * inv, O.y * inv, O.z * inv, O.w * inv));
    if (a.lse && tid == 0) a.lse[orow] = (ref + log2f(L)) * kLn2;
}

template <bool kFp16, int D, bool kFew, bool kMore, bool kSinks>
cudaError_t launch_variant(const AttendArgs &a, int num_sms, cudaStream_t st) {
    using C = Cfg<D>;
    const int grid = (num_sms < kMaxSms ? num_sms : kMaxSms) * C::kPerSm;
    cudaError_t e = allow_smem<decode_kernel<kFp16, D, kFew, kMore, kSinks>>(C::kSmem);
    if (e != cudaSuccess) return e;
    e = launch_pdl(decode_kernel<kFp16, D, kFew, kMore, kSinks>, dim3((unsigned)grid), dim3(kThreads), C::kSmem, st, a);
    if (e != cudaSuccess) return e;
    return launch_pdl(decode_join_kernel<kFp16, D>, dim3((unsigned)(a.kv.num_seqs * a.Hq)),
                      dim3(kJoinThreads), 0, st, a, grid);
}

template <bool kFp16, int D>
cudaError_t launch_type(const AttendArgs &a, int num_sms, cudaStream_t st) {
    // up to 8 query heads a group: half of the fragment's rows carry no weights
    const bool few = a.g <= 8, more = a.softcap > 0.f || a.slopes;
    if (a.sinks) return few ? launch_variant<kFp16, D, true, true, true>(a, num_sms, st)
                            : launch_variant<kFp16, D, false, true, true>(a, num_sms, st);
    if (few) return more ? launch_variant<kFp16, D, true, true, false>(a, num_sms, st)
                         : launch_variant<kFp16, D, true, false, false>(a, num_sms, st);
    return more ? launch_variant<kFp16, D, false, true, false>(a, num_sms, st)
                : launch_variant<kFp16, D, false, false, false>(a, num_sms, st);
}

}  // namespace

size_t decode_workspace(int, int Hq, int Hk, int d) {
    // two parts for every block the grid may have
    return (size_t)2 * kMaxSms * kMaxPerSm * (size_t)(Hq / Hk) * (size_t)(d + 4) * sizeof(float);
}

cudaError_t launch_decode(const AttendArgs &a, int num_sms, cudaStream_t st) {
    switch (a.kv.d) {
        case 64: return a.kv.fp16 ? launch_type<true, 64>(a, num_sms, st) : launch_type<false, 64>(a, num_sms, st);
        case 128: return a.kv.fp16 ? launch_type<true, 128>(a, num_sms, st) : launch_type<false, 128>(a, num_sms, st);
        default: return a.kv.fp16 ? launch_type<true, 256>(a, num_sms, st) : launch_type<false, 256>(a, num_sms, st);
    }
}

}  // namespace up
