// attend_set.cuh -- attention of new tokens that see more than one range of slots: a window and
// the first tokens of the cache that stay visible (sinks), or the cache and a tree of
// drafted tokens at its end.  The plans, and the launches (see attend_tc.cuh for the kernel).
//
// Per row the set is a window [first, end), the slots below `sinks` and, in a tree, one bit for
// each drafted token: its ancestors and itself.  A unit's key tiles are those of the first
// slots and those of its rows' windows; between the two nothing is read.  Only tiles at the
// windows' edges and in the tree take the masked path, where a row's 32 slots are one word.
#pragma once

#include "attend_tc.cuh"

namespace up {

namespace {

// A unit's tiles: those of the first `send` slots, and those of [first, wend) behind them.
__device__ __forceinline__ void set_of(Unit &u, int first, int wend, int send, bool gaps) {
    const int st = (send + kRows - 1) / kRows;
    const int wt = wend > 0 ? (wend + kRows - 1) / kRows - max(first / kRows, st) : 0;
    u.kt0 = gaps ? ~first : first;
    u.edges = (uint32_t)wend;
    u.tiles = st + max(wt, 0);
}

// Block 0 lists the units.  With a tree the other blocks write each token's bits: a thread walks
// its token's line of parents, whose numbers fall at every step.
template <Mask kMask>
__global__ void __launch_bounds__(kPlanThreads) attend_set_plan_kernel(const Params p, uint32_t *bits, int tpu) {
    constexpr bool kIsTree = kMask == kTree;
    __shared__ int64_t sh[32];
    __shared__ int bad, s_wrong, s_off[kPlanThreads];
    const AttendArgs &a = p.a;
    const int B = a.kv.num_seqs, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) bad = s_wrong = 0;
    pdl_wait();
    pdl_trigger();  // what came before is complete: the main kernel's set-up may overlap
    __syncthreads();
    if (kIsTree && blockIdx.x > 0) {
        const int t = ((int)blockIdx.x - 1) * kPlanThreads + tid;
        if (t >= a.T) return;
        const int s = seq_of_token(a.cu_seqlens, B, t, a.T, a.kv.err);
        uint32_t m[kTreeWords] = {};
        if (s >= 0) {
            const int c0 = a.cu_seqlens[s];
            int j = t - c0;
            while (j >= 0 && j < UP_TREE_MAX) {
#pragma unroll
                for (int i = 0; i < kTreeWords; ++i) m[i] |= (j >> 5) == i ? 1u << (j & 31) : 0u;
                const int up = a.parents[c0 + j];
                if (up >= j) break;  // malformed: the sequence has no unit with tiles
                j = up;
            }
        }
        uint4 *dst = reinterpret_cast<uint4 *>(bits + (int64_t)t * kTreeWords);
#pragma unroll
        for (int i = 0; i < kTreeWords / 4; ++i)
            dst[i] = make_uint4(m[4 * i], m[4 * i + 1], m[4 * i + 2], m[4 * i + 3]);
        return;
    }
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
            if (s0 == 0) s_off[s] = p.seq_off[s];
            // (see Pieces::all)
            const int past = kIsTree && n ? a.kv.kv_lens[s] - (a.cu_seqlens[s + 1] - a.cu_seqlens[s]) : 0;
            p.seen[s] = kIsTree ? make_int4(a.kv_start ? max(past, 0) : 0, past + (a.cu_seqlens[s + 1] - a.cu_seqlens[s]),
                                          min(a.sinks, max(past, 0)), 0)
                              : make_int4(INT32_MAX, 0, 0, 0);
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
    if constexpr (kIsTree) {
        // a warp a sequence: every parent comes before its child
        for (int s = warp; s < B; s += kPlanThreads / 32) {
            const int c0 = a.cu_seqlens[s], n = a.cu_seqlens[s + 1] - c0;
            bool wrong = n > UP_TREE_MAX;
            for (int j = lane; j < n && !wrong; j += 32) wrong = a.parents[c0 + j] < -1 || a.parents[c0 + j] >= j;
            if (__any_sync(0xffffffffu, wrong) && lane == 0) {
                s_wrong = 1;
                p.seen[s].y = -1;
                atomicOr(a.kv.err, kErrTree);
            }
        }
        __syncthreads();
    }
    // the unit numbered i, without its tiles (a tree's without windows: with them)
    auto unit_at = [&](int64_t i) {
        int lo = 0, hi = B - 1;  // the last sequence with seq_off <= i
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if ((mid < kPlanThreads ? s_off[mid] : p.seq_off[mid]) <= i) lo = mid; else hi = mid - 1;
        }
        const int c0 = a.cu_seqlens[lo], c1 = a.cu_seqlens[lo + 1];
        Unit u{};
        u.s = lo;
        u.tok0 = c0 + (int)(i - p.seq_off[lo]) * tpu;
        u.ntok = min(tpu, c1 - u.tok0);
        u.kv = kv_len_of(a.kv, lo, c1 - c0);
        if (kIsTree && s_wrong && p.seen[lo].y < 0) u.kv = -1;
        if (kIsTree && u.kv >= 0) {
            u.hi0 = u.kv - (c1 - c0);
            set_of(u, 0, u.kv, min(a.sinks, u.hi0), false);
        }
        return u;
    };
    if (kIsTree && !a.kv_start) {
        for (int64_t i = tid; i < units; i += kPlanThreads) p.units[i] = unit_at(i);
    } else {
        // A warp takes four units at once, a lane each to begin with, then its lanes at their tokens (one at a
        // time 250 units took 14 us; 10 so).
        constexpr int kSame = 4;
        for (int64_t i0 = warp * kSame; i0 < units; i0 += kPlanThreads / 32 * kSame) {
            Unit u = unit_at(min(i0 + (lane & (kSame - 1)), units - 1));
            // (the first token has one before it in its sequence?)
            const bool goes_on = u.tok0 > a.cu_seqlens[u.s];
            int tok0[kSame], ntok[kSame], kv[kSame], first[kSame], end[kSame], some[kSame];
            bool on[kSame], gaps[kSame], torn[kSame];
#pragma unroll
            for (int k = 0; k < kSame; ++k) {
                tok0[k] = __shfl_sync(0xffffffffu, u.tok0, k);
                ntok[k] = __shfl_sync(0xffffffffu, u.ntok, k);
                kv[k] = __shfl_sync(0xffffffffu, u.kv, k);
                if (kv[k] < 0) ntok[k] = 0;
                first[k] = INT32_MAX;
                end[k] = some[k] = 0;
                on[k] = __shfl_sync(0xffffffffu, goes_on, k);
                gaps[k] = torn[k] = false;
            }
            for (int t = lane; t < tpu; t += 32) {
                int2 v[kSame], b[kSame];
#pragma unroll
                for (int k = 0; k < kSame; ++k) {
                    const int at = tok0[k] + min(t, max(ntok[k] - 1, 0));
                    if constexpr (kIsTree) {
                        v[k].x = a.kv_start[at];
                    } else {
                        const int2 *vis = reinterpret_cast<const int2 *>(a.visible) + at;
                        v[k] = *vis;
                        b[k] = vis[(t || on[k]) && t < ntok[k] ? -1 : 0];
                    }
                }
#pragma unroll
                for (int k = 0; k < kSame; ++k) {
                    if (t >= ntok[k]) continue;
                    if constexpr (kIsTree) {
                        first[k] = min(first[k], max(v[k].x, 0));
                    } else {
                        const int2 r = cut_range(v[k], kv[k]), before = cut_range(b[k], kv[k]);
                        first[k] = min(first[k], r.x);
                        end[k] = max(end[k], r.y);
                        some[k] = max(some[k], min(v[k].y, kv[k]));
                        const bool apart = r.y > 0 && max(before.x, r.x) > min(before.y, r.y);
                        torn[k] |= apart;
                        gaps[k] |= apart && t;
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < kSame; ++k) {
                const int lo = __reduce_min_sync(0xffffffffu, first[k]);
                const int hi = __reduce_max_sync(0xffffffffu, end[k]), most = __reduce_max_sync(0xffffffffu, some[k]);
                const bool gap = __any_sync(0xffffffffu, gaps[k]), tear = __any_sync(0xffffffffu, torn[k]);
                if (lane != k || i0 + k >= units) continue;
                if (u.kv >= 0) {
                    if constexpr (kIsTree) {
                        set_of(u, min(lo, u.hi0), u.kv, min(a.sinks, u.hi0), false);
                        atomicMin(&p.seen[u.s].x, lo);
                    } else {
                        u.hi0 = min(a.sinks, most);
                        set_of(u, hi > 0 ? lo : 0, hi, u.hi0, gap);
                        if (hi > 0) {
                            atomicMin(&p.seen[u.s].x, lo);
                            atomicMax(&p.seen[u.s].y, hi);
                        }
                        atomicMax(&p.seen[u.s].z, u.hi0);
                        if (tear) atomicOr(&p.seen[u.s].w, 1);
                    }
                }
                p.units[i0 + k] = u;
            }
        }
    }
    __syncthreads();
    int64_t W = 0;
    for (int64_t u0 = 0; u0 < units; u0 += kPlanThreads) {
        const int64_t i = u0 + tid;
        int64_t total;
        const int64_t at = block_scan(i < units ? width_of(p.units[i]) : 0, &total, sh);
        if (i < units) p.units[i].prefix = W + at;
        W += total;
    }
    if (tid == 0) *p.plan = Plan{W, (int)units, 0, 0};
}

template <Mask kMask, bool kFp16, int D>
cudaError_t launch_type(const AttendArgs &a, int num_sms, cudaStream_t st) {
    using C = Cfg<D>;
    Params p{};
    CUtensorMap qm, km, vm;
    const size_t used = params_of<D>(a, num_sms, p);
    uint32_t *bits = kMask == kTree ? reinterpret_cast<uint32_t *>(static_cast<char *>(a.workspace) + used) : nullptr;
    p.bits = bits;
    if (!encode_maps(a, p.tpt, p.box, &qm, &km, &vm)) return cudaErrorInvalidValue;
    const bool more = a.softcap > 0.f || a.slopes || !(a.scale > 0.f);
    auto kernel = more ? attend_kernel<kFp16, D, true, kMask> : attend_kernel<kFp16, D, false, kMask>;
    cudaError_t e = more ? allow_smem<attend_kernel<kFp16, D, true, kMask>>(C::kSmem)
                         : allow_smem<attend_kernel<kFp16, D, false, kMask>>(C::kSmem);
    if (e != cudaSuccess) return e;
    const unsigned blocks = kMask == kTree ? 1 + (unsigned)((a.T + kPlanThreads - 1) / kPlanThreads) : 1;
    e = launch_pdl(attend_set_plan_kernel<kMask>, dim3(blocks), dim3(kPlanThreads), 0, st, p, bits, C::kTiles * p.tpt);
    if (e != cudaSuccess) return e;
    e = launch_pdl(kernel, dim3((unsigned)p.grid), dim3(C::kThreads), C::kSmem, st, qm, km, vm, p);
    if (e != cudaSuccess) return e;
    return launch_pdl(attend_join_kernel<kFp16, D, kMask>, dim3((unsigned)p.grid * kJoinPerSm), dim3(kJoinThreads), 0, st, p);
}

template <Mask kMask>
cudaError_t launch_set(const AttendArgs &a, int num_sms, cudaStream_t st) {
    switch (a.kv.d) {
        case 64: return a.kv.fp16 ? launch_type<kMask, true, 64>(a, num_sms, st) : launch_type<kMask, false, 64>(a, num_sms, st);
        case 128: return a.kv.fp16 ? launch_type<kMask, true, 128>(a, num_sms, st) : launch_type<kMask, false, 128>(a, num_sms, st);
        default: return a.kv.fp16 ? launch_type<kMask, true, 256>(a, num_sms, st) : launch_type<kMask, false, 256>(a, num_sms, st);
    }
}

}  // namespace

}  // namespace up
