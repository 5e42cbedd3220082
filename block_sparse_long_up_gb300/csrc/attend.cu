// attend.cu -- attention of new tokens whose visible slots are one range each: the plan, which
// lists the work, and the launches (see attend_tc.cuh for the kernel).
#include "attend_tc.cuh"

namespace up {

namespace {

// ---------------------------------------------------------------- the plan

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

// ---------------------------------------------------------------- host

template <bool kFp16, int D>
cudaError_t launch_type(const AttendArgs &a, int num_sms, cudaStream_t st) {
    using C = Cfg<D>;
    Params p{};
    params_of<D>(a, num_sms, p);
    CUtensorMap qm, km, vm;
    if (!encode_maps(a, p.tpt, p.box, &qm, &km, &vm)) return cudaErrorInvalidValue;
    // a scale that is not positive turns the maximum around: the general path
    // scales before it compares
    const bool more = a.softcap > 0.f || a.slopes || !(a.scale > 0.f);
    auto kernel = more ? attend_kernel<kFp16, D, true, kRanges> : attend_kernel<kFp16, D, false, kRanges>;
    cudaError_t e = more ? allow_smem<attend_kernel<kFp16, D, true, kRanges>>(C::kSmem)
                         : allow_smem<attend_kernel<kFp16, D, false, kRanges>>(C::kSmem);
    if (e == cudaSuccess && a.visible) e = allow_smem<attend_kernel<kFp16, D, true, kGaps>>(C::kSmem);
    if (e != cudaSuccess) return e;
    e = launch_pdl(a.visible ? attend_plan_kernel<true> : attend_plan_kernel<false>, dim3(1), dim3(kPlanThreads), 0, st, p, C::kTiles * p.tpt);
    if (e != cudaSuccess) return e;
    e = launch_pdl(kernel, dim3((unsigned)p.grid), dim3(C::kThreads), C::kSmem, st, qm, km, vm, p);
    if (e == cudaSuccess && a.visible)
        e = launch_pdl(attend_kernel<kFp16, D, true, kGaps>, dim3((unsigned)p.grid), dim3(C::kThreads), C::kSmem, st, qm,
                       km, vm, p);
    if (e != cudaSuccess) return e;
    return launch_pdl(attend_join_kernel<kFp16, D, kRanges>, dim3((unsigned)p.grid * kJoinPerSm), dim3(kJoinThreads), 0, st, p);
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
