// attend.cu -- attention over the paged cache, the plainest form: one warp per
// (new token, query head).  A lane holds d/32 dims of the query and of the
// output; each visible slot costs one product summed over the warp, and the
// softmax's maximum and sum run along (everything in fp32, one rounding at the
// end).  Reads the keys once per query head, so the cache's bandwidth and the
// shuffles bound it.
#include "paged.cuh"

namespace up {

namespace {

constexpr int kWarps = 8;

template <bool kFp16>
__device__ __forceinline__ float load1(const void *p, int64_t i) {
    if constexpr (kFp16) return __half2float(static_cast<const __half *>(p)[i]);
    else return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
}

template <bool kFp16, int kD>
__global__ void attend_rows_kernel(const AttendArgs a) {
    constexpr int kE = kD / 32;
    pdl_wait();
    const int64_t row = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (row >= (int64_t)a.T * a.Hq) return;
    const int lane = threadIdx.x & 31, h = (int)(row % a.Hq), t = (int)(row / a.Hq);
    const int j = h / a.g;
    int s = t, fresh = 0, back = 1;  // back: tokens of the sequence from this one on
    if (a.cu_seqlens) {
        s = seq_of_token(a.cu_seqlens, a.kv.num_seqs, t, a.T, a.kv.err);
        if (s >= 0) {
            fresh = a.cu_seqlens[s + 1] - a.cu_seqlens[s];
            back = a.cu_seqlens[s + 1] - t;
        }
    }
    const int kv = s >= 0 ? kv_len_of(a.kv, s, fresh) : -1;
    int lo = 0, hi = 0;
    if (kv >= 0) {
        hi = kv - back + 1;
        if (a.kv_start) lo = max(a.kv_start[s], 0);
        if (a.visible) {
            lo = max(a.visible[2 * (int64_t)t], 0);
            hi = min(a.visible[2 * (int64_t)t + 1], kv);
        }
    }
    float q[kE], o[kE], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < kE; ++e) {
        q[e] = load1<kFp16>(a.q, row * kD + e * 32 + lane);
        o[e] = 0.f;
    }
    const float slope = a.slopes ? a.slopes[h] : 0.f;
    const int qp = a.slopes ? a.q_pos[t] : 0;
    for (int i = lo; i < hi; ++i) {
        const int pg = page_of(a.kv, s, i), in_page = i % a.kv.page_size;
        const int64_t at = (((int64_t)pg * a.kv.Hk + j) * a.kv.page_size + in_page) * kD;
        float x = 0.f;
        if (pg >= 0)
#pragma unroll
            for (int e = 0; e < kE; ++e) x = fmaf(q[e], load1<kFp16>(a.kv.k, at + e * 32 + lane), x);
#pragma unroll
        for (int k = 16; k; k >>= 1) x += __shfl_xor_sync(0xffffffffu, x, k);
        x *= a.scale;
        if (a.softcap > 0.f) x = a.softcap * tanhf(x / a.softcap);
        if (a.slopes) {
            const int kp = pg >= 0 ? a.kv.pos[(int64_t)pg * a.kv.page_size + in_page] : 0;
            x -= slope * fabsf((float)(qp - kp));
        }
        const float mn = fmaxf(m, x);
        const float back_m = mn == -INFINITY ? 0.f : mn;
        const float p = expf(x - back_m), c = expf(m - back_m);
        l = l * c + p;
        m = mn;
#pragma unroll
        for (int e = 0; e < kE; ++e)
            o[e] = o[e] * c + (pg >= 0 ? p * load1<kFp16>(a.kv.v, at + e * 32 + lane) : 0.f);
    }
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
#pragma unroll
    for (int e = 0; e < kE; ++e) {
        if constexpr (kFp16)
            static_cast<__half *>(a.out)[row * kD + e * 32 + lane] = __float2half_rn(o[e] * inv);
        else
            static_cast<__nv_bfloat16 *>(a.out)[row * kD + e * 32 + lane] =
                __float2bfloat16_rn(o[e] * inv);
    }
    if (a.lse && lane == 0) a.lse[row] = (m == -INFINITY ? 0.f : m) + logf(l);
}

template <bool kFp16>
cudaError_t launch_rows(const AttendArgs &a, cudaStream_t st) {
    const dim3 grid((unsigned)(((int64_t)a.T * a.Hq + kWarps - 1) / kWarps)), block(32 * kWarps);
    switch (a.kv.d) {
        case 64: return launch_pdl(attend_rows_kernel<kFp16, 64>, grid, block, 0, st, a);
        case 128: return launch_pdl(attend_rows_kernel<kFp16, 128>, grid, block, 0, st, a);
        default: return launch_pdl(attend_rows_kernel<kFp16, 256>, grid, block, 0, st, a);
    }
}

}  // namespace

size_t attend_workspace(int64_t, int, int, int, int) { return 256; }

cudaError_t launch_attend(const AttendArgs &a, int, cudaStream_t st) {
    return a.kv.fp16 ? launch_rows<true>(a, st) : launch_rows<false>(a, st);
}

}  // namespace up
