// append.cu -- rotary positions and the append to the paged cache, in one kernel.
//
// Every new token's query, key and value rows are read once and written once:
// 2 * (Hq + 2*Hk) * d * 2 bytes a token, which is all there is to do beside
// rot/2 sines and cosines a token; so memory bounds a prompt and latency a step (32768
// tokens of 32 + 16 rows of 128: 129 us at 6.2 TB/s; one token: 3.9 us in a graph, 20 us
// a call, the host's).
//
// A block takes a tile of consecutive tokens.  Their angles come first, one
// thread per (token, frequency), into shared memory: computed once per token and
// used by its Hq + Hk rows.  Then a thread moves 32 bytes at a time (one "unit"
// of a row): for a rotated row the 8 dims [8u, 8u+8) and their partners half a
// rotation away (or 16 adjacent dims when pairs are interleaved), for the rest
// 16 adjacent dims, so both members of every pair are in one thread and no
// element is exchanged.
#include "paged.cuh"

namespace up {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 32;   // tokens of a tile
constexpr int kMaxHalf = 128;    // rot / 2
constexpr int kAngles = 2048;    // angles of a tile
constexpr int kUnits = 12 * kThreads;  // units of a tile
constexpr int kInFlight = 4;     // units a thread loads before it stores any

// inv_freq in turns a position, as a multiple of 2^-64 turns (rounded once, to 2^-56 of a
// turn for up to 1 radian); its product with a position wraps at whole turns by itself, so
// nothing is lost beside that rounding for every 32-bit position.  (Once a frequency and
// block: 64-bit floats are slow here.)
__device__ __forceinline__ unsigned long long turn_step(float inv_freq) {
    double t = (double)inv_freq * 0.15915494309189533577;  // 1 / (2 pi)
    t -= rint(t);
    return (unsigned long long)__double2ll_rn(t * 18446744073709551616.0);
}
// The angle at a position as a fraction of half a turn in [-1, 1).
__device__ __forceinline__ float half_turns(unsigned long long step, int pos) {
    const unsigned long long at = step * (unsigned long long)(long long)pos;
    return (float)(int)(at >> 32) * 4.656612873077392578125e-10f;  // 2^-31
}

template <typename T2>
__device__ __forceinline__ float2 to_f2(uint32_t w);
template <>
__device__ __forceinline__ float2 to_f2<__nv_bfloat162>(uint32_t w) {
    return __bfloat1622float2(*reinterpret_cast<__nv_bfloat162 *>(&w));
}
template <>
__device__ __forceinline__ float2 to_f2<__half2>(uint32_t w) {
    return __half22float2(*reinterpret_cast<__half2 *>(&w));
}
template <typename T2>
__device__ __forceinline__ uint32_t from_f2(float a, float b);
template <>
__device__ __forceinline__ uint32_t from_f2<__nv_bfloat162>(float a, float b) {
    const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&r);
}
template <>
__device__ __forceinline__ uint32_t from_f2<__half2>(float a, float b) {
    const __half2 r = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&r);
}

// Turns the 8 pairs of a unit: (x[i], y[i]) when split in halves, adjacent
// elements of x then y when interleaved.  fp32 products, one rounding at the end.
template <typename T2, bool kInterleaved>
__device__ __forceinline__ void turn_unit(uint4 &x, uint4 &y, const float *cs, const float *sn) {
    uint32_t *xw = reinterpret_cast<uint32_t *>(&x), *yw = reinterpret_cast<uint32_t *>(&y);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 a = to_f2<T2>(xw[i]), b = to_f2<T2>(yw[i]);
        if constexpr (kInterleaved) {
            xw[i] = from_f2<T2>(a.x * cs[i] - a.y * sn[i], a.y * cs[i] + a.x * sn[i]);
            yw[i] = from_f2<T2>(b.x * cs[4 + i] - b.y * sn[4 + i], b.y * cs[4 + i] + b.x * sn[4 + i]);
        } else {
            xw[i] = from_f2<T2>(a.x * cs[2 * i] - b.x * sn[2 * i],
                                a.y * cs[2 * i + 1] - b.y * sn[2 * i + 1]);
            yw[i] = from_f2<T2>(b.x * cs[2 * i] + a.x * sn[2 * i],
                                b.y * cs[2 * i + 1] + a.y * sn[2 * i + 1]);
        }
    }
}

template <typename T2, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, 4) append_kernel(const AppendArgs a, int tile) {
    __shared__ __align__(16) float s_cos[kAngles], s_sin[kAngles];
    __shared__ unsigned long long s_step[kMaxHalf];
    __shared__ int64_t s_row[kMaxTokens];
    const int tid = threadIdx.x;
    const int t0 = blockIdx.x * tile, nt = min(tile, a.T - t0);
    const int half = a.rot >> 1, page_size = a.kv.page_size;
    pdl_wait();
    for (int f = tid; f < half; f += kThreads) s_step[f] = turn_step(a.inv_freq[f]);
    // one thread per token (the last warp's) finds its slot and records its position there
    const int finder = kThreads - 1 - tid;
    if (finder < nt) {
        const int t = t0 + finder;
        const int s = seq_of_token(a.cu_seqlens, a.kv.num_seqs, t, a.T, a.kv.err);
        int64_t row = -1;
        if (s >= 0) {
            const int end = a.cu_seqlens[s + 1];
            const int kv = kv_len_of(a.kv, s, end - a.cu_seqlens[s]);
            if (kv >= 0) {
                const int slot = kv - (end - t), in_page = slot % page_size;
                const int pg = page_of(a.kv, s, slot);
                if (pg >= 0) {
                    row = (int64_t)pg * a.kv.Hk * page_size + in_page;
                    if (a.kv.pos) a.kv.pos[(int64_t)pg * page_size + in_page] = a.pos[t];
                }
            }
        }
        s_row[finder] = row;
    }
    __syncthreads();
    for (int i = tid; i < nt * half; i += kThreads) {
        const int tl = i / half, f = i - tl * half;
        int ax = a.axes ? a.axes[f] : 0;
        if (ax < 0 || ax >= a.num_axes) ax = 0;
        float sn, cs;
        sincospif(half_turns(s_step[f], a.pos[(int64_t)ax * a.T + t0 + tl]), &sn, &cs);
        s_cos[i] = cs;
        s_sin[i] = sn;
    }
    __syncthreads();
    const int d = a.kv.d, Hq = a.Hq, Hk = a.kv.Hk;
    const int upr = d >> 4, turned = a.rot >> 4;  // units of a row, those that turn
    const int R = Hq + 2 * Hk;
    const int total = nt * R * upr;
    for (int base = tid; base < total; base += kThreads * kInFlight) {
        uint4 x[kInFlight], y[kInFlight];
        uint4 *dst[kInFlight];
        int xo[kInFlight], yo[kInFlight], ang[kInFlight];
#pragma unroll
        for (int k = 0; k < kInFlight; ++k) {
            const int i = base + k * kThreads;
            dst[k] = nullptr;
            if (i < total) {
                const int u = i % upr, pr = i / upr, tl = pr / R, r = pr - tl * R;
                const int64_t t = t0 + tl;
                const uint4 *src;
                bool rot = u < turned;
                if (r < Hq) {
                    src = reinterpret_cast<const uint4 *>(
                        static_cast<const uint16_t *>(a.q) + t * a.q_stride + (int64_t)r * d);
                    dst[k] = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.q_out) +
                                                       (t * Hq + r) * d);
                } else {
                    const bool is_k = r < Hq + Hk;
                    const int j = r - Hq - (is_k ? 0 : Hk);
                    src = reinterpret_cast<const uint4 *>(
                        static_cast<const uint16_t *>(is_k ? a.k : a.v) +
                        t * (is_k ? a.k_stride : a.v_stride) + (int64_t)j * d);
                    if (s_row[tl] >= 0)
                        dst[k] = reinterpret_cast<uint4 *>(
                            static_cast<uint16_t *>(is_k ? a.kv.k : a.kv.v) +
                            (s_row[tl] + (int64_t)j * page_size) * d);
                    rot = rot && is_k;
                }
                const bool split = u < turned && !kInterleaved;
                xo[k] = split ? u : 2 * u;
                yo[k] = split ? u + turned : 2 * u + 1;
                ang[k] = rot ? tl * half + 8 * u : -1;
                x[k] = src[xo[k]];
                y[k] = src[yo[k]];
            }
        }
#pragma unroll
        for (int k = 0; k < kInFlight; ++k) {
            if (!dst[k]) continue;
            if (ang[k] >= 0) {
                float cs[8], sn[8];
                const float4 *c4 = reinterpret_cast<const float4 *>(s_cos + ang[k]);
                const float4 *s4 = reinterpret_cast<const float4 *>(s_sin + ang[k]);
                *reinterpret_cast<float4 *>(cs) = c4[0];
                *reinterpret_cast<float4 *>(cs + 4) = c4[1];
                *reinterpret_cast<float4 *>(sn) = s4[0];
                *reinterpret_cast<float4 *>(sn + 4) = s4[1];
                turn_unit<T2, kInterleaved>(x[k], y[k], cs, sn);
            }
            dst[k][xo[k]] = x[k];
            dst[k][yo[k]] = y[k];
        }
    }
}

}  // namespace

cudaError_t launch_append(const AppendArgs &a, int num_sms, cudaStream_t st) {
    // tokens per block: a step's few tokens spread one to a block; a prompt's fill a block
    // (kUnits or kAngles of them) once there are four blocks for every SM.  Eight tokens
    // of 12 rows of 64 left blocks that were all lookups: 21 us for 19K tokens against
    // 15 with 32.
    int tile = (a.T + 4 * num_sms - 1) / (4 * num_sms);
    const int units = (a.Hq + 2 * a.kv.Hk) * (a.kv.d >> 4);
    if (tile > kUnits / units) tile = kUnits / units;
    if (a.rot > 0 && tile > kAngles / (a.rot >> 1)) tile = kAngles / (a.rot >> 1);
    tile = tile < 1 ? 1 : tile > kMaxTokens ? kMaxTokens : tile;
    const unsigned grid = (unsigned)((a.T + tile - 1) / tile);
    if (a.kv.fp16)
        return a.interleaved
                   ? launch_pdl(append_kernel<__half2, true>, dim3(grid), dim3(kThreads), 0, st, a, tile)
                   : launch_pdl(append_kernel<__half2, false>, dim3(grid), dim3(kThreads), 0, st, a, tile);
    return a.interleaved
               ? launch_pdl(append_kernel<__nv_bfloat162, true>, dim3(grid), dim3(kThreads), 0, st, a, tile)
               : launch_pdl(append_kernel<__nv_bfloat162, false>, dim3(grid), dim3(kThreads), 0, st, a, tile);
}

}  // namespace up
