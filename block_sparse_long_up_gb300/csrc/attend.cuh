// attend.cuh -- what the two attention kernels share: the cut of the work into equal
// shares, the capped logit and the output rows.
#pragma once

#include "paged.cuh"
#include "sm100.cuh"

namespace up {

constexpr int kMaxSms = 160;  // workspaces are sized for this many
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// The W key tiles of a call, laid end to end, cut into n equal shares wherever they
// fall: block c takes tiles [W*c/n, W*(c+1)/n).
struct Shares {
    int64_t W;
    int n;
};
__device__ __forceinline__ Shares shares_of(int64_t W, int grid, int min_tiles) {
    const int64_t most = (W + min_tiles - 1) / min_tiles;
    return Shares{W, (int)(most < grid ? most : grid)};
}
__device__ __forceinline__ int64_t share_begin(const Shares &h, int c) { return h.W * c / h.n; }
// the block whose share holds tile x
__device__ __forceinline__ int share_of(const Shares &h, int64_t x) {
    int c = (int)(x * h.n / h.W);
    while (c + 1 < h.n && share_begin(h, c + 1) <= x) ++c;
    while (c > 0 && share_begin(h, c) > x) --c;
    return c;
}

// softcap * tanh(x / softcap) as softcap * (1 - 2 / (e^(2x/softcap) + 1)): exact at
// both ends, off by about 2^-22 of softcap in between.
__device__ __forceinline__ float capped(float x, float two_log2e_over_cap, float cap) {
    const float e = sm100::ex2_approx(x * two_log2e_over_cap);
    return cap - __fdividef(2.f * cap, e + 1.f);
}

template <bool kFp16>
__device__ __forceinline__ void store_row4(void *out, int64_t at, float4 v) {
    uint2 w;
    if constexpr (kFp16) {
        const __half2 x = __floats2half2_rn(v.x, v.y), y = __floats2half2_rn(v.z, v.w);
        w = make_uint2(*reinterpret_cast<const uint32_t *>(&x), *reinterpret_cast<const uint32_t *>(&y));
    } else {
        const __nv_bfloat162 x = __floats2bfloat162_rn(v.x, v.y), y = __floats2bfloat162_rn(v.z, v.w);
        w = make_uint2(*reinterpret_cast<const uint32_t *>(&x), *reinterpret_cast<const uint32_t *>(&y));
    }
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(out) + at) = w;
}

}  // namespace up
