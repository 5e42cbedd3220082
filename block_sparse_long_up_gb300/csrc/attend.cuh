// attend.cuh -- what the two attention kernels share: the cut of the work into equal
// shares, the capped logit and the output rows.
#pragma once

#include <atomic>

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

// A capped logit, softcap * tanh(scale * x / softcap), in log2 units.  Where the
// argument of tanh is small (most logits of most models) its Taylor series: 4 terms up
// to 0.2 and 8 up to 0.5 leave less than 2^-23 of the result; elsewhere
// (1 - t) / (1 + t) with t = e^(-2|y|), off by about 2^-23 of softcap.  The series' coefficients
// hold powers of scale / softcap up to the 14th; where these pass fp32 (a softcap below about
// 1/900 of the scale) the general form serves small arguments too.
struct Cap {
    float in, out;   // scale / softcap, softcap * log2(e)
    float reach;     // |in|, or infinite where there is no series: product * reach bounds its argument
    uint64_t c[8];   // the series in powers of x, for two logits at once
    __device__ __forceinline__ void set(float scale, float softcap) {
        constexpr float k[8] = {1.f, -1.f / 3.f, 2.f / 15.f, -17.f / 315.f, 62.f / 2835.f, -1382.f / 155925.f,
                                21844.f / 6081075.f, -929569.f / 638512875.f};
        in = fmaxf(fminf(scale / softcap, 3.0e38f), -3.0e38f);
        out = softcap * kLog2e;
        float f = scale * kLog2e;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            c[i] = sm100::pack2(k[i] * f, k[i] * f);
            f *= in * in;
        }
        float last, same;
        sm100::unpack2(c[7], last, same);
        reach = fabsf(last) <= 3.0e38f ? fabsf(in) : INFINITY;
    }
    template <int kTerms>
    __device__ __forceinline__ void small(float &x, float &y) const {
        const uint64_t t = sm100::pack2(x, y), t2 = sm100::mul2(t, t);
        uint64_t r = c[kTerms - 1];
#pragma unroll
        for (int i = kTerms - 2; i >= 0; --i) r = sm100::fma2(r, t2, c[i]);
        sm100::unpack2(sm100::mul2(r, t), x, y);
    }
    __device__ __forceinline__ float any(float x) const {
        const float t = sm100::ex2_approx(fabsf(x * in) * (-2.f * kLog2e));
        return copysignf(__fdividef(1.f - t, 1.f + t) * out, x * in);
    }
};

// The running reference of a row's weights: a maximum less kLift, replaced when the maximum has grown by
// more than kSlack (both log2), so that outputs are seldom rescaled.  Weights stay
// below 2^(kSlack + kLift).  Fp16 ends at 2^16 and loses bits below 2^-14: lifted by 2^7,
// weights keep them down to 2^-21 of the maximum's and lose 2^-32 of it at most below
// (unlifted, a first token that draws all the weight left 2^-24 of itself as the smallest
// weight of the others, which the sum counted in full).
constexpr float kSlack = 8.f;
template <bool kFp16>
constexpr float kLift = kFp16 ? 7.f : 0.f;

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

// Lets a kernel use `bytes` of dynamic shared memory, once per device.
template <auto kKernel>
cudaError_t allow_smem(int bytes) {
    static std::atomic<uint64_t> done{0};  // a bit per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
}

}  // namespace up
