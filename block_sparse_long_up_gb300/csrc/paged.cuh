// paged.cuh -- the paged KV cache as the append and attention kernels see it.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace up {

// Error bits the paged kernels set (see UP_DEVERR_* in include/up.h).
constexpr unsigned int kErrCuSeqlens = 0x1u;
constexpr unsigned int kErrTimeout = 0x4u;
constexpr unsigned int kErrPage = 0x8u;
constexpr unsigned int kErrKvLens = 0x40u;

struct PagedKv {
    void *k;
    void *v;
    int32_t *pos;  // may be null
    const int32_t *block_table;
    const int32_t *kv_lens;
    int64_t num_pages;
    int num_seqs, max_pages, page_size, Hk, d;
    bool fp16;
    unsigned int *err;
};

// Page of slot `slot` of sequence s, or -1 when the table names a page outside the
// pool.  0 <= slot < max_pages * page_size.
__device__ __forceinline__ int find_page(const PagedKv &c, int s, int slot) {
    const int pg = c.block_table[(int64_t)s * c.max_pages + slot / c.page_size];
    return pg < 0 || pg >= c.num_pages ? -1 : pg;
}
// The same, and a page outside the pool sets UP_DEVERR_BAD_PAGE.
__device__ __forceinline__ int page_of(const PagedKv &c, int s, int slot) {
    const int pg = find_page(c, s, slot);
    if (pg < 0) atomicOr(c.err, kErrPage);
    return pg;
}

// Cached tokens of sequence s, of which `fresh` are new; -1 (UP_DEVERR_BAD_KV_LENS
// set) when the length cannot be one.
__device__ __forceinline__ int kv_len_of(const PagedKv &c, int s, int fresh) {
    const int kv = c.kv_lens[s];
    // (the last 2^16 lengths are left out so that rounding up to tiles stays in 32 bits)
    if (kv < fresh || kv < 0 || kv > INT32_MAX - 65536 || kv > (int64_t)c.max_pages * c.page_size) {
        atomicOr(c.err, kErrKvLens);
        return -1;
    }
    return kv;
}

// The sequence of packed token t (0 <= t < total): the last s with cu[s] <= t.
// Sets UP_DEVERR_BAD_CU_SEQLENS and returns -1 when cu does not cover t, or the
// sequence would end past the total.
__device__ __forceinline__ int seq_of_token(const int32_t *cu, int num_seqs, int t, int total,
                                            unsigned int *err) {
    int lo = 0, hi = num_seqs - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cu[mid] <= t) lo = mid; else hi = mid - 1;
    }
    if (cu[lo] < 0 || cu[lo] > t || cu[lo + 1] <= t || cu[lo + 1] > total) {
        atomicOr(err, kErrCuSeqlens);
        return -1;
    }
    return lo;
}

struct AppendArgs {
    PagedKv kv;
    const void *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;
    const int32_t *pos, *axes;
    const float *inv_freq;
    const int32_t *cu_seqlens;
    void *q_out;
    int num_axes, rot, Hq, T;
    bool interleaved;
};
cudaError_t launch_append(const AppendArgs &a, int num_sms, cudaStream_t st);

struct AttendArgs {
    PagedKv kv;
    const void *q;
    const int32_t *cu_seqlens;  // null: one token per sequence (decode)
    const int32_t *visible;     // attend: [T][2] or null
    const int32_t *kv_start;    // decode: [num_seqs] or null
    const float *slopes;        // [Hq] or null
    const int32_t *q_pos;       // [T] or null
    void *out;
    float *lse;  // may be null
    void *workspace;
    float scale, softcap;
    int T, Hq, g;
    long long wait_limit;
};
size_t attend_workspace(int64_t T, int num_seqs, int Hq, int Hk, int d);
size_t decode_workspace(int num_seqs, int Hq, int Hk, int d);
cudaError_t launch_attend(const AttendArgs &a, int num_sms, cudaStream_t st);
cudaError_t launch_decode(const AttendArgs &a, int num_sms, cudaStream_t st);

}  // namespace up
