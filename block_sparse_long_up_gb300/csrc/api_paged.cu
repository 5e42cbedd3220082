// api_paged.cu -- the C ABI of the paged-cache calls declared in include/up.h:
// argument validation and launches.  No compute happens here.
#include <math.h>

#include "../../include/up.h"
#include "api_util.cuh"
#include "pages.cuh"

namespace {

using up::aligned;

up_status check_cache(const up_paged_kv *c, int Hq_multiple_of) {
    if (!c || c->num_seqs < 0 || c->Hk < 1 || c->num_pages < 0 || c->max_pages < 1 ||
        c->page_size < 16 || c->page_size % 16 != 0)
        return UP_ERR_INVALID_ARG;
    if (c->num_seqs > 0 &&
        (!c->k_pages || !c->v_pages || !c->block_table || !c->kv_lens || c->num_pages < 1))
        return UP_ERR_INVALID_ARG;
    // page indexes, the rows of one page over all heads and the heads of all pages are 32-bit
    if (c->num_pages > INT32_MAX || (int64_t)c->Hk * c->page_size > INT32_MAX ||
        c->num_pages * c->Hk >= INT32_MAX)
        return UP_ERR_INVALID_ARG;
    if (!aligned(c->k_pages, 16) || !aligned(c->v_pages, 16) || !aligned(c->pos_pages, 16) ||
        !aligned(c->block_table, 4) || !aligned(c->kv_lens, 4))
        return UP_ERR_INVALID_ARG;
    if (c->d != 64 && c->d != 128 && c->d != 256) return UP_ERR_UNSUPPORTED;
    if (c->dtype != UP_BF16 && c->dtype != UP_FP16) return UP_ERR_UNSUPPORTED;
    if (Hq_multiple_of >= 0) {
        if (Hq_multiple_of < 1 || Hq_multiple_of % c->Hk != 0) return UP_ERR_INVALID_ARG;
        if (Hq_multiple_of / c->Hk > 16) return UP_ERR_UNSUPPORTED;
    }
    return UP_OK;
}

up::PagedKv device_view(const up_paged_kv *c, unsigned int *err) {
    up::PagedKv k{};
    k.k = c->k_pages;
    k.v = c->v_pages;
    k.pos = c->pos_pages;
    k.block_table = c->block_table;
    k.kv_lens = c->kv_lens;
    k.num_pages = c->num_pages;
    k.num_seqs = c->num_seqs;
    k.max_pages = c->max_pages;
    k.page_size = c->page_size;
    k.Hk = c->Hk;
    k.d = c->d;
    k.fp16 = c->dtype == UP_FP16;
    k.err = err;
    return k;
}

up_status check_logits(const up_logits *l, const up_paged_kv *c) {
    if (!l || !isfinite(l->scale) || !isfinite(l->softcap) || l->softcap < 0.f ||
        (l->softcap > 0.f && l->softcap < 1e-6f))
        return UP_ERR_INVALID_ARG;
    if (l->slopes && (!l->q_pos || !c->pos_pages)) return UP_ERR_INVALID_ARG;
    return UP_OK;
}

// what a pool call takes, before its pointers to rows
up_status check_table(const up_page_pool *p, int num_seqs, int max_pages, int page_size) {
    if (!p || !p->refs || !p->free_pages || !p->num_free || p->num_pages < 1 || p->num_pages > INT32_MAX ||
        !aligned(p->refs, 4) || !aligned(p->free_pages, 4) || !aligned(p->num_free, 4))
        return UP_ERR_INVALID_ARG;
    if (num_seqs < 0 || max_pages < 1 || page_size < 16 || page_size % 16 != 0 ||
        (int64_t)num_seqs * max_pages > INT32_MAX)
        return UP_ERR_INVALID_ARG;
    return UP_OK;
}

up::PagePool pool_view(const up_page_pool *p, unsigned int *err) {
    return up::PagePool{p->refs, p->free_pages, p->num_free, (int)p->num_pages, err};
}

bool overlap(const int32_t *a, int64_t na, const int32_t *b, int64_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + 4 * (uint64_t)nb && y < x + 4 * (uint64_t)na;
}

// the tiles of a compaction (32 rows and more each, of every head's keys and values) have 32-bit numbers
bool few_tiles(int64_t T, int num_seqs, int Hk) { return (T / 32 + num_seqs) * 2 * Hk <= INT32_MAX; }

up_status check_sinks(int sinks) {
    return sinks < 0 ? UP_ERR_INVALID_ARG : sinks > UP_SINKS_MAX ? UP_ERR_UNSUPPORTED : UP_OK;
}

up::AttendArgs attend_args(const void *q, int Hq, int64_t T, const up_paged_kv *c,
                           const up_logits *l, void *out, float *lse, void *ws,
                           const up::DeviceInfo &di) {
    up::AttendArgs a{};
    a.kv = device_view(c, di.err);
    a.q = q;
    a.slopes = l->slopes;
    a.q_pos = l->q_pos;
    a.out = out;
    a.lse = lse;
    a.workspace = ws;
    a.scale = l->scale;
    a.softcap = l->softcap;
    a.T = (int)T;
    a.Hq = Hq;
    a.g = Hq / c->Hk;
    a.wait_limit = di.wait_limit;
    return a;
}

// sizes that the workspace calls answer for
bool known_sizes(int64_t T, int num_seqs, int Hq, int Hk, int d) {
    return T >= 0 && T <= INT32_MAX && num_seqs >= 0 && Hk >= 1 && Hq >= 1 && Hq % Hk == 0 &&
           Hq / Hk <= 16 && (d == 64 || d == 128 || d == 256) && T * Hq <= INT32_MAX;
}

}  // namespace

extern "C" {

up_status up_append_kv(const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                       const void *v, int64_t v_stride, const int32_t *pos, int num_axes,
                       const int32_t *axes, const float *inv_freq, int rot_dim, uint32_t flags,
                       const int32_t *cu_seqlens, int64_t total_tokens, int Hq,
                       const up_paged_kv *cache, void *q_out, up_stream_t stream) {
    const up::CallRange range("up_append_kv");
    up_status st = check_cache(cache, -1);
    if (st != UP_OK) return st;
    if (total_tokens < 0 || total_tokens > INT32_MAX || Hq < 0 || num_axes < 1 || rot_dim < 0 ||
        rot_dim > cache->d || rot_dim % 16 != 0 || (flags & ~UP_ROPE_INTERLEAVED) != 0)
        return UP_ERR_INVALID_ARG;
    if (total_tokens == 0) return UP_OK;
    if (cache->num_seqs < 1 || !k || !v || !pos || !cu_seqlens || (rot_dim > 0 && !inv_freq) ||
        (Hq > 0 && (!q || !q_out)))
        return UP_ERR_INVALID_ARG;
    const int64_t wk = (int64_t)cache->Hk * cache->d, wq = (int64_t)Hq * cache->d;
    if (k_stride < wk || v_stride < wk || k_stride % 8 != 0 || v_stride % 8 != 0 ||
        (Hq > 0 && (q_stride < wq || q_stride % 8 != 0 || (q_out == q && q_stride != wq))))
        return UP_ERR_INVALID_ARG;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(q, 16) || !aligned(q_out, 16) ||
        !aligned(pos, 4) || !aligned(axes, 4) || !aligned(inv_freq, 4) || !aligned(cu_seqlens, 4))
        return UP_ERR_INVALID_ARG;
    up::DeviceInfo di{};
    if ((st = up::device_info(&di)) != UP_OK) return st;
    up::AppendArgs a{};
    a.kv = device_view(cache, di.err);
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.pos = pos;
    a.axes = axes;
    a.inv_freq = inv_freq;
    a.cu_seqlens = cu_seqlens;
    a.q_out = q_out;
    a.num_axes = num_axes;
    a.rot = rot_dim;
    a.Hq = Hq;
    a.T = (int)total_tokens;
    a.interleaved = (flags & UP_ROPE_INTERLEAVED) != 0;
    if (up::launch_append(a, di.sms, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
        return UP_ERR_CUDA;
    return UP_OK;
}

size_t up_attend_paged_workspace(int64_t total_tokens, int num_seqs, int Hq, int Hk, int d) {
    if (!known_sizes(total_tokens, num_seqs, Hq, Hk, d)) return 0;
    return up::attend_workspace(total_tokens, num_seqs, Hq, Hk, d);
}

size_t up_attend_tree_workspace(int64_t total_tokens, int num_seqs, int Hq, int Hk, int d) {
    if (!known_sizes(total_tokens, num_seqs, Hq, Hk, d)) return 0;
    return up::attend_tree_workspace(total_tokens, num_seqs, Hq, Hk, d);
}

size_t up_decode_attend_workspace(int num_seqs, int Hq, int Hk, int d) {
    if (!known_sizes(num_seqs, num_seqs, Hq, Hk, d)) return 0;
    return up::decode_workspace(num_seqs, Hq, Hk, d);
}

}  // extern "C"

namespace {

// up_attend_paged, up_attend_sinks and (with parents) up_attend_tree.
up_status attend(const void *q, const int32_t *cu_seqlens, const int32_t *parents, int64_t total_tokens,
                 int Hq, const up_paged_kv *cache, const up_logits *logits, const int32_t *visible,
                 const int32_t *kv_start, int sinks, bool tree, void *out, float *lse, void *workspace,
                 size_t workspace_bytes, up_stream_t stream) {
    up_status st = check_cache(cache, Hq);
    if (st != UP_OK) return st;
    if ((st = check_logits(logits, cache)) != UP_OK) return st;
    if ((st = check_sinks(sinks)) != UP_OK) return st;
    if (!known_sizes(total_tokens, cache->num_seqs, Hq, cache->Hk, cache->d))
        return UP_ERR_INVALID_ARG;
    if (total_tokens == 0) return UP_OK;
    if (cache->num_seqs < 1 || !q || !cu_seqlens || !out || (tree && !parents)) return UP_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(visible, 8) ||
        !aligned(cu_seqlens, 4) || !aligned(parents, 4) || !aligned(kv_start, 4))
        return UP_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, 256) ||
        workspace_bytes <
            (tree ? up::attend_tree_workspace : up::attend_workspace)(total_tokens, cache->num_seqs, Hq,
                                                                      cache->Hk, cache->d))
        return UP_ERR_WORKSPACE;
    up::DeviceInfo di{};
    if ((st = up::device_info(&di)) != UP_OK) return st;
    up::AttendArgs a = attend_args(q, Hq, total_tokens, cache, logits, out, lse, workspace, di);
    a.cu_seqlens = cu_seqlens;
    a.visible = visible;
    a.kv_start = kv_start;
    a.parents = parents;
    // without a window nothing lies between the first tokens and the others
    a.sinks = visible || kv_start ? sinks : 0;
    const auto launch = tree ? up::launch_attend_tree : a.sinks ? up::launch_attend_sinks : up::launch_attend;
    if (launch(a, di.sms, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) return UP_ERR_CUDA;
    return UP_OK;
}

up_status decode(const void *q, int Hq, const up_paged_kv *cache, const up_logits *logits,
                 const int32_t *kv_start, int sinks, void *out, float *lse, void *workspace,
                 size_t workspace_bytes, up_stream_t stream) {
    up_status st = check_cache(cache, Hq);
    if (st != UP_OK) return st;
    if ((st = check_logits(logits, cache)) != UP_OK) return st;
    if ((st = check_sinks(sinks)) != UP_OK) return st;
    if (!known_sizes(cache->num_seqs, cache->num_seqs, Hq, cache->Hk, cache->d))
        return UP_ERR_INVALID_ARG;
    if (cache->num_seqs == 0) return UP_OK;
    if (!q || !out) return UP_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(kv_start, 4))
        return UP_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, 256) ||
        workspace_bytes < up::decode_workspace(cache->num_seqs, Hq, cache->Hk, cache->d))
        return UP_ERR_WORKSPACE;
    up::DeviceInfo di{};
    if ((st = up::device_info(&di)) != UP_OK) return st;
    up::AttendArgs a =
        attend_args(q, Hq, cache->num_seqs, cache, logits, out, lse, workspace, di);
    a.kv_start = kv_start;
    a.sinks = kv_start ? sinks : 0;
    if (up::launch_decode(a, di.sms, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
        return UP_ERR_CUDA;
    return UP_OK;
}

}  // namespace

extern "C" {

up_status up_attend_paged(const void *q, const int32_t *cu_seqlens, int64_t total_tokens, int Hq,
                          const up_paged_kv *cache, const up_logits *logits,
                          const int32_t *visible, void *out, float *lse, void *workspace,
                          size_t workspace_bytes, up_stream_t stream) {
    const up::CallRange range("up_attend_paged");
    return attend(q, cu_seqlens, nullptr, total_tokens, Hq, cache, logits, visible, nullptr, 0, false, out, lse,
                  workspace, workspace_bytes, stream);
}

up_status up_attend_sinks(const void *q, const int32_t *cu_seqlens, int64_t total_tokens, int Hq,
                          const up_paged_kv *cache, const up_logits *logits,
                          const int32_t *visible, int sinks, void *out, float *lse,
                          void *workspace, size_t workspace_bytes, up_stream_t stream) {
    const up::CallRange range("up_attend_sinks");
    return attend(q, cu_seqlens, nullptr, total_tokens, Hq, cache, logits, visible, nullptr, sinks, false, out,
                  lse, workspace, workspace_bytes, stream);
}

up_status up_attend_tree(const void *q, const int32_t *cu_seqlens, const int32_t *parents,
                         int64_t total_tokens, int Hq, const up_paged_kv *cache,
                         const up_logits *logits, const int32_t *kv_start, int sinks, void *out,
                         float *lse, void *workspace, size_t workspace_bytes,
                         up_stream_t stream) {
    const up::CallRange range("up_attend_tree");
    return attend(q, cu_seqlens, parents, total_tokens, Hq, cache, logits, nullptr, kv_start, sinks, true, out,
                  lse, workspace, workspace_bytes, stream);
}

up_status up_decode_attend(const void *q, int Hq, const up_paged_kv *cache,
                           const up_logits *logits, const int32_t *kv_start, void *out,
                           float *lse, void *workspace, size_t workspace_bytes,
                           up_stream_t stream) {
    const up::CallRange range("up_decode_attend");
    return decode(q, Hq, cache, logits, kv_start, 0, out, lse, workspace, workspace_bytes, stream);
}

up_status up_decode_sinks(const void *q, int Hq, const up_paged_kv *cache,
                          const up_logits *logits, const int32_t *kv_start, int sinks, void *out,
                          float *lse, void *workspace, size_t workspace_bytes,
                          up_stream_t stream) {
    const up::CallRange range("up_decode_sinks");
    return decode(q, Hq, cache, logits, kv_start, sinks, out, lse, workspace, workspace_bytes, stream);
}

size_t up_compact_kv_workspace(int64_t max_tokens, int num_seqs, int Hk, int d) {
    if (max_tokens < 0 || max_tokens > INT32_MAX || num_seqs < 0 || Hk < 1 ||
        (d != 64 && d != 128 && d != 256) || !few_tiles(max_tokens, num_seqs, Hk))
        return 0;
    return up::kv_compact_workspace(max_tokens, num_seqs, Hk, d);
}

up_status up_compact_kv(const up_paged_kv *cache, const int32_t *cu_seqlens, int64_t max_tokens,
                        const uint8_t *keep, int64_t num_flags, const int32_t *cu_blocks, int G,
                        int32_t *kv_lens_out, void *workspace, size_t workspace_bytes,
                        up_stream_t stream) {
    const up::CallRange range("up_compact_kv");
    up_status st = check_cache(cache, -1);
    if (st != UP_OK) return st;
    if (max_tokens < 0 || max_tokens > INT32_MAX || num_flags < 0 || G < 1 || (!cu_blocks && G > 1) ||
        !few_tiles(max_tokens, cache->num_seqs, cache->Hk))
        return UP_ERR_INVALID_ARG;
    if (cache->num_seqs == 0) return UP_OK;
    if (!cu_seqlens || !kv_lens_out || (num_flags > 0 && !keep)) return UP_ERR_INVALID_ARG;
    if (!aligned(cu_seqlens, 4) || !aligned(cu_blocks, 4) || !aligned(kv_lens_out, 4)) return UP_ERR_INVALID_ARG;
    const int64_t n = cache->num_seqs;
    if ((kv_lens_out != cache->kv_lens && overlap(kv_lens_out, n, cache->kv_lens, n)) ||
        overlap(kv_lens_out, n, cu_seqlens, n + 1) || (cu_blocks && overlap(kv_lens_out, n, cu_blocks, n + 1)))
        return UP_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, 256) ||
        workspace_bytes < up::kv_compact_workspace(max_tokens, cache->num_seqs, cache->Hk, cache->d))
        return UP_ERR_WORKSPACE;
    up::DeviceInfo di{};
    if ((st = up::device_info(&di)) != UP_OK) return st;
    up::KvCompactArgs a{};
    a.kv = device_view(cache, di.err);
    a.cu_seqlens = cu_seqlens;
    a.cu_blocks = cu_blocks ? cu_blocks : cu_seqlens;
    a.keep = keep;
    a.lens_out = kv_lens_out;
    a.workspace = workspace;
    a.num_flags = num_flags;
    a.T = (int)max_tokens;
    a.G = G;
    a.wait_limit = di.wait_limit;
    if (up::launch_kv_compact(a, di.sms, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
        return UP_ERR_CUDA;
    return UP_OK;
}

up_status up_reserve_pages(const up_page_pool *pool, int32_t *block_table, int num_seqs,
                           int max_pages, int page_size, const int32_t *have, const int32_t *want,
                           up_stream_t stream) {
    const up::CallRange range("up_reserve_pages");
    up_status st = check_table(pool, num_seqs, max_pages, page_size);
    if (st != UP_OK) return st;
    if (num_seqs == 0) return UP_OK;
    if (!block_table || !have || !want || !aligned(block_table, 4) || !aligned(have, 4) || !aligned(want, 4))
        return UP_ERR_INVALID_ARG;
    up::DeviceInfo di{};
    if ((st = up::device_info(&di)) != UP_OK) return st;
    const up::PageTable t{block_table, num_seqs, max_pages, page_size};
    if (up::launch_reserve(pool_view(pool, di.err), t, have, want, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
        return UP_ERR_CUDA;
    return UP_OK;
}

up_status up_release_pages(const up_page_pool *pool, int32_t *block_table, int num_seqs,
                           int max_pages, int page_size, const int32_t *first, const int32_t *end,
                           up_stream_t stream) {
    const up::CallRange range("up_release_pages");
    up_status st = check_table(pool, num_seqs, max_pages, page_size);
    if (st != UP_OK) return st;
    if (num_seqs == 0) return UP_OK;
    if (!block_table || !end || !aligned(block_table, 4) || !aligned(first, 4) || !aligned(end, 4))
        return UP_ERR_INVALID_ARG;
    up::DeviceInfo di{};
    if ((st = up::device_info(&di)) != UP_OK) return st;
    const up::PageTable t{block_table, num_seqs, max_pages, page_size};
    if (up::launch_release(pool_view(pool, di.err), t, first, end, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
        return UP_ERR_CUDA;
    return UP_OK;
}

up_status up_fork_pages(const up_page_pool *pool, const int32_t *block_table,
                        const int32_t *kv_lens, int num_seqs, int max_pages, int page_size,
                        const int32_t *parents, int num_children, int32_t *table_out,
                        int32_t *lens_out, int32_t *copies, up_stream_t stream) {
    const up::CallRange range("up_fork_pages");
    up_status st = check_table(pool, num_seqs, max_pages, page_size);
    if (st != UP_OK) return st;
    if (num_children < 0 || (int64_t)num_children * max_pages > INT32_MAX || (int64_t)num_children * 3 > INT32_MAX)
        return UP_ERR_INVALID_ARG;
    if (num_children == 0) return UP_OK;
    if (num_seqs < 1 || !block_table || !kv_lens || !parents || !table_out || !lens_out || !copies)
        return UP_ERR_INVALID_ARG;
    if (!aligned(block_table, 4) || !aligned(kv_lens, 4) || !aligned(parents, 4) || !aligned(table_out, 4) ||
        !aligned(lens_out, 4) || !aligned(copies, 4))
        return UP_ERR_INVALID_ARG;
    // nothing is written over what other children, or other blocks, still read
    const struct { const int32_t *at; int64_t n; } all[6] = {
        {table_out, (int64_t)num_children * max_pages}, {lens_out, num_children}, {copies, (int64_t)num_children * 3},
        {block_table, (int64_t)num_seqs * max_pages},   {kv_lens, num_seqs},      {parents, num_children}};
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 6; ++j)
            if (overlap(all[i].at, all[i].n, all[j].at, all[j].n)) return UP_ERR_INVALID_ARG;
    up::DeviceInfo di{};
    if ((st = up::device_info(&di)) != UP_OK) return st;
    up::ForkArgs a{};
    a.pool = pool_view(pool, di.err);
    a.from = up::PageTable{const_cast<int32_t *>(block_table), num_seqs, max_pages, page_size};
    a.kv_lens = kv_lens;
    a.parents = parents;
    a.children = num_children;
    a.table = table_out;
    a.lens = lens_out;
    a.copies = copies;
    if (up::launch_fork(a, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) return UP_ERR_CUDA;
    return UP_OK;
}

up_status up_copy_pages(const up_paged_kv *cache, const int32_t *copies, int num_copies,
                        up_stream_t stream) {
    const up::CallRange range("up_copy_pages");
    up_status st = check_cache(cache, -1);
    if (st != UP_OK) return st;
    // (the kernel's indexes into copies are 32-bit)
    if (num_copies < 0 || (int64_t)num_copies * 3 > INT32_MAX) return UP_ERR_INVALID_ARG;
    if (num_copies == 0) return UP_OK;
    if (!copies || !aligned(copies, 4) || !cache->k_pages || !cache->v_pages || cache->num_pages < 1)
        return UP_ERR_INVALID_ARG;
    if (up::copy_blocks(device_view(cache, nullptr), num_copies) > INT32_MAX) return UP_ERR_INVALID_ARG;
    up::DeviceInfo di{};
    if ((st = up::device_info(&di)) != UP_OK) return st;
    const up::PagedKv kv = device_view(cache, di.err);
    if (up::launch_copy_pages(kv, copies, num_copies, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
        return UP_ERR_CUDA;
    return UP_OK;
}

}  // extern "C"
