// kv4_api.cu -- the C ABI of the paged 4-bit cache (include/dkv.h, dkv_kv4_*):
// argument validation and the launches.
#include <cstdint>
#include <cstring>

#include "../../include/dkv.h"
#include "dkv_internal.h"
#include "kv4_common.cuh"
#include "kv4_internal.h"

namespace {

using dkv::kv4::Query;
using dkv::kv4::View;

inline bool aligned(const void *p, uintptr_t a) {
    return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}
inline bool valid_dtype(int32_t t) { return t == DKV_F32 || t == DKV_F16 || t == DKV_BF16; }
inline dkv_status cuda_status(cudaError_t e) { return e == cudaSuccess ? DKV_OK : DKV_ECUDA; }
inline bool valid_scale(float s) { return s > 0.f && s < 1e30f; }   // finite, > 0

constexpr int32_t kMaxQueries = 16;
constexpr int64_t kMaxPositions = (int64_t)1 << 30;
constexpr int64_t kMaxRows = (int64_t)1 << 33;       // rows x kv heads: grids stay in range
constexpr int32_t kMaxTokens = INT32_MAX - 1023;     // a row's number and a warp's share, summed
constexpr int64_t kMaxQueryRows = (int64_t)1 << 30;  // prompt: rows x query heads
constexpr int64_t kMaxRuns = (int64_t)1 << 24;       // decode: batch x kv heads x head groups

int64_t decode_runs(int32_t batch, int32_t H, int32_t Hq, int32_t nq) {
    return (int64_t)batch * H * (((int64_t)nq * (Hq / H) + 7) / 8);
}

dkv_status check_desc(const dkv_kv4_desc *d) {
    if (!d) return DKV_EINVAL;
    if (d->n_kv_heads < 1 || d->n_kv_heads > 4096) return DKV_EINVAL;
    if (d->page_size < 16 || d->page_size > 65536 || d->page_size % 16 != 0) return DKV_EINVAL;
    if (d->head_dim != 64 && d->head_dim != 128) return DKV_EUNSUPPORTED;
    if (d->group != 32 && d->group != 64) return DKV_EUNSUPPORTED;
    return DKV_OK;
}

size_t page_bytes_of(const dkv_kv4_desc *d) {
    return (size_t)d->n_kv_heads * (size_t)(d->page_size / dkv::kv4::RT) *
           (size_t)dkv::kv4::rec_bytes(d->head_dim, d->group);
}

dkv_status check_pool(const dkv_kv4_pool *p) {
    if (!p || !p->base || !p->status) return DKV_EINVAL;
    const dkv_status s = check_desc(&p->desc);
    if (s != DKV_OK) return s;
    if (p->n_pages < 1 || p->n_pages > INT32_MAX || p->page_bytes != page_bytes_of(&p->desc))
        return DKV_EINVAL;
    if (!aligned(p->base, 256) || !aligned(p->status, 4)) return DKV_EALIGN;
    return DKV_OK;
}

dkv_status check_geometry(const dkv_kv4_desc *d, int32_t batch, int32_t max_pages) {
    if (batch < 1 || batch > 16384 || max_pages < 1) return DKV_EINVAL;
    if ((int64_t)max_pages * d->page_size > kMaxPositions) return DKV_ECAPACITY;
    return DKV_OK;
}

// The checks and the view of one call.
dkv_status make_view(const dkv_kv4_pool *p, const dkv_kv4_batch *b, int32_t n_rows, bool ragged,
                     View *v) {
    dkv_status s = check_pool(p);
    if (s != DKV_OK) return s;
    if (!b || !b->block_table || !b->seq_lens || n_rows < 1) return DKV_EINVAL;
    s = check_geometry(&p->desc, b->batch, b->max_pages);
    if (s != DKV_OK) return s;
    const int32_t *starts = ragged ? b->starts : nullptr;
    if (!starts && n_rows % b->batch != 0) return DKV_EINVAL;
    if (n_rows > kMaxTokens || (int64_t)n_rows * p->desc.n_kv_heads > kMaxRows)
        return DKV_ECAPACITY;
    if (!aligned(b->block_table, 4) || !aligned(b->seq_lens, 4) || !aligned(starts, 4))
        return DKV_EALIGN;
    v->pool = static_cast<uint8_t *>(p->base);
    v->n_pages = p->n_pages;
    v->page_bytes = (int64_t)p->page_bytes;
    v->status = p->status;
    v->H = p->desc.n_kv_heads;
    v->page_size = p->desc.page_size;
    v->rpp = p->desc.page_size / dkv::kv4::RT;
    v->table = b->block_table;
    v->lens = b->seq_lens;
    v->starts = starts;
    v->B = b->batch;
    v->max_pages = b->max_pages;
    v->n_rows = n_rows;
    v->n_uniform = starts ? 0 : n_rows / b->batch;
    return DKV_OK;
}

// Strided rows [n_rows][heads][D]: base and strides in whole 16-byte pieces.
dkv_status check_rows(const void *p, int32_t dtype, int64_t row, int64_t head) {
    const int64_t size = dtype == DKV_F32 ? 4 : 2;
    if (row < 0 || head < 0) return DKV_EINVAL;
    if (!aligned(p, 16) || row * size % 16 != 0 || head * size % 16 != 0) return DKV_EALIGN;
    return DKV_OK;
}

dkv_status check_query(const View &v, const void *Q, int32_t q_dtype, int32_t Hq, int64_t row,
                       int64_t head, float scale, int32_t window, const void *out,
                       const float *lse, const void *ws, Query *q) {
    if (!Q || !out || !ws || !valid_dtype(q_dtype) || !valid_scale(scale) || window < 0)
        return DKV_EINVAL;
    if (Hq < 1 || Hq % v.H != 0) return DKV_EINVAL;
    if (q_dtype == DKV_F32) return DKV_EUNSUPPORTED;
    const dkv_status s = check_rows(Q, q_dtype, row, head);
    if (s != DKV_OK) return s;
    if (!aligned(out, 16) || !aligned(lse, 4) || !aligned(ws, 16)) return DKV_EALIGN;
    // a window past every position is none (and sums with it stay in 32 bits)
    *q = Query{Q, const_cast<void *>(out), const_cast<float *>(lse), row, head, q_dtype, Hq,
               window > kMaxPositions ? 0 : window, scale};
    return DKV_OK;
}

}  // namespace

extern "C" {

size_t dkv_kv4_page_bytes(const dkv_kv4_desc *desc) {
    return check_desc(desc) == DKV_OK ? page_bytes_of(desc) : 0;
}

dkv_status dkv_kv4_init(const dkv_kv4_desc *desc, void *pool, int64_t n_pages, int32_t *status,
                        dkv_kv4_pool *out, void *stream) {
    dkv_status s = check_desc(desc);
    if (s != DKV_OK) return s;
    if (!out) return DKV_EINVAL;
    dkv_kv4_pool p;
    std::memset(&p, 0, sizeof(p));
    p.desc = *desc;
    p.base = pool;
    p.n_pages = n_pages;
    p.page_bytes = page_bytes_of(desc);
    p.status = status;
    s = check_pool(&p);
    if (s != DKV_OK) return s;
    *out = p;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaMemsetAsync(pool, 0, (size_t)n_pages * p.page_bytes, st);
    if (e == cudaSuccess) e = cudaMemsetAsync(status, 0, sizeof(int32_t), st);
    return cuda_status(e);
}

dkv_status dkv_kv4_get_device_status(const dkv_kv4_pool *pool, int32_t *host_out, void *stream) {
    const dkv_status s = check_pool(pool);
    if (s != DKV_OK) return s;
    if (!host_out) return DKV_EINVAL;
    if (dkv::take_status(pool->status, host_out, static_cast<cudaStream_t>(stream)) != cudaSuccess)
        return DKV_ECUDA;
    return *host_out ? DKV_EDEVICE : DKV_OK;
}

dkv_status dkv_kv4_append(const dkv_kv4_pool *pool, const dkv_kv4_batch *seqs, const void *K,
                          const void *V, int32_t dtype, int32_t n_rows, int64_t k_row_stride,
                          int64_t k_head_stride, int64_t v_row_stride, int64_t v_head_stride,
                          void *stream) {
    View v;
    dkv_status s = make_view(pool, seqs, n_rows, true, &v);
    if (s != DKV_OK) return s;
    if (!K || !V || !valid_dtype(dtype)) return DKV_EINVAL;
    s = check_rows(K, dtype, k_row_stride, k_head_stride);
    if (s == DKV_OK) s = check_rows(V, dtype, v_row_stride, v_head_stride);
    if (s != DKV_OK) return s;
    return cuda_status(dkv::kv4::launch_append(v, pool->desc.head_dim, pool->desc.group, K, V,
                                               dtype, k_row_stride, k_head_stride, v_row_stride,
                                               v_head_stride, static_cast<cudaStream_t>(stream)));
}

dkv_status dkv_kv4_read(const dkv_kv4_pool *pool, const dkv_kv4_batch *seqs, void *K_out,
                        void *V_out, int32_t dtype, int32_t n_rows, void *stream) {
    View v;
    const dkv_status s = make_view(pool, seqs, n_rows, true, &v);
    if (s != DKV_OK) return s;
    if (!K_out || !V_out || !valid_dtype(dtype)) return DKV_EINVAL;
    if (!aligned(K_out, 16) || !aligned(V_out, 16)) return DKV_EALIGN;
    return cuda_status(dkv::kv4::launch_read(v, pool->desc.head_dim, pool->desc.group, K_out,
                                             V_out, dtype, static_cast<cudaStream_t>(stream)));
}

size_t dkv_kv4_decode_workspace_bytes(const dkv_kv4_desc *desc, int32_t batch, int32_t max_pages,
                                      int32_t n_q_heads, int32_t n_queries) {
    if (check_desc(desc) != DKV_OK || check_geometry(desc, batch, max_pages) != DKV_OK) return 0;
    if (n_q_heads < 1 || n_q_heads % desc->n_kv_heads != 0 || n_queries < 1 ||
        n_queries > kMaxQueries ||
        decode_runs(batch, desc->n_kv_heads, n_q_heads, n_queries) > kMaxRuns)
        return 0;
    View v;
    std::memset(&v, 0, sizeof(v));
    v.H = desc->n_kv_heads;
    v.page_size = desc->page_size;
    v.B = batch;
    v.max_pages = max_pages;
    int64_t f = 0;
    if (dkv::kv4::decode_workspace_floats(v, desc->head_dim, n_q_heads, n_queries, &f) !=
        cudaSuccess)
        return 0;
    return (size_t)f * sizeof(float);
}

dkv_status dkv_kv4_decode_attn(const dkv_kv4_pool *pool, const dkv_kv4_batch *seqs, const void *Q,
                               int32_t q_dtype, int32_t n_q_heads, int32_t n_queries,
                               int64_t q_row_stride, int64_t q_head_stride, float softmax_scale,
                               int32_t window, void *out, float *lse, void *workspace,
                               size_t ws_bytes, void *stream) {
    if (n_queries < 1 || n_queries > kMaxQueries) return DKV_EINVAL;
    View v;
    const int32_t batch = seqs ? seqs->batch : 0;
    if (batch < 1 || batch > 16384) return DKV_EINVAL;
    dkv_status s = make_view(pool, seqs, batch * n_queries, false, &v);
    if (s != DKV_OK) return s;
    Query q;
    s = check_query(v, Q, q_dtype, n_q_heads, q_row_stride, q_head_stride, softmax_scale, window,
                    out, lse, workspace, &q);
    if (s != DKV_OK) return s;
    if (decode_runs(batch, v.H, n_q_heads, n_queries) > kMaxRuns) return DKV_ECAPACITY;
    int64_t need = 0;
    if (dkv::kv4::decode_workspace_floats(v, pool->desc.head_dim, n_q_heads, n_queries, &need) !=
        cudaSuccess)
        return DKV_ECUDA;
    if (ws_bytes < (size_t)need * sizeof(float)) return DKV_ECAPACITY;
    return cuda_status(dkv::kv4::launch_decode(v, pool->desc.head_dim, pool->desc.group, q,
                                               n_queries, static_cast<float *>(workspace), need,
                                               dkv::debug_fault(),
                                               static_cast<cudaStream_t>(stream)));
}

size_t dkv_kv4_prompt_workspace_bytes(const dkv_kv4_desc *desc, int32_t batch, int32_t max_pages,
                                      int32_t n_q_heads, int32_t n_rows, int32_t ragged) {
    if (check_desc(desc) != DKV_OK || check_geometry(desc, batch, max_pages) != DKV_OK) return 0;
    if (n_q_heads < 1 || n_q_heads % desc->n_kv_heads != 0 || n_rows < 1 ||
        (int64_t)n_rows * n_q_heads > kMaxQueryRows || (!ragged && n_rows % batch != 0))
        return 0;
    View v;
    std::memset(&v, 0, sizeof(v));
    v.H = desc->n_kv_heads;
    v.page_size = desc->page_size;
    v.B = batch;
    v.max_pages = max_pages;
    v.n_rows = n_rows;
    int64_t f = 0;
    if (dkv::kv4::prompt_workspace_floats(v, desc->head_dim, n_q_heads, &f) !=
        cudaSuccess)
        return 0;
    return (size_t)f * sizeof(float);
}

dkv_status dkv_kv4_prompt_attn(const dkv_kv4_pool *pool, const dkv_kv4_batch *seqs, const void *Q,
                               int32_t q_dtype, int32_t n_q_heads, int32_t n_rows,
                               int64_t q_row_stride, int64_t q_head_stride, float softmax_scale,
                               int32_t window, void *out, float *lse, void *workspace,
                               size_t ws_bytes, void *stream) {
    View v;
    dkv_status s = make_view(pool, seqs, n_rows, true, &v);
    if (s != DKV_OK) return s;
    Query q;
    s = check_query(v, Q, q_dtype, n_q_heads, q_row_stride, q_head_stride, softmax_scale, window,
                    out, lse, workspace, &q);
    if (s != DKV_OK) return s;
    if ((int64_t)n_rows * n_q_heads > kMaxQueryRows) return DKV_ECAPACITY;
    int64_t need = 0;
    if (dkv::kv4::prompt_workspace_floats(v, pool->desc.head_dim, n_q_heads, &need) != cudaSuccess)
        return DKV_ECUDA;
    if (ws_bytes < (size_t)need * sizeof(float)) return DKV_ECAPACITY;
    return cuda_status(dkv::kv4::launch_prompt(v, pool->desc.head_dim, pool->desc.group, q,
                                               static_cast<float *>(workspace), need,
                                               static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
