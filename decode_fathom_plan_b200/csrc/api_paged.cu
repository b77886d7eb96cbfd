// C ABI of the calls on a paged cache: argument validation and the arguments
// of their launchers.  The operations are documented in include/fathom.h.
#include <math.h>

#include "common.cuh"
#include "internal.h"
#include "paged.cuh"

using namespace fathom;

namespace {

constexpr int kMaxHeads = 65535;      // also the y and z extent of a grid
constexpr int kMaxSequences = 65535;
constexpr int kMaxList = 1 << 28;     // listed keys of a query
// Keys of a sequence: numbers of keys are int, and run up to a block past the last one; so is the
// number of a block of 64 among those of all KV heads.
constexpr int kMaxLength = INT32_MAX - 65535;
bool length_ok(int max_len, int n_kv_heads)
{
    return max_len >= 1 && max_len <= kMaxLength && (max_len / 64 + 1ll) * n_kv_heads <= INT32_MAX;
}

fathom_status cuda_status(cudaError_t e) { return e == cudaSuccess ? FATHOM_OK : FATHOM_ERR_CUDA; }

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool dtype_ok(int dtype) { return dtype == FATHOM_F32 || dtype == FATHOM_BF16 || dtype == FATHOM_F16; }

int elem_size(int dtype) { return dtype == FATHOM_F32 ? 4 : 2; }

bool head_dim_ok(int d) { return d >= 32 && d <= kMaxHeadDim && d % 32 == 0; }

// No data is needed for no tokens (an empty tensor has none).
bool rows_ok(const fathom_rows *r, int n_tokens)
{
    return r && (r->data || n_tokens == 0) && r->n_heads >= 1 && r->n_heads <= kMaxHeads && dtype_ok(r->dtype) &&
           reinterpret_cast<uintptr_t>(r->data) % elem_size(r->dtype) == 0;
}

// Whether rows can be moved 16 bytes (8 elements, for float32 two times 4) at a time.
bool rows_vector(const fathom_rows *r)
{
    const int step = 16 / elem_size(r->dtype);
    return aligned16(r->data) && r->token_stride % step == 0 && r->head_stride % step == 0;
}

bool rotary_ok(const fathom_rotary *r, int head_dim)
{
    return r->turns && reinterpret_cast<uintptr_t>(r->turns) % 8 == 0 && r->rotary_dim >= 2 &&
           r->rotary_dim <= head_dim && r->rotary_dim % 2 == 0 &&
           (r->interleaved == 0 || r->interleaved == 1) && isfinite(r->magnitude);
}

// A stride over n > 1 rows that are read or written in words of up to `words` elements.
bool stride_ok(int64_t stride, int n, int words) { return n == 1 || (stride > 0 && stride % words == 0); }
// The rows of a cache are read in words of 32 bytes.
constexpr int kCacheWord = 16;

bool cache_ok(const fathom_kv_cache *c)
{
    return c && c->n_pages >= 1 && c->page_size >= 8 && c->page_size <= 1024 &&
           (c->page_size & (c->page_size - 1)) == 0 && c->n_kv_heads >= 1 &&
           c->n_kv_heads <= kMaxHeads && head_dim_ok(c->head_dim) &&
           (c->dtype == FATHOM_BF16 || c->dtype == FATHOM_F16) &&
           stride_ok(c->page_stride, c->n_pages, kCacheWord) &&
           stride_ok(c->head_stride, c->n_kv_heads, kCacheWord) &&
           stride_ok(c->token_stride, c->page_size, kCacheWord);
}

int log2_of(int x)
{
    int s = 0;
    while ((1 << s) < x) ++s;
    return s;
}

// A device-usable address of a cache array: the current device's or managed memory as is,
// pinned host memory through its device mapping where host_ok.
fathom_status resolve_cache(void *p, bool host_ok, void **out)
{
    if (!p || reinterpret_cast<uintptr_t>(p) % (2 * kCacheWord)) return FATHOM_ERR_INVALID_ARG;
    cudaPointerAttributes attr{};
    if (cudaPointerGetAttributes(&attr, p) != cudaSuccess) {
        cudaGetLastError();
        return FATHOM_ERR_INVALID_ARG;
    }
    int device = 0;
    if (attr.type == cudaMemoryTypeDevice && (cudaGetDevice(&device) != cudaSuccess || attr.device != device))
        return FATHOM_ERR_INVALID_ARG;
    if (attr.type == cudaMemoryTypeDevice || attr.type == cudaMemoryTypeManaged) {
        *out = p;
        return FATHOM_OK;
    }
    if (attr.type == cudaMemoryTypeHost && host_ok) {
        if (cudaHostGetDevicePointer(out, p, 0) == cudaSuccess && *out) return FATHOM_OK;
        cudaGetLastError();
    }
    return FATHOM_ERR_INVALID_ARG;
}

fathom_status paged_view(const fathom_kv_cache *c, bool host_ok, const int32_t *table,
                         int32_t table_stride, PagedView *v)
{
    void *k = nullptr, *val = nullptr;
    fathom_status st = resolve_cache(c->k, host_ok, &k);
    if (st != FATHOM_OK) return st;
    if ((st = resolve_cache(c->v, host_ok, &val)) != FATHOM_OK) return st;
    *v = PagedView{k, val, c->page_stride, c->head_stride, c->token_stride, c->n_pages,
                   log2_of(c->page_size), c->n_kv_heads, c->head_dim, c->dtype, table, table_stride};
    return FATHOM_OK;
}

void set_rotary(RowsArgs *a, const fathom_rotary *r)
{
    if (!r) return;
    a->turns = r->turns;
    a->magnitude = r->magnitude;
    a->rotary_dim = r->rotary_dim;
    a->interleaved = r->interleaved;
}

// Checks that the two attentions share; 0 heads per KV head where the rows do not fit.
int query_group(const fathom_kv_cache *c, const fathom_rows *q, const fathom_rows *out,
                int32_t n_seqs, float scale, float softcap)
{
    if (!rows_ok(q, n_seqs) || !rows_ok(out, n_seqs) || q->dtype != c->dtype || out->dtype != c->dtype) return 0;
    if (!aligned16(q->data) || !aligned16(out->data) || q->n_heads != out->n_heads) return 0;
    for (const fathom_rows *r : {q, out})
        if (!stride_ok(r->token_stride, n_seqs, 8) || !stride_ok(r->head_stride, r->n_heads, 8)) return 0;
    if (q->n_heads % c->n_kv_heads || q->n_heads / c->n_kv_heads > kMaxGroup) return 0;
    if (n_seqs < 1 || n_seqs > kMaxSequences || (long long)n_seqs * q->n_heads >= (1ll << 31)) return 0;
    if (!(softcap >= 0.0f && softcap <= kMaxSoftcap)) return 0;
    if (!isfinite(scale) || !isfinite(score_args(scale, softcap).scale)) return 0;
    return q->n_heads / c->n_kv_heads;
}

PagedQuery paged_query(const fathom_rows *q, const fathom_rows *out, const int32_t *seq_lens,
                       const float *slopes, float scale, float softcap, int n_seqs, int group)
{
    return PagedQuery{q->data, out->data, q->token_stride, q->head_stride, out->token_stride,
                      out->head_stride, seq_lens, slopes, scale, softcap, n_seqs, group};
}

}  // namespace

extern "C" {

fathom_status fathom_rotary_turns(double *turns, float *magnitude, int32_t rotary_dim, double base,
                                  int32_t scaling, double factor, int64_t original_len,
                                  double beta_fast, double beta_slow)
{
    if (!turns || !magnitude || rotary_dim < 2 || rotary_dim % 2 || !(base > 0.0) || !isfinite(base))
        return FATHOM_ERR_INVALID_ARG;
    if (scaling < FATHOM_ROTARY_PLAIN || scaling > FATHOM_ROTARY_YARN_INDEX) return FATHOM_ERR_INVALID_ARG;
    if (scaling != FATHOM_ROTARY_PLAIN && !(factor >= 1.0 && isfinite(factor)))
        return FATHOM_ERR_INVALID_ARG;
    if (scaling == FATHOM_ROTARY_NTK && rotary_dim < 4) return FATHOM_ERR_INVALID_ARG;
    const bool by_index = scaling == FATHOM_ROTARY_YARN_INDEX, yarn = by_index || scaling == FATHOM_ROTARY_YARN;
    if (by_index && !(base > 1.0 && beta_slow > 0.0)) return FATHOM_ERR_INVALID_ARG;
    if (yarn &&
        (original_len < 1 || !(beta_fast > beta_slow) || !isfinite(beta_fast) || !isfinite(beta_slow)))
        return FATHOM_ERR_INVALID_ARG;
    const double pi2 = 6.283185307179586476925286766559;
    if (scaling == FATHOM_ROTARY_NTK) base *= pow(factor, rotary_dim / (rotary_dim - 2.0));
    double low = 0.0, high = 0.0;             // pairs between which YARN_INDEX changes over
    if (by_index) {
        const auto pair = [&](double r) { return rotary_dim * log(original_len / (pi2 * r)) / (2.0 * log(base)); };
        low = fmax(floor(pair(beta_fast)), 0.0);
        high = fmin(ceil(pair(beta_slow)), rotary_dim - 1.0);
        if (high < low) return FATHOM_ERR_INVALID_ARG;
        if (low == high) high += 0.001;
    }
    for (int i = 0; i < rotary_dim / 2; ++i) {
        double turn = pow(base, -2.0 * i / rotary_dim) / pi2;
        if (scaling == FATHOM_ROTARY_LINEAR) turn /= factor;
        if (yarn) {
            const double r = (double)original_len * turn;
            const double at = by_index ? 1.0 - (i - low) / (high - low) : (r - beta_slow) / (beta_fast - beta_slow);
            const double g = fmin(1.0, fmax(0.0, at));
            turn = turn * g + turn / factor * (1.0 - g);
        }
        turns[i] = turn;
    }
    *magnitude = yarn ? (float)(0.1 * log(factor) + 1.0) : 1.0f;
    return FATHOM_OK;
}

fathom_status fathom_qk_norm_rope(int32_t n_tokens, int32_t head_dim, const int32_t *pos,
                                  const fathom_rotary *rotary, const void *q_weight,
                                  const void *k_weight, float eps, const fathom_rows *q,
                                  const fathom_rows *q_out, const fathom_rows *k,
                                  const fathom_rows *k_out, cudaStream_t stream)
{
    NvtxRange range("fathom_qk_norm_rope");
    if (n_tokens < 0 || !head_dim_ok(head_dim) || (!q && !k) || !q != !q_out || !k != !k_out)
        return FATHOM_ERR_INVALID_ARG;
    if (rotary && (!rotary_ok(rotary, head_dim) || (!pos && n_tokens))) return FATHOM_ERR_INVALID_ARG;
    if (!isfinite(eps) || eps < 0.0f) return FATHOM_ERR_INVALID_ARG;
    RowsArgs a{};
    a.pos = pos;
    a.eps = eps;
    a.n_tokens = n_tokens;
    a.head_dim = head_dim;
    set_rotary(&a, rotary);
    bool vector = a.rotary_dim % 16 == 0;
    int sets = 0, dtype = 0;
    const fathom_rows *in[2] = {q, k}, *out[2] = {q_out, k_out};
    const void *weight[2] = {q_weight, k_weight};
    for (int i = 0; i < 2; ++i) {
        if (!in[i]) {
            if (weight[i]) return FATHOM_ERR_INVALID_ARG;
            continue;
        }
        if (!rows_ok(in[i], n_tokens) || !rows_ok(out[i], n_tokens) || in[i]->n_heads != out[i]->n_heads)
            return FATHOM_ERR_INVALID_ARG;
        if (sets && in[i]->dtype != dtype) return FATHOM_ERR_INVALID_ARG;
        dtype = in[i]->dtype;
        vector = vector && rows_vector(in[i]) && rows_vector(out[i]) && aligned16(weight[i]);
        a.set[sets++] = RowSet{in[i]->data, out[i]->data, weight[i], in[i]->token_stride,
                               in[i]->head_stride, out[i]->token_stride, out[i]->head_stride,
                               in[i]->n_heads, out[i]->dtype, 1};
    }
    if (n_tokens == 0) return FATHOM_OK;
    return cuda_status(launch_rows(a, dtype, vector, stream));
}

fathom_status fathom_append_kv(const fathom_kv_cache *cache, int32_t n_tokens, const fathom_rows *k,
                               const fathom_rows *v, const int32_t *seq, const int32_t *pos,
                               const int32_t *page_table, int32_t n_seqs, int32_t table_stride,
                               const fathom_rotary *rotary, const void *k_weight, float eps,
                               cudaStream_t stream)
{
    NvtxRange range("fathom_append_kv");
    if (!cache_ok(cache) || n_tokens < 0 || !rows_ok(k, n_tokens) || !rows_ok(v, n_tokens))
        return FATHOM_ERR_INVALID_ARG;
    if (k->n_heads != cache->n_kv_heads || v->n_heads != cache->n_kv_heads || k->dtype != v->dtype)
        return FATHOM_ERR_INVALID_ARG;
    if (((!seq || !pos) && n_tokens) || !page_table || n_seqs < 1 || table_stride < 1) return FATHOM_ERR_INVALID_ARG;
    if (rotary && !rotary_ok(rotary, cache->head_dim)) return FATHOM_ERR_INVALID_ARG;
    if (!isfinite(eps) || eps < 0.0f) return FATHOM_ERR_INVALID_ARG;
    PagedView view{};
    const fathom_status st = paged_view(cache, true, page_table, table_stride, &view);
    if (st != FATHOM_OK) return st;
    if (n_tokens == 0) return FATHOM_OK;
    RowsArgs a{};
    a.set[0] = RowSet{k->data, const_cast<void *>(view.k), k_weight, k->token_stride, k->head_stride,
                      0, cache->head_stride, k->n_heads, cache->dtype, 1};
    a.set[1] = RowSet{v->data, const_cast<void *>(view.v), nullptr, v->token_stride, v->head_stride,
                      0, cache->head_stride, v->n_heads, cache->dtype, 0};
    a.pos = pos;
    a.eps = eps;
    a.n_tokens = n_tokens;
    a.head_dim = cache->head_dim;
    set_rotary(&a, rotary);
    a.paged = 1;
    a.seq = seq;
    a.table = page_table;
    a.n_seqs = n_seqs;
    a.table_stride = table_stride;
    a.n_pages = cache->n_pages;
    a.page_shift = view.page_shift;
    a.page_stride = cache->page_stride;
    a.slot_stride = cache->token_stride;
    const bool vector = a.rotary_dim % 16 == 0 && rows_vector(k) && rows_vector(v) && aligned16(k_weight);
    return cuda_status(launch_rows(a, k->dtype, vector, stream));
}

size_t fathom_paged_attention_workspace_bytes(const fathom_kv_cache *cache, int32_t n_seqs,
                                              int32_t group, int32_t max_len, int32_t prefix_len)
{
    if (!cache_ok(cache) || n_seqs < 1 || n_seqs > kMaxSequences || group < 1 || group > kMaxGroup ||
        !length_ok(max_len, cache->n_kv_heads) || prefix_len < 0 || prefix_len > max_len || prefix_len % cache->page_size)
        return 0;
    return paged_attention_most_bytes(cache->n_kv_heads, cache->head_dim, n_seqs, group, max_len, prefix_len);
}

fathom_status fathom_paged_attention(const fathom_kv_cache *cache, const fathom_rows *q,
                                     const int32_t *page_table, int32_t table_stride,
                                     const int32_t *seq_lens, int32_t n_seqs, int32_t max_len,
                                     int32_t prefix_len, float softmax_scale, float softcap,
                                     const float *slopes, const fathom_rows *out, void *workspace,
                                     size_t workspace_bytes, cudaStream_t stream)
{
    NvtxRange range("fathom_paged_attention");
    if (!cache_ok(cache) || !page_table || !seq_lens) return FATHOM_ERR_INVALID_ARG;
    const int group = query_group(cache, q, out, n_seqs, softmax_scale, softcap);
    if (!group || !length_ok(max_len, cache->n_kv_heads) || prefix_len < 0 || prefix_len > max_len ||
        prefix_len % cache->page_size || table_stride < 1 ||
        (long long)table_stride * cache->page_size < max_len)
        return FATHOM_ERR_INVALID_ARG;
    const size_t need = paged_attention_bytes(cache->n_kv_heads, cache->head_dim, n_seqs, group,
                                              max_len, prefix_len);
    if (need && (!workspace || !aligned16(workspace) || workspace_bytes < need))
        return FATHOM_ERR_WORKSPACE;
    PagedView view{};
    const fathom_status st = paged_view(cache, false, page_table, table_stride, &view);
    if (st != FATHOM_OK) return st;
    return cuda_status(launch_paged_attention(
        view, paged_query(q, out, seq_lens, slopes, softmax_scale, softcap, n_seqs, group), max_len,
        prefix_len, workspace, stream));
}

size_t fathom_sparse_attention_paged_workspace_bytes(int32_t n_seqs, int32_t n_heads,
                                                     int32_t head_dim, int32_t k)
{
    if (n_seqs < 1 || n_seqs > kMaxSequences || n_heads < 1 || n_heads > kMaxHeads || k < 1 ||
        k > kMaxList || !head_dim_ok(head_dim) || (long long)n_seqs * n_heads >= (1ll << 31))
        return 0;
    return paged_sparse_most_bytes(n_seqs * n_heads, head_dim, k);
}

fathom_status fathom_sparse_attention_paged(const fathom_kv_cache *cache, const fathom_rows *q,
                                            const int32_t *idx, int32_t k,
                                            const int32_t *page_table, int32_t table_stride,
                                            const int32_t *seq_lens, int32_t n_seqs,
                                            float softmax_scale, float softcap, const float *slopes,
                                            const fathom_rows *out, void *workspace,
                                            size_t workspace_bytes, cudaStream_t stream)
{
    NvtxRange range("fathom_sparse_attention_paged");
    if (!cache_ok(cache) || !page_table || !seq_lens || !idx || k < 1 || k > kMaxList || table_stride < 1)
        return FATHOM_ERR_INVALID_ARG;
    const int group = query_group(cache, q, out, n_seqs, softmax_scale, softcap);
    if (!group) return FATHOM_ERR_INVALID_ARG;
    const size_t need = paged_sparse_bytes(n_seqs * q->n_heads, cache->head_dim, k);
    if (need && (!workspace || !aligned16(workspace) || workspace_bytes < need))
        return FATHOM_ERR_WORKSPACE;
    PagedView view{};
    const fathom_status st = paged_view(cache, true, page_table, table_stride, &view);
    if (st != FATHOM_OK) return st;
    return cuda_status(launch_paged_sparse(
        view, paged_query(q, out, seq_lens, slopes, softmax_scale, softcap, n_seqs, group), idx, k,
        workspace, stream));
}

}  // extern "C"
