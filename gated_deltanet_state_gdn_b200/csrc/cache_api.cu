// cache_api.cu -- the C ABI of the paged key-value cache: host-side validation and dispatch.
//
// As in gdn_api.cu nothing reads tensor contents or synchronises: every check uses the scalars
// and pointer values the caller passes.
#include <string.h>

#include <algorithm>

#include "cache.cuh"
#include "host_checks.cuh"

using gdn::aligned;
using gdn::overlaps;

namespace {

constexpr int64_t kMostPositions = (int64_t)1 << 30;   // of a row: positions are 32-bit numbers

gdn_status done(cudaError_t e, const char *where)
{
    return e == cudaSuccess ? GDN_OK : gdn_report_cuda_failure(e, where);
}

int elem_size(int32_t dtype) { return dtype == GDN_E4M3 ? 1 : 2; }

// bytes from the first to past the last element of k (or v)
int64_t cache_bytes(const gdn_paged_cache &c)
{
    return ((c.num_pages - 1) * c.page_stride + (c.page_size - 1) * c.token_stride +
            (c.heads - 1) * c.head_stride + c.head_dim) * elem_size(c.dtype);
}

size_t table_bytes(int32_t rows, int64_t stride, int32_t width)
{
    return ((size_t)(rows - 1) * stride + width) * 4;
}

// no two vectors of the cache share an element: heads inside tokens or tokens inside heads,
// both inside pages (here and below, the stride of a dimension of one does not matter)
bool apart(const gdn_paged_cache &c)
{
    const int64_t D = c.head_dim, H = c.heads, S = c.page_size;
    const int64_t hs = H > 1 ? c.head_stride : 0, ts = S > 1 ? c.token_stride : 0;
    const bool heads_in = (H == 1 || hs >= D) && (S == 1 || ts >= (H - 1) * hs + D);
    const bool tokens_in = (S == 1 || ts >= D) && (H == 1 || hs >= (S - 1) * ts + D);
    return (heads_in || tokens_in) &&
           (c.num_pages == 1 || c.page_stride >= (H - 1) * hs + (S - 1) * ts + D);
}

// Whether two rows of bytes `delta` apart meet when either may be moved by whole numbers of steps: by
// less than dim[i].n of dim[i].step each, a step at least what the dimensions after it span.  The
// first row is of `a` bytes, the second of `b`.
struct Steps {
    int64_t n, step;
};
bool rows_meet(int64_t delta, int64_t a, int64_t b, const Steps *dim, int dims)
{
    if (dims == 0) return delta < a && -delta < b;
    // (what is left after the right number of steps is less than one)
    const int64_t near = dim->n > 1 ? delta / dim->step : 0;
    for (int64_t k = near - 1; k <= near + 1; ++k)
        if (-dim->n < k && k < dim->n &&
            rows_meet(delta - (dim->n > 1 ? k * dim->step : 0), a, b, dim + 1, dims - 1))
            return true;
    return false;
}

// a vector of k and one of v share an element; the vectors of either are apart
bool keys_meet_values(const gdn_paged_cache &c)
{
    const int64_t es = elem_size(c.dtype), row = c.head_dim * es;
    const Steps page = {c.num_pages, c.page_stride * es}, token = {c.page_size, c.token_stride * es},
                head = {c.heads, c.head_stride * es};
    const bool heads_in = c.heads == 1 || (c.page_size > 1 && c.head_stride < c.token_stride);
    const Steps dim[3] = {page, heads_in ? token : head, heads_in ? head : token};
    return rows_meet((int64_t)((uintptr_t)c.v - (uintptr_t)c.k), row, row, dim, 3);
}

gdn_status check_cache(const gdn_paged_cache *c)
{
    if (!c) return GDN_ERR_NULL;
    if (c->dtype != GDN_BF16 && c->dtype != GDN_F16 && c->dtype != GDN_E4M3) return GDN_ERR_DTYPE;
    if (c->rows < 1 || c->width < 1 || c->num_pages < 1 || c->page_size < 1 || c->heads < 1 ||
        c->head_dim < 1 || c->page_stride < 0 || c->token_stride < 0 || c->head_stride < 0 ||
        (c->rows > 1 && c->table_stride < c->width))
        return GDN_ERR_SHAPE;
    // (an expanded view: a box of a tensor map has no steps of zero)
    if ((c->num_pages > 1 && c->page_stride == 0) || (c->page_size > 1 && c->token_stride == 0) ||
        (c->heads > 1 && c->head_stride == 0))
        return GDN_ERR_SHAPE;
    const int es = elem_size(c->dtype);
    if (c->head_dim > 256 || c->head_dim * es % 16 != 0) return GDN_ERR_UNSUPPORTED;
    if ((int64_t)c->width * c->page_size > kMostPositions) return GDN_ERR_UNSUPPORTED;
    if (c->dtype != GDN_E4M3 && (c->k_scale || c->v_scale)) return GDN_ERR_DTYPE;
    if (!c->k || !c->v || !c->block_table || !c->seq_lens) return GDN_ERR_NULL;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || (c->num_pages > 1 && c->page_stride * es % 16) ||
        (c->page_size > 1 && c->token_stride * es % 16) || (c->heads > 1 && c->head_stride * es % 16) ||
        !aligned(c->block_table, 4) ||
        !aligned(c->seq_lens, 4) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
        return GDN_ERR_ALIGN;
    return GDN_OK;
}

gdn_status check_table(const gdn_page_table *t)
{
    if (!t) return GDN_ERR_NULL;
    if (t->rows < 1 || t->width < 1 || t->num_pages < 1 || t->page_size < 1 ||
        (t->rows > 1 && t->table_stride < t->width))
        return GDN_ERR_SHAPE;
    if ((int64_t)t->width * t->page_size > kMostPositions) return GDN_ERR_UNSUPPORTED;
    if (!t->block_table || !t->ref_count || !t->seq_lens) return GDN_ERR_NULL;
    if (!aligned(t->block_table, 4) || !aligned(t->ref_count, 4) || !aligned(t->seq_lens, 4))
        return GDN_ERR_ALIGN;
    const size_t tb = table_bytes(t->rows, t->table_stride, t->width), pb = (size_t)t->num_pages * 4,
                 sb = (size_t)t->rows * 4;
    if (overlaps(t->block_table, tb, t->ref_count, pb) || overlaps(t->block_table, tb, t->seq_lens, sb) ||
        overlaps(t->ref_count, pb, t->seq_lens, sb))
        return GDN_ERR_ALIAS;
    return GDN_OK;
}

// a buffer of the call against the table's three
bool meets_table(const gdn_page_table &t, const void *p, size_t bytes)
{
    return overlaps(p, bytes, t.block_table, table_bytes(t.rows, t.table_stride, t.width)) ||
           overlaps(p, bytes, t.ref_count, (size_t)t.num_pages * 4) ||
           overlaps(p, bytes, t.seq_lens, (size_t)t.rows * 4);
}

int64_t pool_span(const gdn_pool &p, int32_t rows) { return (int64_t)(rows - 1) * p.row_stride + p.row_bytes; }

// a row of p and one of q share a byte
bool pools_meet(const gdn_pool &p, const gdn_pool &q, int32_t rows)
{
    if (!overlaps(p.data, (size_t)pool_span(p, rows), q.data, (size_t)pool_span(q, rows))) return false;
    const int64_t delta = (int64_t)((uintptr_t)q.data - (uintptr_t)p.data);
    if (rows == 1 || p.row_stride == q.row_stride) {
        const Steps dim = {rows, p.row_stride};
        return rows_meet(delta, p.row_bytes, q.row_bytes, &dim, 1);
    }
    // rows of two spacings in one place: row by row, against the first of q's that ends past it
    for (int64_t i = 0; i < rows; ++i) {
        const int64_t at = i * p.row_stride - delta;        // of p's row, from q's first
        const int64_t k = at < q.row_bytes ? 0 : (at - q.row_bytes) / q.row_stride + 1;
        if (k < rows && k * q.row_stride < at + p.row_bytes && k * q.row_stride + q.row_bytes > at) return true;
    }
    return false;
}

// Whether two of the pools share bytes, which two blocks would copy at the same time.  Spans may
// interleave: keys and values of one tensor, its layers.  Up to kSorted pools are gone through in
// the order of their addresses: a pool past all before it, or beside the last one in rows of the
// same spacing, need not be compared with each.
bool any_pools_meet(const gdn_pool *pools, int32_t n, int32_t rows)
{
    constexpr int kSorted = 512;
    int order[kSorted];
    const bool sorted = n <= kSorted;
    if (sorted) {
        for (int i = 0; i < n; ++i) order[i] = i;
        std::sort(order, order + n,
                  [&](int i, int j) { return (uintptr_t)pools[i].data < (uintptr_t)pools[j].data; });
    }
    auto at = [&](int k) -> const gdn_pool & { return pools[sorted ? order[k] : k]; };
    auto end = [](const gdn_pool &p, int64_t bytes) { return (uintptr_t)p.data + (uintptr_t)bytes; };
    int first = 0;              // those from here on reach past one another's beginnings
    uintptr_t reach = 0;
    bool beside = true;         // all of them lie side by side, between two rows of the first
    for (int k = 0; k < n; ++k) {
        const gdn_pool &q = at(k);
        const uintptr_t q_end = end(q, pool_span(q, rows));
        if (sorted && (uintptr_t)q.data >= reach) {
            first = k;
            reach = q_end;
            beside = true;
            continue;
        }
        const gdn_pool &f = at(first);
        beside = beside && sorted && q.row_stride == f.row_stride &&
                 (uintptr_t)q.data >= end(at(k - 1), at(k - 1).row_bytes) &&
                 end(q, q.row_bytes) <= end(f, f.row_stride);
        for (int j = first; j < k && !beside; ++j)
            if (pools_meet(at(j), q, rows)) return true;
        reach = std::max(reach, q_end);
    }
    return false;
}

// Pools of `rows` rows.
gdn_status check_pools(const gdn_page_table &t, const gdn_pool *pools, int32_t n, int32_t rows)
{
    if (n < 0) return GDN_ERR_SHAPE;
    if (n > 0 && !pools) return GDN_ERR_NULL;
    for (int i = 0; i < n; ++i) {
        const gdn_pool &p = pools[i];
        if (p.row_bytes < 1 || (rows > 1 && p.row_stride < p.row_bytes)) return GDN_ERR_SHAPE;
        if (p.row_bytes >= (int64_t)1 << 36) return GDN_ERR_UNSUPPORTED;
        if (!p.data) return GDN_ERR_NULL;
        if (meets_table(t, p.data, (size_t)pool_span(p, rows))) return GDN_ERR_ALIAS;
    }
    return any_pools_meet(pools, n, rows) ? GDN_ERR_ALIAS : GDN_OK;
}

bool meets_pools(const gdn_pool *pools, int32_t n, int32_t rows, const void *p, size_t bytes)
{
    for (int i = 0; i < n; ++i)
        if (overlaps(p, bytes, pools[i].data, (size_t)pool_span(pools[i], rows))) return true;
    return false;
}

}  // namespace

extern "C" {

gdn_status gdn_kv_append(const void *k, const void *v, int64_t k_token_stride,
                         int64_t k_head_stride, int64_t v_token_stride, int64_t v_head_stride,
                         const gdn_paged_cache *cache, const int32_t *slots,
                         const int32_t *row_offsets, int32_t B, int64_t N, gdn_dtype dtype,
                         int32_t *dev_status, void *stream)
{
    if (dtype != GDN_BF16 && dtype != GDN_F16) return GDN_ERR_DTYPE;
    const gdn_status st = check_cache(cache);
    if (st != GDN_OK) return st;
    if (cache->dtype != GDN_E4M3 && cache->dtype != (int32_t)dtype) return GDN_ERR_DTYPE;
    if (!apart(*cache)) return GDN_ERR_SHAPE;
    if (keys_meet_values(*cache)) return GDN_ERR_ALIAS;
    if (B < 0 || N < 0 || k_token_stride < 0 || k_head_stride < 0 || v_token_stride < 0 ||
        v_head_stride < 0)
        return GDN_ERR_SHAPE;
    if (B == 0) return N == 0 ? GDN_OK : GDN_ERR_SHAPE;
    if (!row_offsets && N % B != 0) return GDN_ERR_SHAPE;
    if (!slots && B > cache->rows) return GDN_ERR_SHAPE;
    if (N > ((int64_t)1 << 31) - 1) return GDN_ERR_UNSUPPORTED;
    if (N == 0) return GDN_OK;
    if (!k || !v) return GDN_ERR_NULL;
    if (!aligned(k, 16) || !aligned(v, 16) ||
        (N > 1 && (k_token_stride % 8 || v_token_stride % 8)) ||
        (cache->heads > 1 && (k_head_stride % 8 || v_head_stride % 8)) || !aligned(slots, 4) ||
        !aligned(row_offsets, 4))
        return GDN_ERR_ALIGN;
    const size_t cb = (size_t)cache_bytes(*cache);
    const size_t kb = (size_t)((N - 1) * k_token_stride + (cache->heads - 1) * k_head_stride + cache->head_dim) * 2;
    const size_t vb = (size_t)((N - 1) * v_token_stride + (cache->heads - 1) * v_head_stride + cache->head_dim) * 2;
    for (const void *c : {(const void *)cache->k, (const void *)cache->v})
        if (overlaps(c, cb, k, kb) || overlaps(c, cb, v, vb) ||
            overlaps(c, cb, cache->block_table, table_bytes(cache->rows, cache->table_stride, cache->width)) ||
            overlaps(c, cb, cache->seq_lens, (size_t)cache->rows * 4) ||
            overlaps(c, cb, slots, (size_t)B * 4) || overlaps(c, cb, row_offsets, (size_t)(B + 1) * 4) ||
            overlaps(c, cb, cache->k_scale, (size_t)cache->heads * 4) ||
            overlaps(c, cb, cache->v_scale, (size_t)cache->heads * 4))
            return GDN_ERR_ALIAS;

    GdnAppendArgs a;
    a.k = k; a.v = v;
    a.k_token_stride = k_token_stride; a.k_head_stride = k_head_stride;
    a.v_token_stride = v_token_stride; a.v_head_stride = v_head_stride;
    a.cache = *cache; a.slots = slots; a.row_offsets = row_offsets; a.B = B; a.N = N;
    a.bf16 = dtype == GDN_BF16; a.dev_status = dev_status;
    return done(launch_kv_append(a, (cudaStream_t)stream), "gdn_kv_append launch");
}

uint64_t gdn_paged_attn_workspace_size(int32_t B, int32_t T, int32_t Hq, int32_t heads,
                                       int32_t head_dim, gdn_dtype cache_dtype)
{
    if (B < 1 || T < 1 || T > 16 || Hq < 1 || heads < 1 || Hq % heads != 0 || head_dim < 1 ||
        head_dim > 256)
        return 0;
    return paged_attn_workspace_bytes(B, T, Hq, heads, head_dim, (int32_t)cache_dtype);
}

gdn_status gdn_paged_attn(const void *q, int64_t q_token_stride, int64_t q_head_stride,
                          const gdn_paged_cache *cache, const int32_t *slots, int32_t B, int32_t T,
                          int32_t Hq, gdn_dtype dtype, float scale, int32_t window, void *out,
                          float *lse, uint32_t flags, void *workspace, uint64_t workspace_bytes,
                          int32_t *dev_status, void *stream)
{
    if (dtype != GDN_BF16 && dtype != GDN_F16) return GDN_ERR_DTYPE;
    if (flags & ~(uint32_t)GDN_ZERO_PADDING) return GDN_ERR_UNSUPPORTED;
    const gdn_status st = check_cache(cache);
    if (st != GDN_OK) return st;
    if (cache->dtype != GDN_E4M3 && cache->dtype != (int32_t)dtype) return GDN_ERR_DTYPE;
    if (B < 0 || T < 1 || Hq < 1 || Hq % cache->heads != 0 || window < 0 || q_token_stride < 0 ||
        q_head_stride < 0)
        return GDN_ERR_SHAPE;
    if (T > 16 || Hq > 65536) return GDN_ERR_UNSUPPORTED;
    if (B == 0) return GDN_OK;
    if (!slots && B > cache->rows) return GDN_ERR_SHAPE;
    if (!q || !out || !workspace) return GDN_ERR_NULL;
    if (!aligned(q, 4) || !aligned(out, 4) || ((int64_t)B * T > 1 && q_token_stride % 2) ||
        (Hq > 1 && q_head_stride % 2) ||
        !aligned(lse, 4) || !aligned(slots, 4) || !aligned(workspace, 16))
        return GDN_ERR_ALIGN;
    const uint64_t need = paged_attn_workspace_bytes(B, T, Hq, cache->heads, cache->head_dim, cache->dtype);
    if (workspace_bytes < need) return GDN_ERR_SHAPE;
    const size_t rows = (size_t)B * T * Hq, ob = rows * cache->head_dim * 2, lb = rows * 4;
    const size_t qb = (size_t)(((int64_t)B * T - 1) * q_token_stride + (Hq - 1) * q_head_stride + cache->head_dim) * 2;
    const size_t cb = (size_t)cache_bytes(*cache);
    const size_t tb = table_bytes(cache->rows, cache->table_stride, cache->width);
    struct { const void *p; size_t n; } written[3] = {{out, ob}, {lse, lb}, {workspace, (size_t)need}};
    for (int i = 0; i < 3; ++i) {
        const void *p = written[i].p;
        const size_t n = written[i].n;
        if (overlaps(p, n, q, qb) || overlaps(p, n, cache->k, cb) || overlaps(p, n, cache->v, cb) ||
            overlaps(p, n, cache->block_table, tb) || overlaps(p, n, cache->seq_lens, (size_t)cache->rows * 4) ||
            overlaps(p, n, slots, (size_t)B * 4) || overlaps(p, n, cache->k_scale, (size_t)cache->heads * 4) ||
            overlaps(p, n, cache->v_scale, (size_t)cache->heads * 4))
            return GDN_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlaps(p, n, written[j].p, written[j].n)) return GDN_ERR_ALIAS;
    }

    GdnAttnArgs a;
    a.q = q; a.q_token_stride = q_token_stride; a.q_head_stride = q_head_stride;
    a.cache = *cache; a.slots = slots; a.B = B; a.T = T; a.Hq = Hq; a.q_bf16 = dtype == GDN_BF16;
    a.scale = scale; a.window = window; a.out = out; a.lse = lse;
    a.zero_padding = (flags & GDN_ZERO_PADDING) ? 1 : 0;
    a.workspace = workspace; a.workspace_bytes = workspace_bytes; a.dev_status = dev_status;
    return done(launch_paged_attn(a, (cudaStream_t)stream), "gdn_paged_attn launch");
}

uint64_t gdn_page_workspace_size(int32_t num_pages, int32_t n)
{
    return num_pages < 1 || n < 0 ? 0 : page_workspace_bytes(num_pages, n);
}

gdn_status gdn_page_resize(const gdn_page_table *table, const int32_t *row_list,
                           const int32_t *new_lens, int32_t n, const gdn_pool *pools,
                           int32_t n_pools, void *workspace, uint64_t workspace_bytes,
                           int32_t *dev_status, void *stream)
{
    gdn_status st = check_table(table);
    if (st != GDN_OK) return st;
    if (n < 0) return GDN_ERR_SHAPE;
    st = check_pools(*table, pools, n_pools, table->num_pages);
    if (st != GDN_OK) return st;
    if (n == 0) return GDN_OK;
    if (!row_list || !new_lens || !workspace) return GDN_ERR_NULL;
    if (!aligned(row_list, 4) || !aligned(new_lens, 4) || !aligned(workspace, 16)) return GDN_ERR_ALIGN;
    const uint64_t need = page_workspace_bytes(table->num_pages, n);
    if (workspace_bytes < need) return GDN_ERR_SHAPE;
    const size_t nb = (size_t)n * 4;
    if (meets_table(*table, row_list, nb) || meets_table(*table, new_lens, nb) ||
        meets_table(*table, workspace, (size_t)need) || overlaps(workspace, (size_t)need, row_list, nb) ||
        overlaps(workspace, (size_t)need, new_lens, nb) ||
        meets_pools(pools, n_pools, table->num_pages, workspace, (size_t)need) ||
        meets_pools(pools, n_pools, table->num_pages, row_list, nb) ||
        meets_pools(pools, n_pools, table->num_pages, new_lens, nb))
        return GDN_ERR_ALIAS;
    return done(launch_page_resize(*table, row_list, new_lens, n, pools, n_pools, workspace,
                                   dev_status, (cudaStream_t)stream), "gdn_page_resize launch");
}

gdn_status gdn_page_fork(const gdn_page_table *table, const int32_t *parents,
                         const int32_t *children, int32_t n, const gdn_pool *pools,
                         int32_t n_pools, int32_t *dev_status, void *stream)
{
    gdn_status st = check_table(table);
    if (st != GDN_OK) return st;
    if (n < 0) return GDN_ERR_SHAPE;
    st = check_pools(*table, pools, n_pools, table->rows);
    if (st != GDN_OK) return st;
    if (n == 0) return GDN_OK;
    if (!parents || !children) return GDN_ERR_NULL;
    if (!aligned(parents, 4) || !aligned(children, 4)) return GDN_ERR_ALIGN;
    const size_t nb = (size_t)n * 4;
    if (meets_table(*table, parents, nb) || meets_table(*table, children, nb) ||
        meets_pools(pools, n_pools, table->rows, parents, nb) ||
        meets_pools(pools, n_pools, table->rows, children, nb))
        return GDN_ERR_ALIAS;
    return done(launch_page_fork(*table, parents, children, n, pools, n_pools, dev_status,
                                 (cudaStream_t)stream), "gdn_page_fork launch");
}

gdn_status gdn_page_compact(const gdn_page_table *table, int32_t *page_map, const gdn_pool *pools,
                            int32_t n_pools, void *workspace, uint64_t workspace_bytes,
                            int32_t *dev_status, void *stream)
{
    gdn_status st = check_table(table);
    if (st != GDN_OK) return st;
    st = check_pools(*table, pools, n_pools, table->num_pages);
    if (st != GDN_OK) return st;
    if (!page_map || !workspace) return GDN_ERR_NULL;
    if (!aligned(page_map, 4) || !aligned(workspace, 16)) return GDN_ERR_ALIGN;
    const uint64_t need = page_workspace_bytes(table->num_pages, 0);
    if (workspace_bytes < need) return GDN_ERR_SHAPE;
    const size_t mb = (size_t)table->num_pages * 4;
    if (meets_table(*table, page_map, mb) || meets_table(*table, workspace, (size_t)need) ||
        overlaps(workspace, (size_t)need, page_map, mb) ||
        meets_pools(pools, n_pools, table->num_pages, workspace, (size_t)need) ||
        meets_pools(pools, n_pools, table->num_pages, page_map, mb))
        return GDN_ERR_ALIAS;
    return done(launch_page_compact(*table, page_map, pools, n_pools, workspace, dev_status,
                                    (cudaStream_t)stream), "gdn_page_compact launch");
}

}  // extern "C"
