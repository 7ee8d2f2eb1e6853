// libtcq C ABI of the paged cache and the attention over it: argument checks and workspace
// sizes.  The numeric steps run in kernels_cache.hip and kernels_attention.hip.
#include <cmath>

#include "tcq.h"
#include "abi_checks.h"
#include "region.h"
#include "tcq_internal.h"

using namespace tcq;

namespace {

constexpr int kMostHeads = 1024, kMostPage = 4096;
constexpr int64_t kMostSeqs = 1 << 20;

int check_cache(const char *fn, const tcq_cache *c, CacheShape &out) {
    if (!c) {
        set_error("%s: cache is NULL", fn);
        return TCQ_EINVAL;
    }
    const int rc = check_format(fn, c->format);
    if (rc != TCQ_OK) return rc;
    if (c->pages < 0 || c->heads <= 0 || c->page <= 0) {
        set_error("%s: sizes of the cache (pages=%lld heads=%d page=%d) must be positive", fn,
                  (long long)c->pages, c->heads, c->page);
        return TCQ_EINVAL;
    }
    if (c->page & (c->page - 1)) {
        set_error("%s: page=%d is no power of two", fn, c->page);
        return TCQ_EINVAL;
    }
    if ((c->dim != 64 && c->dim != 128 && c->dim != 256) || c->heads > kMostHeads ||
        c->page > kMostPage || c->pages > INT32_MAX) {
        set_error("%s: outside the cache's limits (dim 64, 128 or 256, heads <= %d, page <= %d, "
                  "pages < 2^31): pages=%lld heads=%d page=%d dim=%d",
                  fn, kMostHeads, kMostPage, (long long)c->pages, c->heads, c->page, c->dim);
        return TCQ_EUNSUPPORTED;
    }
    if (c->pages > 0) {
        const void *p[4] = {c->k_codes, c->k_scale, c->v_codes, c->v_scale};
        for (int i = 0; i < 4; ++i) {
            if (!p[i]) {
                set_error("%s: the cache's codes and scale bytes must be non-NULL", fn);
                return TCQ_EINVAL;
            }
            if (i % 2 == 0 && reinterpret_cast<uintptr_t>(p[i]) % 16) {
                set_error("%s: the cache's codes at %p are not aligned to 16 bytes", fn, p[i]);
                return TCQ_EINVAL;
            }
        }
    }
    int log2 = 0;
    while ((1 << log2) < c->page) ++log2;
    out = CacheShape{c->k_codes, c->k_scale, c->v_codes, c->v_scale, c->pages, c->heads, log2,
                     c->dim, c->format};
    return TCQ_OK;
}

int check_batch(const char *fn, const tcq_cache_batch *b, int64_t rows, CacheBatch &out) {
    if (!b) {
        set_error("%s: batch is NULL", fn);
        return TCQ_EINVAL;
    }
    if (b->seqs < 0 || b->width < 0 || rows < 0) {
        set_error("%s: negative size (seqs=%lld width=%lld rows=%lld)", fn, (long long)b->seqs,
                  (long long)b->width, (long long)rows);
        return TCQ_EINVAL;
    }
    if (b->seqs > kMostSeqs || b->width > INT32_MAX || rows > TCQ_LINEAR_MAX_BATCH) {
        set_error("%s: outside the limits (seqs <= %lld, width < 2^31, rows <= %d): seqs=%lld "
                  "width=%lld rows=%lld",
                  fn, (long long)kMostSeqs, TCQ_LINEAR_MAX_BATCH, (long long)b->seqs,
                  (long long)b->width, (long long)rows);
        return TCQ_EUNSUPPORTED;
    }
    if (b->seqs > 0 && (!b->lens || !b->starts || (!b->table && b->width > 0))) {
        set_error("%s: table, lens and starts must be non-NULL", fn);
        return TCQ_EINVAL;
    }
    if (b->seqs > 1 && b->ldt < b->width) {
        set_error("%s: leading dimension %lld of table is below its width %lld", fn,
                  (long long)b->ldt, (long long)b->width);
        return TCQ_EINVAL;
    }
    for (const void *p : {static_cast<const void *>(b->table), static_cast<const void *>(b->lens),
                          static_cast<const void *>(b->starts)})
        if (reinterpret_cast<uintptr_t>(p) % 4) {
            set_error("%s: table, lens and starts must be aligned to 4 bytes (%p)", fn, p);
            return TCQ_EINVAL;
        }
    out = CacheBatch{b->table, b->ldt, b->width, b->lens, b->starts, b->seqs};
    return TCQ_OK;
}

// rows x heads vectors of dim values.
int check_rows(const char *fn, const char *name, const void *p, int64_t row, int64_t head,
               int64_t heads, int64_t dim, size_t size) {
    if (!p) {
        set_error("%s: %s must be non-NULL", fn, name);
        return TCQ_EINVAL;
    }
    if (reinterpret_cast<uintptr_t>(p) % size) {
        set_error("%s: %s at %p is not aligned to its values of %zu bytes", fn, name, p, size);
        return TCQ_EINVAL;
    }
    if (head < dim || row < (heads - 1) * head + dim) {
        set_error("%s: strides of %s (row %lld, head %lld) are below what %lld heads of %lld "
                  "values take", fn, name, (long long)row, (long long)head, (long long)heads,
                  (long long)dim);
        return TCQ_EINVAL;
    }
    return TCQ_OK;
}

// The bytes of rows x heads vectors, without what lies between the rows (the heads' gaps count).
Region rows_region(const char *name, const void *p, int64_t rows, int64_t row, int64_t head,
                   int64_t heads, int64_t dim, size_t size) {
    return region(name, p, rows, row, (heads - 1) * head + dim, size);
}

int check_apart_from_cache(const char *fn, const Region &r, const CacheShape &c) {
    const int64_t vectors = (c.pages * c.heads) << c.page_log2;
    const int64_t codes = c.format == TCQ_FP4 ? c.dim / 2 : c.dim;
    const Region parts[4] = {region("the cache's key codes", c.k_codes, 1, 0, vectors * codes, 1),
                             region("the cache's key scales", c.k_scale, 1, 0,
                                    vectors * (c.dim / 32), 1),
                             region("the cache's value codes", c.v_codes, 1, 0, vectors * codes, 1),
                             region("the cache's value scales", c.v_scale, 1, 0,
                                    vectors * (c.dim / 32), 1)};
    for (const Region &p : parts) {
        const int rc = check_apart(fn, r, p);
        if (rc != TCQ_OK) return rc;
    }
    return TCQ_OK;
}

int check_apart_from_batch(const char *fn, const Region &r, const CacheBatch &b) {
    int rc = check_apart(fn, r, region("table", b.table, b.seqs, b.ldt, b.width, 4));
    if (rc == TCQ_OK) rc = check_apart(fn, r, region("lens", b.lens, 1, 0, b.seqs, 4));
    if (rc == TCQ_OK) rc = check_apart(fn, r, region("starts", b.starts, 1, 0, b.seqs + 1, 4));
    return rc;
}

int cache_move(const char *fn, bool write, const tcq_cache *cache, const tcq_cache_batch *batch,
               int dtype, const void *k, int64_t k_row, int64_t k_head, const void *v,
               int64_t v_row, int64_t v_head, int64_t rows, hipStream_t stream) {
    clear_error();
    CacheShape c;
    CacheBatch b;
    int rc = check_cache(fn, cache, c);
    if (rc == TCQ_OK) rc = check_batch(fn, batch, rows, b);
    if (rc == TCQ_OK) rc = check_dtype(fn, dtype);
    if (rc != TCQ_OK) return rc;
    if (rows == 0 || b.seqs == 0) return TCQ_OK;
    const size_t size = size_of(dtype);
    rc = check_rows(fn, "k", k, k_row, k_head, c.heads, c.dim, size);
    if (rc == TCQ_OK) rc = check_rows(fn, "v", v, v_row, v_head, c.heads, c.dim, size);
    if (rc != TCQ_OK) return rc;
    const Region rk = rows_region("k", k, rows, k_row, k_head, c.heads, c.dim, size);
    const Region rv = rows_region("v", v, rows, v_row, v_head, c.heads, c.dim, size);
    for (const Region *r : {&rk, &rv}) {
        rc = check_apart_from_cache(fn, *r, c);
        if (rc == TCQ_OK && !write) rc = check_apart_from_batch(fn, *r, b);
        if (rc != TCQ_OK) return rc;
    }
    if (!write) {
        rc = check_apart(fn, rk, rv);
        if (rc != TCQ_OK) return rc;
    }
    const hipError_t e = launch_cache_move(write, c, b, dtype, CacheRows{k, k_row, k_head},
                                           CacheRows{v, v_row, v_head}, rows, stream);
    if (e != hipSuccess) return hip_fail(fn, "cache launch", e);
    return TCQ_OK;
}

int check_heads(const char *fn, int q_heads, int heads, int64_t rows, int64_t seqs) {
    if (q_heads <= 0 || q_heads % heads) {
        set_error("%s: q_heads=%d is no multiple of the cache's %d heads", fn, q_heads, heads);
        return TCQ_EINVAL;
    }
    // (workgroups of a launch)
    if (q_heads > kMostHeads || rows * q_heads / 16 + seqs * heads > (1 << 24) - 4096) {
        set_error("%s: outside the limits (q_heads <= %d, rows x q_heads / 16 + seqs x heads below "
                  "2^24): rows=%lld q_heads=%d seqs=%lld", fn, kMostHeads, (long long)rows, q_heads,
                  (long long)seqs);
        return TCQ_EUNSUPPORTED;
    }
    if (attention_threads(q_heads / heads, heads, seqs, rows) > UINT32_MAX) {
        set_error("%s: outside the limits (rows x q_heads / 128 + seqs x heads below 2^23 - 256 with "
                  "more than 16 query rows to a sequence on average): rows=%lld q_heads=%d "
                  "seqs=%lld heads=%d", fn, (long long)rows, q_heads, (long long)seqs, heads);
        return TCQ_EUNSUPPORTED;
    }
    return TCQ_OK;
}

}  // namespace

extern "C" int tcq_cache_write(const tcq_cache *cache, const tcq_cache_batch *batch, int dtype,
                               const void *k, int64_t k_row, int64_t k_head, const void *v,
                               int64_t v_row, int64_t v_head, int64_t rows, hipStream_t stream) {
    return cache_move("tcq_cache_write", true, cache, batch, dtype, k, k_row, k_head, v, v_row,
                      v_head, rows, stream);
}

extern "C" int tcq_cache_read(const tcq_cache *cache, const tcq_cache_batch *batch, int dtype,
                              void *k, int64_t k_row, int64_t k_head, void *v, int64_t v_row,
                              int64_t v_head, int64_t rows, hipStream_t stream) {
    return cache_move("tcq_cache_read", false, cache, batch, dtype, k, k_row, k_head, v, v_row,
                      v_head, rows, stream);
}

extern "C" int tcq_cache_attention_workspace_bytes(int dim, int heads, int q_heads, int64_t seqs,
                                                   int64_t rows, size_t *bytes) {
    clear_error();
    const char *fn = "tcq_cache_attention_workspace_bytes";
    if (heads <= 0 || heads > kMostHeads || seqs < 0 || seqs > kMostSeqs || rows < 0 ||
        rows > TCQ_LINEAR_MAX_BATCH || (dim != 64 && dim != 128 && dim != 256)) {
        set_error("%s: outside the limits (dim 64, 128 or 256, heads <= %d, seqs <= %lld, rows <= "
                  "%d): dim=%d heads=%d seqs=%lld rows=%lld", fn, kMostHeads,
                  (long long)kMostSeqs, TCQ_LINEAR_MAX_BATCH, dim, heads, (long long)seqs,
                  (long long)rows);
        return TCQ_EUNSUPPORTED;
    }
    const int rc = check_heads(fn, q_heads, heads, rows, seqs);
    if (rc != TCQ_OK) return rc;
    if (!bytes) {
        set_error("%s: bytes is NULL", fn);
        return TCQ_EINVAL;
    }
    *bytes = attention_most_bytes(dim, q_heads / heads, seqs, rows);
    return TCQ_OK;
}

extern "C" int tcq_cache_attention(const tcq_cache *cache, const tcq_cache_batch *batch, int dtype,
                                   const void *q, int64_t q_row, int64_t q_head, int q_heads,
                                   int64_t rows, float scale, void *o, int64_t o_row,
                                   int64_t o_head, void *workspace, size_t workspace_bytes,
                                   hipStream_t stream) {
    clear_error();
    const char *fn = "tcq_cache_attention";
    CacheShape c;
    CacheBatch b;
    int rc = check_cache(fn, cache, c);
    if (rc == TCQ_OK) rc = check_batch(fn, batch, rows, b);
    if (rc == TCQ_OK) rc = check_dtype(fn, dtype);
    if (rc == TCQ_OK) rc = check_heads(fn, q_heads, c.heads, rows, b.seqs);
    if (rc != TCQ_OK) return rc;
    if (!(scale >= 0x1p-60f && scale <= 0x1p60f)) {
        set_error("%s: scale=%g is not between 2^-60 and 2^60", fn, static_cast<double>(scale));
        return TCQ_EINVAL;
    }
    if (rows == 0 || b.seqs == 0) return TCQ_OK;
    const size_t size = size_of(dtype);
    rc = check_rows(fn, "q", q, q_row, q_head, q_heads, c.dim, size);
    if (rc == TCQ_OK) rc = check_rows(fn, "o", o, o_row, o_head, q_heads, c.dim, size);
    if (rc != TCQ_OK) return rc;
    rc = check_workspace(fn, workspace, workspace_bytes,
                         attention_bytes(c.dim, q_heads / c.heads, b.seqs, rows));
    if (rc != TCQ_OK) return rc;
    const Region ro = rows_region("o", o, rows, o_row, o_head, q_heads, c.dim, size);
    rc = check_apart(fn, ro, rows_region("q", q, rows, q_row, q_head, q_heads, c.dim, size));
    if (rc == TCQ_OK) rc = check_apart_from_cache(fn, ro, c);
    if (rc == TCQ_OK) rc = check_apart_from_batch(fn, ro, b);
    if (rc != TCQ_OK) return rc;
    const AttentionCall call{c, b, dtype, CacheRows{q, q_row, q_head}, CacheRows{o, o_row, o_head},
                             q_heads / c.heads, rows, scale};
    const hipError_t e = launch_attention(call, static_cast<char *>(workspace), stream);
    if (e != hipSuccess) return hip_fail(fn, "attention launch", e);
    return TCQ_OK;
}
