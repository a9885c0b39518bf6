// C ABI of the paged pool (include/dflash_paged.h): argument checks, the pool's
// memory layout, and the launches of each call.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>

#include "../../include/dflash_paged.h"
#include "paged.cuh"

using namespace df;

struct dflash_pool {
    dflash_pool_config cfg;
    int device, num_sms;
    PoolView v;
    CUtensorMap tmap, tmap_half;   // bf16: the slab's rows (encode_kv_rows)
    uint8_t* scratch;          // attention partials and counters
    long long launches;
};

namespace {

inline size_t al(size_t x, size_t a = 256) { return (x + a - 1) / a * a; }
inline cudaStream_t S(dflash_stream s) { return (cudaStream_t)s; }
inline bool aligned16(const void* p) { return p && (((uintptr_t)p) & 15) == 0; }

struct PoolLayout {
    size_t len, table, refs, freelist, movers, recs, copies, n_copies, counters, cleared, partial, slab, total;
    int max_pages;
    long long page_bytes;
};

int pool_layout(const dflash_pool_config* c, PoolLayout& L) {
    if (!c || c->n_layers < 1 || c->n_q_heads < 1 || c->n_kv_heads < 1 || c->n_pages < 1 || c->max_seqs < 1 ||
        c->max_seqs > kPoolMaxSeqs || c->max_len < 1 || c->max_len > (1 << 30) || c->n_q_heads % c->n_kv_heads ||
        (c->dtype != DFLASH_BF16 && c->dtype != DFLASH_F32))
        return DFLASH_INVALID_ARG;
    if (c->head_dim != 64 && c->head_dim != 128) return DFLASH_UNSUPPORTED;
    const int ps = c->page_size;
    if (ps != 16 && ps != 32 && ps != 64 && ps != 128 && ps != 256) return DFLASH_UNSUPPORTED;
    if (c->n_q_heads / c->n_kv_heads > kPagedRowsTc) return DFLASH_UNSUPPORTED;
    // rows of one head in the slab are 32-bit coordinates; products stay in 64 bits by these bounds
    const long long runs = 2LL * c->n_layers * c->n_kv_heads;
    if (runs > (1LL << 31) / ps || (long long)c->n_pages * ps * runs >= (1LL << 31)) return DFLASH_UNSUPPORTED;
    L.max_pages = (int)(((long long)c->max_len + ps - 1) / ps);
    if ((long long)c->max_seqs * L.max_pages >= (1LL << 31)) return DFLASH_UNSUPPORTED;
    const size_t es = c->dtype == DFLASH_BF16 ? 2 : 4;
    L.page_bytes = runs * ps * c->head_dim * (long long)es;
    const size_t np = (size_t)c->n_pages;
    size_t o = 256;                                        // status word
    L.len = o; o = al(o + (size_t)c->max_seqs * 4);
    L.refs = o; o = al(o + np * 4);
    L.n_copies = o; o = al(o + 32);
    L.counters = o; o = al(o + kPagedCounterBytes);
    L.cleared = o;                                         // [0, cleared) starts at zero, the tables at -1
    L.table = o; o = al(o + (size_t)c->max_seqs * L.max_pages * 4);
    L.freelist = o; o = al(o + np * 4);
    L.movers = o; o = al(o + np * 4);
    L.recs = o; o = al(o + std::max(np, (size_t)kPoolMaxSeqs) * 16);
    L.copies = o; o = al(o + np * 16);
    L.partial = o; o = al(o + paged_scratch_bytes() - kPagedCounterBytes, 1024);
    L.slab = o; o += np * (size_t)L.page_bytes;
    L.total = o;
    return DFLASH_OK;
}

// The pool's device is current and the call can list n sequences.
int check(const dflash_pool* p, int n) {
    if (!p || n < 0 || n > p->cfg.max_seqs) return DFLASH_INVALID_ARG;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return DFLASH_CUDA;
    return dev == p->device ? DFLASH_OK : DFLASH_INVALID_ARG;
}

int done(dflash_pool* p, int e, int launches) {
    if (e != 0) {
        cudaGetLastError();
        return DFLASH_CUDA;
    }
    p->launches += launches;
    return DFLASH_OK;
}

// The cache has the pool's device, layers, heads and type.
bool same_shape(const dflash_pool* p, const CacheView& c) {
    return c.device == p->device && c.n_layers == p->cfg.n_layers && c.n_kv_heads == p->cfg.n_kv_heads && c.head_dim == p->cfg.head_dim &&
           c.dtype == p->cfg.dtype;
}

}  // namespace

extern "C" {

int dflash_pool_bytes(const dflash_pool_config* cfg, size_t* bytes) {
    PoolLayout L;
    const int e = pool_layout(cfg, L);
    if (e) return e;
    if (!bytes) return DFLASH_INVALID_ARG;
    *bytes = L.total;
    return DFLASH_OK;
}

int dflash_pool_init(const dflash_pool_config* cfg, void* mem, size_t bytes, dflash_pool** out, dflash_stream stream) {
    PoolLayout L;
    const int e = pool_layout(cfg, L);
    if (e) return e;
    if (!mem || !out || ((uintptr_t)mem & 1023)) return DFLASH_INVALID_ARG;
    if (bytes < L.total) return DFLASH_WORKSPACE;
    int dev = 0, sms = 0, major = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess)
        return DFLASH_CUDA;
    if (major != 10) return DFLASH_UNSUPPORTED;
    dflash_pool* p = new (std::nothrow) dflash_pool();
    if (!p) return DFLASH_CUDA;
    const dflash_pool_config& c = *cfg;
    uint8_t* b = (uint8_t*)mem;
    p->cfg = c;
    p->device = dev;
    p->num_sms = sms;
    p->launches = 0;
    p->scratch = b + L.partial;
    PoolView& v = p->v;
    v.status = (int*)b;
    v.len = (int*)(b + L.len);
    v.table = (int*)(b + L.table);
    v.refs = (int*)(b + L.refs);
    v.n_pages = c.n_pages;
    v.ps = c.page_size;
    v.ps_log2 = 0;
    while ((1 << v.ps_log2) < c.page_size) ++v.ps_log2;
    v.max_seqs = c.max_seqs;
    v.max_pages = L.max_pages;
    v.max_len = c.max_len;
    v.slab = b + L.slab;
    v.page_bytes = L.page_bytes;
    v.n_layers = c.n_layers;
    v.nkv = c.n_kv_heads;
    v.row_bytes = c.head_dim * (c.dtype == DFLASH_BF16 ? 2 : 4);
    v.freelist = (int*)(b + L.freelist);
    v.movers = (int*)(b + L.movers);
    v.recs = (int4*)(b + L.recs);
    v.copies = (int4*)(b + L.copies);
    v.n_copies = (int*)(b + L.n_copies);
    v.counters = (int*)(b + L.counters);
    if (c.dtype == DFLASH_BF16) {
        const uint64_t rows = (uint64_t)c.n_pages * 2 * c.n_layers * c.n_kv_heads * c.page_size;
        const int box = std::min(c.page_size, 64), halves = c.head_dim / 64;
        if (!encode_kv_rows(&p->tmap, v.slab, rows, c.head_dim, box, halves) ||
            !encode_kv_rows(&p->tmap_half, v.slab, rows, c.head_dim, box, 1)) {
            delete p;
            return DFLASH_CUDA;
        }
    }
    if (cudaMemsetAsync(b, 0, L.cleared, S(stream)) != cudaSuccess ||
        cudaMemsetAsync(v.table, 0xff, (size_t)c.max_seqs * L.max_pages * 4, S(stream)) != cudaSuccess) {
        delete p;
        return DFLASH_CUDA;
    }
    *out = p;
    return DFLASH_OK;
}

void dflash_pool_release(dflash_pool* p) { delete p; }

int dflash_pool_get_info(const dflash_pool* p, dflash_pool_info* info) {
    if (!p || !info) return DFLASH_INVALID_ARG;
    info->max_pages = p->v.max_pages;
    info->status = p->v.status;
    info->len = p->v.len;
    info->table = p->v.table;
    info->refs = p->v.refs;
    info->slab = p->v.slab;
    info->stride_kv = (int64_t)p->cfg.page_size * p->cfg.head_dim;
    info->stride_kind = info->stride_kv * p->cfg.n_kv_heads;
    info->stride_layer = info->stride_kind * 2;
    info->stride_page = info->stride_layer * p->cfg.n_layers;
    return DFLASH_OK;
}

int dflash_pool_status(dflash_pool* p, dflash_stream stream) {
    const int e = check(p, 0);
    if (e) return e;
    int s = 0;
    if (cudaMemcpyAsync(&s, p->v.status, 4, cudaMemcpyDeviceToHost, S(stream)) != cudaSuccess) return DFLASH_CUDA;
    if (cudaMemsetAsync(p->v.status, 0, 4, S(stream)) != cudaSuccess) return DFLASH_CUDA;
    if (cudaStreamSynchronize(S(stream)) != cudaSuccess) return DFLASH_CUDA;
    return s;
}

int64_t dflash_pool_launch_count(const dflash_pool* p) { return p ? p->launches : 0; }

int dflash_pool_set_tables(dflash_pool* p, const int32_t* lens, const int32_t* table, dflash_stream stream) {
    const int e = check(p, 0);
    if (e) return e;
    if (!lens || !table) return DFLASH_INVALID_ARG;
    int launches = 0;
    const int r = launch_pool_set_tables(p->v, lens, table, S(stream), &launches);
    return done(p, r, launches);
}

int dflash_pages_reserve(dflash_pool* p, const int32_t* seqs, const int32_t* grow, int n, dflash_stream stream) {
    const int e = check(p, n);
    if (e) return e;
    if (n == 0) return DFLASH_OK;
    if (!grow) return DFLASH_INVALID_ARG;
    return done(p, launch_pages_reserve(p->v, seqs, grow, n, S(stream)), 2);
}

int dflash_pages_fork(dflash_pool* p, const int32_t* src, const int32_t* dst, int n, int deep, dflash_stream stream) {
    const int e = check(p, n);
    if (e) return e;
    if (n == 0) return DFLASH_OK;
    if (!src || !dst) return DFLASH_INVALID_ARG;
    return done(p, launch_pages_fork(p->v, src, dst, n, deep, S(stream)), deep ? 2 : 1);
}

int dflash_pages_free(dflash_pool* p, const int32_t* seqs, const int32_t* keep, int n, dflash_stream stream) {
    const int e = check(p, n);
    if (e) return e;
    if (n == 0) return DFLASH_OK;
    return done(p, launch_pages_free(p->v, seqs, keep, n, S(stream)), 1);
}

int dflash_pages_compact(dflash_pool* p, int32_t* used, dflash_stream stream) {
    const int e = check(p, 0);
    if (e) return e;
    if (!used) return DFLASH_INVALID_ARG;
    int launches = 0;
    const int r = launch_pages_compact(p->v, used, S(stream), &launches);
    return done(p, r, launches);
}

int dflash_pages_write(dflash_pool* p, const int32_t* seqs, int n, int layer, const void* k, const void* v,
                       int64_t stride, const int32_t* row_start, const int32_t* row_count, int total_rows,
                       int max_rows, dflash_stream stream) {
    const int e = check(p, n);
    if (e) return e;
    if (layer < 0 || layer >= p->cfg.n_layers || total_rows < 0 || max_rows < 0 || !row_start != !row_count)
        return DFLASH_INVALID_ARG;
    if (!row_start && (max_rows < 1 || total_rows < n)) return DFLASH_INVALID_ARG;
    if (n == 0 || max_rows == 0 || total_rows == 0) return DFLASH_OK;
    const int es = p->cfg.dtype == DFLASH_BF16 ? 2 : 4;
    const int64_t width = (int64_t)p->cfg.n_kv_heads * p->cfg.head_dim;
    if (!aligned16(k) || !aligned16(v) || stride < width || stride > (INT64_MAX >> 4) || (stride * es) % 16)
        return DFLASH_INVALID_ARG;
    if (!row_start) max_rows = 1;
    return done(p, launch_pages_write(p->v, seqs, n, layer, k, v, stride * es, row_start, row_count, total_rows,
                                      std::min(std::min(max_rows, total_rows), p->cfg.max_len), S(stream)), 1);
}

int dflash_pages_advance(dflash_pool* p, const int32_t* seqs, const int32_t* row_count, int n, dflash_stream stream) {
    const int e = check(p, n);
    if (e) return e;
    if (n == 0) return DFLASH_OK;
    return done(p, launch_pages_advance(p->v, seqs, row_count, n, S(stream)), 1);
}

int dflash_pages_store(dflash_pool* p, const int32_t* seqs, const dflash_cache* c, const int32_t* reqs, int n,
                       dflash_stream stream) {
    const int e = check(p, n);
    if (e) return e;
    CacheView cv;
    if (!cache_view(c, cv) || !same_shape(p, cv) || (!reqs && n > cv.slab.batch)) return DFLASH_INVALID_ARG;
    if (n == 0) return DFLASH_OK;
    return done(p, launch_pages_exchange(p->v, seqs, cv.slab, reqs, n, false, S(stream)), 3);
}

int dflash_pages_load(dflash_pool* p, const int32_t* seqs, dflash_cache* c, const int32_t* reqs, int n,
                      dflash_stream stream) {
    const int e = check(p, n);
    if (e) return e;
    CacheView cv;
    if (!cache_view(c, cv) || !same_shape(p, cv) || (!reqs && n > cv.slab.batch)) return DFLASH_INVALID_ARG;
    if (n == 0) return DFLASH_OK;
    return done(p, launch_pages_exchange(p->v, seqs, cv.slab, reqs, n, true, S(stream)), 3);
}

int dflash_paged_attention(dflash_pool* p, const int32_t* seqs, int n, int layer, const void* q, int64_t q_stride,
                           const int32_t* row_start, const int32_t* row_count, int total_rows, int max_rows,
                           int causal, int window, int sinks, void* out, dflash_stream stream) {
    // entries of a read-only call may repeat a sequence, so their number has its own bound
    const int e = check(p, 0);
    if (e) return e;
    const dflash_pool_config& c = p->cfg;
    if (n < 0 || n > kPoolMaxSeqs || (!seqs && n > c.max_seqs) || layer < 0 || layer >= c.n_layers || total_rows < 0 ||
        max_rows < 0 || !row_start != !row_count || window < 0 || sinks < 0)
        return DFLASH_INVALID_ARG;
    if (!row_start && (max_rows < 1 || total_rows < n)) return DFLASH_INVALID_ARG;
    if (n == 0 || max_rows == 0 || total_rows == 0) return DFLASH_OK;
    const int es = c.dtype == DFLASH_BF16 ? 2 : 4;
    if (!aligned16(q) || !aligned16(out) || q_stride < (int64_t)c.n_q_heads * c.head_dim ||
        q_stride > (INT64_MAX >> 4) || (q_stride * es) % 16)
        return DFLASH_INVALID_ARG;
    PagedAttnParams a;
    std::memset(&a, 0, sizeof(a));
    a.tmap = p->tmap;
    a.tmap_half = p->tmap_half;
    a.slab = p->v.slab;
    a.q = q;
    a.q_stride = q_stride;
    a.out = out;
    a.seqs = seqs;
    a.len = p->v.len;
    a.table = p->v.table;
    a.n = n;
    a.max_seqs = c.max_seqs;
    a.max_pages = p->v.max_pages;
    a.ps_log2 = p->v.ps_log2;
    a.row_start = row_start;
    a.row_count = row_count;
    a.uniform = 1;
    a.total_rows = total_rows;
    a.max_rows = row_start ? std::min(std::min(max_rows, total_rows), c.max_len) : 1;
    a.G = c.n_q_heads / c.n_kv_heads;
    a.nq = c.n_q_heads;
    a.nkv = c.n_kv_heads;
    a.causal = causal ? 1 : 0;
    a.window = window;
    a.sinks = window > 0 ? sinks : 0;
    a.rows_kv = c.page_size;
    a.rows_kind = a.rows_kv * c.n_kv_heads;
    a.rows_page = a.rows_kind * 2 * c.n_layers;
    a.row_layer = a.rows_kind * 2 * layer;
    a.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)c.head_dim));
    a.partial = (float*)p->scratch;
    a.counters = p->v.counters;
    a.status = p->v.status;
    a.wait_status = p->v.status;
    const int r = c.dtype == DFLASH_BF16 ? launch_paged_attn_bf16(a, c.head_dim, p->num_sms, S(stream))
                                         : launch_paged_attn_f32(a, c.head_dim, p->num_sms, S(stream));
    return done(p, r, a.launches);
}

int dflash_window_scratch_bytes(size_t* bytes) {
    if (!bytes) return DFLASH_INVALID_ARG;
    *bytes = paged_scratch_bytes();
    return DFLASH_OK;
}

}  // extern "C"
