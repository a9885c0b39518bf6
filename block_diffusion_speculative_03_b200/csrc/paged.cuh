// The paged key/value pool: views, launchers of the page operations (pages.cu)
// and of attention over pages or over a cache slab (paged_attn.cu, paged_attn_tc.cu).
#pragma once
#include "common.cuh"

namespace df {

constexpr int kPoolMaxSeqs = 1024;      // the plan kernels hold one sequence per thread of one block
constexpr int kPagedCtas = 160;         // most CTAs of an attention launch with partials (>= SMs of any B200)
constexpr int kPagedRowsTc = 128;       // query rows of a tensor-core row tile

// Device view of a pool.
struct PoolView {
    int* status;
    int* len;             // [max_seqs]
    int* table;           // [max_seqs][max_pages]
    int* refs;            // [n_pages]
    int n_pages, ps, ps_log2, max_seqs, max_pages, max_len;
    uint8_t* slab;
    long long page_bytes; // n_layers * 2 * nkv * ps * row_bytes
    int n_layers, nkv, row_bytes;
    // scratch of the page operations
    int* freelist;        // [n_pages]
    int* movers;          // [n_pages]: compact's sources, then the map old id -> new id
    int4* recs;           // [n_pages]: planned new entries (sequence, index, old page, new page)
    int4* copies;         // [n_pages]: (source page, destination page, rows, 0)
    int* n_copies;        // [8]: copies of the running operation; compact's page count; set_tables' error flag
    int* counters;        // attention: arrivals per split item, zero between launches
};

// A request's rows in a dflash_cache, as bytes.
struct SlabView {
    uint8_t* slab;
    long long s_req, s_layer, s_kind, s_kv;   // bytes
    int* len;
    int* committed;
    int batch, capacity;
};

// What abi.cu knows of a cache (its struct is private to it).
struct CacheView {
    SlabView slab;
    int n_layers, n_kv_heads, head_dim, dtype;
};
bool cache_view(const dflash_cache* c, CacheView& v);

int launch_pool_set_tables(const PoolView& v, const int* lens, const int* table, cudaStream_t st);
int launch_pages_reserve(const PoolView& v, const int* seqs, const int* grow, int n, cudaStream_t st);
int launch_pages_fork(const PoolView& v, const int* src, const int* dst, int n, int deep, cudaStream_t st);
int launch_pages_free(const PoolView& v, const int* seqs, const int* keep, int n, cudaStream_t st);
int launch_pages_compact(const PoolView& v, int* used, cudaStream_t st);
int launch_pages_write(const PoolView& v, const int* seqs, int n, int layer, const void* k, const void* vv,
                       long long stride_bytes, const int* row_start, const int* row_count, int total_rows, int max_rows,
                       cudaStream_t st);
int launch_pages_advance(const PoolView& v, const int* seqs, const int* row_count, int n, cudaStream_t st);
int launch_pages_exchange(const PoolView& v, const int* seqs, const SlabView& c, const int* reqs, int n, bool load,
                          cudaStream_t st);

// ---------------------------------------------------------------------------
// Attention
// ---------------------------------------------------------------------------

struct PagedAttnParams {
    CUtensorMap tmap;        // bf16: slab rows as [head_dim / 64][rows][64], 128-byte swizzle, box
                             // {64, min(page_size, 64), head_dim / 64}
    const void* slab;        // fp32: the slab itself
    const void* q;
    long long q_stride;      // elements
    void* out;               // [total_rows][nq][d]
    const int* seqs;         // null: 0..n-1
    const int* len;
    const int* table;        // null: the slab of a dflash_cache
    const int* req_ok;       // slab: requests to skip (0); null: none
    int n, max_seqs, max_pages, ps_log2;
    const int* row_start;    // null: entry i owns rows [i * uniform, (i+1) * uniform)
    const int* row_count;
    int uniform;             // rows per entry when row_start is null
    int total_rows, max_rows, row_tiles;
    int rt;                  // positions per row tile: query rows of a tile = rt * G
    int G, nq, nkv;
    int causal, window, sinks;
    // slab rows (units of one head's row): page (or request), kind and kv-head strides, the layer's first row
    long long rows_page, rows_kind, rows_kv, row_layer;
    float scale_log2;
    float* partial;          // split items' partials
    int* counters;           // [kPagedCtas], zero between launches
    int splits;              // fp32 kernel: key splits per item
    int* status;             // null: the slab path (requests are checked by the draft step)
    int* wait_status;        // DFLASH_TIMEOUT of a bounded wait
};

// Key tiles of TK keys that the rows [r0, r1) (positions len + r) of an entry with
// `count` rows can see: `ns` leading tiles that hold sinks, then tiles from t0;
// nt in all.
struct KeySpan {
    int ns, t0, nt;
    __host__ __device__ int tile(int i) const { return i < ns ? i : t0 + (i - ns); }
};
__host__ __device__ inline KeySpan key_span(int len, int count, int r0, int r1, int causal, int window, int sinks,
                                            int tk) {
    const int hi = causal ? len + r1 : len + count;
    int lo = 0;
    if (window > 0) {
        lo = len + r0 - window + 1;
        if (lo < 0) lo = 0;
    }
    const int a = sinks < lo ? sinks : lo;
    KeySpan s;
    s.ns = (a + tk - 1) / tk;
    s.t0 = lo / tk;
    if (s.t0 < s.ns) s.t0 = s.ns;
    const int te = (hi + tk - 1) / tk;
    s.nt = s.ns + (te > s.t0 ? te - s.t0 : 0);
    return s;
}

// What an entry of the call stands for; count 0: nothing to do.
struct AttnEntry {
    int seq, start, count, len;
    int bad;                 // its rows are to be zeroed: [start, start + count)
};
DF_DEV AttnEntry attn_entry(const PagedAttnParams& p, int i) {
    AttnEntry e;
    e.seq = p.seqs ? p.seqs[i] : i;
    e.start = p.row_start ? p.row_start[i] : i * p.uniform;
    e.count = p.row_start ? p.row_count[i] : p.uniform;
    e.len = 0;
    e.bad = 0;
    if (e.seq == -1 || e.count == 0) {
        e.count = 0;
        return e;
    }
    if (e.count < 0 || e.count > p.max_rows || e.start < 0 || e.start > p.total_rows - e.count) {
        e.count = 0;
        e.bad = DFLASH_INVALID_ARG;   // not a row range: nothing can be zeroed
        return e;
    }
    if (e.seq < 0 || e.seq >= p.max_seqs) {
        e.bad = DFLASH_INVALID_ARG;
        return e;
    }
    e.len = p.len[e.seq];
    if (p.table) {
        const long long last = ((long long)e.len + e.count - 1) >> p.ps_log2;
        if (last >= p.max_pages || p.table[(size_t)e.seq * p.max_pages + last] < 0) e.bad = DFLASH_CAPACITY;
    } else if (p.req_ok && !p.req_ok[e.seq]) {
        e.bad = DFLASH_STATE;
    }
    return e;
}
DF_DEV bool key_visible(int k, int pos, int hi, int window, int sinks) {
    return k < hi && (window <= 0 || k < sinks || k > pos - window);
}

// Tensor map of a bf16 slab of `rows` rows of d elements for the kernels (abi.cu); false
// when the driver's encoder rejects it.
bool encode_kv_rows(CUtensorMap* m, const void* slab, uint64_t rows, int d, int box_rows);

size_t paged_scratch_bytes();    // partials and counters of an attention launch
constexpr size_t kPagedCounterBytes = 8192;

// At most 16 query rows per kv head (paged_decode.cu).
int launch_paged_decode(const PagedAttnParams& p, int d, int num_sms, cudaStream_t st);
int launch_paged_attn_f32(PagedAttnParams& p, int d, int num_sms, cudaStream_t st);
int launch_paged_attn_bf16(PagedAttnParams& p, int d, int num_sms, cudaStream_t st);

}  // namespace df
