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
    CUtensorMap tmap_half;   // the same with box {64, min(page_size, 64), 1}
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
    int launches;            // set by the launchers: kernels of this call
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

// ---------------------------------------------------------------------------
// Equal shares of a call's work (the tensor-core kernels).  An item is one (entry, row
// tile, kv head) with nt key tiles.  All items lie on one line, each nt + ovh units long
// (ovh: what starting and ending an item costs, in tiles), in the order entry, row tile,
// head.  CTA c of P takes the units [c U / P, (c+1) U / P), U the line's length, so all
// CTAs finish together whatever the lengths; a share may start or end inside an item.
// ---------------------------------------------------------------------------
constexpr int kLineTile = 64;     // keys of a tile

// Shared memory of a CTA: the entries and the units before each.
struct Line {
    int4* ent;          // [n]: sequence, first row, rows (0: nothing to do), length
    long long* pre;     // [n + 1], per kv head
    int n, rt, ovh, nkv, causal, window, sinks;

    DF_DEV int row_tiles(int i) const { return (ent[i].z + rt - 1) / rt; }
    DF_DEV KeySpan span(const int4& e, int t) const {
        const int r0 = t * rt, r1 = min(e.z, r0 + rt);
        return key_span(e.w, e.z, r0, r1, causal, window, sinks, kLineTile);
    }
};
constexpr int kLineBytes = kPoolMaxSeqs * 16 + (kPoolMaxSeqs + 2) * 8;

// Fill the line (the whole block; sums: THREADS / 32 long longs of shared memory).  Rows of
// bad entries are zeroed, each entry by one CTA.  Returns U.
template <int THREADS, int D>
DF_DEV long long line_plan(const PagedAttnParams& p, Line& L, uint8_t* mem, long long* sums, int ovh) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    L.ent = (int4*)mem;
    L.pre = (long long*)(mem + kPoolMaxSeqs * 16);
    L.n = p.n;
    L.rt = p.rt;
    L.ovh = ovh;
    L.nkv = p.nkv;
    L.causal = p.causal;
    L.window = p.window;
    L.sinks = p.sinks;
    for (int i = tid; i < p.n; i += THREADS) {
        AttnEntry e = attn_entry(p, i);
        if (e.bad) {
            if (i % (int)gridDim.x == (int)blockIdx.x) {
                if (p.status) set_error(p.status, e.bad);
                uint4* o = (uint4*)((__nv_bfloat16*)p.out + (size_t)e.start * p.nq * D);
                const size_t nz = (size_t)e.count * p.nq * D / 8;
                for (size_t x = 0; x < nz; ++x) o[x] = make_uint4(0, 0, 0, 0);
            }
            e.count = 0;
        }
        L.ent[i] = make_int4(e.seq, e.start, e.count, e.len);
        if (p.row_tiles == 1) L.pre[i] = e.count > 0 ? L.span(L.ent[i], 0).nt + ovh : 0;
    }
    __syncthreads();
    if (p.row_tiles > 1) {
        for (int i = warp; i < p.n; i += THREADS / 32) {
            const int4 e = L.ent[i];
            const int T = L.row_tiles(i);
            long long w = 0;
            for (int t = lane; t < T; t += 32) w += L.span(e, t).nt + ovh;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
            if (lane == 0) L.pre[i] = w;
        }
        __syncthreads();
    }
    long long run = 0;
    for (int base = 0; base < p.n; base += THREADS) {
        const int i = base + tid;
        const long long w = i < p.n ? L.pre[i] : 0;
        long long inc = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += u;
        }
        if (lane == 31) sums[warp] = inc;
        __syncthreads();
        long long before = run;
        for (int k = 0; k < THREADS / 32; ++k) {
            if (k < warp) before += sums[k];
            run += sums[k];
        }
        if (i < p.n) L.pre[i] = before + inc - w;
        __syncthreads();
    }
    if (tid == 0) L.pre[p.n] = run;
    __syncthreads();
    return run * p.nkv;
}

// A CTA's stretch of one item: key tiles [t0, t1) of span.nt for rows [r0, r1) of entry i.
struct Stretch {
    int i, g, r0, r1, t0, t1;
    KeySpan span;
    long long v0;       // the item's first unit
    DF_DEV bool whole() const { return t0 == 0 && t1 == span.nt; }
};
struct Walker {
    long long v, end;   // units still to come
    int i, t, g, off;   // item and units of it that lie before v

    // The calling warp as a whole; v < end <= U.
    DF_DEV void start(const Line& L, long long begin, long long end_) {
        v = begin;
        end = end_;
        int lo = 0;
        for (int hi = L.n; hi - lo > 1;) {
            const int mid = (lo + hi) >> 1;
            if (L.pre[mid] * L.nkv <= v) lo = mid;
            else hi = mid;
        }
        i = lo;
        while (L.pre[i + 1] * L.nkv <= v) ++i;     // entries without units share their start
        long long local = v - L.pre[i] * L.nkv;
        const int4 e = L.ent[i];
        const int T = L.row_tiles(i), lane = threadIdx.x & 31;
        t = 0;
        if (T > 1) {
            for (int tb = 0;; tb += 32) {
                const int tt = tb + lane;
                const long long w = tt < T ? (long long)(L.span(e, tt).nt + L.ovh) * L.nkv : 0;
                long long inc = w;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const long long u = __shfl_up_sync(0xffffffffu, inc, o);
                    if (lane >= o) inc += u;
                }
                const unsigned m = __ballot_sync(0xffffffffu, inc > local);
                if (m) {
                    const int src = __ffs(m) - 1;
                    t = tb + src;
                    local -= __shfl_sync(0xffffffffu, inc - w, src);
                    break;
                }
                local -= __shfl_sync(0xffffffffu, inc, 31);
            }
        }
        const int size = L.span(e, t).nt + L.ovh;
        g = (int)(local / size);
        off = (int)(local % size);
    }
    // The next stretch with tiles; false when the share is done.
    DF_DEV bool next(const Line& L, Stretch& s) {
        while (v < end) {
            const int4 e = L.ent[i];
            s.span = L.span(e, t);
            const int size = s.span.nt + L.ovh;
            const int take = (int)min((long long)(size - off), end - v);
            s.i = i;
            s.g = g;
            s.r0 = t * L.rt;
            s.r1 = min(e.z, s.r0 + L.rt);
            s.t0 = max(0, off - L.ovh);
            s.t1 = max(0, off + take - L.ovh);
            s.v0 = v - off;
            v += take;
            off += take;
            if (off == size) {
                off = 0;
                if (++g == L.nkv) {
                    g = 0;
                    if (++t >= L.row_tiles(i)) {
                        t = 0;
                        while (++i < L.n && L.ent[i].z == 0) {}
                    }
                }
            }
            if (s.t1 > s.t0) return true;
        }
        return false;
    }
};
// True for one lane of a converged warp, the same one every time.
DF_DEV bool elect_one() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r != 0;
}
// Whether an mbarrier phase has completed, without waiting.
DF_DEV bool mbar_test(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
// CTA that holds unit u.
DF_DEV int line_owner(long long u, long long U, int P) { return (int)(((u + 1) * P - 1) / U); }

// Issue the TMA loads of one 64-key tile of K and V by a whole warp: pages looked up 32 at
// a time.  A box is min(page_size, 64) rows; boxes in which no row sees a key are not loaded.
struct PageLookup {
    int first, page;    // pages first .. first + 31 of the sequence, one per lane
    DF_DEV void reset() { first = -(1 << 30); }
    DF_DEV int at(const PagedAttnParams& p, int seq, int k0, int kb, int boxes, int lane) {
        if (!p.table) return seq;
        const int pf = k0 >> p.ps_log2;
        if (pf < first || pf + boxes > first + 32) {
            first = pf;
            page = first + lane < p.max_pages ? p.table[(size_t)seq * p.max_pages + first + lane] : -1;
        }
        return __shfl_sync(0xffffffffu, page, ((kb >> p.ps_log2) - first) & 31);
    }
};

// Tensor map of a bf16 slab of `rows` rows of d elements for the kernels (abi.cu); false
// when the driver's encoder rejects it.
bool encode_kv_rows(CUtensorMap* m, const void* slab, uint64_t rows, int d, int box_rows, int halves);

size_t paged_scratch_bytes();    // partials and counters of an attention launch
constexpr size_t kPagedCounterBytes = 8192;
constexpr size_t kJoinRecords = 2048;   // in them: 32 bytes per CTA, what paged_block.cu has to join

// At most 16 query rows per kv head (paged_decode.cu).
int launch_paged_decode(PagedAttnParams& p, int d, int num_sms, cudaStream_t st);
// Any number of rows (paged_block.cu).
int launch_paged_block(PagedAttnParams& p, int d, int num_sms, cudaStream_t st);
int launch_paged_attn_f32(PagedAttnParams& p, int d, int num_sms, cudaStream_t st);
int launch_paged_attn_bf16(PagedAttnParams& p, int d, int num_sms, cudaStream_t st);

}  // namespace df
