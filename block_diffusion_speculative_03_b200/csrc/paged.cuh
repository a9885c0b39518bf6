// The paged key/value pool: views, launchers of the page operations (pages.cu)
// and of attention over pages or over a cache slab (paged_decode.cu: few rows, paged_block.cu:
// many; paged_attn.cu: fp32 storage).
#pragma once
#include <atomic>

#include "common.cuh"

namespace df {

constexpr int kPoolMaxSeqs = 1024;      // the plan kernels hold one sequence per thread of one block
constexpr int kPagedCtas = 160;         // most CTAs of an attention launch with partials (>= SMs of any B200)
constexpr int kPagedRowsTc = 128;       // query rows of a tensor-core row tile

// Let a kernel use `bytes` of dynamic shared memory, once per kernel (ID: one number per
// kernel) and device.
template <int ID> bool allow_smem(const void* fn, int bytes) {
    static std::atomic<unsigned long long> done{0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    const unsigned long long bit = 1ull << (dev & 63);
    if (dev < 64 && (done.load(std::memory_order_relaxed) & bit)) return true;
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
    if (dev < 64) done.fetch_or(bit, std::memory_order_relaxed);
    return true;
}

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
    int n_layers, n_kv_heads, head_dim, dtype, device;
};
bool cache_view(const dflash_cache* c, CacheView& v);

int launch_pool_set_tables(const PoolView& v, const int* lens, const int* table, cudaStream_t st, int* launches);
int launch_pages_reserve(const PoolView& v, const int* seqs, const int* grow, int n, cudaStream_t st);
int launch_pages_fork(const PoolView& v, const int* src, const int* dst, int n, int deep, cudaStream_t st);
int launch_pages_free(const PoolView& v, const int* seqs, const int* keep, int n, cudaStream_t st);
int launch_pages_compact(const PoolView& v, int* used, cudaStream_t st, int* launches);
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
    int g_magic;             // v / G = v * g_magic >> 16 for v < 512 (set by the launchers)
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
    // the loads that do not depend on one another together
    AttnEntry e;
    e.start = p.row_start ? p.row_start[i] : i * p.uniform;
    e.count = p.row_start ? p.row_count[i] : p.uniform;
    e.seq = p.seqs ? p.seqs[i] : i;
    const bool exists = e.seq >= 0 && e.seq < p.max_seqs;
    e.len = p.len[exists ? e.seq : 0];
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
    if (!exists) {
        e.bad = DFLASH_INVALID_ARG;
        return e;
    }
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

// A row's integer base b moves when the floor of its running maximum passes b + kBaseLag, to
// kBaseLead above it: P stays below 2^(kBaseLag + 1), and after its first tile a row's scores
// have to rise by 2^16 before O is rescaled again (with the base at the maximum itself, rows
// whose first tile shows only a few sinks rescaled in most tiles, 700 cycles each time).  A
// weight that vanishes for the lead is below 2^-118 of the row's largest.
constexpr float kBaseLag = 8.0f, kBaseLead = 8.0f;

// Shared memory of a CTA: the entries and the units before each.  Units are 32-bit (2^31 of them
// are two hours of work for a whole device; a call with more records DFLASH_UNSUPPORTED).
struct Line {
    int4* ent;          // [n]: sequence, first row, rows (0: nothing to do), length (-r: r rows to zero)
    int* pre;           // [n + 1]
    int n, rt, ovh, nkv, causal, window, sinks;

    DF_DEV int row_tiles(int i) const {
        const int z = ent[i].z;
        return z <= rt ? (z > 0) : (z + rt - 1) / rt;
    }
    DF_DEV KeySpan span(const int4& e, int t) const {
        const int r0 = t * rt, r1 = min(e.z, r0 + rt);
        return key_span(e.w, e.z, r0, r1, causal, window, sinks, kLineTile);
    }
};
constexpr int kLineBytes = kPoolMaxSeqs * 16 + (kPoolMaxSeqs + 4) * 4;

// Zero the rows of refused entries: the whole device, 16 bytes a thread at a time.  (A function of its own:
// inline, its code on the way to a CTA's first load cost calls that refuse nothing 0.2 us.)
template <int THREADS, int D> __device__ __noinline__ void zero_rows(void* out, int nq, const int4* ent, int n) {
    for (int i = 0; i < n; ++i) {
        const int4 e = ent[i];
        if (e.z != 0 || e.w >= 0) continue;
        uint4* o = (uint4*)((__nv_bfloat16*)out + (size_t)e.y * nq * D);
        const size_t nz = (size_t)-e.w * nq * D / 8;
        for (size_t x = (size_t)blockIdx.x * THREADS + threadIdx.x; x < nz; x += (size_t)gridDim.x * THREADS)
            o[x] = make_uint4(0, 0, 0, 0);
    }
}

// Fill the line (the whole block; sums: THREADS / 32 long longs of shared memory).  Rows of
// bad entries are zeroed.  Returns U, 0 when there is nothing to do.
template <int THREADS, int D>
DF_DEV int line_plan(const PagedAttnParams& p, Line& L, uint8_t* mem, long long* sums, int ovh) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    L.ent = (int4*)mem;
    L.pre = (int*)(mem + kPoolMaxSeqs * 16);
    L.n = p.n;
    L.rt = p.rt;
    L.ovh = ovh;
    L.nkv = p.nkv;
    L.causal = p.causal;
    L.window = p.window;
    L.sinks = p.sinks;
    long long w = 0;              // units of entry tid, in the one-row-tile case of the first THREADS entries
    const bool quick = p.n <= 32 && p.row_tiles == 1;      // one warp scans
    bool refused = false;         // this thread has an entry whose rows are to be zeroed
    for (int i = tid; i < p.n; i += THREADS) {
        AttnEntry e = attn_entry(p, i);
        if (e.bad) {
            if (p.status && i % (int)gridDim.x == (int)blockIdx.x) set_error(p.status, e.bad);
            refused |= e.count > 0;
            e.len = -e.count;
            e.count = 0;
        } else if (e.count == 0) {
            e.len = 0;
        }
        L.ent[i] = make_int4(e.seq, e.start, e.count, e.len);
        if (p.row_tiles == 1) {
            w = e.count > 0 ? (long long)(L.span(L.ent[i], 0).nt + ovh) * p.nkv : 0;
            L.pre[i] = (int)min(w, 0x7fffffffll);
        }
    }
    if (quick) {
        if (warp == 0) {
            long long inc = w;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long u = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += u;
            }
            if (lane < p.n) L.pre[lane] = (int)min(inc - w, 0x7fffffffll);
            if (lane == p.n - 1) sums[0] = inc;
        }
        if (__syncthreads_or(refused)) zero_rows<THREADS, D>(p.out, p.nq, L.ent, p.n);
        const long long all = sums[0];
        if (tid == 0) L.pre[p.n] = (int)min(all, 0x7fffffffll);
        __syncthreads();
        if (all >= 0x7fffffffll && tid == 0 && p.wait_status) set_error(p.wait_status, DFLASH_UNSUPPORTED);
        return all < 0x7fffffffll ? (int)all : 0;
    }
    if (__syncthreads_or(refused)) zero_rows<THREADS, D>(p.out, p.nq, L.ent, p.n);
    if (p.row_tiles > 1) {
        for (int i = warp; i < p.n; i += THREADS / 32) {
            const int4 e = L.ent[i];
            const int T = L.row_tiles(i);
            long long x = 0;
            for (int t = lane; t < T; t += 32) x += L.span(e, t).nt + ovh;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
            if (lane == 0) L.pre[i] = (int)min(x * p.nkv, 0x7fffffffll);
        }
        __syncthreads();
    }
    long long run = 0;
    for (int base = 0; base < p.n; base += THREADS) {
        const int i = base + tid;
        const long long x = i < p.n ? L.pre[i] : 0;
        long long inc = x;
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
        if (i < p.n) L.pre[i] = (int)min(before + inc - x, 0x7fffffffll);
        __syncthreads();
    }
    if (tid == 0) L.pre[p.n] = (int)min(run, 0x7fffffffll);
    __syncthreads();
    if (run >= 0x7fffffffll && tid == 0 && p.wait_status) set_error(p.wait_status, DFLASH_UNSUPPORTED);
    return run < 0x7fffffffll ? (int)run : 0;
}

// A CTA's stretch of one item: key tiles [t0, t1) of span.nt for rows [r0, r1) of entry i.
struct Stretch {
    int i, g, r0, r1, t0, t1;
    KeySpan span;
    int v0;             // the item's first unit
    DF_DEV bool whole() const { return t0 == 0 && t1 == span.nt; }
};
// TILES: entries may have several row tiles.
template <bool TILES> struct Walker {
    int v, end;         // units still to come
    int i, t, g, off;   // item and units of it that lie before v
    int T;              // row tiles of entry i

    // The calling warp as a whole; v < end <= U.
    DF_DEV void start(const Line& L, int begin, int end_) {
        v = begin;
        end = end_;
        const int lane = threadIdx.x & 31;
        if (L.n <= 32) {      // entries without units share their start: the last that starts at or before v
            const int x = lane < L.n ? L.pre[lane] : 0x7fffffff;
            i = 31 - __clz(__ballot_sync(0xffffffffu, x <= v));
        } else {
            int lo = 0;
            for (int hi = L.n; hi - lo > 1;) {
                const int mid = (lo + hi) >> 1;
                if (L.pre[mid] <= v) lo = mid;
                else hi = mid;
            }
            i = lo;
            while (L.pre[i + 1] <= v) ++i;
        }
        int local = v - L.pre[i];
        const int4 e = L.ent[i];
        t = 0;
        T = 1;
        int size;
        if constexpr (!TILES) {
            size = (L.pre[i + 1] - L.pre[i]) / L.nkv;
        } else {
            T = L.row_tiles(i);
            size = L.span(e, 0).nt + L.ovh;
        }
        if (TILES && T > 1) {
            for (int tb = 0;; tb += 32) {
                const int tt = tb + lane;
                const int sz = tt < T ? L.span(e, tt).nt + L.ovh : 0;
                int inc = sz * L.nkv;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int u = __shfl_up_sync(0xffffffffu, inc, o);
                    if (lane >= o) inc += u;
                }
                const unsigned m = __ballot_sync(0xffffffffu, inc > local);
                if (m) {
                    const int src = __ffs(m) - 1;
                    t = tb + src;
                    size = __shfl_sync(0xffffffffu, sz, src);
                    local -= __shfl_sync(0xffffffffu, inc, src) - size * L.nkv;
                    break;
                }
                local -= __shfl_sync(0xffffffffu, inc, 31);
            }
        }
        g = local / size;
        off = local - g * size;
    }
    // The next stretch with tiles; false when the share is done.
    DF_DEV bool next(const Line& L, Stretch& s) {
        while (v < end) {
            const int4 e = L.ent[i];
            s.r0 = TILES ? t * L.rt : 0;
            s.r1 = TILES ? min(e.z, s.r0 + L.rt) : e.z;
            s.span = key_span(e.w, e.z, s.r0, s.r1, L.causal, L.window, L.sinks, kLineTile);
            const int size = s.span.nt + L.ovh;
            const int take = min(size - off, end - v);
            s.i = i;
            s.g = g;
            s.t0 = max(0, off - L.ovh);
            s.t1 = max(0, off + take - L.ovh);
            s.v0 = v - off;
            v += take;
            off += take;
            if (off == size) {
                off = 0;
                if (++g == L.nkv) {
                    g = 0;
                    if (!TILES || ++t >= T) {
                        t = 0;
                        while (++i < L.n && L.ent[i].z == 0) {}
                        if (TILES && i < L.n) T = L.row_tiles(i);
                    }
                }
            }
            if (s.t1 > s.t0) return true;
        }
        return false;
    }
};

// Bounded wait on an mbarrier phase by a converged warp, as mbar_wait, for waits that are short and
// many: a try may suspend the warp for up to 20 us (a warp that spins takes issue slots from the
// softmax warps beside it), the clock is first read after 32 of them, and the lanes leave together,
// by branches on votes only (lanes that leave one by one cost 100 cycles and more of reconvergence).
DF_DEV bool mbar_wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* status) {
    uint64_t t0 = 0;
    for (uint32_t it = 1;; ++it) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_u32(bar)), "r"(parity), "r"(20000u)
            : "memory");
        if (__all_sync(0xffffffffu, ok)) return true;
        if ((it & 31u) == 0) {
            if (__any_sync(0xffffffffu, *abort_flag)) return false;
            const uint64_t now = globaltimer_ns();
            if (t0 == 0) t0 = now;
            if (__any_sync(0xffffffffu, now - t0 > kWaitLimitNs)) {
                *abort_flag = 1;
                if (status) atomicCAS(status, 0, DFLASH_TIMEOUT);
                return false;
            }
        }
    }
}
DF_DEV int atom_add_acq_rel(int* p, int v) {
    int old;
    asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
    return old;
}
// 2^x for an integer x <= 0 (0 below -126), exactly; bases differ by integers.
DF_DEV float pow2_int(float x) { return __int_as_float(((int)fmaxf(x, -127.f) + 127) << 23); }
// Arrive without a branch.
DF_DEV void mbar_arrive_if(bool pred, uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}"
        ::"r"(smem_u32(bar)), "r"((uint32_t)pred)
        : "memory");
}
// Pairs of fp32 operations in one instruction, and the maximum of three.
DF_DEV float2 fma_x2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, c, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\t"
        "mov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
DF_DEV float2 add_x2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 d, a, b;\n\t"
        "mov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
DF_DEV float fmax3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
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
// 32 lanes x 64 consecutive 32-bit columns of tensor memory, waited for in the same statement.
DF_DEV void tmem_ld64w(uint32_t taddr, float* v) {
    uint32_t r[64];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%64];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 64; ++i) v[i] = __uint_as_float(r[i]);
}
// The shares of P CTAs of a line of U units: CTA c has the units [c U / P, (c+1) U / P).  In 32 bits
// (with 64-bit divisions each call took 0.1 us longer): with U = q P + r the share
// starts at c q + floor(c r / P), and c r stays below 160^2, where fp32 gives the floor exactly (the
// quotient's distance from an integer is 0.5 / P at least, once 0.5 is added to c r).
struct Shares {
    int q, r, P;
    float inv, per;
    DF_DEV Shares(int U, int P_) : P(P_) {
        q = U / P;
        r = U - q * P;
        inv = 1.0f / (float)P;
        per = (float)P / (float)U;
    }
    DF_DEV int begin(int c) const { return c * q + (int)(((float)(c * r) + 0.5f) * inv); }
    // CTA that holds unit u: the estimate is off by one at most
    DF_DEV int owner(int u) const {
        int c = min((int)((float)u * per), P - 1);
        if (begin(c) > u) --c;
        if (begin(c + 1) <= u) ++c;
        return c;
    }
};

// The pages of a sequence, looked up 32 at a time by a whole warp.
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
// What its joins of `rows` query rows per kv head write to shared memory, and the room for it: (base,
// sum) pairs, their room, floats of O, their room.  False: no such shape.
bool paged_decode_join_room(int d, int rows, int* room);
// Any number of rows (paged_block.cu).
int launch_paged_block(PagedAttnParams& p, int d, int num_sms, cudaStream_t st);
int launch_paged_attn_f32(PagedAttnParams& p, int d, int num_sms, cudaStream_t st);
int launch_paged_attn_bf16(PagedAttnParams& p, int d, int num_sms, cudaStream_t st);

}  // namespace df
