// Operations on the pages of a key/value pool: growing with copy on write,
// forking, freeing, compacting, and moving rows in and out.
//
// Tables, counts and lengths live in device memory and every operation is a fixed
// sequence of launches, so that a captured cycle can grow and fork sequences whose
// lengths only the device knows.  The planning kernels are one block: a call lists
// at most 1024 sequences and usually a handful of pages, and what has to be ordered
// (free pages ascending, served in list order) is a prefix sum over the block.  The
// page data is moved by separate kernels that spread over the device.
//
// The plans are bound by latency: a chain of launches and of dependent reads (list, length, table,
// count).  32 sequences, in a captured graph: free 2.0 us, shared fork 2.8, reserve 4.8 with nothing
// new (its copy launch included), 6.7 with two new pages each, write of one row each 2.9, advance 1.
// Moving pages is bound by HBM, see there.
#include "paged.cuh"

namespace df {

namespace {

constexpr int kPlan = 1024;   // threads of a planning block
constexpr int kCopyWarps = 8;

// Exclusive prefix sum of one int per thread over the block; total in *total.
// sums: 33 ints of shared memory.  Ends with a barrier after which sums may be reused.
DF_DEV int block_scan(int v, int* sums, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    int inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += u;
    }
    if (lane == 31) sums[warp] = inc;
    __syncthreads();
    if (warp == 0) {
        int s = lane < nw ? sums[lane] : 0;
        int si = s;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, si, o);
            if (lane >= o) si += u;
        }
        sums[lane] = si - s;
        if (lane == 31) sums[32] = si;
    }
    __syncthreads();
    const int r = sums[warp] + inc - v;
    *total = sums[32];
    __syncthreads();
    return r;
}

// The lowest-numbered free pages (count 0), in order, into out[0..want): how many
// there are, at most want.  The whole block takes part.
DF_DEV int find_free(const PoolView& v, int want, int* out, int* sums) {
    int found = 0;
    for (int base = 0; base < v.n_pages && found < want; base += kPlan * 4) {
        const int id0 = base + threadIdx.x * 4;
        bool f[4];
        int c = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            f[k] = id0 + k < v.n_pages && v.refs[id0 + k] == 0;
            c += f[k];
        }
        int total;
        int at = found + block_scan(c, sums, &total);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (f[k]) {
                if (at < want) out[at] = id0 + k;
                ++at;
            }
        found += total;
    }
    return found < want ? found : want;
}

// Sequence of entry i: -1 for padding, -2 for an id that does not exist.
DF_DEV int entry_seq(const PoolView& v, const int* seqs, int i) {
    const int s = seqs ? seqs[i] : i;
    if (s == -1) return -1;
    return s >= 0 && s < v.max_seqs ? s : -2;
}
// Whether entry i's sequence stands earlier in the list (the calling threads share the search).
// partner: the other list of a pair, or null; beside a -1 there a sequence is not listed.
DF_DEV bool listed_before(const int* seqs, const int* partner, int i, int s, int first, int step) {
    bool d = false;
    if (seqs)
        for (int j = first; j < i; j += step) d |= seqs[j] == s && !(partner && partner[j] == -1);
    return d;
}

DF_DEV int pages_for(long long positions, int ps_log2) {
    return (int)((positions + (1 << ps_log2) - 1) >> ps_log2);
}

// ---------------------------------------------------------------------------
// reserve, deep fork: plan
// ---------------------------------------------------------------------------
// Entry i wants the table indices [first, past) of its sequence (`sid`).  reserve: an index needs a
// new page when it has none, or when others hold its page too, but for one case: when all holders
// of a page are entries of this call that write it, the last of them keeps it.  So per shared page
// the writers are counted and the last is found: two atomics an index (128 forks of one page, all
// reserved at once: 16 us, against 77 with every entry searching the ones before it; 1023: 89,
// against 6900).  deep fork: every index needs one.
// Decisions are made twice (counted, then written) from the same tables, which stay as they are
// until all are made: no list of candidates has to fit anywhere.
template <bool FORK>
__global__ void __launch_bounds__(kPlan) k_pages_plan(PoolView v, const int* __restrict__ seqs,
                                                      const int* __restrict__ grow, const int* __restrict__ src, int n) {
    __shared__ int sid[kPoolMaxSeqs], first[kPoolMaxSeqs], past[kPoolMaxSeqs], cnt[kPoolMaxSeqs];
    __shared__ int owner[kPoolMaxSeqs];      // the first entry that lists a sequence
    __shared__ int sums[33];
    griddep_wait();
    griddep_launch();
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    if (t == 0) *v.n_copies = 0;
    owner[t] = kPlan;
    __syncthreads();
    if (t < n) {
        const int s = FORK && src[t] == -1 ? -1 : entry_seq(v, seqs, t);
        sid[t] = s;
        first[t] = past[t] = 0;
        if (s >= 0) atomicMin(&owner[s], t);
    }
    __syncthreads();
    if (t < n) {
        const int s = sid[t];
        int err = 0;
        if (s == -2) {
            err = DFLASH_INVALID_ARG;
        } else if (s >= 0) {
            if (owner[s] < t) err = DFLASH_INVALID_ARG;
            if (FORK) {
                const int a = src[t];
                if (a < 0 || a >= v.max_seqs) {
                    err = DFLASH_INVALID_ARG;
                } else {
                    for (int j = 0; j < n; ++j)
                        if (src[j] == s) err = DFLASH_INVALID_ARG;   // a destination that is a source too
                    if (!err && (v.len[s] != 0 || v.table[(size_t)s * v.max_pages] >= 0)) err = DFLASH_STATE;
                    if (!err) past[t] = pages_for(v.len[a], v.ps_log2);
                }
            } else if (!err) {
                const int g = grow[t];
                const long long ln = v.len[s];
                if (g < 0) err = DFLASH_INVALID_ARG;
                else if (ln + g > v.max_len) err = DFLASH_CAPACITY;
                else if (g > 0) {
                    first[t] = (int)(ln >> v.ps_log2);
                    past[t] = pages_for(ln + g, v.ps_log2);
                }
            }
        }
        if (err) {
            set_error(v.status, err);
            first[t] = past[t] = 0;
        }
    }
    __syncthreads();

    // (writers, last writer) of the shared pages stand in v.copies until the decisions are made
    auto needs_new = [&](int i, int c) -> bool {
        if (FORK) return true;
        const int x = v.table[(size_t)sid[i] * v.max_pages + c];
        if (x < 0) return true;
        const int holders = v.refs[x];
        if (holders <= 1) return false;
        return !(__ldcg(&v.copies[x].x) == holders && __ldcg(&v.copies[x].y) == i);
    };
    if (!FORK) {
        bool shared = false;
        for (int i = warp; i < n; i += kPlan / 32)
            for (int c = first[i] + lane; c < past[i]; c += 32) {
                const int x = v.table[(size_t)sid[i] * v.max_pages + c];
                if (x >= 0 && v.refs[x] > 1) {
                    shared = true;
                    v.copies[x] = make_int4(0, -1, 0, 0);
                }
            }
        if (__syncthreads_or(shared)) {
            for (int i = warp; i < n; i += kPlan / 32)
                for (int c = first[i] + lane; c < past[i]; c += 32) {
                    const int x = v.table[(size_t)sid[i] * v.max_pages + c];
                    if (x >= 0 && v.refs[x] > 1) {
                        atomicAdd(&v.copies[x].x, 1);
                        atomicMax(&v.copies[x].y, i);
                    }
                }
            __syncthreads();
        }
    }
    for (int i = warp; i < n; i += kPlan / 32) {
        int total = 0;
        for (int c0 = first[i]; c0 < past[i]; c0 += 32)
            total += __popc(__ballot_sync(0xffffffffu, c0 + lane < past[i] && needs_new(i, c0 + lane)));
        if (lane == 0) cnt[i] = total;
    }
    __syncthreads();
    int total;
    const int off = block_scan(t < n ? cnt[t] : 0, sums, &total);
    if (t < n) cnt[t] = off;
    if (total == 0) {
        // a deep fork of empty sequences has nothing to allocate, and their length is 0
        return;
    }
    const bool fits = total <= v.n_pages && find_free(v, total, v.freelist, sums) == total;
    if (!fits) {
        if (t == 0) set_error(v.status, DFLASH_CAPACITY);
        return;
    }
    __syncthreads();
    // planned entries, in order; the tables stay as they are until all decisions are made
    for (int i = warp; i < n; i += kPlan / 32) {
        int at = cnt[i];
        for (int c0 = first[i]; c0 < past[i]; c0 += 32) {
            const int c = c0 + lane;
            const bool nw = c < past[i] && needs_new(i, c);
            const unsigned m = __ballot_sync(0xffffffffu, nw);
            if (nw) {
                const int j = at + __popc(m & ((1u << lane) - 1));
                const int old = FORK ? v.table[(size_t)src[i] * v.max_pages + c]
                                     : v.table[(size_t)sid[i] * v.max_pages + c];
                v.recs[j] = make_int4(i, c, old, v.freelist[j]);
            }
            at += __popc(m);
        }
    }
    __syncthreads();
    for (int j = t; j < total; j += kPlan) {
        const int4 r = v.recs[j];
        const int s = sid[r.x];
        v.table[(size_t)s * v.max_pages + r.y] = r.w;
        v.refs[r.w] = 1;
        int rows = 0;
        if (FORK) {
            rows = v.ps;
            if (r.y == 0) v.len[s] = v.len[src[r.x]];
        } else if (r.z >= 0) {
            atomicSub(&v.refs[r.z], 1);
            if (r.y == first[r.x]) rows = v.len[s] & (v.ps - 1);
        }
        if (rows > 0) {
            const int k = atomicAdd(v.n_copies, 1);   // the order of the copies does not matter
            v.copies[k] = make_int4(r.z, r.w, rows, 0);
        }
    }
}

// ---------------------------------------------------------------------------
// Copies of pages
// ---------------------------------------------------------------------------
// Bound by HBM: every byte is read once and written once.
//
// Parts of pages (copy on write).  Unit: up to 4 KB of one (layer, kind, head) run of one
// copied page, one warp, its eight 16-byte loads per lane issued before the first store.
__global__ void __launch_bounds__(kCopyWarps * 32) k_pages_copy(PoolView v) {
    griddep_wait();
    griddep_launch();
    const int nc = *v.n_copies;
    const int runs = v.n_layers * 2 * v.nkv;
    const int run_bytes = v.ps * v.row_bytes;
    const int subs = (run_bytes + 4095) >> 12;
    const int lane = threadIdx.x & 31;
    const long long warps = (long long)gridDim.x * kCopyWarps;
    const long long units = (long long)nc * runs * subs;
    for (long long u = (long long)blockIdx.x * kCopyWarps + (threadIdx.x >> 5); u < units; u += warps) {
        const int c = (int)(u / (runs * subs)), rem = (int)(u % (runs * subs));
        const int4 rec = v.copies[c];
        const int run = rem / subs, b0 = (rem % subs) << 12;
        const int bytes = rec.z * v.row_bytes - b0;     // of this run past b0
        if (bytes <= 0) continue;
        const size_t o = (size_t)run * run_bytes + b0;
        const uint4* a = reinterpret_cast<const uint4*>(v.slab + (size_t)rec.x * v.page_bytes + o);
        uint4* b = reinterpret_cast<uint4*>(v.slab + (size_t)rec.y * v.page_bytes + o);
        const int nv = min(bytes, 4096) >> 4;
        uint4 r[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (lane + 32 * k < nv) r[k] = __ldcs(a + lane + 32 * k);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (lane + 32 * k < nv) __stcs(b + lane + 32 * k, r[k]);
    }
}

// Whole pages (deep fork, compact): one warp per SM keeps kBulkStages chunks of 32 KB in flight
// through shared memory with bulk copies, in and out; no registers, no address arithmetic
// beside one record per chunk.  32 contexts of 2048 positions, 5 layers, 8 heads of 128 (2.7 GB read
// and written): 435 us, 6.2 TB/s, 95 % of a copy; the warp-per-4-KB kernel above on the same kind of
// pages reached 79 %.  (That one stays for copy on write, whose rows end inside every run.)
constexpr int kBulkStages = 6, kBulkChunk = 32768;
__global__ void __launch_bounds__(32) k_pages_copy_whole(PoolView v) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = smem_align_up<uint8_t>(smem_raw, 128);
    __shared__ uint64_t full[kBulkStages];
    __shared__ int abort_s;
    griddep_wait();
    griddep_launch();
    if (threadIdx.x != 0) return;
    abort_s = 0;
    for (int i = 0; i < kBulkStages; ++i) mbar_init(&full[i], 1);
    fence_mbar_init();
    const int cpp = (int)((v.page_bytes + kBulkChunk - 1) / kBulkChunk);      // chunks of a page
    const long long chunks = (long long)*v.n_copies * cpp;
    const long long mine = chunks > blockIdx.x ? (chunks - blockIdx.x + gridDim.x - 1) / gridDim.x : 0;
    const uint64_t once = make_l2_policy_evict_first();
    auto place = [&](long long i, size_t& from, size_t& to) -> uint32_t {
        const long long u = blockIdx.x + i * gridDim.x;
        const int4 rec = v.copies[u / cpp];
        const long long o = (u % cpp) * kBulkChunk;
        from = (size_t)rec.x * v.page_bytes + o;
        to = (size_t)rec.y * v.page_bytes + o;
        return (uint32_t)min((long long)kBulkChunk, v.page_bytes - o);
    };
    auto load = [&](long long i) {
        size_t from, to;
        const uint32_t n = place(i, from, to);
        const int st = (int)(i % kBulkStages);
        mbar_arrive_expect_tx(&full[st], n);
        asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;"
                     ::"r"(smem_u32(ring + st * kBulkChunk)), "l"((uint64_t)(v.slab + from)), "r"(n), "r"(smem_u32(&full[st])),
                       "l"(once)
                     : "memory");
    };
    long long loaded = 0;
    while (loaded < kBulkStages && loaded < mine) load(loaded++);
    for (long long i = 0; i < mine; ++i) {
        const int st = (int)(i % kBulkStages);
        if (!mbar_wait(&full[st], (uint32_t)((i / kBulkStages) & 1), &abort_s, v.status)) break;
        size_t from, to;
        const uint32_t n = place(i, from, to);
        asm volatile("cp.async.bulk.global.shared::cta.bulk_group.L2::cache_hint [%0], [%1], %2, %3;"
                     ::"l"((uint64_t)(v.slab + to)), "r"(smem_u32(ring + st * kBulkChunk)), "r"(n), "l"(once) : "memory");
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        if (i >= 1 && loaded < mine) {
            // the stage of the chunk before is free once its store has read it
            asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
            load(loaded++);
        }
    }
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    if (abort_s) {      // copies in land before the block exits
        volatile int never = 0;
        for (long long k = loaded < kBulkStages ? 0 : loaded - kBulkStages; k < loaded; ++k)
            mbar_wait(&full[k % kBulkStages], (uint32_t)((k / kBulkStages) & 1), &never, nullptr);
    }
}

// ---------------------------------------------------------------------------
// fork (shared), free
// ---------------------------------------------------------------------------
__global__ void k_pages_fork(PoolView v, const int* __restrict__ src, const int* __restrict__ dst) {
    griddep_wait();
    griddep_launch();
    const int i = blockIdx.x, t = threadIdx.x, n = gridDim.x;
    const int d = entry_seq(v, dst, i), a = src[i];
    if (d == -1 || a == -1) return;
    bool bad = d == -2 || a < 0 || a >= v.max_seqs;
    bad |= listed_before(dst, src, i, d, t, blockDim.x);
    for (int j = t; j < n; j += blockDim.x) bad |= src[j] == d;
    if (__syncthreads_or(bad)) {
        if (t == 0) set_error(v.status, DFLASH_INVALID_ARG);
        return;
    }
    int* to = v.table + (size_t)d * v.max_pages;
    const bool full = v.len[d] != 0 || to[0] >= 0;
    if (__syncthreads_or(full)) {          // read before any thread writes
        if (t == 0) set_error(v.status, DFLASH_STATE);
        return;
    }
    const int ln = v.len[a], np = pages_for(ln, v.ps_log2);
    const int* from = v.table + (size_t)a * v.max_pages;
    for (int c = t; c < np; c += blockDim.x) {
        const int x = from[c];
        to[c] = x;
        atomicAdd(&v.refs[x], 1);
    }
    if (t == 0) v.len[d] = ln;
}

__global__ void k_pages_free(PoolView v, const int* __restrict__ seqs, const int* __restrict__ keep) {
    griddep_wait();
    griddep_launch();
    const int i = blockIdx.x, t = threadIdx.x;
    const int s = entry_seq(v, seqs, i);
    if (s == -1) return;
    bool bad = s == -2 || listed_before(seqs, nullptr, i, s, t, blockDim.x);
    const int k = keep ? keep[i] : 0;
    if (!bad) bad = k < 0 || k > v.len[s];
    if (__syncthreads_or(bad)) {           // len is read before it is written below
        if (t == 0) set_error(v.status, DFLASH_INVALID_ARG);
        return;
    }
    int* row = v.table + (size_t)s * v.max_pages;
    // entries are a prefix: a stretch of blockDim.x indices without a page ends it
    for (int c0 = pages_for(k, v.ps_log2); c0 < v.max_pages; c0 += blockDim.x) {
        const int c = c0 + t;
        const int x = c < v.max_pages ? row[c] : -1;
        if (x >= 0) {
            atomicSub(&v.refs[x], 1);
            row[c] = -1;
        }
        if (!__syncthreads_or(x >= 0)) break;
    }
    if (t == 0) v.len[s] = k;
}

// ---------------------------------------------------------------------------
// compact
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kPlan) k_pages_compact(PoolView v, int* __restrict__ used_out, int remap) {
    __shared__ int sums[33];
    griddep_wait();
    griddep_launch();
    const int t = threadIdx.x;
    int mine = 0;
    for (int i = t; i < v.n_pages; i += kPlan) mine += v.refs[i] > 0;
    int used;
    block_scan(mine, sums, &used);
    // holes below `used` and pages in use from `used` on: equally many
    int holes = 0, moves = 0;
    for (int base = 0; base < v.n_pages; base += kPlan * 4) {
        const int id0 = base + t * 4;
        bool f[4];
        int ch = 0, cm = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int id = id0 + k;
            const bool in = id < v.n_pages, u = in && v.refs[id] > 0;
            f[k] = in && (id < used ? !u : u);
            if (f[k]) {
                if (id < used) ++ch;
                else ++cm;
            }
        }
        // both counts in one scan: at most 4096 of each per stretch
        int total;
        const int both = block_scan(ch | (cm << 16), sums, &total);
        int ah = holes + (both & 0xffff), am = moves + (both >> 16);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (f[k]) {
                if (id0 + k < used) v.freelist[ah++] = id0 + k;
                else v.recs[am++].x = id0 + k;
            }
        holes += total & 0xffff;
        moves += total >> 16;
    }
    __syncthreads();
    for (int j = t; j < moves; j += kPlan) {
        const int from = v.recs[j].x, to = v.freelist[j];
        v.movers[from] = to;
        v.refs[to] = v.refs[from];
        v.refs[from] = 0;
        v.copies[j] = make_int4(from, to, v.ps, 0);
    }
    if (t == 0) {
        v.n_copies[0] = moves;
        v.n_copies[1] = used;
        *used_out = used;
    }
    if (!remap || moves == 0) return;
    __syncthreads();
    for (int e = t; e < v.max_seqs * v.max_pages; e += kPlan) {
        const int x = v.table[e];
        if (x >= used) v.table[e] = v.movers[x];
    }
}

__global__ void k_pages_remap(PoolView v) {
    griddep_wait();
    griddep_launch();
    if (v.n_copies[0] == 0) return;
    const int used = v.n_copies[1];
    const size_t n = (size_t)v.max_seqs * v.max_pages;
    for (size_t e = (size_t)blockIdx.x * blockDim.x + threadIdx.x; e < n; e += (size_t)gridDim.x * blockDim.x) {
        const int x = v.table[e];
        if (x >= used) v.table[e] = v.movers[x];
    }
}

// ---------------------------------------------------------------------------
// set_tables
// ---------------------------------------------------------------------------
__global__ void k_tables_begin(PoolView v) {
    griddep_wait();
    griddep_launch();
    for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < v.n_pages; i += gridDim.x * blockDim.x) {
        v.refs[i] = 0;
        v.movers[i] = -1;      // the index a page stands at
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) v.n_copies[2] = 0;
}
// Whether table entry e can stand; counts its page.
DF_DEV bool count_entry(const PoolView& v, const int* lens, const int* table, size_t e) {
    const int s = (int)(e / v.max_pages), c = (int)(e % v.max_pages);
    const int ln = lens[s], x = table[e];
    if (ln < 0 || ln > v.max_len || x < -1 || x >= v.n_pages) return false;
    if (x < 0) return c >= pages_for(ln, v.ps_log2);
    if (c > 0 && table[e - 1] < 0) return false;
    const int at = atomicCAS(&v.movers[x], -1, c);
    atomicAdd(&v.refs[x], 1);
    return at == -1 || at == c;
}
__global__ void k_tables_count(PoolView v, const int* lens, const int* table) {
    griddep_wait();
    griddep_launch();
    const size_t n = (size_t)v.max_seqs * v.max_pages;
    bool bad = false;
    for (size_t e = (size_t)blockIdx.x * blockDim.x + threadIdx.x; e < n; e += (size_t)gridDim.x * blockDim.x)
        bad |= !count_entry(v, lens, table, e);
    if (bad) v.n_copies[2] = 1;
}
__global__ void k_tables_apply(PoolView v, const int* lens, const int* table) {
    griddep_wait();
    griddep_launch();
    const bool bad = v.n_copies[2] != 0;
    const size_t n = (size_t)v.max_seqs * v.max_pages;
    const size_t t = (size_t)blockIdx.x * blockDim.x + threadIdx.x, step = (size_t)gridDim.x * blockDim.x;
    for (size_t e = t; e < n; e += step) v.table[e] = bad ? -1 : table[e];
    for (size_t s = t; s < (size_t)v.max_seqs; s += step) v.len[s] = bad ? 0 : lens[s];
    if (bad) {
        for (size_t i = t; i < (size_t)v.n_pages; i += step) v.refs[i] = 0;
        if (t == 0) set_error(v.status, DFLASH_INVALID_ARG);
    }
}

// The three steps in one block, for tables that it goes through faster than two more launches
// take (1024 entries: 2.7 us against 3.5 on the device; 2048: 3.8 both; 4096: 5.5 against 4.0, which
// the host pays for with two more launches; 8192: 9.5).
constexpr int kSmallTables = 4096;
__global__ void __launch_bounds__(kPlan) k_tables_small(PoolView v, const int* lens, const int* table) {
    griddep_wait();
    griddep_launch();
    const int t = threadIdx.x, n = v.max_seqs * v.max_pages;
    for (int i = t; i < v.n_pages; i += kPlan) {
        v.refs[i] = 0;
        v.movers[i] = -1;
    }
    __syncthreads();
    bool bad = false;
    for (int e = t; e < n; e += kPlan) bad |= !count_entry(v, lens, table, e);
    bad = __syncthreads_or(bad);
    for (int e = t; e < n; e += kPlan) v.table[e] = bad ? -1 : table[e];
    if (t < v.max_seqs) v.len[t] = bad ? 0 : lens[t];
    if (bad) {
        for (int i = t; i < v.n_pages; i += kPlan) v.refs[i] = 0;
        if (t == 0) set_error(v.status, DFLASH_INVALID_ARG);
    }
}

// ---------------------------------------------------------------------------
// write, advance, store, load
// ---------------------------------------------------------------------------
// Whether the positions [from, to) of sequence s have pages that only s holds
// (0, or the error).  The threads of the block share the look.
DF_DEV int writable(const PoolView& v, int s, long long from, long long to) {
    int err = 0;
    if (to > v.max_len) {
        err = DFLASH_CAPACITY;
    } else {
        const int* row = v.table + (size_t)s * v.max_pages;
        const int c1 = pages_for(to, v.ps_log2);
        for (int c = (int)(from >> v.ps_log2) + threadIdx.x; c < c1; c += blockDim.x) {
            const int x = row[c];
            if (x < 0) err = DFLASH_CAPACITY;
            else if (v.refs[x] > 1 && !err) err = DFLASH_STATE;
        }
    }
    if (__syncthreads_or(err == DFLASH_CAPACITY)) return DFLASH_CAPACITY;
    return __syncthreads_or(err) ? DFLASH_STATE : 0;
}

// Block (x, i): rows x * kWriteRows.. of entry i.  Each block looks at the entry's pages itself (a
// launch for the checks alone would cost as much as the writing).  2048 rows of 8 heads of 128 to one
// sequence: 7.9 us (16.8 MB).
constexpr int kWriteRows = 4;
__global__ void __launch_bounds__(256) k_pages_write(PoolView v, const int* __restrict__ seqs, int layer,
                                                     const uint8_t* __restrict__ k, const uint8_t* __restrict__ vv,
                                                     long long stride, const int* __restrict__ row_start,
                                                     const int* __restrict__ row_count, int total_rows, int max_rows) {
    griddep_wait();
    griddep_launch();
    const int i = blockIdx.y, t = threadIdx.x;
    const int s = entry_seq(v, seqs, i);
    const int start = row_start ? row_start[i] : i, count = row_start ? row_count[i] : 1;
    if (s == -1 || count == 0) return;
    bool bad = s == -2 || count < 0 || count > max_rows || start < 0 || start > total_rows - count;
    bad |= listed_before(seqs, nullptr, i, s, t, blockDim.x);
    if (__syncthreads_or(bad)) {
        if (t == 0) set_error(v.status, DFLASH_INVALID_ARG);
        return;
    }
    const int r0 = blockIdx.x * kWriteRows;
    if (r0 >= count) return;
    const long long ln = v.len[s];
    const int err = writable(v, s, ln, ln + count);
    if (err) {
        if (t == 0) set_error(v.status, err);
        return;
    }
    const int hv = v.row_bytes >> 4, rv = v.nkv * hv;        // 16-byte pieces of a head's row, of a row
    const int rows = min(kWriteRows, count - r0);
    for (int e = t; e < rows * 2 * rv; e += blockDim.x) {
        const int r = e / (2 * rv), rem = e % (2 * rv), kind = rem / rv, w = rem % rv;
        const long long pos = ln + r0 + r;
        const int page = v.table[(size_t)s * v.max_pages + (pos >> v.ps_log2)];
        const uint8_t* from = (kind ? vv : k) + (size_t)(start + r0 + r) * stride + (size_t)w * 16;
        uint8_t* to = v.slab + (size_t)page * v.page_bytes +
                      (((size_t)layer * 2 + kind) * v.nkv + w / hv) * ((size_t)v.ps * v.row_bytes) +
                      (size_t)(pos & (v.ps - 1)) * v.row_bytes + (size_t)(w % hv) * 16;
        *reinterpret_cast<uint4*>(to) = *reinterpret_cast<const uint4*>(from);
    }
}

__global__ void __launch_bounds__(kPlan) k_pages_advance(PoolView v, const int* __restrict__ seqs,
                                                         const int* __restrict__ row_count, int n) {
    griddep_wait();
    griddep_launch();
    __shared__ int owner[kPoolMaxSeqs];      // the first entry that lists a sequence
    const int t = threadIdx.x;
    owner[t] = kPlan;
    __syncthreads();
    const int s = t < n ? entry_seq(v, seqs, t) : -1;
    if (s >= 0) atomicMin(&owner[s], t);
    __syncthreads();
    if (s == -1) return;
    const int c = row_count ? row_count[t] : 1;
    int err = 0;
    if (s == -2 || c < 0 || owner[s] < t) {
        err = DFLASH_INVALID_ARG;
    } else if (c > 0) {
        const long long to = (long long)v.len[s] + c;
        if (to > v.max_len || v.table[(size_t)s * v.max_pages + ((to - 1) >> v.ps_log2)] < 0) err = DFLASH_CAPACITY;
        else v.len[s] = (int)to;
    }
    if (err) set_error(v.status, err);
}

// store / load, step 1: what entry i copies, as recs[i] = (sequence, request, from, to).
__global__ void k_exchange_plan(PoolView v, const int* __restrict__ seqs, SlabView c, const int* __restrict__ reqs,
                                int load) {
    griddep_wait();
    griddep_launch();
    const int i = blockIdx.x, t = threadIdx.x;
    const int s = entry_seq(v, seqs, i), b = reqs ? reqs[i] : i;
    if (t == 0) v.recs[i] = make_int4(s, b, 0, 0);
    if (s == -1 || b == -1) return;
    bool bad = s == -2 || b < 0 || b >= c.batch;
    bad |= load ? listed_before(reqs, seqs, i, b, t, blockDim.x) : listed_before(seqs, reqs, i, s, t, blockDim.x);
    if (__syncthreads_or(bad)) {
        if (t == 0) set_error(v.status, DFLASH_INVALID_ARG);
        return;
    }
    const int from = load ? c.len[b] : v.len[s], to = load ? v.len[s] : c.len[b];
    if (to <= from) return;
    int err = 0;
    if (load) err = to > c.capacity ? DFLASH_CAPACITY : 0;
    else err = writable(v, s, from, to);
    if (t == 0) {
        if (err) set_error(v.status, err);
        else v.recs[i] = make_int4(s, b, from, to);
    }
}
// Step 2: bound by HBM, every byte read once and written once.  A run of positions of one (layer, kind,
// head) is contiguous in a page and in the cache, so it moves as bulk copies through shared memory
// (chunks of at most 16 KB and one page, 2^lp positions), kExStages of them in flight; two
// one-warp blocks on an SM.  Lanes look the addresses of 32 chunks up together.  (A warp per 4 KB
// through registers: 5.2 TB/s at 32 contexts of 2048 of 5 layers and 8 heads of 128.)
constexpr int kExStages = 6, kExChunk = 16384;
__global__ void __launch_bounds__(32) k_exchange_copy(PoolView v, SlabView c, int load, int lp) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = smem_align_up<uint8_t>(smem_raw, 128);
    __shared__ uint64_t full[kExStages];
    __shared__ uint8_t *from_s[64], *to_s[64];
    __shared__ uint32_t bytes_s[64];
    __shared__ int abort_s;
    griddep_wait();
    griddep_launch();
    const int4 r = v.recs[blockIdx.y];
    if (r.w <= r.z) return;
    const int lane = threadIdx.x;
    const int u0 = r.z >> lp, nb = ((r.w + (1 << lp) - 1) >> lp) - u0;
    const long long units = (long long)nb * v.n_layers * 2 * v.nkv;
    const long long mine = units > blockIdx.x ? (units - blockIdx.x + gridDim.x - 1) / gridDim.x : 0;
    if (mine == 0) return;
    if (lane == 0) {
        abort_s = 0;
        for (int i = 0; i < kExStages; ++i) mbar_init(&full[i], 1);
        fence_mbar_init();
    }
    const uint64_t once = make_l2_policy_evict_first();
    auto issue = [&](long long i) {       // the load of this block's chunk i
        if ((i & 31) == 0) {
            if (i + lane < mine) {
                const long long u = blockIdx.x + (i + lane) * gridDim.x;
                const int run = (int)(u / nb), blk = u0 + (int)(u % nb);
                const int g = run % v.nkv, kind = run / v.nkv % 2, layer = run / v.nkv / 2;
                const int p0 = max(r.z, blk << lp), p1 = min((long long)r.w, (long long)(blk + 1) << lp);
                const int page = v.table[(size_t)r.x * v.max_pages + (p0 >> v.ps_log2)];
                uint8_t* a = v.slab + (size_t)page * v.page_bytes + (size_t)run * v.ps * v.row_bytes +
                             (size_t)(p0 & (v.ps - 1)) * v.row_bytes;
                uint8_t* b = c.slab + (size_t)r.y * c.s_req + (size_t)layer * c.s_layer + (size_t)kind * c.s_kind +
                             (size_t)g * c.s_kv + (size_t)p0 * v.row_bytes;
                const int at = (int)(i + lane) & 63;
                from_s[at] = load ? a : b;
                to_s[at] = load ? b : a;
                bytes_s[at] = (uint32_t)(p1 - p0) * v.row_bytes;
            }
            __syncwarp();
        }
        if (lane == 0) {
            const int st = (int)(i % kExStages), at = (int)(i & 63);
            mbar_arrive_expect_tx(&full[st], bytes_s[at]);
            asm volatile(
                "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;"
                ::"r"(smem_u32(ring + st * kExChunk)), "l"((uint64_t)from_s[at]), "r"(bytes_s[at]),
                  "r"(smem_u32(&full[st])), "l"(once)
                : "memory");
        }
    };
    __syncwarp();
    long long loaded = 0;
    while (loaded < kExStages && loaded < mine) issue(loaded++);
    for (long long i = 0; i < mine; ++i) {
        const int st = (int)(i % kExStages), at = (int)(i & 63);
        const bool ok = mbar_wait(&full[st], (uint32_t)((i / kExStages) & 1), &abort_s, v.status);
        if (!__all_sync(0xffffffffu, ok)) break;
        if (lane == 0) {
            asm volatile("cp.async.bulk.global.shared::cta.bulk_group.L2::cache_hint [%0], [%1], %2, %3;"
                         ::"l"((uint64_t)to_s[at]), "r"(smem_u32(ring + st * kExChunk)), "r"(bytes_s[at]), "l"(once)
                         : "memory");
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        }
        if (i >= 1 && loaded < mine) {
            // the stage of the chunk before is free once its store has read it
            if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
            issue(loaded++);
        }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    if (abort_s && lane == 0) {      // copies in land before the block exits
        volatile int never = 0;
        for (long long k = loaded < kExStages ? 0 : loaded - kExStages; k < loaded; ++k)
            mbar_wait(&full[k % kExStages], (uint32_t)((k / kExStages) & 1), &never, nullptr);
    }
}
// Step 3: the lengths.
__global__ void __launch_bounds__(kPlan) k_exchange_end(PoolView v, SlabView c, int n, int load) {
    griddep_wait();
    griddep_launch();
    if ((int)threadIdx.x >= n) return;
    const int4 r = v.recs[threadIdx.x];
    if (r.w <= r.z) return;
    if (load) c.len[r.y] = c.committed[r.y] = r.w;
    else v.len[r.x] = r.w;
}

int copy_blocks(const PoolView& v, long long most_copies) {
    const long long per = (long long)v.n_layers * 2 * v.nkv * (((long long)v.ps * v.row_bytes + 4095) >> 12);
    const long long b = (most_copies * per + kCopyWarps - 1) / kCopyWarps;
    return (int)(b < 1 ? 1 : b > 148 * 8 ? 148 * 8 : b);
}
cudaError_t copy_whole(const PoolView& v, cudaStream_t st) {
    constexpr int smem = kBulkStages * kBulkChunk + 128;
    if (!allow_smem<1>((const void*)k_pages_copy_whole, smem)) return cudaErrorInvalidValue;
    return launch_k(k_pages_copy_whole, dim3(148), dim3(32), smem, st, v);
}
int blocks_for(size_t n) { return (int)(n + 255 < 256 * 592 ? (n + 255) / 256 : 592); }

}  // namespace

int launch_pool_set_tables(const PoolView& v, const int* lens, const int* table, cudaStream_t st, int* launches) {
    const size_t n = (size_t)v.max_seqs * v.max_pages;
    if (n <= kSmallTables && v.n_pages <= kSmallTables) {
        *launches = 1;
        return (int)launch_k(k_tables_small, dim3(1), dim3(kPlan), 0, st, v, lens, table);
    }
    *launches = 3;
    cudaError_t e = launch_k(k_tables_begin, dim3(blocks_for(v.n_pages)), dim3(256), 0, st, v);
    if (e == cudaSuccess) e = launch_k(k_tables_count, dim3(blocks_for(n)), dim3(256), 0, st, v, lens, table);
    if (e == cudaSuccess) e = launch_k(k_tables_apply, dim3(blocks_for(n)), dim3(256), 0, st, v, lens, table);
    return (int)e;
}

int launch_pages_reserve(const PoolView& v, const int* seqs, const int* grow, int n, cudaStream_t st) {
    cudaError_t e = launch_k(k_pages_plan<false>, dim3(1), dim3(kPlan), 0, st, v, seqs, grow, (const int*)nullptr, n);
    if (e == cudaSuccess) e = launch_k(k_pages_copy, dim3(copy_blocks(v, n)), dim3(kCopyWarps * 32), 0, st, v);
    return (int)e;
}

int launch_pages_fork(const PoolView& v, const int* src, const int* dst, int n, int deep, cudaStream_t st) {
    if (!deep) return (int)launch_k(k_pages_fork, dim3(n), dim3(256), 0, st, v, src, dst);
    cudaError_t e = launch_k(k_pages_plan<true>, dim3(1), dim3(kPlan), 0, st, v, dst, (const int*)nullptr, src, n);
    if (e == cudaSuccess) e = copy_whole(v, st);
    return (int)e;
}

int launch_pages_free(const PoolView& v, const int* seqs, const int* keep, int n, cudaStream_t st) {
    return (int)launch_k(k_pages_free, dim3(n), dim3(256), 0, st, v, seqs, keep);
}

int launch_pages_compact(const PoolView& v, int* used, cudaStream_t st, int* launches) {
    // small tables are followed up by the planning block itself (2048 entries: 5.6 us against 6.0 with
    // a launch for it; 16384: 11.4 against 11.1)
    const bool small = (size_t)v.max_seqs * v.max_pages <= 8192;
    *launches = small ? 2 : 3;
    cudaError_t e = launch_k(k_pages_compact, dim3(1), dim3(kPlan), 0, st, v, used, small ? 1 : 0);
    if (e == cudaSuccess && !small)
        e = launch_k(k_pages_remap, dim3(blocks_for((size_t)v.max_seqs * v.max_pages)), dim3(256), 0, st, v);
    if (e == cudaSuccess) e = copy_whole(v, st);
    return (int)e;
}

int launch_pages_write(const PoolView& v, const int* seqs, int n, int layer, const void* k, const void* vv,
                       long long stride_bytes, const int* row_start, const int* row_count, int total_rows, int max_rows,
                       cudaStream_t st) {
    return (int)launch_k(k_pages_write, dim3((max_rows + kWriteRows - 1) / kWriteRows, n), dim3(256), 0, st, v, seqs,
                         layer, (const uint8_t*)k, (const uint8_t*)vv, stride_bytes, row_start, row_count, total_rows,
                         max_rows);
}

int launch_pages_advance(const PoolView& v, const int* seqs, const int* row_count, int n, cudaStream_t st) {
    return (int)launch_k(k_pages_advance, dim3(1), dim3(kPlan), 0, st, v, seqs, row_count, n);
}

int launch_pages_exchange(const PoolView& v, const int* seqs, const SlabView& c, const int* reqs, int n, bool load,
                          cudaStream_t st) {
    constexpr int smem = kExStages * kExChunk + 128;
    if (!allow_smem<2>((const void*)k_exchange_copy, smem)) return 1;
    int lp = v.ps_log2;
    while (v.row_bytes << lp > kExChunk) --lp;
    const int bx = (2 * 148 + n - 1) / n;
    cudaError_t e = launch_k(k_exchange_plan, dim3(n), dim3(256), 0, st, v, seqs, c, reqs, load ? 1 : 0);
    if (e == cudaSuccess) e = launch_k(k_exchange_copy, dim3(bx, n), dim3(32), smem, st, v, c, load ? 1 : 0, lp);
    if (e == cudaSuccess) e = launch_k(k_exchange_end, dim3(1), dim3(kPlan), 0, st, v, c, n, load ? 1 : 0);
    return (int)e;
}

}  // namespace df
