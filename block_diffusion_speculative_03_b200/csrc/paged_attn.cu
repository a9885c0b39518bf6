// Attention over a paged pool (or a cache slab) on the CUDA cores, fp32 storage.
//
// With t_k = q.k log2(e) / sqrt(d) over the keys a row sees, out = sum 2^(t_k - m) v_k
// / sum 2^(t_k - m) for the running maximum m: one pass over K and V, everything in
// fp32 and nothing rounded in between.
//
// A block takes 2, 4 or 8 query vectors of one (entry, kv head): the vectors v = row * G + head
// of the entry, in order, share every key and value that is read.  Its four groups of two warps
// walk 32-key tiles through their part of shared memory, each warp with half of the vectors: K of
// the next tile comes in (asynchronous copies) while the values of this one are weighted, V while
// its scores are formed.  Each lane forms one key's dot products with the warp's vectors (K rows
// padded by 16 bytes, so the 32 lanes' 16-byte reads of one column hit all banks once), the
// weights go to shared memory, and each lane accumulates its D / 32 columns of the output over the
// tile's V rows.  The groups' (m, l, o) are joined in shared memory; with few items the keys are
// also split over blocks, whose partials the last one to arrive joins in split order.
//
// A tile of 32 keys fills 33 KB at head_dim 128, so four groups are what an SM holds: with a single
// warp each, one warp per scheduler ran a chain of dependent instructions (16 sequences of 1000,
// 8 heads of 128, 8 rows: 85 us against 58 with two; four warps with a quarter of the vectors each:
// 58 there, but 171 against 124 at 32 of 3000 with head_dim 64, the reads of K from shared memory
// repeated by each).  Bound by latency at few keys (2 x 4 heads of 64, 300 keys: 9.7 us), by
// shared-memory reads and fp32 instructions at many (32 sequences of 3000, 8 heads of 64: 393 MB
// in 71 us, 5.5 TB/s, at one row; 125 us at eight).  16 sequences of 16000, one row, 8 heads of 128 with a
// window of 1024: 43 us (135 MB, 3.1 TB/s).  A prompt reads K and V once for every eight vectors: 512
// rows of 8 heads on 2 of 128 behind 1000 positions take 207 us (13 TFLOP/s), 2048 rows of 32 heads on 8
// with a window of 2048 4.2 ms (16 TFLOP/s).
#include <algorithm>

#include "paged.cuh"

namespace df {

namespace {

constexpr int kGroups = 4;    // groups of warps that take the tiles in turn
constexpr int kTile = 32;     // keys of a tile
constexpr int kMaxSplits = 32;

constexpr int kShare = 2;     // warps of a group: they share its tiles and have half of the vectors each
constexpr int kThreads = kGroups * kShare * 32;

constexpr int smem_bytes(int d, int v) {
    return v * d * 4 + kGroups * kTile * (2 * d + 4) * 4 + kGroups * v * kTile * 4 + kGroups * v * 8;
}

// Grid: (vector blocks * nkv * splits, entries); V: query vectors of a block.
template <int D, int V>
__global__ void __launch_bounds__(kThreads) k_paged_attn_f32(const __grid_constant__ PagedAttnParams p) {
    constexpr int C = D / 32;                   // output columns per lane
    constexpr int GW = kShare, VW = V / GW;     // vectors of a warp
    extern __shared__ __align__(16) float sm[];
    float* sq = sm;                             // [V][D], scaled to log2 units
    float* sk = sq + V * D;                     // [kGroups][kTile][D + 4]
    float* sv = sk + kGroups * kTile * (D + 4); // [kGroups][kTile][D]
    float* sp = sv + kGroups * kTile * D;       // [kGroups][V][kTile]
    float2* sml = reinterpret_cast<float2*>(sp + kGroups * V * kTile);   // [kGroups][V]
    __shared__ int last;
    griddep_wait();
    griddep_launch();
    const int tid = threadIdx.x, group = (tid >> 5) / GW, sub = (tid >> 5) % GW, lane = tid & 31;
    const int split = blockIdx.x % p.splits, item_x = blockIdx.x / p.splits, i = blockIdx.y;
    const int vb = item_x / p.nkv, g = item_x % p.nkv;
    const AttnEntry e = attn_entry(p, i);
    if (e.bad && p.status && tid == 0) set_error(p.status, e.bad);
    const int nvec = min(V, e.count * p.G - vb * V);
    if (nvec <= 0) return;
    const int v0 = vb * V;
    float* out = (float*)p.out;
    auto out_row = [&](int j) {   // vector j of this block
        const int r = (v0 + j) / p.G, h = (v0 + j) % p.G;
        return out + ((size_t)(e.start + r) * p.nq + (size_t)g * p.G + h) * D;
    };
    if (e.bad) {
        if (split == 0)
            for (int x = tid; x < nvec * D; x += blockDim.x) out_row(x / D)[x % D] = 0.f;
        return;
    }
    const int r0 = v0 / p.G, r1 = (v0 + nvec - 1) / p.G + 1;
    const KeySpan span = key_span(e.len, e.count, r0, r1, p.causal, p.window, p.sinks, kTile);
    // at least a tile for each group of a split
    const int splits = min(p.splits, max(1, span.nt / kGroups));
    if (split >= splits) return;
    const int t_lo = (int)((long long)span.nt * split / splits), t_hi = (int)((long long)span.nt * (split + 1) / splits);
    // the positions that exist for any row of the block
    const int hi_all = p.causal ? e.len + r1 : e.len + e.count;

    for (int x = tid; x < nvec * (D / 4); x += blockDim.x) {
        const int j = x / (D / 4), c = x % (D / 4) * 4, r = (v0 + j) / p.G, h = (v0 + j) % p.G;
        const float4 f = *reinterpret_cast<const float4*>((const float*)p.q + (size_t)(e.start + r) * p.q_stride +
                                                          ((size_t)g * p.G + h) * D + c);
        *reinterpret_cast<float4*>(sq + j * D + c) =
            make_float4(f.x * p.scale_log2, f.y * p.scale_log2, f.z * p.scale_log2, f.w * p.scale_log2);
    }
    __syncthreads();

    const int j0 = sub * VW, mine = max(0, min(VW, nvec - j0));   // this warp's vectors
    float m[VW], l[VW], acc[VW][C];
#pragma unroll
    for (int j = 0; j < VW; ++j) {
        m[j] = -INFINITY;
        l[j] = 0.f;
#pragma unroll
        for (int c = 0; c < C; ++c) acc[j][c] = 0.f;
    }
    float* gk = sk + group * kTile * (D + 4);
    float* gv = sv + group * kTile * D;
    float* wp = sp + (group * V + j0) * kTile;
    const float* wq = sq + j0 * D;
    auto group_sync = [&]() { named_bar_sync(1 + group, GW * 32); };
    const float* slab = (const float*)p.slab;
    // The group's next tile from t on in which some row sees a key: its first key, the keys that
    // any row sees (the others are neither read nor weighted), and this lane's key's slab row.
    struct Tile { int t, k0; unsigned seen; long long row; };
    auto find = [&](int t) -> Tile {
        for (; t < t_hi; t += kGroups) {
            const int k0 = span.tile(t) * kTile, key = k0 + lane;
            bool any = false;
            for (int r = r0; r < r1; ++r)
                any |= key_visible(key, e.len + r, p.causal ? e.len + r + 1 : hi_all, p.window, p.sinks);
            const unsigned seen = __ballot_sync(0xffffffffu, any);
            if (!seen) continue;
            long long row = 0;
            if (any) {
                const long long pg = p.table ? p.table[(size_t)e.seq * p.max_pages + (key >> p.ps_log2)] : e.seq;
                const int in = p.table ? key & ((1 << p.ps_log2) - 1) : key;
                row = pg * p.rows_page + p.row_layer + (long long)g * p.rows_kv + in;
            }
            return {t, k0, seen, row};
        }
        return {t_hi, 0, 0u, 0};
    };
    // this warp's share of a tile's rows
    auto fetch = [&](const Tile& x, float* to, int ld, long long kind) {
        constexpr int PER = 128 / D;      // rows per instruction
#pragma unroll
        for (int i = sub * PER; i < kTile; i += GW * PER) {
            const int k = i + lane / (D / 4), c = lane % (D / 4) * 4;
            const long long rk = __shfl_sync(0xffffffffu, x.row, k) + kind;
            if ((x.seen >> k) & 1)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                             ::"r"(smem_u32(to + k * ld + c)), "l"((uint64_t)(slab + rk * D + c)) : "memory");
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto weigh = [&](int k, const float* w) {     // += w[j] * (row k of V)
        float v[C];
        if constexpr (C == 4) {
            const float4 f = *reinterpret_cast<const float4*>(gv + k * D + lane * 4);
            v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
        } else {
            const float2 f = *reinterpret_cast<const float2*>(gv + k * D + lane * 2);
            v[0] = f.x; v[1] = f.y;
        }
#pragma unroll
        for (int j = 0; j < VW; ++j)
#pragma unroll
            for (int c = 0; c < C; ++c) acc[j][c] = fmaf(w[j], v[c], acc[j][c]);
    };
    Tile cur = find(t_lo + group);
    if (cur.seen) {
        fetch(cur, gk, D + 4, 0);
        fetch(cur, gv, D, p.rows_kind);
    }
    while (cur.seen) {        // the same for all warps of the group
        const int key = cur.k0 + lane;
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        group_sync();                                             // K is there
        if (mine > 0) {
            float4 s4[VW];                                        // four chains per vector
#pragma unroll
            for (int j = 0; j < VW; ++j) s4[j] = make_float4(0.f, 0.f, 0.f, 0.f);
            if ((cur.seen >> lane) & 1) {
#pragma unroll 8
                for (int c = 0; c < D; c += 4) {
                    const float4 kv = *reinterpret_cast<const float4*>(gk + lane * (D + 4) + c);
#pragma unroll
                    for (int j = 0; j < VW; ++j) {                // (vectors past the last: whatever stands there)
                        const float4 qv = *reinterpret_cast<const float4*>(wq + j * D + c);
                        s4[j].x = fmaf(qv.x, kv.x, s4[j].x);
                        s4[j].y = fmaf(qv.y, kv.y, s4[j].y);
                        s4[j].z = fmaf(qv.z, kv.z, s4[j].z);
                        s4[j].w = fmaf(qv.w, kv.w, s4[j].w);
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < VW; ++j) {
                const int r = (v0 + j0 + j) / p.G;
                const bool vis = j < mine && key_visible(key, e.len + r, p.causal ? e.len + r + 1 : hi_all, p.window, p.sinks);
                const float x = vis ? (s4[j].x + s4[j].y) + (s4[j].z + s4[j].w) : -INFINITY;
                float mx = x;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                const float mn = fmaxf(m[j], mx);
                const float base = mn == -INFINITY ? 0.f : mn;
                const float f = exp2f(m[j] - base);               // 0 while nothing has been seen
                const float w = vis ? exp2f(x - base) : 0.f;
                wp[j * kTile + lane] = w;
                l[j] = l[j] * f + w;                              // this lane's keys; the lanes are added at the end
                m[j] = mn;
#pragma unroll
                for (int c = 0; c < C; ++c) acc[j][c] *= f;
            }
        }
        const Tile next = find(cur.t + kGroups);
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        group_sync();                                             // K has been read, V is there, the weights are written
        if (next.seen) fetch(next, gk, D + 4, 0);
        if (mine > 0) {
            if (cur.seen == 0xffffffffu) {
#pragma unroll 2
                for (int k = 0; k < kTile; k += 4) {
                    float4 w4[VW];
#pragma unroll
                    for (int j = 0; j < VW; ++j) w4[j] = *reinterpret_cast<const float4*>(wp + j * kTile + k);
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        float w[VW];
#pragma unroll
                        for (int j = 0; j < VW; ++j) w[j] = x == 0 ? w4[j].x : x == 1 ? w4[j].y : x == 2 ? w4[j].z : w4[j].w;
                        weigh(k + x, w);
                    }
                }
            } else {
                for (int k = 0; k < kTile; ++k) {
                    if (!((cur.seen >> k) & 1)) continue;         // not read
                    float w[VW];
#pragma unroll
                    for (int j = 0; j < VW; ++j) w[j] = wp[j * kTile + k];
                    weigh(k, w);
                }
            }
        }
        group_sync();                                             // V has been read
        if (next.seen) fetch(next, gv, D, p.rows_kind);
        cur = next;
    }
    // join the groups: o over the K staging, [group][vector][D]
    __syncthreads();
#pragma unroll
    for (int j = 0; j < VW; ++j) {
        float s = l[j];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == 0) sml[group * V + j0 + j] = make_float2(m[j], s);
#pragma unroll
        for (int c = 0; c < C; ++c) sk[(group * V + j0 + j) * D + lane * C + c] = acc[j][c];
    }
    __syncthreads();
    const size_t item = (size_t)i * (gridDim.x / p.splits) + item_x;
    constexpr int SLOT = V * (D + 2);
    float* part = p.partial + (item * p.splits + split) * SLOT;
    for (int x = tid; x < nvec * D; x += blockDim.x) {
        const int j = x / D;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kGroups; ++w) M = fmaxf(M, sml[w * V + j].x);
        const float base = M == -INFINITY ? 0.f : M;
        float L = 0.f, o = 0.f;
#pragma unroll
        for (int w = 0; w < kGroups; ++w) {
            const float f = exp2f(sml[w * V + j].x - base);
            L += f * sml[w * V + j].y;
            o += f * sk[(w * V + j) * D + x % D];
        }
        if (splits == 1) {
            out_row(j)[x % D] = L == 0.f ? 0.f : o / L;   // a NaN sum stays one
        } else {
            part[j * (D + 2) + 2 + x % D] = o;
            if (x % D == 0) {
                part[j * (D + 2)] = M;
                part[j * (D + 2) + 1] = L;
            }
        }
    }
    if (splits == 1) return;
    __syncthreads();
    if (tid == 0) last = atom_add_acq_rel(&p.counters[item], 1) == splits - 1;
    __syncthreads();
    if (!last) return;
    const float* all = p.partial + item * p.splits * SLOT;
    for (int x = tid; x < nvec * D; x += blockDim.x) {
        const int j = x / D;
        const float* q = all + j * (D + 2);
        float M = -INFINITY, L = 0.f, o = 0.f;
        for (int s0 = 0; s0 < splits; s0 += 8) {      // eight partials' loads in flight
            float m8[8], l8[8], o8[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float* z = q + min(s0 + k, splits - 1) * SLOT;
                m8[k] = __ldcg(z);
                l8[k] = __ldcg(z + 1);
                o8[k] = __ldcg(z + 2 + x % D);
            }
            float nm = M;
#pragma unroll
            for (int k = 0; k < 8; ++k) nm = fmaxf(nm, m8[k]);
            const float base = nm == -INFINITY ? 0.f : nm, g = exp2f(M - base);
            M = nm;
            L *= g;
            o *= g;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if (s0 + k >= splits) break;
                const float f = exp2f(m8[k] - base);
                L += f * l8[k];
                o += f * o8[k];
            }
        }
        out_row(j)[x % D] = L == 0.f ? 0.f : o / L;
    }
    if (tid == 0) p.counters[item] = 0;
}

// CTAs of a launch that run at the same time.
template <int D> int resident(int num_sms) { return std::min(num_sms, kPagedCtas) * (D == 128 ? 1 : 3); }
long long items_of(const PagedAttnParams& p, int v) {
    return ((long long)p.max_rows * p.G + v - 1) / v * p.nkv * p.n;
}
template <int D, int V>
int launch_dv(PagedAttnParams& p, int num_sms, cudaStream_t st) {
    constexpr int smem = smem_bytes(D, V);
    if (!allow_smem<D * 100 + V>((const void*)k_paged_attn_f32<D, V>, smem)) return 1;
    const long long items = items_of(p, V);
    // Two waves of blocks, so that every SM has work and entries of different lengths even out:
    // fewer items are split.
    p.splits = (int)std::max(1LL, std::min<long long>(kMaxSplits, 2LL * resident<D>(num_sms) / items));
    return (int)launch_k(k_paged_attn_f32<D, V>, dim3((unsigned)(items / p.n * p.splits), p.n),
                         dim3(kThreads), smem, st, p);
}
// Vectors a block: more share K and V (whose reads from shared memory and from L2 bound large calls),
// fewer make more blocks, which small calls lack.  8 kv heads, one query head each:
//   1 sequence of 500, head_dim 128, 8 rows: 11.7 us with 2, 13.4 with 4, 18.1 with 8
//   16 of 1000, head_dim 64, 4 rows: 30.3, 24.7, 32.1; head_dim 128, 8 rows: 117, 64.5, 58.0
//   32 of 3000, head_dim 64, 8 rows: 215, 157, 124; 1 row: 70, 73, 92
//   the same with head_dim 128, 2 rows: 173, 146 (one warp of a group has both), 193
template <int D>
int launch_d(PagedAttnParams& p, int num_sms, cudaStream_t st) {
    const long long vectors = (long long)p.max_rows * p.G;
    if (vectors <= 128 / D || 2 * items_of(p, 2) <= resident<D>(num_sms)) return launch_dv<D, 2>(p, num_sms, st);
    if (vectors <= 4 || items_of(p, 4) <= resident<D>(num_sms)) return launch_dv<D, 4>(p, num_sms, st);
    return launch_dv<D, 8>(p, num_sms, st);
}

}  // namespace

size_t paged_scratch_bytes() {
    return kPagedCounterBytes + (size_t)2 * kPagedCtas * kPagedRowsTc * (128 + 2) * sizeof(float);
}

int launch_paged_attn_f32(PagedAttnParams& p, int d, int num_sms, cudaStream_t st) {
    p.launches = 1;
    return d == 128 ? launch_d<128>(p, num_sms, st) : launch_d<64>(p, num_sms, st);
}
// Up to 16 vectors fit one register tile.  At 16 (16 rows of 8 heads of 128), this side and the other:
// 1 sequence of 2000: 14.7 us, 13.3; 4 of 8000: 30.8, 33.3; 32 of 4000: 89.2, 97.4.  At 4: 10.1, 13.2;
// 27.5, 33.5; 86.6, 95.9.
int launch_paged_attn_bf16(PagedAttnParams& p, int d, int num_sms, cudaStream_t st) {
    return p.max_rows * p.G <= 16 ? launch_paged_decode(p, d, num_sms, st) : launch_paged_block(p, d, num_sms, st);
}

}  // namespace df
