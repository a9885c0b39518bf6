// Attention over a paged pool (or a cache slab) on the CUDA cores, fp32 storage.
//
// With t_k = q.k log2(e) / sqrt(d) over the keys a row sees, out = sum 2^(t_k - m) v_k
// / sum 2^(t_k - m) for the running maximum m: one pass over K and V, everything in
// fp32 and nothing rounded in between.
//
// One block of 4 warps takes up to 8 query vectors of one (entry, kv head): the vectors
// v = row * G + head of the entry, in order, share every key and value that is read.  A
// warp walks 32-key tiles through its part of shared memory: K of the next tile comes in
// (asynchronous copies) while the values of this one are weighted, V while its scores are
// formed.  Each lane forms one key's dot products with the 8 vectors (K rows padded by 16
// bytes, so the 32 lanes' 16-byte reads of one column hit all banks once), the weights go to
// shared memory, and each lane accumulates its D / 32 columns of the output over the tile's
// V rows.  The four warps' (m, l, o) are joined in shared memory; with few items the keys are
// also split over `splits` blocks, whose partials the last one to arrive joins in split order.
// Bound by latency at few keys (two memory round trips per 32 keys of a warp), by HBM at many.
#include <algorithm>

#include "paged.cuh"

namespace df {

namespace {

constexpr int kWarps = 4;
constexpr int kTile = 32;     // keys of a warp's tile
constexpr int kMaxSplits = 32;

constexpr int smem_bytes(int d, int kVec) {
    return kVec * d * 4 + kWarps * kTile * (2 * d + 4) * 4 + kWarps * kVec * kTile * 4 + kWarps * kVec * 8;
}

// Grid: (vector blocks * nkv * splits, entries).
// kVec: query vectors per block.
template <int D, int kVec>
__global__ void __launch_bounds__(kWarps * 32) k_paged_attn_f32(const __grid_constant__ PagedAttnParams p) {
    constexpr int C = D / 32;                   // output columns per lane
    extern __shared__ __align__(16) float sm[];
    float* sq = sm;                             // [kVec][D], scaled to log2 units
    float* sk = sq + kVec * D;                  // [kWarps][kTile][D + 4]
    float* sv = sk + kWarps * kTile * (D + 4);  // [kWarps][kTile][D]
    float* sp = sv + kWarps * kTile * D;        // [kWarps][kVec][kTile]
    float2* sml = reinterpret_cast<float2*>(sp + kWarps * kVec * kTile);   // [kWarps][kVec]
    __shared__ int last;
    griddep_wait();
    griddep_launch();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int split = blockIdx.x % p.splits, item_x = blockIdx.x / p.splits, i = blockIdx.y;
    const int vb = item_x / p.nkv, g = item_x % p.nkv;
    const AttnEntry e = attn_entry(p, i);
    if (e.bad && p.status && tid == 0) set_error(p.status, e.bad);
    const int nvec = min(kVec, e.count * p.G - vb * kVec);
    if (nvec <= 0) return;
    const int v0 = vb * kVec;
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
    // at least a tile for each warp of a split
    const int splits = min(p.splits, max(1, span.nt / kWarps));
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

    float m[kVec], l[kVec], acc[kVec][C];
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
        m[j] = -INFINITY;
        l[j] = 0.f;
#pragma unroll
        for (int c = 0; c < C; ++c) acc[j][c] = 0.f;
    }
    float* wk = sk + warp * kTile * (D + 4);
    float* wv = sv + warp * kTile * D;
    float* wp = sp + warp * kVec * kTile;
    const float* slab = (const float*)p.slab;
    // The warp's next tile from t on in which some row sees a key: its first key, the keys that
    // any row sees (the others are neither read nor weighted), and this lane's key's slab row.
    struct Tile { int t, k0; unsigned seen; long long row; };
    auto find = [&](int t) -> Tile {
        for (; t < t_hi; t += kWarps) {
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
    auto fetch = [&](const Tile& x, float* to, int ld, long long kind) {
#pragma unroll 8
        for (int i = 0; i < kTile; i += 128 / D) {
            const int k = i + lane / (D / 4), c = lane % (D / 4) * 4;
            const long long rk = __shfl_sync(0xffffffffu, x.row, k) + kind;
            if ((x.seen >> k) & 1)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                             ::"r"(smem_u32(to + k * ld + c)), "l"((uint64_t)(slab + rk * D + c)) : "memory");
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    Tile cur = find(t_lo + warp);
    if (cur.seen) {
        fetch(cur, wk, D + 4, 0);
        fetch(cur, wv, D, p.rows_kind);
    }
    while (cur.seen) {
        const int key = cur.k0 + lane;
        const bool any = (cur.seen >> lane) & 1;
        asm volatile("cp.async.wait_group 1;" ::: "memory");      // K
        __syncwarp();
        float s[kVec];
#pragma unroll
        for (int j = 0; j < kVec; ++j) s[j] = 0.f;
        if (any) {
#pragma unroll 4
            for (int c = 0; c < D; c += 4) {
                const float4 kv = *reinterpret_cast<const float4*>(wk + lane * (D + 4) + c);
#pragma unroll
                for (int j = 0; j < kVec; ++j)
                    if (j < nvec) {
                        const float4 qv = *reinterpret_cast<const float4*>(sq + j * D + c);
                        s[j] = fmaf(qv.x, kv.x, fmaf(qv.y, kv.y, fmaf(qv.z, kv.z, fmaf(qv.w, kv.w, s[j]))));
                    }
            }
        }
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            if (j >= nvec) break;
            const int r = (v0 + j) / p.G;
            const bool vis = key_visible(key, e.len + r, p.causal ? e.len + r + 1 : hi_all, p.window, p.sinks);
            const float x = vis ? s[j] : -INFINITY;
            float mx = x;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            const float mn = fmaxf(m[j], mx);
            const float base = mn == -INFINITY ? 0.f : mn;
            const float f = exp2f(m[j] - base);           // 0 while nothing has been seen
            const float w = vis ? exp2f(x - base) : 0.f;
            wp[j * kTile + lane] = w;
            l[j] = l[j] * f + w;                           // this lane's keys; the lanes are added at the end
            m[j] = mn;
#pragma unroll
            for (int c = 0; c < C; ++c) acc[j][c] *= f;
        }
        const Tile next = find(cur.t + kWarps);
        __syncwarp();                                             // K and the weights: read, written
        if (next.seen) {
            fetch(next, wk, D + 4, 0);
            asm volatile("cp.async.wait_group 1;" ::: "memory");  // V
        } else {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
        }
        __syncwarp();
#pragma unroll 4
        for (int k = 0; k < kTile; ++k) {
            if (!((cur.seen >> k) & 1)) continue;
            float v[C];
            if constexpr (C == 4) {
                const float4 f = *reinterpret_cast<const float4*>(wv + k * D + lane * 4);
                v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
            } else {
                const float2 f = *reinterpret_cast<const float2*>(wv + k * D + lane * 2);
                v[0] = f.x; v[1] = f.y;
            }
#pragma unroll
            for (int j = 0; j < kVec; ++j)
                if (j < nvec) {
                    const float w = wp[j * kTile + k];
#pragma unroll
                    for (int c = 0; c < C; ++c) acc[j][c] = fmaf(w, v[c], acc[j][c]);
                }
        }
        __syncwarp();                                             // V has been read
        if (next.seen) fetch(next, wv, D, p.rows_kind);
        cur = next;
    }
    // join the warps: o over the K staging, [warp][vector][D]
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
        float s = l[j];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == 0) sml[warp * kVec + j] = make_float2(m[j], s);
#pragma unroll
        for (int c = 0; c < C; ++c) sk[(warp * kVec + j) * D + lane * C + c] = acc[j][c];
    }
    __syncthreads();
    const size_t item = (size_t)i * (gridDim.x / p.splits) + item_x;
    constexpr int SLOT = kVec * (D + 2);
    float* part = p.partial + (item * p.splits + split) * SLOT;
    for (int x = tid; x < nvec * D; x += blockDim.x) {
        const int j = x / D;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sml[w * kVec + j].x);
        const float base = M == -INFINITY ? 0.f : M;
        float L = 0.f, o = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = exp2f(sml[w * kVec + j].x - base);
            L += f * sml[w * kVec + j].y;
            o += f * sk[(w * kVec + j) * D + x % D];
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

template <int D, int V>
int launch_dv(PagedAttnParams& p, int num_sms, cudaStream_t st) {
    constexpr int smem = smem_bytes(D, V);
    if (!allow_smem<D * 100 + V>((const void*)k_paged_attn_f32<D, V>, smem)) return 1;
    const long long vbs = ((long long)p.max_rows * p.G + V - 1) / V;
    const long long items = vbs * p.nkv * p.n;
    // Two waves of blocks (3 fit on an SM at 64, 1 at 128), so that every SM has work and entries
    // of different lengths even out: fewer items are split (80 items of 1 to 2235 keys: 118 us
    // with one wave, 72 with two).
    const long long target = 2LL * std::min(num_sms, kPagedCtas) * (D == 64 ? 3 : 1);
    p.splits = (int)std::max(1LL, std::min<long long>(kMaxSplits, target / items));
    return (int)launch_k(k_paged_attn_f32<D, V>, dim3((unsigned)(vbs * p.nkv * p.splits), p.n), dim3(kWarps * 32), smem,
                         st, p);
}
// 8 vectors a block share K and V; with fewer in all, loops over the missing ones cost as much as
// the others (2 vectors: 11.7 us with room for 8).
template <int D>
int launch_d(PagedAttnParams& p, int num_sms, cudaStream_t st) {
    const long long vectors = (long long)p.max_rows * p.G;
    if (vectors <= 2) return launch_dv<D, 2>(p, num_sms, st);
    if (vectors <= 4) return launch_dv<D, 4>(p, num_sms, st);
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
int launch_paged_attn_bf16(PagedAttnParams& p, int d, int num_sms, cudaStream_t st) {
    return p.max_rows * p.G <= 16 ? launch_paged_decode(p, d, num_sms, st) : launch_paged_block(p, d, num_sms, st);
}

}  // namespace df
