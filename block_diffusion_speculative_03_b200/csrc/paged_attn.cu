// Attention over a paged pool (or a cache slab) on the CUDA cores, fp32 storage.
//
// With t_k = q.k log2(e) / sqrt(d) over the keys a row sees, out = sum 2^(t_k - m) v_k
// / sum 2^(t_k - m) for the running maximum m: one pass over K and V, everything in
// fp32 and nothing rounded in between.
//
// One block of 4 warps takes up to 8 query vectors of one (entry, kv head): the vectors
// v = row * G + head of the entry, in order, share every key and value that is read.  A
// warp walks 32-key tiles: it stages the K rows in its part of shared memory, each lane
// forms one key's dot products with the 8 vectors (K rows padded by 16 bytes, so the 32
// lanes' 16-byte reads of one column hit all banks once), the weights go to shared
// memory, and each lane accumulates its D / 32 columns of the output over the tile's V
// rows, read straight from global memory.  The four warps' (m, l, o) are joined in shared
// memory; with few items the keys are also split over `splits` blocks, whose partials the
// last one to arrive joins in split order.
#include <algorithm>

#include "paged.cuh"

namespace df {

namespace {

constexpr int kVec = 8;       // query vectors per block
constexpr int kWarps = 4;
constexpr int kTile = 32;     // keys of a warp's tile
constexpr int kMaxSplits = 32;

template <typename T> struct F32Smem {
    static constexpr int bytes(int d) {
        return kVec * d * 4 + kWarps * kTile * (d + 4) * 4 + kWarps * kVec * kTile * 4 + kWarps * kVec * 8;
    }
};

template <typename T> DF_DEV void load4(const T* p, float* v);
template <> DF_DEV void load4<float>(const float* p, float* v) {
    const float4 f = *reinterpret_cast<const float4*>(p);
    v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
}

// Grid: (vector blocks * nkv * splits, entries).
template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32) k_paged_attn_simt(const __grid_constant__ PagedAttnParams p) {
    constexpr int C = D / 32;                   // output columns per lane
    extern __shared__ __align__(16) float sm[];
    float* sq = sm;                             // [kVec][D], scaled to log2 units
    float* sk = sq + kVec * D;                  // [kWarps][kTile][D + 4]
    float* sp = sk + kWarps * kTile * (D + 4);  // [kWarps][kVec][kTile]
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
    T* out = (T*)p.out;
    auto out_row = [&](int j) {   // vector j of this block
        const int r = (v0 + j) / p.G, h = (v0 + j) % p.G;
        return out + ((size_t)(e.start + r) * p.nq + (size_t)g * p.G + h) * D;
    };
    if (e.bad) {
        if (split == 0)
            for (int x = tid; x < nvec * D; x += blockDim.x) stf(out_row(x / D) + x % D, 0.f);
        return;
    }
    const int r0 = v0 / p.G, r1 = (v0 + nvec - 1) / p.G + 1;
    const KeySpan span = key_span(e.len, e.count, r0, r1, p.causal, p.window, p.sinks, kTile);
    const int t_lo = (int)((long long)span.nt * split / p.splits), t_hi = (int)((long long)span.nt * (split + 1) / p.splits);
    // the positions that exist for any row of the block
    const int hi_all = p.causal ? e.len + r1 : e.len + e.count;

    for (int x = tid; x < nvec * (D / 4); x += blockDim.x) {
        const int j = x / (D / 4), c = x % (D / 4) * 4, r = (v0 + j) / p.G, h = (v0 + j) % p.G;
        float f[4];
        load4((const T*)p.q + (size_t)(e.start + r) * p.q_stride + ((size_t)g * p.G + h) * D + c, f);
#pragma unroll
        for (int k = 0; k < 4; ++k) sq[j * D + c + k] = f[k] * p.scale_log2;
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
    float* wp = sp + warp * kVec * kTile;
    const T* slab = (const T*)p.slab;
    for (int t = t_lo + warp; t < t_hi; t += kWarps) {
        const int k0 = span.tile(t) * kTile, key = k0 + lane;
        // which of the tile's keys any row sees; the others are neither read nor weighted
        bool any = false;
        for (int r = r0; r < r1; ++r)
            any |= key_visible(key, e.len + r, p.causal ? e.len + r + 1 : hi_all, p.window, p.sinks);
        const unsigned seen = __ballot_sync(0xffffffffu, any);
        if (!seen) continue;
        long long row = 0;    // slab row of this lane's key
        if (any) {
            const long long pg = p.table ? p.table[(size_t)e.seq * p.max_pages + (key >> p.ps_log2)] : e.seq;
            const int in = p.table ? key & ((1 << p.ps_log2) - 1) : key;
            row = pg * p.rows_page + p.row_layer + (long long)g * p.rows_kv + in;
        }
#pragma unroll 4
        for (int k = 0; k < kTile; ++k) {
            const long long rk = __shfl_sync(0xffffffffu, row, k);
            if (!((seen >> k) & 1)) continue;
            if (lane * 4 < D) {
                float f[4];
                load4(slab + rk * D + lane * 4, f);
                *reinterpret_cast<float4*>(wk + k * (D + 4) + lane * 4) = make_float4(f[0], f[1], f[2], f[3]);
            }
        }
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
        __syncwarp();
#pragma unroll 4
        for (int k = 0; k < kTile; ++k) {
            const long long rk = __shfl_sync(0xffffffffu, row, k) + p.rows_kind;
            if (!((seen >> k) & 1)) continue;
            float v[C];
            if constexpr (C == 4) {
                load4(slab + rk * D + lane * 4, v);
            } else {
                v[0] = ldf(slab + rk * D + lane * 2);
                v[1] = ldf(slab + rk * D + lane * 2 + 1);
            }
#pragma unroll
            for (int j = 0; j < kVec; ++j)
                if (j < nvec) {
                    const float w = wp[j * kTile + k];
#pragma unroll
                    for (int c = 0; c < C; ++c) acc[j][c] = fmaf(w, v[c], acc[j][c]);
                }
        }
        __syncwarp();
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
        if (p.splits == 1) {
            stf(out_row(j) + x % D, L == 0.f ? 0.f : o / L);   // a NaN sum stays one
        } else {
            part[j * (D + 2) + 2 + x % D] = o;
            if (x % D == 0) {
                part[j * (D + 2)] = M;
                part[j * (D + 2) + 1] = L;
            }
        }
    }
    if (p.splits == 1) return;
    __threadfence();
    __syncthreads();
    if (tid == 0) last = atomicAdd(&p.counters[item], 1) == p.splits - 1;
    __syncthreads();
    if (!last) return;
    __threadfence();
    const float* all = p.partial + item * p.splits * SLOT;
    for (int x = tid; x < nvec * D; x += blockDim.x) {
        const int j = x / D;
        float M = -INFINITY;
        for (int s = 0; s < p.splits; ++s) M = fmaxf(M, __ldcg(all + s * SLOT + j * (D + 2)));
        const float base = M == -INFINITY ? 0.f : M;
        float L = 0.f, o = 0.f;
        for (int s = 0; s < p.splits; ++s) {
            const float f = exp2f(__ldcg(all + s * SLOT + j * (D + 2)) - base);
            L += f * __ldcg(all + s * SLOT + j * (D + 2) + 1);
            o += f * __ldcg(all + s * SLOT + j * (D + 2) + 2 + x % D);
        }
        stf(out_row(j) + x % D, L == 0.f ? 0.f : o / L);
    }
    if (tid == 0) p.counters[item] = 0;
}

template <typename T, int D>
int launch_simt(PagedAttnParams& p, int num_sms, cudaStream_t st) {
    const int smem = F32Smem<T>::bytes(D);
    auto kern = k_paged_attn_simt<T, D>;
    if (!allow_smem<D * 8 + 7>((const void*)kern, smem)) return 1;
    const long long vbs = ((long long)p.max_rows * p.G + kVec - 1) / kVec;
    const long long items = vbs * p.nkv * p.n;
    // two blocks' worth of items per SM, no item split into less than its tiles
    p.splits = 1;
    if (items < 2 * num_sms) p.splits = (int)std::min<long long>(kMaxSplits, 2LL * std::min(num_sms, kPagedCtas) / items);
    if (p.splits < 1) p.splits = 1;
    return (int)launch_k(kern, dim3((unsigned)(vbs * p.nkv * p.splits), p.n), dim3(kWarps * 32), smem, st, p);
}

}  // namespace

size_t paged_scratch_bytes() {
    return kPagedCounterBytes + (size_t)2 * kPagedCtas * kPagedRowsTc * (128 + 2) * sizeof(float);
}

int launch_paged_attn_f32(PagedAttnParams& p, int d, int num_sms, cudaStream_t st) {
    p.launches = 1;
    return d == 128 ? launch_simt<float, 128>(p, num_sms, st) : launch_simt<float, 64>(p, num_sms, st);
}
int launch_paged_attn_bf16(PagedAttnParams& p, int d, int num_sms, cudaStream_t st) {
    return p.max_rows * p.G <= 16 ? launch_paged_decode(p, d, num_sms, st) : launch_paged_block(p, d, num_sms, st);
}

}  // namespace df
