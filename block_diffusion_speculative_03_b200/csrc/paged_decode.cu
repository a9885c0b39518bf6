// Attention of few query rows (at most 16 per kv head: one new token of up to 16
// query heads per kv head, or a short block) over pages, bf16: split over the keys and
// joined.
//
// With t_k = q.k log2(e) / sqrt(d), out = sum_k P_k v_k / sum_k 2^(t_k - b), P_k =
// 2^(t_k - b) in two bf16 terms, for an integer b per row.  (One term costs 2^-9 of each weight:
// 0.0025 off in all, against 0.0017 for rounding the output alone; the second term's products
// fit beside the loads: 4 x 32768 keys take the same time, one of 2048 0.4 us more.)  b follows the running maximum (kBaseLag,
// kBaseLead): moving b scales everything by an exact power of two, so the split points
// and the order of the keys change no rounding of P.
//
// Bound by HBM: every K and V byte is read once, and there are only 2 * rows flops for
// each.  So all SMs stream equal shares whatever the lengths (Line in paged.cuh).  An
// item held by one CTA is finished there; otherwise its CTAs write partials (b, l, o) and
// the last to arrive adds them in the order of the keys (nobody waits).
//
//   warp 0     TMA: K and V boxes of min(page_size, 64) rows (both 64-column halves of a
//              row group in one box) into a ring; pages are looked up 32 at a time.
//              Boxes in which no row sees a key are not loaded.
//   warps 1-8  two groups of four that take the tiles in turn, 16 keys of a tile per warp, with
//              their own running state: S = Q K^T and
//              O += P V on m16n8k16 tensor instructions, P's terms staying in registers (the
//              accumulator layout of S is the operand layout of P).  No barrier between
//              the warps until the end of the item.  (At 16 rows the tensor work is 1/8 of
//              what the loads leave time for, so the register path wins over tensor memory:
//              no hand-offs between issuing, softmax and correction.)
//
// Measured in a captured graph, one token, 32 heads on 8 of 128: 4 sequences of 32768 85.2 us (537 MB,
// 6.3 TB/s, 97 % of a copy; 88 us, 94 %, as calls one after another); one of 2048 10.0 us (10.9), of which
// 1.3 are HBM: the launch, the dependent reads of the plan (list, length, table), the first load, and
// the join of 3-tile shares make up the rest.
#include <algorithm>

#include "paged.cuh"

namespace df {

namespace {

constexpr int kConsumers = 8;      // two groups of four warps take the tiles in turn
constexpr int kThreads = 32 + 32 * kConsumers;
constexpr int kTileKeys = kLineTile;
// Units that starting and joining an item costs, in tiles (32 sequences of 1 to 8191, 4 kv heads: 18.2 us
// with 4, 18.8 with 6, 19.0 with 3, 19.2 with 2).
constexpr int kOverhead = 4;
// Smallest share of a CTA, in units (one sequence of 2048, 8 kv heads: 9.9 us with 3, 9.3 with 4, 9.7 with
// 5, 10.3 with 7; one of 512, one head: 7.0, 7.2, 7.9, 7.2).
constexpr int kMinShare = 3;

template <int D> struct DecodeCfg {
    static constexpr int TILE = kTileKeys * D * 2;           // bytes of a K (or V) tile
    static constexpr int STAGES = D == 128 ? 4 : 8;
    static constexpr int RING = STAGES * 2 * TILE;
    static constexpr int OLD = D + 4;                        // row stride of the join buffer (floats)
    static constexpr int JOIN = kConsumers * 16 * OLD * 4;
    // (base, sum) pairs: a warp's 16 rows each, or one for every consumer thread (a long join's teams)
    static constexpr int PAIRS = kConsumers * 32;
    // offsets from the aligned start: ring, join buffer, pairs, plan, barriers
    static constexpr int JOIN_AT = RING, PAIRS_AT = JOIN_AT + JOIN, LINE_AT = PAIRS_AT + PAIRS * 8;
    static constexpr int BARS_AT = LINE_AT + kLineBytes, SMEM = 1024 + BARS_AT + 256;
    static constexpr int SLOT = 16 * (D + 2);                // floats of a partial
    static_assert(LINE_AT - PAIRS_AT >= kConsumers * 32 * 8 && JOIN >= kConsumers * 32 * 16,
                  "a long join keeps a pair and four columns of every consumer thread");
    static_assert(2 * STAGES * 8 <= 256 && SMEM <= 227 * 1024, "shared memory");
};
// Teams of E = rows * D / 4 threads that share a long join.
__host__ __device__ constexpr int join_teams(int E) { return kConsumers * 32 / E < 8 ? kConsumers * 32 / E : 8; }

DF_DEV void ldsm4(uint32_t a, uint32_t* r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
DF_DEV void ldsm4t(uint32_t a, uint32_t* r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
DF_DEV void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
DF_DEV void tma_load_3d(void* dst, const CUtensorMap* m, uint64_t* bar, int x, int y, int z, uint64_t pol) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint "
        "[%0], [%1, {%2, %3, %4}], [%5], %6;"
        ::"r"(smem_u32(dst)), "l"((uint64_t)m), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar)), "l"(pol)
        : "memory");
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) k_paged_decode(const __grid_constant__ PagedAttnParams p) {
    using C = DecodeCfg<D>;
    constexpr int S = C::STAGES, NT8 = D / 8;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = smem_align_up<uint8_t>(smem_raw, 1024);
    float* join = (float*)(ring + C::JOIN_AT);                       // [kConsumers][16][OLD]; long join: [threads][4]
    float2* join_ml = (float2*)(ring + C::PAIRS_AT);                 // [kConsumers][16]; long join: [threads]
    uint8_t* line_mem = ring + C::LINE_AT;
    uint64_t* full = (uint64_t*)(ring + C::BARS_AT);
    uint64_t* empty = full + S;
    __shared__ int abort_s, flag_s;
    __shared__ long long sums[kThreads / 32];
    volatile int* abort_flag = &abort_s;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], kConsumers / 2);
        }
        abort_s = 0;
        fence_mbar_init();
        tma_prefetch_desc(&p.tmap);
    }
    griddep_wait();
    griddep_launch();

    Line line;
    const int U = line_plan<kThreads, D>(p, line, line_mem, sums, kOverhead);
    const int P = min((int)gridDim.x, max(1, U / kMinShare));
    if (U == 0 || (int)blockIdx.x >= P) return;
    const Shares shares(U, P);
    Walker<false> walk;
    walk.start(line, shares.begin(blockIdx.x), shares.begin(blockIdx.x + 1));
    Stretch s;
    const int bl = p.table ? min(p.ps_log2, 6) : 6;          // log2 rows of a TMA box
    const int box_rows = 1 << bl, boxes = kTileKeys >> bl;

    if (warp == 0) {
        // ------------------------------------------------------------ TMA producer
        const uint64_t pol = make_l2_policy_evict_first();
        int it = 0;
        bool ok = true;
        while (ok && walk.next(line, s)) {
            const int4 e = line.ent[s.i];
            const int hi = e.w + e.z, lo = p.window > 0 ? max(0, e.w - p.window + 1) : 0;
            PageLookup look;
            look.reset();
            for (int t = s.t0; t < s.t1; ++t, ++it) {
                const int k0 = s.span.tile(t) * kTileKeys, st = it % S;
                // lane b: box b of K, lane boxes + b: box b of V
                const int b = lane & (boxes - 1), kind = lane / boxes, kb = k0 + b * box_rows;
                const bool want = kind < 2 && kb < hi && (kb < p.sinks || kb + box_rows > lo);
                const int page = look.at(p, e.x, k0, kb, boxes, lane);
                ok = mbar_wait_warp(&empty[st], (uint32_t)(((it / S) & 1) ^ 1), abort_flag, p.wait_status);
                if (!ok) break;
                const int n_want = __popc(__ballot_sync(0xffffffffu, want && page >= 0));
                if (lane == 0) mbar_arrive_expect_tx(&full[st], (uint32_t)(n_want * box_rows * D * 2));
                __syncwarp();
                if (want && page >= 0) {
                    const long long row = (long long)page * p.rows_page + p.row_layer + (long long)s.g * p.rows_kv +
                                          kind * p.rows_kind + (p.table ? kb & ((1 << p.ps_log2) - 1) : kb);
                    tma_load_3d(ring + st * 2 * C::TILE + kind * C::TILE + b * box_rows * D * 2, &p.tmap, &full[st], 0,
                                (int)row, 0, pol);
                }
            }
        }
        if (!ok) {
            // an abandoned launch: its copies land before the CTA exits
            volatile int never = 0;
            for (int k = max(0, it - S); k < it; ++k) mbar_wait_warp(&full[k % S], (uint32_t)((k / S) & 1), &never, nullptr);
        }
        return;
    }

    // ---------------------------------------------------------------- consumers
    const int cw = (warp - 1) & 3, group = (warp - 1) >> 2, jw = warp - 1, c_tid = tid - 32;
    const int qr = lane >> 2, qc = (lane & 3) * 2;            // accumulator row and first column of this lane
    // ldmatrix row of this lane: K: matrices (keys 0-7, 8 columns), (keys 0-7, next 8), (keys 8-15, ..), ..;
    // V transposed: (keys 0-7, columns), (keys 8-15, columns), (keys 0-7, next 8), ..
    const int kk = cw * 16 + (lane & 7) + ((lane >> 4) << 3);
    const int vk = cw * 16 + (lane & 7) + (((lane >> 3) & 1) << 3);
    const int kc8 = (lane >> 3) & 1, vc8 = lane >> 4;         // which 16-byte column of a pair
    auto row_addr = [&](int k) -> uint32_t {                  // byte offset of key k's first half in a tile
        return (uint32_t)((k >> bl) * box_rows * D * 2 + (k & (box_rows - 1)) * 128);
    };
    const uint32_t k_off = row_addr(kk), v_off = row_addr(vk), half = (uint32_t)box_rows * 128;
    const uint32_t ring_a = smem_u32(ring);

    int it0 = 0;                                              // tiles before this stretch
    bool ok = true;
    while (walk.next(line, s)) {
        const int4 e = line.ent[s.i];
        const int R = e.z * p.G, hi = e.w + e.z, lo = p.window > 0 ? max(0, e.w - p.window + 1) : 0;
        // this lane's two rows: vector v = row * G + head
        const int ra = qr * p.g_magic >> 16, rb = (qr + 8) * p.g_magic >> 16;
        const int pos_a = e.w + ra, pos_b = e.w + rb;
        const int hi_a = qr < R ? (p.causal ? pos_a + 1 : hi) : 0, hi_b = qr + 8 < R ? (p.causal ? pos_b + 1 : hi) : 0;
        uint32_t qf[D / 16][4];
        {
            const __nv_bfloat16* q = (const __nv_bfloat16*)p.q;
            const __nv_bfloat16* qa = q + (size_t)(e.y + ra) * p.q_stride + (size_t)(s.g * p.G + qr - ra * p.G) * D + qc;
            const __nv_bfloat16* qb = q + (size_t)(e.y + rb) * p.q_stride + (size_t)(s.g * p.G + qr + 8 - rb * p.G) * D + qc;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                qf[k][0] = qr < R ? *reinterpret_cast<const uint32_t*>(qa + k * 16) : 0u;
                qf[k][2] = qr < R ? *reinterpret_cast<const uint32_t*>(qa + k * 16 + 8) : 0u;
                qf[k][1] = qr + 8 < R ? *reinterpret_cast<const uint32_t*>(qb + k * 16) : 0u;
                qf[k][3] = qr + 8 < R ? *reinterpret_cast<const uint32_t*>(qb + k * 16 + 8) : 0u;
            }
        }
        float o[NT8][4];
#pragma unroll
        for (int j = 0; j < NT8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
        float base_a = -INFINITY, base_b = -INFINITY, l_a = 0.f, l_b = 0.f;

        for (int t = s.t0 + ((it0 ^ group) & 1); t < s.t1; t += 2) {
            const int it = it0 + t - s.t0, st = it % S;
            if (ok) ok = mbar_wait_warp(&full[st], (uint32_t)((it / S) & 1), abort_flag, p.wait_status);
            if (!ok) continue;
            const int kw = s.span.tile(t) * kTileKeys + cw * 16;          // this warp's first key
            const uint32_t sk = ring_a + st * 2 * C::TILE, sv = sk + C::TILE;
            float sc[2][4];
#pragma unroll
            for (int j = 0; j < 2; ++j) sc[j][0] = sc[j][1] = sc[j][2] = sc[j][3] = 0.f;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                uint32_t b[4];
                ldsm4(sk + k_off + (k >> 2) * half + ((((k & 3) * 2 + kc8) ^ (kk & 7)) << 4), b);
                mma16816(sc[0], qf[k], b[0], b[1]);
                mma16816(sc[1], qf[k], b[2], b[3]);
            }
            // keys that some row does not see: the last ones, and with a window those before it
            if (kw + 16 > (p.causal ? e.w + 1 : hi) ||
                (p.window > 0 && kw + 16 > p.sinks && kw <= hi - 1 - p.window)) {
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int key = kw + j * 8 + qc + c;
                        if (!key_visible(key, pos_a, hi_a, p.window, p.sinks)) sc[j][c] = -INFINITY;
                        if (!key_visible(key, pos_b, hi_b, p.window, p.sinks)) sc[j][2 + c] = -INFINITY;
                    }
                // V rows that no row sees may hold anything (0 * NaN is NaN): zero them
                const int key = kw + (lane >> 1);
                const bool dead = key >= hi || (p.window > 0 && key >= p.sinks && key < lo);
                if (dead) {
                    uint8_t* vr = ring + st * 2 * C::TILE + C::TILE + row_addr(cw * 16 + (lane >> 1));
#pragma unroll
                    for (int h = 0; h < D / 64; ++h)
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            *reinterpret_cast<uint4*>(vr + h * half + ((lane & 1) * 4 + c) * 16) = make_uint4(0, 0, 0, 0);
                }
                __syncwarp();
            }
            const float ma = fmaxf(fmaxf(sc[0][0], sc[0][1]), fmaxf(sc[1][0], sc[1][1])) * p.scale_log2;
            const float mb = fmaxf(fmaxf(sc[0][2], sc[0][3]), fmaxf(sc[1][2], sc[1][3])) * p.scale_log2;
            if (__any_sync(0xffffffffu, floorf(ma) > base_a + kBaseLag || floorf(mb) > base_b + kBaseLag)) {
                float xa = fmaxf(ma, __shfl_xor_sync(0xffffffffu, ma, 1));
                float xb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, 1));
                xa = floorf(fmaxf(xa, __shfl_xor_sync(0xffffffffu, xa, 2)));
                xb = floorf(fmaxf(xb, __shfl_xor_sync(0xffffffffu, xb, 2)));
                const float na = xa > base_a + kBaseLag ? xa + kBaseLead : base_a;
                const float nb = xb > base_b + kBaseLag ? xb + kBaseLead : base_b;
                const float fa = na == base_a ? 1.f : pow2_int(base_a - na), fb = nb == base_b ? 1.f : pow2_int(base_b - nb);
                base_a = na;
                base_b = nb;
                l_a *= fa;
                l_b *= fb;
#pragma unroll
                for (int j = 0; j < NT8; ++j) {
                    o[j][0] *= fa;
                    o[j][1] *= fa;
                    o[j][2] *= fb;
                    o[j][3] *= fb;
                }
            }
            const float za = base_a == -INFINITY ? 0.f : base_a, zb = base_b == -INFINITY ? 0.f : base_b;
            // P in two terms, bf16(P) and bf16(P - bf16(P)): 16 bits of it
            uint32_t pf[4], pl[4];
            auto rest = [](float x, float y, uint32_t hi) {
                return pack_bf16(x - __uint_as_float(hi << 16), y - __uint_as_float(hi & 0xffff0000u));
            };
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float p0 = ex2_fast(fmaf(sc[j][0], p.scale_log2, -za)), p1 = ex2_fast(fmaf(sc[j][1], p.scale_log2, -za));
                const float p2 = ex2_fast(fmaf(sc[j][2], p.scale_log2, -zb)), p3 = ex2_fast(fmaf(sc[j][3], p.scale_log2, -zb));
                l_a += p0 + p1;
                l_b += p2 + p3;
                pf[j * 2] = pack_bf16(p0, p1);
                pf[j * 2 + 1] = pack_bf16(p2, p3);
                pl[j * 2] = rest(p0, p1, pf[j * 2]);
                pl[j * 2 + 1] = rest(p2, p3, pf[j * 2 + 1]);
            }
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
                uint32_t b[4];
                ldsm4t(sv + v_off + (j >> 2) * half + ((((j & 3) * 2 + vc8) ^ (vk & 7)) << 4), b);
                mma16816(o[2 * j], pf, b[0], b[1]);
                mma16816(o[2 * j + 1], pf, b[2], b[3]);
                mma16816(o[2 * j], pl, b[0], b[1]);
                mma16816(o[2 * j + 1], pl, b[2], b[3]);
            }
            // The reads of V come before the next tile's copy (another proxy): without the fence the compiler
            // may leave one for after the arrive, and where the loop ends and new code has to be fetched
            // the copy overtook it (10^-10 of all reads: 14 of 250000 calls on 4 x 32768 keys were off
            // in their last bits).
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[st]);
        }
        // ---- join the warps
        l_a += __shfl_xor_sync(0xffffffffu, l_a, 1);
        l_b += __shfl_xor_sync(0xffffffffu, l_b, 1);
        l_a += __shfl_xor_sync(0xffffffffu, l_a, 2);
        l_b += __shfl_xor_sync(0xffffffffu, l_b, 2);
        if ((lane & 3) == 0) {
            join_ml[jw * 16 + qr] = make_float2(base_a, l_a);
            join_ml[jw * 16 + qr + 8] = make_float2(base_b, l_b);
        }
#pragma unroll
        for (int j = 0; j < NT8; ++j) {
            if (qr < R) *reinterpret_cast<float2*>(join + (jw * 16 + qr) * C::OLD + j * 8 + qc) = make_float2(o[j][0], o[j][1]);
            if (qr + 8 < R)
                *reinterpret_cast<float2*>(join + (jw * 16 + qr + 8) * C::OLD + j * 8 + qc) = make_float2(o[j][2], o[j][3]);
        }
        named_bar_sync(1, kConsumers * 32);
        const bool whole = s.whole(), head = s.t0 == 0;   // head: holds the item's first tile
        float* slot = p.partial + (size_t)(2 * blockIdx.x + (head ? 1 : 0)) * C::SLOT;
        for (int x = c_tid; x < R * (D / 4); x += kConsumers * 32) {
            const int r = x / (D / 4), c = (x % (D / 4)) * 4;
            float B = -INFINITY;
#pragma unroll
            for (int w = 0; w < kConsumers; ++w) B = fmaxf(B, join_ml[w * 16 + r].x);
            const float z = B == -INFINITY ? 0.f : B;
            float L = 0.f;
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kConsumers; ++w) {
                const float2 ml = join_ml[w * 16 + r];
                const float f = pow2_int(ml.x - z);
                const float4 v = *reinterpret_cast<const float4*>(join + (w * 16 + r) * C::OLD + c);
                L += f * ml.y;
                a.x += f * v.x;
                a.y += f * v.y;
                a.z += f * v.z;
                a.w += f * v.w;
            }
            if (whole) {
                const float inv = L == 0.f ? 0.f : 1.0f / L;
                __nv_bfloat16* dst = (__nv_bfloat16*)p.out + ((size_t)(e.y + (r * p.g_magic >> 16)) * p.nq + (size_t)s.g * p.G + r - (r * p.g_magic >> 16) * p.G) * D + c;
                *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16(a.x * inv, a.y * inv), pack_bf16(a.z * inv, a.w * inv));
            } else {
                *reinterpret_cast<float4*>(slot + 32 + r * D + c) = a;
                if (c == 0) *reinterpret_cast<float2*>(slot + 2 * r) = make_float2(B, L);
            }
        }
        if (!whole) {
            // the CTAs that hold the item's first and last tile
            const int c0 = shares.owner(s.v0 + kOverhead), c1 = shares.owner(s.v0 + kOverhead + s.span.nt - 1);
            named_bar_sync(1, kConsumers * 32);
            if (c_tid == 0) {
                // releases the block's partial (the barrier above) and acquires the others'
                const int before = atom_add_acq_rel(&p.counters[c0], 1);
                flag_s = before == c1 - c0;
                if (before == c1 - c0) p.counters[c0] = 0;      // ready for the next launch
            }
            named_bar_sync(1, kConsumers * 32);
            if (flag_s) {
                auto part = [&](int c) { return p.partial + (size_t)(2 * c + (c == c0 ? 1 : 0)) * C::SLOT; };
                // adds the partials of CTAs k, k + 1, .. k + 7, k + step, .. to (B, L, a)
                auto gather = [&](int r, int c, int k, int step, float& B, float& L, float4& a) {
                    for (int k0 = k; k0 <= c1; k0 += step) {      // eight partials' loads in flight
                        float2 ml[8];
                        float4 v[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float* q = part(min(k0 + j, c1));
                            ml[j] = __ldcg(reinterpret_cast<const float2*>(q + 2 * r));
                            v[j] = __ldcg(reinterpret_cast<const float4*>(q + 32 + r * D + c));
                        }
                        float nb = B;
#pragma unroll
                        for (int j = 0; j < 8; ++j) nb = fmaxf(nb, ml[j].x);
                        const float z = nb == -INFINITY ? 0.f : nb, g = pow2_int(B - z);
                        B = nb;
                        L *= g;
                        a.x *= g;
                        a.y *= g;
                        a.z *= g;
                        a.w *= g;
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            if (k0 + j > c1) break;
                            const float f = pow2_int(ml[j].x - z);
                            L += f * ml[j].y;
                            a.x += f * v[j].x;
                            a.y += f * v[j].y;
                            a.z += f * v[j].z;
                            a.w += f * v[j].w;
                        }
                    }
                };
                auto store = [&](int r, int c, float L, const float4& a) {
                    const float inv = L == 0.f ? 0.f : 1.0f / L;
                    const int v = r * p.g_magic >> 16;
                    __nv_bfloat16* dst = (__nv_bfloat16*)p.out +
                                         ((size_t)(e.y + v) * p.nq + (size_t)s.g * p.G + r - v * p.G) * D + c;
                    *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16(a.x * inv, a.y * inv), pack_bf16(a.z * inv, a.w * inv));
                };
                const int E = R * (D / 4), teams = join_teams(E);
                if (c1 - c0 < 8 || teams < 2) {
                    for (int x = c_tid; x < E; x += kConsumers * 32) {
                        float B = -INFINITY, L = 0.f;
                        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
                        gather(x / (D / 4), (x % (D / 4)) * 4, c0, 8, B, L, a);
                        store(x / (D / 4), (x % (D / 4)) * 4, L, a);
                    }
                } else {
                    // few rows, many partials: teams of threads take eight partials each in turn (one
                    // sequence of 32768, one kv head, 4 rows, 148 partials: 26.4 us, 43.2 without; one row:
                    // 14.5, 44.0; of 2048, 8 kv heads of 4 rows, 12 partials: 9.9, 10.0)
                    const int team = c_tid / E, x = c_tid - team * E, r = x / (D / 4), c = (x % (D / 4)) * 4;
                    float B = -INFINITY, L = 0.f;
                    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (team < teams) {
                        gather(r, c, c0 + team * 8, teams * 8, B, L, a);
                        join_ml[c_tid] = make_float2(B, L);
                        *reinterpret_cast<float4*>(join + c_tid * 4) = a;
                    }
                    named_bar_sync(1, kConsumers * 32);
                    if (team == 0) {
                        float M = B;
                        for (int k = 1; k < teams; ++k) M = fmaxf(M, join_ml[k * E + x].x);
                        const float z = M == -INFINITY ? 0.f : M, f0 = pow2_int(B - z);
                        L *= f0;
                        a.x *= f0;
                        a.y *= f0;
                        a.z *= f0;
                        a.w *= f0;
                        for (int k = 1; k < teams; ++k) {
                            const float2 ml = join_ml[k * E + x];
                            const float4 v = *reinterpret_cast<const float4*>(join + (k * E + x) * 4);
                            const float f = pow2_int(ml.x - z);
                            L += f * ml.y;
                            a.x += f * v.x;
                            a.y += f * v.y;
                            a.z += f * v.z;
                            a.w += f * v.w;
                        }
                        store(r, c, L, a);
                    }
                }
            }
        }
        it0 += s.t1 - s.t0;
        named_bar_sync(1, kConsumers * 32);          // the join buffer and flag_s are free again
    }
}

template <int D>
int launch_d(const PagedAttnParams& p, int num_sms, cudaStream_t st) {
    auto kern = k_paged_decode<D>;
    if (!allow_smem<D * 8>((const void*)kern, DecodeCfg<D>::SMEM)) return 1;
    return (int)launch_k(kern, dim3(std::min(num_sms, kPagedCtas)), dim3(kThreads), DecodeCfg<D>::SMEM, st, p);
}

template <int D> void join_room(int rows, int* room) {
    using C = DecodeCfg<D>;
    const int E = rows * (D / 4), threads = join_teams(E) * E;
    room[0] = std::max(kConsumers * 16, threads);
    room[1] = (C::LINE_AT - C::PAIRS_AT) / 8;
    room[2] = std::max(((kConsumers - 1) * 16 + rows) * C::OLD, threads * 4);
    room[3] = (C::PAIRS_AT - C::JOIN_AT) / 4;
}

}  // namespace

bool paged_decode_join_room(int d, int rows, int* room) {
    if ((d != 64 && d != 128) || rows < 1 || rows > 16) return false;
    d == 128 ? join_room<128>(rows, room) : join_room<64>(rows, room);
    return true;
}

int launch_paged_decode(PagedAttnParams& p, int d, int num_sms, cudaStream_t st) {
    p.rt = p.max_rows;
    p.row_tiles = 1;
    p.g_magic = (65536 + p.G - 1) / p.G;
    p.launches = 1;
    return d == 128 ? launch_d<128>(p, num_sms, st) : launch_d<64>(p, num_sms, st);
}

}  // namespace df
