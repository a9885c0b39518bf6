// Attention of many query rows (draft blocks, prompt chunks) over pages or a cache slab,
// bf16, on the 5th-generation tensor cores.
//
// The mathematics, the integer base and the equal shares are those of paged_decode.cu; here
// a row tile is up to 128 query vectors of one kv head (vector v = row * G + head), and S, P
// and O live in tensor memory.  Up to 64 (32) vectors fill CS = 2 (4) copies of a window of
// RW = 128 / CS lanes: lane l holds vector l % RW and takes key slice l / RW (64 / CS keys)
// of every tile, so all softmax warps have work.
//
//   warps 2-9  softmax, two groups of four warps that take the tiles in turn, each with its
//              own S and O in tensor memory and its own running base and sum per lane (they are
//              joined once per stretch: two chains hide each other's latencies, and nothing is
//              exchanged between warps inside a stretch).  Per tile: read the lane's slice of S,
//              mask it where the tile has keys that some row does not see, write P =
//              bf16(2^(t - b)), rescale O by an exact power of two when b moves.
//   warp 0     TMA: K and V tiles of 64 keys, one box per page and 64-column half.
//   warp 1     tcgen05.mma: S = Q K^T of a group's next tile once it has read the one before.
//   warp 10    tcgen05.mma: O += P V once P is there.  (Two issuers that each wait for one thing:
//              one that polled for both took 300 to 700 cycles to notice either.)
//
// An item that several CTAs hold is joined by a second launch (k_paged_join): adding up to 18
// partials of 32 KB took one CTA 15 us, all SMs together 2 us.
#include <algorithm>

#include "paged.cuh"

namespace df {

namespace {

constexpr int kThreads = 352;
constexpr int kSoftmax = 256;    // threads of the two softmax groups
constexpr float kBaseLag = 8.0f;
constexpr int kOverhead = 4;   // units that starting and ending an item costs, in tiles
constexpr int kMinShare = 8;   // smallest share of a CTA, in units

template <int D> struct BlockCfg {
    static constexpr int HALVES = D / 64;
    static constexpr int KV = HALVES * 64 * 128;             // bytes of a K (or V) tile
    static constexpr int STAGES = D == 128 ? 4 : 8;
    static constexpr int RING = STAGES * 2 * KV;
    static constexpr int OLD = D + 4;
    static constexpr int HLD = D / 2 + 4;
    static constexpr int JOIN = 256 * HLD * 4;               // >= 128 * OLD * 4
    static constexpr int SMEM = 1024 + RING + JOIN + 2 * 128 * 8 + kLineBytes + 512;
    static constexpr int SLOT = 128 * (D + 2);               // floats of a partial
    // tensor memory columns: S[2] (64 each), P[2] (32 bf16 pairs each), Q (D / 2), O[2] (D each)
    static constexpr uint32_t T_S = 0, T_P = 128, T_Q = 192, T_O = 256, COLS = 512;
};

template <int D, int CS>
__global__ void __launch_bounds__(kThreads, 1) k_paged_block(const __grid_constant__ PagedAttnParams p) {
    using C = BlockCfg<D>;
    constexpr int S = C::STAGES;
    constexpr int RW = 128 / CS, KC = 64 / CS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = smem_align_up<uint8_t>(smem_raw, 1024);          // [S][K, V]
    float* join = (float*)(ring + C::RING);                          // [128][OLD]
    float2* ml = (float2*)(ring + C::RING + C::JOIN);                // [2][128] base and sum per group and lane
    uint8_t* line_mem = (uint8_t*)(ml + 256);
    uint64_t* kv_full = (uint64_t*)(line_mem + kLineBytes);          // [S]
    uint64_t* kv_empty = kv_full + S;                                // [S]
    uint64_t* s_full = kv_empty + S;                                 // [2]
    uint64_t* p_full = s_full + 2;                                   // [2]
    uint64_t* o_done = p_full + 2;                                   // [2]
    uint64_t* s_read = o_done + 2;                                   // [2]
    uint64_t* q_full = s_read + 2;
    uint64_t* q_free = q_full + 1;
    uint64_t* drain = q_free + 1;                                    // [2]
    uint32_t* tmem_slot = (uint32_t*)(drain + 2);
    __shared__ int abort_s;
    __shared__ long long sums[kThreads / 32];
    volatile int* abort_flag = &abort_s;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int4* rec = (int4*)((uint8_t*)p.counters + kJoinRecords) + 2 * blockIdx.x;
    if (tid == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(&kv_full[i], 1);
            mbar_init(&kv_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&s_read[i], 4);
            mbar_init(&p_full[i], 4);
            mbar_init(&o_done[i], 1);
            mbar_init(&drain[i], 1);
        }
        mbar_init(q_full, 4);
        mbar_init(q_free, 8);
        abort_s = 0;
        fence_mbar_init();
        tma_prefetch_desc(&p.tmap_half);
    }
    griddep_wait();
    Line line;
    const long long U = line_plan<kThreads, D>(p, line, line_mem, sums, kOverhead);
    const int P = (int)min((long long)gridDim.x, max(1ll, U / kMinShare));
    if (tid == 64) rec[0] = make_int4(-1, 0, 0, 0);      // no item to join from here, so far
    if (U == 0 || (int)blockIdx.x >= P) return;
    Walker walk;
    walk.start(line, blockIdx.x * U / P, (blockIdx.x + 1) * U / P);
    Stretch s;
    uint32_t tmem = 0;
    if (warp > 0) {      // the producer does not wait for the tensor memory
        if (warp == 1) {
            tmem_alloc(tmem_slot, C::COLS);
            // The next kernel may start only once this CTA holds its tensor memory: a dependent
            // CTA on this SM that allocated first and then waited for this grid would never let go.
            griddep_launch();
        }
        tc_fence_before();
        named_bar_sync(2, kThreads - 32);
        tc_fence_after();
        tmem = *tmem_slot;
    }
    const uint32_t tS = tmem + C::T_S, tP = tmem + C::T_P, tQ = tmem + C::T_Q, tO = tmem + C::T_O;

    if (warp == 0) {
        // ------------------------------------------------------------ TMA producer
        const int bl = p.table ? min(p.ps_log2, 6) : 6;          // log2 rows of a box
        const int box_rows = 1 << bl, boxes = 64 >> bl;
        int it = 0;
        bool ok = true;
        while (ok && walk.next(line, s)) {
            const int4 e = line.ent[s.i];
            const int hi = p.causal ? e.w + s.r1 : e.w + e.z;
            const int lo = p.window > 0 ? max(0, e.w + s.r0 - p.window + 1) : 0;
            PageLookup look;
            look.reset();
            for (int t = s.t0; t < s.t1; ++t, ++it) {
                const int k0 = s.span.tile(t) * 64, st = it % S;
                // lane (kind, half, box)
                const int b = lane & (boxes - 1), h = lane / boxes % C::HALVES, kind = lane / boxes / C::HALVES;
                const int kb = k0 + b * box_rows;
                const int page = look.at(p, e.x, k0, kb, boxes, lane);
                const bool want = kind < 2 && kb < hi && (kb < p.sinks || kb + box_rows > lo) && page >= 0;
                ok = mbar_wait(&kv_empty[st], (uint32_t)(((it / S) & 1) ^ 1), abort_flag, p.wait_status);
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    break;
                }
                const int n_want = __popc(__ballot_sync(0xffffffffu, want));
                if (lane == 0) mbar_arrive_expect_tx(&kv_full[st], (uint32_t)(n_want * box_rows * 128));
                __syncwarp();
                if (want) {
                    const long long row = (long long)page * p.rows_page + p.row_layer + (long long)s.g * p.rows_kv +
                                          kind * p.rows_kind + (p.table ? kb & ((1 << p.ps_log2) - 1) : kb);
                    uint8_t* dst = ring + (st * 2 + kind) * C::KV + h * 8192 + b * box_rows * 128;
                    asm volatile(
                        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes "
                        "[%0], [%1, {%2, %3, %4}], [%5];"
                        ::"r"(smem_u32(dst)), "l"((uint64_t)&p.tmap_half), "r"(0), "r"((int)row), "r"(h),
                          "r"(smem_u32(&kv_full[st]))
                        : "memory");
                }
            }
        }
        if (!ok) {
            // an abandoned launch: its copies land before the CTA exits
            volatile int never = 0;
            for (int k = max(0, it - S); k < it; ++k) mbar_wait(&kv_full[k % S], (uint32_t)((k / S) & 1), &never, nullptr);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ S = Q K^T
        // The whole warp walks and waits, one elected lane issues: in code that the warp runs
        // together the operands stay in uniform registers (128 x 64 x 16 measured 33 cycles an
        // instruction against 47-70 in a branch of one lane).  S of tile j + 2 goes where S of
        // tile j was, as soon as the softmax has read that, so a group finds its next S waiting.
        constexpr uint32_t IDESC_S = idesc_bf16_f32(128, 64);
        const bool leader = elect_one();
        int it = 0, seg = 0;
        bool ok = true;
        for (; ok && walk.next(line, s); ++seg) {
            ok = __all_sync(0xffffffffu, mbar_wait(q_full, (uint32_t)(seg & 1), abort_flag, p.wait_status));
            for (int t = s.t0; t < s.t1 && ok; ++t, ++it) {
                const int st = it % S;
                ok = mbar_wait(&kv_full[st], (uint32_t)((it / S) & 1), abort_flag, p.wait_status);
                if (ok && it >= 2) ok = mbar_wait(&s_read[it & 1], (uint32_t)(((it - 2) >> 1) & 1), abort_flag, p.wait_status);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                const uint32_t ka = smem_u32(ring + st * 2 * C::KV), d = tS + (it & 1) * 64;
                if (leader) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        tc_mma_bf16_ts(d, tQ + kk * 8, umma_desc_sw128(ka + (kk >> 2) * 8192) + 2 * (kk & 3), IDESC_S,
                                       kk > 0 ? 1u : 0u);
                    tc_commit(&s_full[it & 1]);
                }
                __syncwarp();
            }
        }
        if (__any_sync(0xffffffffu, *abort_flag)) {
            if (leader) tc_commit(&drain[0]);   // the issued MMAs finish before the tensor memory is released
            __syncwarp();
            volatile int never = 0;
            mbar_wait(&drain[0], 0, &never, nullptr);
        }
    } else if (warp == 10) {
        // ------------------------------------------------------------ O += P V
        constexpr uint32_t IDESC_PV = idesc_bf16_f32(128, D, true);
        const bool leader = elect_one();
        int it = 0;
        bool ok = true;
        while (ok && walk.next(line, s)) {
            for (int t = s.t0; t < s.t1; ++t, ++it) {
                const int pb = it & 1;
                ok = mbar_wait(&p_full[pb], (uint32_t)((it >> 1) & 1), abort_flag, p.wait_status);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                const uint32_t va = smem_u32(ring + ((it % S) * 2 + 1) * C::KV), d = tO + pb * 128, a = tP + pb * 32;
                const uint32_t add = t >= s.t0 + 2 ? 1u : 0u;
                if (leader) {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        tc_mma_bf16_ts(d, a + kk * 8, umma_desc_sw128_mn(va + kk * 2048, 8192, 1024), IDESC_PV,
                                       kk > 0 ? 1u : add);
                    tc_commit(&o_done[pb]);
                    tc_commit(&kv_empty[it % S]);      // S of this tile was done before its P
                }
                __syncwarp();
            }
        }
        if (__any_sync(0xffffffffu, *abort_flag)) {
            if (leader) tc_commit(&drain[1]);
            __syncwarp();
            volatile int never = 0;
            mbar_wait(&drain[1], 0, &never, nullptr);
        }
    } else {
        // ------------------------------------------------------------ softmax
        const int w = (warp - 2) >> 2, q4 = warp & 3, rl = q4 * 32 + lane;
        const int row = rl % RW, cs = rl / RW;                 // vector of the tile, key slice (warp-uniform)
        const int e256 = tid - 64;
        const uint32_t lanes = (uint32_t)(q4 * 32) << 16;
        const uint32_t my_s = tS + lanes + w * 64, my_p = tP + lanes + w * 32, my_o = tO + lanes + w * 128;
        // the lane's vector of stretch x into the Q operand (zero past the tile's vectors)
        auto put_q = [&](const Stretch& x) {
            const int4 e = line.ent[x.i];
            const bool have = row < (x.r1 - x.r0) * p.G;
            const __nv_bfloat16* src = (const __nv_bfloat16*)p.q + (size_t)(e.y + x.r0 + row / p.G) * p.q_stride +
                                       (size_t)(x.g * p.G + row % p.G) * D;
            uint4 qv[D / 8];
#pragma unroll
            for (int k = 0; k < D / 8; ++k)
                qv[k] = have ? *reinterpret_cast<const uint4*>(src + 8 * k) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int c0 = 0; c0 < D / 2; c0 += 16) {
                float v[16];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint4 u = qv[c0 / 4 + k];
                    v[4 * k + 0] = __uint_as_float(u.x);
                    v[4 * k + 1] = __uint_as_float(u.y);
                    v[4 * k + 2] = __uint_as_float(u.z);
                    v[4 * k + 3] = __uint_as_float(u.w);
                }
                tmem_st16(tQ + lanes + c0, v);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full);
        };
        Stretch nx;
        bool more = walk.next(line, nx);
        if constexpr (CS > 1) {           // the other slices' columns of this lane's P stay zero
            const uint32_t z[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
            for (int c0 = 0; c0 < 32; c0 += 8) tmem_st8u(my_p + c0, z);
            tmem_wait_st();
        }
        if (more && w == 0) put_q(nx);
        int it0 = 0, seg = 0;             // tiles and stretches before this one
        bool ok = true;
        while (more && ok) {
            s = nx;
            more = walk.next(line, nx);
            const int4 e = line.ent[s.i];
            const int nvec = (s.r1 - s.r0) * p.G;
            const int pos = e.w + s.r0 + row / p.G;                    // this lane's position (padding lanes: any)
            const int hi_tile = p.causal ? e.w + s.r1 : e.w + e.z;     // keys that exist for some row
            const int lo_tile = p.window > 0 ? max(0, e.w + s.r0 - p.window + 1) : 0;
            const int hi_all = p.causal ? e.w + s.r0 + 1 : hi_tile;    // keys below are seen by all rows ..
            const int lo_all = p.window > 0 ? e.w + s.r1 - p.window : 0;   // .. from here on
            const int hi_row = p.causal ? min(pos + 1, hi_tile) : hi_tile;
            const int lo_row = p.window > 0 ? pos - p.window + 1 : 0;
            float base = -INFINITY, l = 0.f;
            int last = -1;                                             // this group's last tile
            for (int t = s.t0 + ((it0 ^ w) & 1); t < s.t1; t += 2) {
                const int it = it0 + t - s.t0;
                last = it;
                ok = mbar_wait(&s_full[w], (uint32_t)((it >> 1) & 1), abort_flag, p.wait_status);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                // the product of the group's tile before has read P and written O (looked at early,
                // waited for where it matters)
                const bool o_ready = it < 2 || mbar_test(&o_done[w], (uint32_t)(((it - 2) >> 1) & 1));
                const int k0 = s.span.tile(t) * 64, kvb = k0 + cs * KC;
                float x[KC];
                if constexpr (KC == 64) {
                    tmem_ld32w(my_s, x);
                    tmem_ld32w(my_s + 32, x + 32);
                } else if constexpr (KC == 32) {
                    tmem_ld32w(my_s + cs * KC, x);
                } else {
                    tmem_ld16w(my_s + cs * KC, x);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s_read[w]);
                // tiles with keys that some row does not see
                if (k0 + 64 > hi_all || (k0 < lo_all && k0 + 64 > p.sinks)) {
#pragma unroll
                    for (int i = 0; i < KC; ++i) {
                        const int k = kvb + i;
                        if (!(k < hi_row && (k >= lo_row || k < p.sinks))) x[i] = -INFINITY;
                    }
                    // V rows that no row sees may hold anything (0 * NaN is NaN): zero them
                    uint8_t* vs = ring + ((it % S) * 2 + 1) * C::KV;
                    for (int idx = rl; idx < 64 * C::HALVES * 8; idx += 128) {
                        const int r = idx / (C::HALVES * 8), rem = idx % (C::HALVES * 8), k = k0 + r;
                        if (k >= hi_tile || (k < lo_tile && k >= p.sinks))
                            *reinterpret_cast<uint4*>(vs + (rem / 8) * 8192 + r * 128 + (rem % 8) * 16) = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async();   // the product reads these rows through the async proxy
                }
                float m8[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) m8[k] = x[k];
#pragma unroll
                for (int i = 8; i < KC; ++i) m8[i & 7] = fmaxf(m8[i & 7], x[i]);
                const float nb = floorf(fmaxf(fmaxf(fmaxf(m8[0], m8[1]), fmaxf(m8[2], m8[3])),
                                              fmaxf(fmaxf(m8[4], m8[5]), fmaxf(m8[6], m8[7]))) * p.scale_log2);
                const bool grow = nb > base + kBaseLag;
                if (!__all_sync(0xffffffffu, o_ready)) {
                    ok = mbar_wait(&o_done[w], (uint32_t)(((it - 2) >> 1) & 1), abort_flag, p.wait_status);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                }
                tc_fence_after();
                if (__any_sync(0xffffffffu, grow)) {
                    if (t >= s.t0 + 2) {   // O holds earlier tiles
                        const float f = grow ? exp2f(base - nb) : 1.0f;
#pragma unroll 1
                        for (int c0 = 0; c0 < D; c0 += 16) {
                            float v[16];
                            tmem_ld16w(my_o + c0, v);
#pragma unroll
                            for (int i = 0; i < 16; ++i) v[i] *= f;
                            tmem_st16(my_o + c0, v);
                        }
                        l *= f;
                    }
                    if (grow) base = nb;
                }
                const float bb = (base == -INFINITY) ? 0.f : base;
                float ls[KC / 16];
#pragma unroll
                for (int c0 = 0; c0 < KC; c0 += 16) {
                    float s2 = 0.f;
                    uint32_t pk[8];
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        const float e0 = ex2_fast(fmaf(x[c0 + i], p.scale_log2, -bb));
                        const float e1 = ex2_fast(fmaf(x[c0 + i + 1], p.scale_log2, -bb));
                        s2 += e0 + e1;
                        pk[i / 2] = pack_bf16(e0, e1);
                    }
                    ls[c0 >> 4] = s2;
                    tmem_st8u(my_p + cs * (KC / 2) + c0 / 2, pk);
                }
#pragma unroll
                for (int i = 0; i < KC / 16; ++i) l += ls[i];
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[w]);
            }
            // this warp has read its last S of the stretch; when all have, Q may change
            __syncwarp();
            if (lane == 0) mbar_arrive(q_free);
            if (ok && more && w == 0) {
                ok = mbar_wait(q_free, (uint32_t)(seg & 1), abort_flag, p.wait_status);
                ok = __all_sync(0xffffffffu, ok);
                if (ok) put_q(nx);
            }
            ++seg;
            if (ok && last >= 0)
                ok = mbar_wait(&o_done[w], (uint32_t)((last >> 1) & 1), abort_flag, p.wait_status);
            ml[w * 128 + rl] = make_float2(base, l);
            if (named_bar_or(1, kSoftmax, !ok)) {
                ok = false;
                break;
            }
            tc_fence_after();
            // ---- the stretch's rows: the groups' O are added, then the copies of a vector.  Bases
            // differ by integers, so all factors are exact powers of two.
            const bool whole = s.whole(), head = s.t0 == 0;   // head: holds the item's first tile
            float* slot = p.partial + (size_t)(2 * blockIdx.x + (head ? 1 : 0)) * C::SLOT;
            if constexpr (CS == 1) {
                // each group finishes half the columns: it gives the other half away
                const float2 other = ml[(w ^ 1) * 128 + rl];
                const float B = fmaxf(base, other.x), z = B == -INFINITY ? 0.f : B;
                const float f0 = last >= 0 ? exp2f(base - z) : 0.f, f1 = exp2f(other.x - z);
                const float L = f0 * l + f1 * other.y, inv = L == 0.f ? 0.f : 1.0f / L;
                float* mine = join + (w * 128 + rl) * C::HLD;
                const float* theirs = join + ((w ^ 1) * 128 + rl) * C::HLD;
                const uint32_t keep = my_o + w * (D / 2), give = my_o + (w ^ 1) * (D / 2);
#pragma unroll
                for (int c0 = 0; c0 < D / 2; c0 += 32) {
                    float v[32];
                    tmem_ld32w(give + c0, v);
#pragma unroll
                    for (int i = 0; i < 32; i += 4)
                        *reinterpret_cast<float4*>(mine + c0 + i) =
                            last >= 0 ? make_float4(f0 * v[i], f0 * v[i + 1], f0 * v[i + 2], f0 * v[i + 3])
                                      : make_float4(0.f, 0.f, 0.f, 0.f);
                }
                named_bar_sync(1, kSoftmax);
                __nv_bfloat16* dst = (__nv_bfloat16*)p.out +
                                     ((size_t)(e.y + s.r0 + row / p.G) * p.nq + (size_t)s.g * p.G + row % p.G) * D + w * (D / 2);
                float* part = slot + 256 + row * D + w * (D / 2);
#pragma unroll
                for (int c0 = 0; c0 < D / 2; c0 += 32) {
                    float v[32];
                    tmem_ld32w(keep + c0, v);
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        const float4 o = *reinterpret_cast<const float4*>(theirs + c0 + i);
                        v[i] = (last >= 0 ? f0 * v[i] : 0.f) + o.x;
                        v[i + 1] = (last >= 0 ? f0 * v[i + 1] : 0.f) + o.y;
                        v[i + 2] = (last >= 0 ? f0 * v[i + 2] : 0.f) + o.z;
                        v[i + 3] = (last >= 0 ? f0 * v[i + 3] : 0.f) + o.w;
                    }
                    if (row < nvec) {
                        if (whole) {
#pragma unroll
                            for (int i = 0; i < 32; i += 8)
                                *reinterpret_cast<uint4*>(dst + c0 + i) =
                                    make_uint4(pack_bf16(v[i] * inv, v[i + 1] * inv), pack_bf16(v[i + 2] * inv, v[i + 3] * inv),
                                               pack_bf16(v[i + 4] * inv, v[i + 5] * inv), pack_bf16(v[i + 6] * inv, v[i + 7] * inv));
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; i += 4)
                                *reinterpret_cast<float4*>(part + c0 + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                        }
                    }
                }
                if (!whole && w == 0 && row < nvec) *reinterpret_cast<float2*>(slot + 2 * row) = make_float2(B, L);
            } else {
                // group 1's O to shared memory, group 0 adds its own
                if (w == 1) {
#pragma unroll 1
                    for (int c0 = 0; c0 < D; c0 += 32) {
                        float v[32];
                        tmem_ld32w(my_o + c0, v);
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
                            *reinterpret_cast<float4*>(join + rl * C::OLD + c0 + i) =
                                last >= 0 ? make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]) : make_float4(0.f, 0.f, 0.f, 0.f);
                    }
                }
                named_bar_sync(1, kSoftmax);
                if (w == 0) {
                    const float2 other = ml[128 + rl];
                    const float B = fmaxf(base, other.x), z = B == -INFINITY ? 0.f : B;
                    const float f0 = exp2f(base - z), f1 = exp2f(other.x - z);
#pragma unroll 1
                    for (int c0 = 0; c0 < D; c0 += 32) {
                        float v[32];
                        tmem_ld32w(my_o + c0, v);
#pragma unroll
                        for (int i = 0; i < 32; i += 4) {
                            float4* d4 = reinterpret_cast<float4*>(join + rl * C::OLD + c0 + i);
                            float4 o = *d4;
                            o.x = (last >= 0 ? f0 * v[i] : 0.f) + f1 * o.x;
                            o.y = (last >= 0 ? f0 * v[i + 1] : 0.f) + f1 * o.y;
                            o.z = (last >= 0 ? f0 * v[i + 2] : 0.f) + f1 * o.z;
                            o.w = (last >= 0 ? f0 * v[i + 3] : 0.f) + f1 * o.w;
                            *d4 = o;
                        }
                    }
                    ml[rl] = make_float2(B, f0 * l + f1 * other.y);
                }
                named_bar_sync(1, kSoftmax);
            for (int i = e256; i < nvec * (D / 8); i += kSoftmax) {
                const int v = i / (D / 8), c = (i % (D / 8)) * 8;
                float B = -INFINITY, L = 0.f, a[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int k = 0; k < CS; ++k) B = fmaxf(B, ml[v + k * RW].x);
                const float z = B == -INFINITY ? 0.f : B;
#pragma unroll
                for (int k = 0; k < CS; ++k) {
                    const float2 m = ml[v + k * RW];
                    const float f = exp2f(m.x - z);
                    const float4 w0 = *reinterpret_cast<const float4*>(join + (v + k * RW) * C::OLD + c);
                    const float4 w1 = *reinterpret_cast<const float4*>(join + (v + k * RW) * C::OLD + c + 4);
                    L += f * m.y;
                    a[0] += f * w0.x; a[1] += f * w0.y; a[2] += f * w0.z; a[3] += f * w0.w;
                    a[4] += f * w1.x; a[5] += f * w1.y; a[6] += f * w1.z; a[7] += f * w1.w;
                }
                if (whole) {
                    const float inv = L == 0.f ? 0.f : 1.0f / L;
                    __nv_bfloat16* dst = (__nv_bfloat16*)p.out +
                                         ((size_t)(e.y + s.r0 + v / p.G) * p.nq + (size_t)s.g * p.G + v % p.G) * D + c;
                    *reinterpret_cast<uint4*>(dst) =
                        make_uint4(pack_bf16(a[0] * inv, a[1] * inv), pack_bf16(a[2] * inv, a[3] * inv),
                                   pack_bf16(a[4] * inv, a[5] * inv), pack_bf16(a[6] * inv, a[7] * inv));
                } else {
                    *reinterpret_cast<float4*>(slot + 256 + v * D + c) = make_float4(a[0], a[1], a[2], a[3]);
                    *reinterpret_cast<float4*>(slot + 256 + v * D + c + 4) = make_float4(a[4], a[5], a[6], a[7]);
                    if (c == 0) *reinterpret_cast<float2*>(slot + 2 * v) = make_float2(B, L);
                }
            }
            }
            if (!whole && head && e256 == 0) {
                rec[0] = make_int4(line_owner(s.v0 + kOverhead + s.span.nt - 1, U, P), nvec, e.y + s.r0, s.g);
            }
            it0 += s.t1 - s.t0;
            named_bar_sync(1, kSoftmax);      // join and ml are free again
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::COLS);
    }
}

// Join of the items that several CTAs hold: block (c, y) takes 256 of the 8-column pieces of
// the item whose first tile CTA c held, and adds the partials of CTAs c .. rec.x in order.
template <int D>
__global__ void __launch_bounds__(256) k_paged_join(const __grid_constant__ PagedAttnParams p) {
    constexpr int SLOT = BlockCfg<D>::SLOT;
    griddep_wait();
    griddep_launch();
    const int c0 = blockIdx.x;
    const int4 rec = *((const int4*)((const uint8_t*)p.counters + kJoinRecords) + 2 * c0);
    const int i = blockIdx.y * 256 + threadIdx.x;
    if (rec.x < 0 || i >= rec.y * (D / 8)) return;
    const int v = i / (D / 8), c = (i % (D / 8)) * 8;
    float B = -INFINITY, L = 0.f, a[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int k0 = c0; k0 <= rec.x; k0 += 4) {     // four partials' loads in flight
        float2 m[4];
        float4 w0[4], w1[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int cta = min(k0 + k, rec.x);
            const float* q = p.partial + (size_t)(2 * cta + (cta == c0 ? 1 : 0)) * SLOT;
            m[k] = *reinterpret_cast<const float2*>(q + 2 * v);
            w0[k] = *reinterpret_cast<const float4*>(q + 256 + v * D + c);
            w1[k] = *reinterpret_cast<const float4*>(q + 256 + v * D + c + 4);
        }
        float nb = B;
#pragma unroll
        for (int k = 0; k < 4; ++k) nb = fmaxf(nb, m[k].x);
        const float z = nb == -INFINITY ? 0.f : nb;
        const float f0 = exp2f(B - z);
        B = nb;
        L *= f0;
#pragma unroll
        for (int j = 0; j < 8; ++j) a[j] *= f0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (k0 + k > rec.x) break;
            const float f = exp2f(m[k].x - z);
            L += f * m[k].y;
            a[0] += f * w0[k].x; a[1] += f * w0[k].y; a[2] += f * w0[k].z; a[3] += f * w0[k].w;
            a[4] += f * w1[k].x; a[5] += f * w1[k].y; a[6] += f * w1[k].z; a[7] += f * w1[k].w;
        }
    }
    const float inv = L == 0.f ? 0.f : 1.0f / L;
    __nv_bfloat16* dst = (__nv_bfloat16*)p.out + ((size_t)(rec.z + v / p.G) * p.nq + (size_t)rec.w * p.G + v % p.G) * D + c;
    *reinterpret_cast<uint4*>(dst) =
        make_uint4(pack_bf16(a[0] * inv, a[1] * inv), pack_bf16(a[2] * inv, a[3] * inv),
                   pack_bf16(a[4] * inv, a[5] * inv), pack_bf16(a[6] * inv, a[7] * inv));
}

template <int D, int CS>
int launch_dc(const PagedAttnParams& p, int num_sms, cudaStream_t st) {
    auto kern = k_paged_block<D, CS>;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, BlockCfg<D>::SMEM) != cudaSuccess) return 1;
    const int ctas = std::min(num_sms, kPagedCtas), pieces = p.rt * p.G * (D / 8);
    cudaError_t e = launch_k(kern, dim3(ctas), dim3(kThreads), BlockCfg<D>::SMEM, st, p);
    if (e == cudaSuccess) e = launch_k(k_paged_join<D>, dim3(ctas, (pieces + 255) / 256), dim3(256), 0, st, p);
    return (int)e;
}
template <int D>
int launch_d(const PagedAttnParams& p, int vectors, int num_sms, cudaStream_t st) {
    if (vectors <= 32) return launch_dc<D, 4>(p, num_sms, st);
    if (vectors <= 64) return launch_dc<D, 2>(p, num_sms, st);
    return launch_dc<D, 1>(p, num_sms, st);
}

}  // namespace

int launch_paged_block(PagedAttnParams& p, int d, int num_sms, cudaStream_t st) {
    p.launches = 2;
    p.rt = std::min(p.max_rows, kPagedRowsTc / p.G);
    p.row_tiles = (p.max_rows + p.rt - 1) / p.rt;
    return d == 128 ? launch_d<128>(p, p.rt * p.G, num_sms, st) : launch_d<64>(p, p.rt * p.G, num_sms, st);
}

}  // namespace df
