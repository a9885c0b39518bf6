// Attention of many query rows (draft blocks, prompt chunks) over pages or a cache slab,
// bf16, on the 5th-generation tensor cores.
//
// The mathematics, the integer base and the equal shares are those of paged_decode.cu; here
// a row tile is up to 128 query vectors of one kv head (vector v = row * G + head), and S and
// O live in tensor memory.  Up to 64 (32) vectors fill CS = 2 (4) copies of a window of
// RW = 128 / CS lanes: lane l holds vector l % RW and takes key slice l / RW (64 / CS keys)
// of every tile, so all four softmax warps have work.
//
//   warps 2-5  softmax, one lane per thread: read the lane's slice of S, mask it where the
//              tile has keys that some row does not see, write P = bf16(2^(t - b)) as the
//              next product's operand, rescale O by an exact power of two when b moves; at
//              the end of a stretch join the copies in shared memory and write the rows, or a
//              partial that the last CTA to arrive adds to the others in key order.
//   warp 0     TMA: K and V tiles of 64 keys, one box per page and 64-column half.
//   warp 1     tcgen05.mma: S = Q K^T up to three tiles ahead of the softmax (across the end
//              of a stretch too: the next stretch's Q is already in the other Q buffer), and
//              O += P V.
#include <algorithm>

#include "paged.cuh"

namespace df {

namespace {

constexpr int kThreads = 192;
constexpr float kBaseLag = 8.0f;
constexpr int kOverhead = 4;   // units that starting and ending an item costs, in tiles
constexpr int kMinShare = 8;   // smallest share of a CTA, in units

template <int D> struct BlockCfg {
    static constexpr int HALVES = D / 64;
    static constexpr int KV = HALVES * 64 * 128;             // bytes of a K (or V) tile
    static constexpr int STAGES = D == 128 ? 4 : 8;
    static constexpr int RING = STAGES * 2 * KV;
    static constexpr int NS = 3;                             // S buffers in tensor memory
    static constexpr int OLD = D + 4;
    static constexpr int JOIN = 128 * OLD * 4;
    static constexpr int SMEM = 1024 + RING + JOIN + 128 * 8 + 128 * 4 + kLineBytes + 512;
    static constexpr int SLOT = 128 * (D + 2);               // floats of a partial
    // tensor memory columns: S[NS] (64 each), Q[2] (D / 2 bf16 pairs), O (D), P[2] (32)
    static constexpr uint32_t T_S = 0, T_Q0 = 192, T_O = 256, T_P = 384, T_Q1 = 448, COLS = 512;
    static_assert(T_Q0 + D / 2 <= T_O && T_O + D <= T_P && T_P + 64 <= T_Q1 && T_Q1 + D / 2 <= COLS, "tensor memory");
};

template <int D, int CS>
__global__ void __launch_bounds__(kThreads, 1) k_paged_block(const __grid_constant__ PagedAttnParams p) {
    using C = BlockCfg<D>;
    constexpr int S = C::STAGES, NS = C::NS;
    constexpr int RW = 128 / CS, KC = 64 / CS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = smem_align_up<uint8_t>(smem_raw, 1024);          // [S][K, V]
    float* join = (float*)(ring + C::RING);                          // [128][OLD]
    float2* ml = (float2*)(ring + C::RING + C::JOIN);                // [128] base, sum per vector
    float* xch = (float*)(ml + 128);                                 // [128] per lane: maximum, then sum
    uint8_t* line_mem = (uint8_t*)(xch + 128);
    uint64_t* kv_full = (uint64_t*)(line_mem + kLineBytes);          // [S]
    uint64_t* kv_empty = kv_full + S;                                // [S]
    uint64_t* s_full = kv_empty + S;                                 // [NS]
    uint64_t* p_full = s_full + NS;                                  // [2]
    uint64_t* o_done = p_full + 2;                                   // [2]
    uint64_t* q_full = o_done + 2;                                   // [2]
    uint64_t* drain = q_full + 2;
    uint32_t* tmem_slot = (uint32_t*)(drain + 1);
    __shared__ int abort_s, flag_s;
    __shared__ long long sums[kThreads / 32];
    volatile int* abort_flag = &abort_s;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(&kv_full[i], 1);
            mbar_init(&kv_empty[i], 1);
        }
        for (int i = 0; i < NS; ++i) mbar_init(&s_full[i], 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&p_full[i], 128);
            mbar_init(&o_done[i], 1);
            mbar_init(&q_full[i], 128);
        }
        mbar_init(drain, 1);
        abort_s = 0;
        fence_mbar_init();
        tma_prefetch_desc(&p.tmap_half);
    }
    griddep_wait();
    Line line;
    const long long U = line_plan<kThreads, D>(p, line, line_mem, sums, kOverhead);
    const int P = (int)min((long long)gridDim.x, max(1ll, U / kMinShare));
    if (U == 0 || (int)blockIdx.x >= P) return;
    if (warp == 1) tmem_alloc(tmem_slot, C::COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // The next kernel may start only once this CTA holds its tensor memory: a dependent CTA
    // on this SM that allocated first and then waited for this grid would never let go.
    griddep_launch();
    const uint32_t tmem = *tmem_slot;
    const uint32_t tS = tmem + C::T_S, tO = tmem + C::T_O, tP = tmem + C::T_P;
    auto tQ = [&](int b) { return tmem + (b ? C::T_Q1 : C::T_Q0); };
    Walker walk;
    walk.start(line, blockIdx.x * U / P, (blockIdx.x + 1) * U / P);
    Stretch s;

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
        // ------------------------------------------------------------ MMA issuer
        if (lane == 0) {
            constexpr uint32_t IDESC_S = idesc_bf16_f32(128, 64);
            constexpr uint32_t IDESC_PV = idesc_bf16_f32(128, D, true);
            // S runs up to NS tiles ahead of the products, on its own walk over the stretches, but
            // at most one stretch ahead: the softmax brings the Q of stretch n + 1 when it begins
            // stretch n, for which the products of stretch n - 1 must have been issued.
            Walker sw = walk;
            Stretch ss;
            int sj = 0, s_seg = -1, s_left = 0, seg = -1, it = 0;
            bool more = true, ok = true;
            auto s_step = [&]() {      // the next tile's S, if its stretch, Q and K are there
                if (s_left == 0) {
                    if (!more || s_seg > seg) return;
                    more = sw.next(line, ss);
                    if (!more) return;
                    ++s_seg;
                    s_left = ss.t1 - ss.t0;
                }
                const int st = sj % S;
                if (!mbar_test(&q_full[s_seg & 1], (uint32_t)((s_seg >> 1) & 1)) ||
                    !mbar_test(&kv_full[st], (uint32_t)((sj / S) & 1)))
                    return;
                tc_fence_after();
                const uint32_t ka = smem_u32(ring + st * 2 * C::KV);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    tc_mma_bf16_ts(tS + (sj % NS) * 64, tQ(s_seg & 1) + kk * 8,
                                   umma_desc_sw128(ka + (kk >> 2) * 8192) + 2 * (kk & 3), IDESC_S, kk > 0 ? 1u : 0u);
                tc_commit(&s_full[sj % NS]);
                ++sj;
                --s_left;
            };
            while (ok && walk.next(line, s)) {
                ++seg;
                for (int t = s.t0; t < s.t1 && ok; ++t, ++it) {
                    const int pb = it & 1;
                    // whichever comes first: K of a tile ahead (its S buffer is free: the softmax has
                    // read S of the tiles before `it`), or P of this tile
                    uint64_t since = 0;
                    for (uint32_t n = 1;; ++n) {
                        if (sj < it + NS) s_step();
                        if (sj > it && mbar_test(&p_full[pb], (uint32_t)((it >> 1) & 1))) break;
                        if ((n & 1023u) == 0) {
                            const uint64_t now = globaltimer_ns();
                            if (!since) since = now;
                            if (!*abort_flag && now - since > kWaitLimitNs) {
                                *abort_flag = 1;
                                if (p.wait_status) atomicCAS(p.wait_status, 0, DFLASH_TIMEOUT);
                            }
                            if (*abort_flag) {
                                ok = false;
                                break;
                            }
                        }
                    }
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t va = smem_u32(ring + ((it % S) * 2 + 1) * C::KV);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        tc_mma_bf16_ts(tO, tP + pb * 32 + kk * 8, umma_desc_sw128_mn(va + kk * 2048, 8192, 1024),
                                       IDESC_PV, (t > s.t0 || kk > 0) ? 1u : 0u);
                    tc_commit(&o_done[pb]);
                    tc_commit(&kv_empty[it % S]);
                }
            }
            if (*abort_flag) {
                tc_commit(drain);   // the issued MMAs finish before the tensor memory is released
                volatile int never = 0;
                mbar_wait(drain, 0, &never, nullptr);
            }
        }
    } else {
        // ------------------------------------------------------------ softmax
        const int q4 = warp & 3, rl = q4 * 32 + lane;
        const int row = rl % RW, cs = rl / RW;                 // vector of the tile, key slice (warp-uniform)
        const int e128 = tid - 64;
        const uint32_t lanes = (uint32_t)(q4 * 32) << 16;
        // the lane's vector of stretch x into Q buffer b (zero past the tile's vectors)
        auto put_q = [&](const Stretch& x, int b) {
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
                    const uint4 w = qv[c0 / 4 + k];
                    v[4 * k + 0] = __uint_as_float(w.x);
                    v[4 * k + 1] = __uint_as_float(w.y);
                    v[4 * k + 2] = __uint_as_float(w.z);
                    v[4 * k + 3] = __uint_as_float(w.w);
                }
                tmem_st16(tQ(b) + lanes + c0, v);
            }
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&q_full[b]);
        };
        Stretch nx;
        bool more = walk.next(line, nx);
        {
            float z[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) z[i] = 0.f;
            // the other slices' columns of this lane's P stay zero
#pragma unroll
            for (int c0 = 0; c0 < 64; c0 += 16) tmem_st16(tP + lanes + c0, z);
            tmem_wait_st();
            if (more) put_q(nx, 0);
        }
        int it = 0, seg = 0;
        bool ok = true;
        while (more && ok) {
            s = nx;
            more = walk.next(line, nx);
            // the other Q buffer is free: the softmax has read all of the stretch before this one
            if (more) put_q(nx, (seg + 1) & 1);
            ++seg;
            const int4 e = line.ent[s.i];
            const int nvec = (s.r1 - s.r0) * p.G;
            const int pos = e.w + s.r0 + row / p.G;                    // this lane's position (padding lanes: any)
            const int hi_tile = p.causal ? e.w + s.r1 : e.w + e.z;     // keys that exist for some row
            const int lo_tile = p.window > 0 ? max(0, e.w + s.r0 - p.window + 1) : 0;
            const int hi_all = p.causal ? e.w + s.r0 + 1 : hi_tile;    // keys below are seen by all rows ..
            const int lo_all = p.window > 0 ? e.w + s.r1 - p.window : 0;   // .. from here on
            const int hi_row = p.causal ? min(pos + 1, hi_tile) : hi_tile;
            const int lo_row = p.window > 0 ? pos - p.window + 1 : 0;
            float base = -INFINITY, mt = -INFINITY, l = 0.f;
            for (int t = s.t0; t < s.t1; ++t, ++it) {
                const int sb = it & 1, sbuf = it % NS;
                ok = mbar_wait(&s_full[sbuf], (uint32_t)((it / NS) & 1), abort_flag, p.wait_status);
                tc_fence_after();
                const int k0 = s.span.tile(t) * 64, kvb = k0 + cs * KC;
                const uint32_t ts = tS + lanes + sbuf * 64 + cs * KC;
                float x[KC];
                if constexpr (KC == 64) {
                    tmem_ld32w(ts, x);
                    tmem_ld32w(ts + 32, x + 32);
                } else if constexpr (KC == 32) {
                    tmem_ld32w(ts, x);
                } else {
                    tmem_ld16w(ts, x);
                }
                // tiles with keys that some row does not see
                const bool edge = k0 + 64 > hi_all || (k0 < lo_all && k0 + 64 > p.sinks);
                if (edge) {
#pragma unroll
                    for (int i = 0; i < KC; ++i) {
                        const int k = kvb + i;
                        if (!(k < hi_row && (k >= lo_row || k < p.sinks))) x[i] = -INFINITY;
                    }
                }
                float m8[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) m8[k] = x[k];
#pragma unroll
                for (int i = 8; i < KC; ++i) m8[i & 7] = fmaxf(m8[i & 7], x[i]);
                const float mx = fmaxf(fmaxf(fmaxf(m8[0], m8[1]), fmaxf(m8[2], m8[3])),
                                       fmaxf(fmaxf(m8[4], m8[5]), fmaxf(m8[6], m8[7])));
                mt = fmaxf(mt, mx * p.scale_log2);
                if (ok && it >= 2)     // the product of tile it - 2 has read this P buffer
                    ok = mbar_wait(&o_done[sb], (uint32_t)(((it - 2) >> 1) & 1), abort_flag, p.wait_status);
                const bool growl = floorf(mt) > base + kBaseLag;
                if (named_bar_or(1, 128, !ok || growl)) {
                    if (named_bar_or(1, 128, !ok)) {
                        ok = false;
                        break;
                    }
                    xch[rl] = mt;
                    named_bar_sync(1, 128);
                    float mrow = mt;
#pragma unroll
                    for (int k = 1; k < CS; ++k) mrow = fmaxf(mrow, xch[(rl + k * RW) & 127]);
                    const float nb = floorf(mrow);
                    const bool grow = nb > base + kBaseLag;
                    if (t > s.t0) {
                        ok = mbar_wait(&o_done[(it - 1) & 1], (uint32_t)(((it - 1) >> 1) & 1), abort_flag, p.wait_status);
                        if (named_bar_or(1, 128, !ok)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const float f = grow ? exp2f(base - nb) : 1.0f;
#pragma unroll 1
                        for (int c0 = 0; c0 < D; c0 += 16) {
                            float v[16];
                            tmem_ld16w(tO + lanes + c0, v);
#pragma unroll
                            for (int i = 0; i < 16; ++i) v[i] *= f;
                            tmem_st16(tO + lanes + c0, v);
                        }
                        tmem_wait_st();
                        l *= f;
                    } else {
                        named_bar_sync(1, 128);     // xch is read before it is written again
                    }
                    if (grow) base = nb;
                }
                if (edge) {
                    // V rows that no row sees may hold anything (0 * NaN is NaN): zero them
                    uint8_t* vs = ring + ((it % S) * 2 + 1) * C::KV;
                    for (int idx = e128; idx < 64 * C::HALVES * 8; idx += 128) {
                        const int r = idx / (C::HALVES * 8), rem = idx % (C::HALVES * 8), k = k0 + r;
                        if (k >= hi_tile || (k < lo_tile && k >= p.sinks))
                            *reinterpret_cast<uint4*>(vs + (rem / 8) * 8192 + r * 128 + (rem % 8) * 16) = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async();   // the product reads these rows through the async proxy
                }
                const float bb = (base == -INFINITY) ? 0.f : base;
                uint32_t pk[KC / 2];
                float ls[KC / 16];
#pragma unroll
                for (int c0 = 0; c0 < KC; c0 += 16) {
                    float s2 = 0.f;
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        const float e0 = ex2_fast(fmaf(x[c0 + i], p.scale_log2, -bb));
                        const float e1 = ex2_fast(fmaf(x[c0 + i + 1], p.scale_log2, -bb));
                        s2 += e0 + e1;
                        pk[(c0 + i) / 2] = pack_bf16(e0, e1);
                    }
                    ls[c0 >> 4] = s2;
                }
                const uint32_t tp = tP + lanes + sb * 32 + cs * (KC / 2);
#pragma unroll
                for (int c0 = 0; c0 < KC / 2; c0 += 8) tmem_st8u(tp + c0, pk + c0);
#pragma unroll
                for (int i = 0; i < KC / 16; ++i) l += ls[i];
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(&p_full[sb]);
            }
            if (ok) ok = mbar_wait(&o_done[(it - 1) & 1], (uint32_t)(((it - 1) >> 1) & 1), abort_flag, p.wait_status);
            if (named_bar_or(1, 128, !ok)) {
                ok = false;
                break;
            }
            tc_fence_after();
            // ---- the stretch's rows: lanes to shared memory, copies of a vector added
            xch[rl] = l;
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 32) {
                float v[32];
                tmem_ld32w(tO + lanes + c0, v);
#pragma unroll
                for (int i = 0; i < 32; i += 4)
                    *reinterpret_cast<float4*>(join + rl * C::OLD + c0 + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
            }
            if (cs == 0) ml[row].x = base;      // the copies of a vector agree on the base
            named_bar_sync(1, 128);
            if (cs == 0) {
                float L = l;
#pragma unroll
                for (int k = 1; k < CS; ++k) L += xch[row + k * RW];
                ml[row].y = L;
            }
            named_bar_sync(1, 128);
            const bool whole = s.whole(), head = s.t0 == 0;
            float* slot = p.partial + (size_t)(2 * blockIdx.x + (head ? 1 : 0)) * C::SLOT;
            __nv_bfloat16* out = (__nv_bfloat16*)p.out;
            auto out_at = [&](int v, int c) {
                return out + ((size_t)(e.y + s.r0 + v / p.G) * p.nq + (size_t)s.g * p.G + v % p.G) * D + c;
            };
            for (int i = e128; i < nvec * (D / 8); i += 128) {
                const int v = i / (D / 8), c = (i % (D / 8)) * 8;
                float a[8];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float4 w = *reinterpret_cast<const float4*>(join + v * C::OLD + c + 4 * h);
#pragma unroll
                    for (int k = 1; k < CS; ++k) {
                        const float4 w2 = *reinterpret_cast<const float4*>(join + (v + k * RW) * C::OLD + c + 4 * h);
                        w.x += w2.x;
                        w.y += w2.y;
                        w.z += w2.z;
                        w.w += w2.w;
                    }
                    a[4 * h] = w.x;
                    a[4 * h + 1] = w.y;
                    a[4 * h + 2] = w.z;
                    a[4 * h + 3] = w.w;
                }
                if (whole) {
                    const float L = ml[v].y, inv = L == 0.f ? 0.f : 1.0f / L;
                    *reinterpret_cast<uint4*>(out_at(v, c)) =
                        make_uint4(pack_bf16(a[0] * inv, a[1] * inv), pack_bf16(a[2] * inv, a[3] * inv),
                                   pack_bf16(a[4] * inv, a[5] * inv), pack_bf16(a[6] * inv, a[7] * inv));
                } else {
                    *reinterpret_cast<float4*>(slot + 256 + v * D + c) = make_float4(a[0], a[1], a[2], a[3]);
                    *reinterpret_cast<float4*>(slot + 256 + v * D + c + 4) = make_float4(a[4], a[5], a[6], a[7]);
                    if (c == 0) *reinterpret_cast<float2*>(slot + 2 * v) = ml[v];
                }
            }
            if (!whole) {
                const int c0 = line_owner(s.v0 + kOverhead, U, P), c1 = line_owner(s.v0 + kOverhead + s.span.nt - 1, U, P);
                __threadfence();
                named_bar_sync(1, 128);
                if (e128 == 0) {
                    const int before = atomicAdd(&p.counters[c0], 1);
                    flag_s = before == c1 - c0;
                    if (before == c1 - c0) p.counters[c0] = 0;      // ready for the next launch
                }
                named_bar_sync(1, 128);
                if (flag_s) {
                    __threadfence();
                    auto part = [&](int c) { return p.partial + (size_t)(2 * c + (c == c0 ? 1 : 0)) * C::SLOT; };
                    for (int i = e128; i < nvec * (D / 8); i += 128) {
                        const int v = i / (D / 8), c = (i % (D / 8)) * 8;
                        float B = -INFINITY;
#pragma unroll 4
                        for (int k = c0; k <= c1; ++k) B = fmaxf(B, __ldcg(part(k) + 2 * v));
                        const float z = B == -INFINITY ? 0.f : B;
                        float L = 0.f, a[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
                        for (int k = c0; k <= c1; ++k) {
                            const float* q = part(k);
                            const float2 m = __ldcg(reinterpret_cast<const float2*>(q + 2 * v));
                            const float4 w0 = __ldcg(reinterpret_cast<const float4*>(q + 256 + v * D + c));
                            const float4 w1 = __ldcg(reinterpret_cast<const float4*>(q + 256 + v * D + c + 4));
                            const float f = exp2f(m.x - z);
                            L += f * m.y;
                            a[0] += f * w0.x; a[1] += f * w0.y; a[2] += f * w0.z; a[3] += f * w0.w;
                            a[4] += f * w1.x; a[5] += f * w1.y; a[6] += f * w1.z; a[7] += f * w1.w;
                        }
                        const float inv = L == 0.f ? 0.f : 1.0f / L;
                        *reinterpret_cast<uint4*>(out_at(v, c)) =
                            make_uint4(pack_bf16(a[0] * inv, a[1] * inv), pack_bf16(a[2] * inv, a[3] * inv),
                                       pack_bf16(a[4] * inv, a[5] * inv), pack_bf16(a[6] * inv, a[7] * inv));
                    }
                }
            }
            named_bar_sync(1, 128);      // join, ml, xch and flag_s are free again
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::COLS);
    }
}

template <int D, int CS>
int launch_dc(const PagedAttnParams& p, int num_sms, cudaStream_t st) {
    auto kern = k_paged_block<D, CS>;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, BlockCfg<D>::SMEM) != cudaSuccess) return 1;
    return (int)launch_k(kern, dim3(std::min(num_sms, kPagedCtas)), dim3(kThreads), BlockCfg<D>::SMEM, st, p);
}
template <int D>
int launch_d(const PagedAttnParams& p, int vectors, int num_sms, cudaStream_t st) {
    if (vectors <= 32) return launch_dc<D, 4>(p, num_sms, st);
    if (vectors <= 64) return launch_dc<D, 2>(p, num_sms, st);
    return launch_dc<D, 1>(p, num_sms, st);
}

}  // namespace

int launch_paged_block(PagedAttnParams& p, int d, int num_sms, cudaStream_t st) {
    p.rt = std::min(p.max_rows, kPagedRowsTc / p.G);
    p.row_tiles = (p.max_rows + p.rt - 1) / p.rt;
    return d == 128 ? launch_d<128>(p, p.rt * p.G, num_sms, st) : launch_d<64>(p, p.rt * p.G, num_sms, st);
}

}  // namespace df
