// Attention of many query rows (draft blocks, prompt chunks) over pages or a cache slab,
// bf16, on the 5th-generation tensor cores.
//
// The mathematics, the integer base and the equal shares are those of paged_decode.cu, with one
// bf16 term of P as in the draft step's attention (a second made prompts 14 % slower, blocks 3 %); here
// a row tile is up to 128 query vectors of one kv head (vector v = row * G + head), and S, P
// and O live in tensor memory.  Up to 64 (32) vectors fill CS = 2 (4) copies of a window of
// RW = 128 / CS lanes: lane l holds vector l % RW and takes key slice l / RW (64 / CS keys)
// of every tile, so all softmax warps have work.
//
//   warps 2-9  softmax, two groups of four warps that take the tiles in turn and hide each
//              other's latencies.  Per tile: read S, mask it where the tile has keys that some
//              row does not see, take over the running base from the tile before (the other
//              group's, through shared memory), move it if a maximum has passed it (then O is
//              rescaled, by an exact power of two), write P = bf16(2^(t - b)).
//   warp 0, 11 TMA: K and V tiles of 64 keys, one box per page and 64-column half; both also
//              stage the next stretch's Q.
//   warp 1     tcgen05.mma: S = Q K^T into the next of kBufs buffers; a tile's P takes the place
//              of its S, so a buffer is free again when the tile's product is done.
//   warp 10    tcgen05.mma: O += P V once P is there.  (Two issuers that each wait for one thing:
//              one that polled for both took 300 to 700 cycles to notice either.)
//
// An item that several CTAs hold is joined by a second launch (k_paged_join): adding up to 18
// partials of 32 KB took one CTA 15 us, all SMs together 2 us.
//
// Few rows on long contexts are bound by HBM (32 sequences of 4000 with 8 heads of 128, 8 rows of
// 4 heads: 98 us for 524 MB, 5.4 TB/s), many rows by the softmax warps: 2048 rows of 32 heads of 128
// behind 6000 positions with a window of 2048 take 86.7 us in a captured graph, 0.79 PFLOP/s of products
// (96.7 us, 0.71, as calls one after another; without the window 212 us, 1.1 PFLOP/s), at 900 cycles a
// tile where the tensor cores need 520 and the exponentials 512, and 6000 cycles more for each
// stretch's end and beginning.  What the time is not: taking out exponentials, conversions or most
// of the products changed it by less than 1 %; it is the waits and the chain read S - maximum -
// exponentials - write P of each group.  Three buffers and an O for each group (the chain then ran
// through the product and back) took 95 us; three groups 89, a thread to half a row 106.
#include <algorithm>

#include "paged.cuh"

namespace df {

namespace {

// Units that starting and ending an item costs, in tiles (9 entries of up to 700 rows, 2 kv heads:
// 16.4 us with 8, 16.8 with 10, 15.9 with 6; 2048 rows of one entry: 86.0, 85.8, 87.5).
constexpr int kOverhead = 8;
// Smallest share of a CTA, in units (the same entries: 15.3 us with 4 or 5, 16.0 with 8, 16.8 with 14; of
// calls of 7 to 18 us most are faster with 5 than with 8, by up to 1.5 us, some slower, by as much).
constexpr int kMinShare = 5;

constexpr int kThreads = 384;
constexpr int kSoftmax = 256;    // threads of the two softmax groups
constexpr int kPvWarp = 10;

constexpr int kBufs = 5;         // buffers of S in tensor memory

template <int D> constexpr int kSlot = 128 * (D + 2);        // floats of a partial

template <int D, int CS> struct BlockCfg {
    static constexpr int HALVES = D / 64;
    static constexpr int KV = HALVES * 64 * 128;             // bytes of a K (or V) tile
    static constexpr int STAGES = D == 64 ? 6 : CS == 1 ? 4 : 3;   // of K and of V
    static constexpr int RING = STAGES * 2 * KV;
    static constexpr int OLD = D + 4;
    static constexpr int QLD = D * 2 + 16;                   // bytes of a staged vector: 16 more, so that lanes hit all banks
    static constexpr int JOIN = CS == 1 ? 128 * QLD : 128 * OLD * 4;
    static constexpr int SMEM = 1024 + RING + JOIN + 4 * 128 * 8 + 128 * QLD + kLineBytes + 512;
    static_assert(SMEM <= 227 * 1024, "shared memory");
    // tensor memory columns: S[kBufs] (64 each; P over the first 32), Q (D / 2), O (D)
    static constexpr uint32_t T_S = 0, T_Q = kBufs * 64, T_O = 384, COLS = 512;
};

// The lowest n bits (n below 0: none, above 32: all).
DF_DEV uint32_t bits_below(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; }

// Floats of a partial: (base, sum) of the 128 vectors, then o, four columns of all vectors after
// one another (a warp's lanes hold consecutive vectors: whole lines per store).
DF_DEV int part_at(int v, int c) { return 256 + ((c >> 2) * 128 + v) * 4 + (c & 3); }

// Vectors [v0, v1) of a stretch's Q to q_stage by thread x of n (a multiple of 32): 16-byte
// pieces, whole rows per group of lanes.  (A softmax lane that read its own 256-byte row from
// global memory touched 32 lines per load: 2500 cycles; one bulk copy per row took 7000.)
template <int D>
DF_DEV void stage_q(const PagedAttnParams& p, const Line& line, const Stretch& s, uint8_t* q_stage, int v0, int v1, int x,
                    int n) {
    const int4 e = line.ent[s.i];
    const int c = x % (D / 8) * 8, step = n / (D / 8);
    v1 = min(v1, (s.r1 - s.r0) * p.G);
#pragma unroll 2
    for (int v = v0 + x / (D / 8); v < v1; v += step) {
        const int r = v * p.g_magic >> 16;
        const __nv_bfloat16* src = (const __nv_bfloat16*)p.q + (size_t)(e.y + s.r0 + r) * p.q_stride +
                                   (s.g * p.G + v - r * p.G) * D + c;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                     ::"r"(smem_u32(q_stage) + v * BlockCfg<D, 1>::QLD + c * 2), "l"((uint64_t)src) : "memory");
    }
}

template <int D, int CS>
__global__ void __launch_bounds__(kThreads, 1) k_paged_block(const __grid_constant__ PagedAttnParams p) {
    using C = BlockCfg<D, CS>;
    constexpr int S = C::STAGES;
    constexpr int RW = 128 / CS, KC = 64 / CS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = smem_align_up<uint8_t>(smem_raw, 1024);          // K [S], V [S]
    uint8_t* join = ring + C::RING;                                  // the stretch's rows on their way out
    float2* ml = (float2*)(join + C::JOIN);                          // [2][128] base and sum per group and lane
    float* base_s = (float*)(ml + 256);                              // [2][128] the base after a group's tile
    uint8_t* q_stage = (uint8_t*)(ml + 512);                         // [128][QLD] the next stretch's Q
    uint8_t* line_mem = q_stage + 128 * C::QLD;
    uint64_t* kv_full = (uint64_t*)(line_mem + kLineBytes);          // [2][S]: K, V
    uint64_t* kv_empty = kv_full + 2 * S;                            // [2][S]
    uint64_t* s_full = kv_empty + 2 * S;                             // [kBufs], as the next two
    uint64_t* p_full = s_full + kBufs;
    uint64_t* pv_done = p_full + kBufs;
    uint64_t* base_set = pv_done + kBufs;                            // [2]
    uint64_t* q_full = base_set + 2;
    uint64_t* q_free = q_full + 1;
    uint64_t* q_staged = q_free + 1;
    uint64_t* drain = q_staged + 1;                                  // [2]
    uint32_t* tmem_slot = (uint32_t*)(drain + 2);
    __shared__ int abort_s;
    __shared__ long long sums[kThreads / 32];
    volatile int* abort_flag = &abort_s;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int4* rec = (int4*)((uint8_t*)p.counters + kJoinRecords) + 2 * blockIdx.x;
    if (tid == 0) {
        for (int i = 0; i < 2 * S; ++i) {
            mbar_init(&kv_full[i], 1);
            mbar_init(&kv_empty[i], 1);
        }
        for (int i = 0; i < kBufs; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);
            mbar_init(&pv_done[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&base_set[i], 4);
            mbar_init(&drain[i], 1);
        }
        mbar_init(q_full, 4);
        mbar_init(q_free, 8);
        mbar_init(q_staged, 64);
        abort_s = 0;
        fence_mbar_init();
        tma_prefetch_desc(&p.tmap_half);
    }
    griddep_wait();
    Line line;
    const int U = line_plan<kThreads, D>(p, line, line_mem, sums, kOverhead);
    const int P = min((int)gridDim.x, max(1, U / kMinShare));
    if (tid == 64) rec[0] = make_int4(-1, 0, 0, 0);      // no item to join from here, so far
    if (U == 0 || (int)blockIdx.x >= P) return;
    const Shares shares(U, P);
    Walker<true> walk;
    walk.start(line, shares.begin(blockIdx.x), shares.begin(blockIdx.x + 1));
    Stretch s;
    uint32_t tmem = 0;
    if (warp > 0 && warp <= kPvWarp) {      // the producers do not wait for the tensor memory
        if (warp == 1) {
            tmem_alloc(tmem_slot, C::COLS);
            // The next kernel may start only once this CTA holds its tensor memory: a dependent
            // CTA on this SM that allocated first and then waited for this grid would never let go.
            griddep_launch();
        }
        tc_fence_before();
        named_bar_sync(2, kThreads - 64);
        tc_fence_after();
        tmem = *tmem_slot;
    }
    const uint32_t tS = tmem + C::T_S, tQ = tmem + C::T_Q, tO = tmem + C::T_O;

    if (warp == 0 || warp > kPvWarp) {
        // ------------------------------------------------------------ TMA producers, K and V
        // Rings of their own: a K tile is free again as soon as its S is done, a V tile when its
        // product is.  Lanes look up the boxes of the next tiles together, one box (both halves)
        // each: what is left to do between a free stage and its load is a few instructions.  (Looked
        // up tile by tile that took 700 cycles, which three stages do not hide.)
        const int kind = warp == 0 ? 0 : 1;
        uint64_t *full = kv_full + kind * S, *empty = kv_empty + kind * S;
        uint8_t* tiles = ring + kind * S * C::KV;
        const int bl = p.table ? min(p.ps_log2, 6) : 6;          // log2 rows of a box
        const int box_rows = 1 << bl, boxes = 64 >> bl;
        const int batch = 32 >> (6 - bl);                         // tiles looked up at a time: 32 boxes
        const int b = lane & (boxes - 1), tile_of = lane >> (6 - bl);   // this lane's box and tile of a batch
        const uint32_t tile_boxes = (1u << boxes) - 1u;
        Stretch nx;
        bool more = walk.next(line, nx);
        int it = 0;
        bool ok = true;
        for (int seg = 0; ok && more; ++seg) {
            s = nx;
            more = walk.next(line, nx);
            int staged = more ? 0 : 128;      // vectors of the next stretch's Q this producer has seen to
            // A few of them after each tile, every other eight by each producer, once the softmax has
            // taken this stretch's Q from there.
            auto stage_some = [&](int until) {
                for (; staged < until; staged += 16)
                    stage_q<D>(p, line, nx, q_stage, staged + kind * 8, staged + kind * 8 + 8, lane, 32);
            };
            const int4 e = line.ent[s.i];
            const int hi = p.causal ? e.w + s.r1 : e.w + e.z;
            const int lo = p.window > 0 ? max(0, e.w + s.r0 - p.window + 1) : 0;
            int row = -1;                                 // slab row of the lane's box, -1: not loaded
            uint32_t wanted = 0;
            for (int t = s.t0; t < s.t1; ++t, ++it) {
                const int j = (t - s.t0) & (batch - 1), st = it % S;
                if (j == 0) {
                    row = -1;
                    const int kb = s.span.tile(t + tile_of) * 64 + b * box_rows;
                    if (t + tile_of < s.t1 && kb < hi && (kb < p.sinks || kb + box_rows > lo)) {
                        const int page = p.table ? p.table[(size_t)e.x * p.max_pages + (kb >> p.ps_log2)] : e.x;
                        if (page >= 0)
                            row = (int)((long long)page * p.rows_page + p.row_layer + (long long)s.g * p.rows_kv +
                                        kind * p.rows_kind + (p.table ? kb & ((1 << p.ps_log2) - 1) : kb));
                    }
                    wanted = __ballot_sync(0xffffffffu, row >= 0);
                }
                const int n_want = __popc((wanted >> (j * boxes)) & tile_boxes);
                ok = mbar_wait_warp(&empty[st], (uint32_t)(((it / S) & 1) ^ 1), abort_flag, p.wait_status);
                if (!ok) break;
                if (tile_of == j) {
                    if (b == 0) mbar_arrive_expect_tx(&full[st], (uint32_t)(n_want * box_rows * 128 * C::HALVES));
                    if (row >= 0) {
#pragma unroll
                        for (int h = 0; h < C::HALVES; ++h)
                            asm volatile(
                                "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes "
                                "[%0], [%1, {%2, %3, %4}], [%5];"
                                ::"r"(smem_u32(tiles + st * C::KV + h * 8192 + b * box_rows * 128)),
                                  "l"((uint64_t)&p.tmap_half), "r"(0), "r"(row), "r"(h), "r"(smem_u32(&full[st]))
                                : "memory");
                    }
                }
                __syncwarp();
                // (with S tiles issued since, the first tile's S is done, and so Q was taken)
                if (t - s.t0 >= S && staged < 128) stage_some(staged + 16);
            }
            if (more && ok) {
                ok = mbar_wait_warp(q_full, (uint32_t)(seg & 1), abort_flag, p.wait_status);
                if (!ok) break;
                stage_some(128);
                asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(q_staged)) : "memory");
            }
        }
        if (!ok) {
            // an abandoned launch: its copies land before the CTA exits
            volatile int never = 0;
            for (int k = max(0, it - S); k < it; ++k) mbar_wait_warp(&full[k % S], (uint32_t)((k / S) & 1), &never, nullptr);
            asm volatile("cp.async.wait_all;" ::: "memory");
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ S = Q K^T
        // The whole warp walks and waits, one elected lane issues: in code that the warp runs
        // together the operands stay in uniform registers (128 x 64 x 16 measured 33 cycles an
        // instruction against 47-70 in a branch of one lane).
        constexpr uint32_t IDESC_S = idesc_bf16_f32(128, 64);
        const bool leader = elect_one();
        int it = 0, seg = 0;
        bool ok = true;
        for (; ok && walk.next(line, s); ++seg) {
            ok = mbar_wait_warp(q_full, (uint32_t)(seg & 1), abort_flag, p.wait_status);
            for (int t = s.t0; t < s.t1 && ok; ++t, ++it) {
                const int st = it % S;
                ok = mbar_wait_warp(&kv_full[st], (uint32_t)((it / S) & 1), abort_flag, p.wait_status);
                if (ok && it >= kBufs)
                    ok = mbar_wait_warp(&pv_done[it % kBufs], (uint32_t)((it / kBufs - 1) & 1), abort_flag, p.wait_status);
                if (!ok) break;
                tc_fence_after();
                const uint32_t ka = smem_u32(ring + st * C::KV), d = tS + (it % kBufs) * 64;
                if (leader) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        tc_mma_bf16_ts(d, tQ + kk * 8, umma_desc_sw128(ka + (kk >> 2) * 8192) + 2 * (kk & 3), IDESC_S,
                                       kk > 0 ? 1u : 0u);
                    tc_commit(&s_full[it % kBufs]);
                    tc_commit(&kv_empty[st]);
                }
                __syncwarp();
            }
        }
        if (__any_sync(0xffffffffu, *abort_flag)) {
            if (leader) tc_commit(&drain[0]);   // the issued MMAs finish before the tensor memory is released
            __syncwarp();
            volatile int never = 0;
            mbar_wait_warp(&drain[0], 0, &never, nullptr);
        }
    } else if (warp == kPvWarp) {
        // ------------------------------------------------------------ O += P V
        constexpr uint32_t IDESC_PV = idesc_bf16_f32(128, D, true);
        const bool leader = elect_one();
        int it = 0;
        bool ok = true;
        while (ok && walk.next(line, s)) {
            for (int t = s.t0; t < s.t1; ++t, ++it) {
                const int sb = it % kBufs;
                ok = mbar_wait_warp(&kv_full[S + it % S], (uint32_t)((it / S) & 1), abort_flag, p.wait_status);
                if (ok) ok = mbar_wait_warp(&p_full[sb], (uint32_t)((it / kBufs) & 1), abort_flag, p.wait_status);
                if (!ok) break;
                tc_fence_after();
                const uint32_t va = smem_u32(ring + (S + it % S) * C::KV), a = tS + sb * 64;
                const uint32_t add = t > s.t0 ? 1u : 0u;
                if (leader) {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        tc_mma_bf16_ts(tO, a + kk * 8, umma_desc_sw128_mn(va + kk * 2048, 8192, 1024), IDESC_PV,
                                       kk > 0 ? 1u : add);
                    tc_commit(&pv_done[sb]);
                    tc_commit(&kv_empty[S + it % S]);
                }
                __syncwarp();
            }
        }
        if (__any_sync(0xffffffffu, *abort_flag)) {
            if (leader) tc_commit(&drain[1]);
            __syncwarp();
            volatile int never = 0;
            mbar_wait_warp(&drain[1], 0, &never, nullptr);
        }
    } else {
        // ------------------------------------------------------------ softmax
        const int w = (warp - 2) >> 2, q4 = warp & 3, rl = q4 * 32 + lane;
        const int row = rl % RW, cs = rl / RW, col = cs * KC;  // vector of the tile, first column (warp-uniform)
        const int e256 = tid - 64;
        const uint32_t lanes = (uint32_t)(q4 * 32) << 16;
        const uint32_t my_o = tO + lanes;
        // the lane's vector of stretch n (staged by the producer) into the Q operand; lanes past the
        // tile's vectors take whatever stands there (their rows are not written)
        auto put_q = [&](int n) -> bool {
            if (n > 0) {
                if (!mbar_wait_warp(q_staged, (uint32_t)((n - 1) & 1), abort_flag, p.wait_status)) return false;
            }
            const uint8_t* src = q_stage + row * C::QLD;
#pragma unroll 1
            for (int c0 = 0; c0 < D / 2; c0 += 16) {
                float v[16];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float4 u = *reinterpret_cast<const float4*>(src + (c0 + 4 * k) * 4);
                    v[4 * k + 0] = u.x;
                    v[4 * k + 1] = u.y;
                    v[4 * k + 2] = u.z;
                    v[4 * k + 3] = u.w;
                }
                tmem_st16(tQ + lanes + c0, v);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            mbar_arrive_if(lane == 0, q_full);
            return true;
        };
        Stretch nx;
        bool more = walk.next(line, nx);
        int it0 = 0, seg = 0;             // tiles and stretches before this one
        bool ok = true;
        if (more) {                       // the first stretch's Q: staged by all softmax threads
            stage_q<D>(p, line, nx, q_stage, 0, 128, e256, kSoftmax);
            asm volatile("cp.async.wait_all;" ::: "memory");
            named_bar_sync(1, kSoftmax);
            if (w == 0) ok = put_q(0);
        }
        while (more) {               // left by all threads together
            s = nx;
            const int4 e = line.ent[s.i];
            const int nvec = (s.r1 - s.r0) * p.G;
            const int pos = e.w + s.r0 + (row * p.g_magic >> 16);                    // this lane's position (padding lanes: any)
            const int hi_tile = p.causal ? e.w + s.r1 : e.w + e.z;     // keys that exist for some row
            const int lo_tile = p.window > 0 ? max(0, e.w + s.r0 - p.window + 1) : 0;
            const int hi_all = p.causal ? e.w + s.r0 + 1 : hi_tile;    // keys below are seen by all rows ..
            const int lo_all = p.window > 0 ? e.w + s.r1 - p.window : 0;   // .. from here on
            const int hi_row = p.causal ? min(pos + 1, hi_tile) : hi_tile;
            const int lo_row = p.window > 0 ? max(0, pos - p.window + 1) : 0;   // (less a key's index stays an int)
            float base = -INFINITY, l = 0.f;
            for (int t = s.t0 + ((it0 ^ w) & 1); ok && t < s.t1; t += 2) {
                const int it = it0 + t - s.t0;
                const int sb = it % kBufs;
                const uint32_t my_s = tS + lanes + sb * 64;            // S, then P
                ok = mbar_wait_warp(&s_full[sb], (uint32_t)((it / kBufs) & 1), abort_flag, p.wait_status);
                if (!ok) break;
                tc_fence_after();
                const int k0 = s.span.tile(t) * 64, kvb = k0 + col;
                float x[KC];
                if constexpr (KC == 64) tmem_ld64w(my_s, x);
                else if constexpr (KC == 32) tmem_ld32w(my_s + col, x);
                else tmem_ld16w(my_s + col, x);
                // tiles with keys that some row does not see
                if (k0 + 64 > hi_all || (k0 < lo_all && k0 + 64 > p.sinks)) {
                    // this thread's keys as bits: below the row's end, and from its window on or a sink
#pragma unroll
                    for (int c0 = 0; c0 < KC; c0 += 32) {
                        const int k = kvb + c0;
                        const uint32_t m = bits_below(hi_row - k) & (~bits_below(lo_row - k) | bits_below(p.sinks - k));
#pragma unroll
                        for (int i = 0; i < (KC < 32 ? KC : 32); ++i)
                            if (!(m & (1u << i))) x[c0 + i] = -INFINITY;
                    }
                    // V rows that no row sees may hold anything (0 * NaN is NaN): zero them
                    if (k0 + 64 > hi_tile || (k0 < lo_tile && k0 + 64 > p.sinks)) {
                        // The softmax may be S tiles and more ahead of the products, and a parity tells two
                        // phases apart, not three: first the product of the stage's tile before (or of
                        // a later tile; tile it - 4 is the last whose barrier cannot have gone on
                        // by another phase), then this tile's V.
                        constexpr int BACK = S < kBufs - 1 ? S : kBufs - 1;
                        if (it >= BACK)
                            mbar_wait_warp(&pv_done[(it - BACK) % kBufs], (uint32_t)(((it - BACK) / kBufs) & 1), abort_flag,
                                           p.wait_status);
                        ok = mbar_wait_warp(&kv_full[S + it % S], (uint32_t)((it / S) & 1), abort_flag, p.wait_status);
                        if (!ok) break;
                        // two threads to a row
                        const int k = k0 + (rl >> 1);
                        if (k >= hi_tile || (k < lo_tile && k >= p.sinks)) {
                            uint8_t* vr = ring + (S + it % S) * C::KV + (rl >> 1) * 128 + (rl & 1) * 64;
#pragma unroll
                            for (int x4 = 0; x4 < C::HALVES * 4; ++x4)
                                *reinterpret_cast<uint4*>(vr + (x4 >> 2) * 8192 + (x4 & 3) * 16) = make_uint4(0, 0, 0, 0);
                        }
                        fence_proxy_async();   // the product reads these rows through the async proxy
                    }
                }
                float m4[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) m4[k] = fmax3(x[3 * k], x[3 * k + 1], x[3 * k + 2]);
#pragma unroll
                for (int i = 12; i + 1 < KC; i += 2) m4[(i >> 1) & 3] = fmax3(m4[(i >> 1) & 3], x[i], x[i + 1]);
                const float nb = floorf(fmax3(fmaxf(m4[0], m4[1]), m4[2], m4[3]) * p.scale_log2);
                // the base that the tile before left (the other group's, half a turn ago), and this tile's
                if (t > s.t0) {
                    ok = mbar_wait_warp(&base_set[w ^ 1], (uint32_t)(((it - 1) >> 1) & 1), abort_flag, p.wait_status);
                    if (!ok) break;
                    const float before = base_s[(w ^ 1) * 128 + rl];
                    if (before != base) {
                        l = base == -INFINITY ? 0.f : l * pow2_int(base - before);
                        base = before;
                    }
                }
                const bool grow = nb > base + kBaseLag;
                const float held = base;
                if (grow) base = nb + kBaseLead;
                base_s[w * 128 + rl] = base;
                __syncwarp();
                mbar_arrive_if(lane == 0, &base_set[w]);
                if (__any_sync(0xffffffffu, grow) && t > s.t0) {
                    // O holds the tiles before: once their products are done
                    ok = mbar_wait_warp(&pv_done[(it - 1) % kBufs], (uint32_t)(((it - 1) / kBufs) & 1), abort_flag,
                                         p.wait_status);
                    if (!ok) break;
                    tc_fence_after();
                    const float f = grow ? pow2_int(held - base) : 1.0f;
#pragma unroll 1
                    for (int c0 = 0; c0 < D; c0 += 32) {
                        float v[32];
                        tmem_ld32w(my_o + c0, v);
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] *= f;
                        tmem_st16(my_o + c0, v);
                        tmem_st16(my_o + c0 + 16, v + 16);
                    }
                    l *= f;
                }
                const float bb = (base == -INFINITY) ? 0.f : base;
                // two at a time where the hardware has it: instructions are what this loop runs out of
                const float2 sc2 = make_float2(p.scale_log2, p.scale_log2), nb2 = make_float2(-bb, -bb);
                float2 sum2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int c0 = 0; c0 < KC; c0 += 16) {
                    uint32_t pk[8];
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        const float2 t2 = fma_x2(make_float2(x[c0 + i], x[c0 + i + 1]), sc2, nb2);
                        const float2 e2 = make_float2(ex2_fast(t2.x), ex2_fast(t2.y));
                        sum2[(i >> 1) & 1] = add_x2(sum2[(i >> 1) & 1], e2);
                        pk[i / 2] = pack_bf16(e2.x, e2.y);
                    }
                    tmem_st8u(my_s + col / 2 + c0 / 2, pk);
                }
                if constexpr (CS > 1) {           // the other slices' columns of this lane's P are zero
                    const uint32_t z[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
                    for (int c0 = 0; c0 < 32; c0 += 8)
                        if (c0 < col / 2 || c0 >= (col + KC) / 2) tmem_st8u(my_s + c0, z);
                }
                sum2[0] = add_x2(sum2[0], sum2[1]);
                l += sum2[0].x + sum2[0].y;
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                mbar_arrive_if(lane == 0, &p_full[sb]);
            }
            // this warp has read its last S of the stretch; when all have, Q may change
            __syncwarp();
            mbar_arrive_if(lane == 0, q_free);
            more = walk.next(line, nx);
            if (ok && more && w == 0) {
                ok = mbar_wait_warp(q_free, (uint32_t)(seg & 1), abort_flag, p.wait_status);
                if (ok) ok = put_q(seg + 1);
            }
            ++seg;
            // by the group that had the last tile: it knows that the barrier's phase before is over
            const int last = it0 + s.t1 - s.t0 - 1;
            if (ok && !((last ^ w) & 1))
                ok = mbar_wait_warp(&pv_done[last % kBufs], (uint32_t)((last / kBufs) & 1), abort_flag, p.wait_status);
            tc_fence_before();
            ml[w * 128 + rl] = make_float2(base, l);
            if (named_bar_or(1, kSoftmax, !ok)) break;
            tc_fence_after();
            // ---- the stretch's rows: O is relative to the last tile's base; bases differ by integers,
            // so all factors are exact powers of two.  Each group has half of the columns.
            const bool whole = s.whole(), head = s.t0 == 0;   // head: holds the item's first tile
            float* slot = p.partial + (size_t)(2 * blockIdx.x + (head ? 1 : 0)) * kSlot<D>;
            constexpr int HC = D / 2;
            const float B = base_s[(last & 1) * 128 + rl], z = B == -INFINITY ? 0.f : B;
            const float2 m0 = ml[rl], m1 = ml[128 + rl];
            const float L = pow2_int(m0.x - z) * m0.y + pow2_int(m1.x - z) * m1.y;
            if constexpr (CS == 1) {
                const float inv = L == 0.f ? 0.f : 1.0f / L;
#pragma unroll 1
                for (int c0 = w * HC; c0 < (w + 1) * HC; c0 += 32) {
                    float v[32];
                    tmem_ld32w(my_o + c0, v);
                    if (whole) {
#pragma unroll
                        for (int i = 0; i < 32; i += 8)
                            *reinterpret_cast<uint4*>(join + rl * C::QLD + (c0 + i) * 2) =
                                make_uint4(pack_bf16(v[i] * inv, v[i + 1] * inv), pack_bf16(v[i + 2] * inv, v[i + 3] * inv),
                                           pack_bf16(v[i + 4] * inv, v[i + 5] * inv), pack_bf16(v[i + 6] * inv, v[i + 7] * inv));
                    } else if (row < nvec) {
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
                            *reinterpret_cast<float4*>(slot + part_at(row, c0 + i)) =
                                make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                    }
                }
                if (whole) {
                    named_bar_sync(1, kSoftmax);
                    // whole 256-byte (128-byte) rows per group of lanes
                    __nv_bfloat16* out0 = (__nv_bfloat16*)p.out + ((size_t)(e.y + s.r0) * p.nq + (size_t)s.g * p.G) * D;
#pragma unroll 4
                    for (int i = e256; i < nvec * (D / 8); i += kSoftmax) {
                        const int v = i / (D / 8), c = (i % (D / 8)) * 8;
                        const uint4 u = *reinterpret_cast<const uint4*>(join + v * C::QLD + c * 2);
                        const int vr = v * p.g_magic >> 16;
                        *reinterpret_cast<uint4*>(out0 + ((size_t)vr * p.nq + (v - vr * p.G)) * D + c) = u;
                    }
                } else if (w == 0 && row < nvec) {
                    *reinterpret_cast<float2*>(slot + 2 * row) = make_float2(B, L);
                }
            } else {
                // the copies of a vector have bases and sums of their own
                float* jf = reinterpret_cast<float*>(join);
#pragma unroll 1
                for (int c0 = w * HC; c0 < (w + 1) * HC; c0 += 32) {
                    float v[32];
                    tmem_ld32w(my_o + c0, v);
#pragma unroll
                    for (int i = 0; i < 32; i += 4)
                        *reinterpret_cast<float4*>(jf + rl * C::OLD + c0 + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                }
                named_bar_sync(1, kSoftmax);             // all have read the groups' sums
                if (w == 0) ml[rl] = make_float2(B, L);
                named_bar_sync(1, kSoftmax);
                // rows in order for the output, columns in order for a partial
#pragma unroll 1
                for (int i = e256; i < RW * (D / 8); i += kSoftmax) {
                    const int v = whole ? i / (D / 8) : i % RW, c = (whole ? i % (D / 8) : i / RW) * 8;
                    if (v >= nvec) continue;
                    float Bv = -INFINITY, Lv = 0.f, a[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int k = 0; k < CS; ++k) Bv = fmaxf(Bv, ml[v + k * RW].x);
                    const float zv = Bv == -INFINITY ? 0.f : Bv;
#pragma unroll
                    for (int k = 0; k < CS; ++k) {
                        const float2 m = ml[v + k * RW];
                        const float f = pow2_int(m.x - zv);
                        const float4 w0 = *reinterpret_cast<const float4*>(jf + (v + k * RW) * C::OLD + c);
                        const float4 w1 = *reinterpret_cast<const float4*>(jf + (v + k * RW) * C::OLD + c + 4);
                        Lv += f * m.y;
                        a[0] += f * w0.x; a[1] += f * w0.y; a[2] += f * w0.z; a[3] += f * w0.w;
                        a[4] += f * w1.x; a[5] += f * w1.y; a[6] += f * w1.z; a[7] += f * w1.w;
                    }
                    if (whole) {
                        const float inv = Lv == 0.f ? 0.f : 1.0f / Lv;
                        __nv_bfloat16* dst = (__nv_bfloat16*)p.out +
                                             ((size_t)(e.y + s.r0 + v / p.G) * p.nq + (size_t)s.g * p.G + v % p.G) * D + c;
                        *reinterpret_cast<uint4*>(dst) =
                            make_uint4(pack_bf16(a[0] * inv, a[1] * inv), pack_bf16(a[2] * inv, a[3] * inv),
                                       pack_bf16(a[4] * inv, a[5] * inv), pack_bf16(a[6] * inv, a[7] * inv));
                    } else {
                        *reinterpret_cast<float4*>(slot + part_at(v, c)) = make_float4(a[0], a[1], a[2], a[3]);
                        *reinterpret_cast<float4*>(slot + part_at(v, c + 4)) = make_float4(a[4], a[5], a[6], a[7]);
                        if (c == 0) *reinterpret_cast<float2*>(slot + 2 * v) = make_float2(Bv, Lv);
                    }
                }
            }
            if (!whole && head && e256 == 0) {
                rec[0] = make_int4(shares.owner(s.v0 + kOverhead + s.span.nt - 1), nvec, e.y + s.r0, s.g);
            }
            it0 += s.t1 - s.t0;
            tc_fence_before();
            named_bar_sync(1, kSoftmax);      // O, join and ml are free again
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
    constexpr int SLOT = kSlot<D>;
    griddep_wait();
    griddep_launch();
    const int c0 = blockIdx.x;
    const int4 rec = *((const int4*)((const uint8_t*)p.counters + kJoinRecords) + 2 * c0);
    const int i = blockIdx.y * 256 + threadIdx.x;
    if (rec.x < 0 || i >= rec.y * (D / 8)) return;
    const int v = i % rec.y, c = i / rec.y * 8;
    float B = -INFINITY, L = 0.f, a[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int k0 = c0; k0 <= rec.x; k0 += 4) {     // four partials' loads in flight
        float2 m[4];
        float4 w0[4], w1[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int cta = min(k0 + k, rec.x);
            const float* q = p.partial + (size_t)(2 * cta + (cta == c0 ? 1 : 0)) * SLOT;
            m[k] = *reinterpret_cast<const float2*>(q + 2 * v);
            w0[k] = *reinterpret_cast<const float4*>(q + part_at(v, c));
            w1[k] = *reinterpret_cast<const float4*>(q + part_at(v, c + 4));
        }
        float nb = B;
#pragma unroll
        for (int k = 0; k < 4; ++k) nb = fmaxf(nb, m[k].x);
        const float z = nb == -INFINITY ? 0.f : nb;
        const float f0 = pow2_int(B - z);
        B = nb;
        L *= f0;
#pragma unroll
        for (int j = 0; j < 8; ++j) a[j] *= f0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (k0 + k > rec.x) break;
            const float f = pow2_int(m[k].x - z);
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
    if (!allow_smem<D * 8 + CS>((const void*)kern, (BlockCfg<D, CS>::SMEM))) return 1;
    const int ctas = std::min(num_sms, kPagedCtas), pieces = p.rt * p.G * (D / 8);
    cudaError_t e = launch_k(kern, dim3(ctas), dim3(kThreads), (BlockCfg<D, CS>::SMEM), st, p);
    if (e == cudaSuccess) e = launch_k(k_paged_join<D>, dim3(ctas, (pieces + 255) / 256), dim3(256), 0, st, p);
    return (int)e;
}
// Copies of the window of vectors: as many as fit.  32 sequences of 4000: one kv head of 64, 32 vectors:
// 15.1 us with 4 copies, 16.1 with 2, 22.9 with 1; 8 kv heads of 128, 64 vectors: 99.8 with 2, 113 with 1.
template <int D>
int launch_d(const PagedAttnParams& p, int vectors, int num_sms, cudaStream_t st) {
    if (vectors <= 32) return launch_dc<D, 4>(p, num_sms, st);
    if (vectors <= 64) return launch_dc<D, 2>(p, num_sms, st);
    return launch_dc<D, 1>(p, num_sms, st);
}

}  // namespace

int launch_paged_block(PagedAttnParams& p, int d, int num_sms, cudaStream_t st) {
    p.g_magic = (65536 + p.G - 1) / p.G;
    p.launches = 2;
    p.rt = std::min(p.max_rows, kPagedRowsTc / p.G);
    p.row_tiles = (p.max_rows + p.rt - 1) / p.rt;
    return d == 128 ? launch_d<128>(p, p.rt * p.G, num_sms, st) : launch_d<64>(p, p.rt * p.G, num_sms, st);
}

}  // namespace df
