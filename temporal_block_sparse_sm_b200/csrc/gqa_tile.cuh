// gqa_tile.cuh -- grouped-query attention of many query rows per key head (prompts, chunks
// of new tokens, video frames) on tcgen05, over packed or paged keys.
//
//   S = Q K^T (32 bits, Tensor Memory), running maximum m and sum l per row,
//   P = 2^(c S - c m) rounded to 16 bits, O += P V, o = O / l,  c = scale log2 e.
//
// A work item is 256 query rows of one key head: two slots of 128 rows, a row being one
// (token, head of the group) pair, so that the G heads of a group share every key and value
// that is loaded, and a slot covers 128 / G whole tokens (one TMA box of G heads by that many
// tokens fills it for any G; rows behind G * (128 / G) hold nothing).  (In a small batch an
// item is a single slot, and the second one idle.)  Each slot owns 128
// TMEM columns of S and D of O; P is written over S and read by the MMA from TMEM.
//
// Blocks are persistent, one per SM, and take whole items or stretches of the batch
// (serving_internal.cuh).  The next item's queries, keys and first product overlap the current
// one's last softmax and its epilogue.
//
// Warps: 0 loads (TMA: Q of a slot when its last product with K is done, 128-key tiles of K
// and V into rings), 1 and 2 issue the MMAs of slot 0 and 1, 3 walks the work items and cleans
// the values of tiles that some row does not see whole; 4-7 and 8-11 are the softmax of slot 0
// and 1, a thread per row.
//
// The softmax goes in steps of 64 keys, and a slot's S has two buffers of 64 columns: the
// product of step u + 2 is issued right behind P V of step u, so that the softmax finds the
// next S ready and neither waits for the other.  With one S of 128 columns per slot, P V and
// the next Q K^T lay between every two softmax steps, 1450 of 3600 cycles per 128 keys.  What
// then counts is how fast a warp can issue: a wait that is already over, a block of MMAs and a
// commit take 100 to 200 cycles each, so each slot has a warp of its own.
//
// What bounds it: the GPU's power.  A causal prompt of 32,760 tokens and 12 heads runs at 1100 to
// 1140 TFLOP/s (2.9 to 3.0 ms) with 1475 cycles a softmax step at about 1.45 GHz; the tensor
// pipe is busy 64% of the cycles, and cuBLAS under the same power cap reaches 1377.  Measured
// and left out: two threads a row on one S of 128 columns (the MMA warp comes late), a second
// set of eight softmax warps, one per S buffer (3196 instead of 2959 us: it reloads and
// rescales more, and energy is what is short), a share of the exponentials as polynomials
// (slower: the issue slots are short too), the rows' sums a step late (no gain).  The epilogue's
// way through shared memory came out even with plain stores; it is kept since its stores are whole lines.
//
// Values that no row sees are zeroed in shared memory, since 0 * NaN is NaN.  In a tile where
// some rows see a key that others do not, values that are not finite are zeroed too and
// noted; the epilogue adds them to the rows that do see them.
#pragma once

#include "gqa_rows.cuh"

namespace lite {

struct TileParams {
    GqaParams a;
    const uint16_t *v;                  // values in global memory (rows of values that are not finite)
    int64_t v_page, v_token, v_head;    // strides, elements (packed: v_token, v_head)
    int slot_tokens;                    // tokens of a slot: 128 / G
};

template <int D, bool F16>
struct TileCfg {
    static constexpr int BN = 128, NSLOT = 2, DCH = D / 64;
    static constexpr int NST = D == 128 ? 2 : 4;               // ring stages of K and of V
    static constexpr int BU = 64;                               // keys of a softmax step
    static constexpr int NSOFT = 8, NTHREADS = 32 * (4 + NSOFT), SLOT_THREADS = 128;
    static constexpr uint32_t REG_LAUNCH = 168, REG_CTRL = 104, REG_SOFTMAX = 200;
    static_assert(128 * REG_CTRL + 256 * REG_SOFTMAX <= NTHREADS * REG_LAUNCH, "register split");
    static constexpr uint32_t Q_CHUNK = 128u * 128u, Q_SLOT = Q_CHUNK * DCH;
    static constexpr uint32_t KV_CHUNK = BN * 128u, KV_BYTES = KV_CHUNK * DCH;
    static constexpr uint32_t K_OFF = NSLOT * Q_SLOT, V_OFF = K_OFF + NST * KV_BYTES;
    static constexpr uint32_t OUT_OFF = V_OFF + NST * KV_BYTES, OUT_WARP = 32u * 64u;   // a softmax warp's rows on their way out
    static constexpr uint32_t SMEM_BYTES = OUT_OFF + NSOFT * OUT_WARP + 1024u;
    static constexpr int NWORK = 4;                             // items known ahead
    static constexpr int NBAR = 6 * NST + 11 * NSLOT + 2 * NWORK + 1;
    static constexpr uint32_t TMEM_COLS = 512;
    __host__ __device__ static constexpr uint32_t s_col(int s) { return s * 128u; }   // two buffers of BU columns
    __host__ __device__ static constexpr uint32_t o_col(int s) { return 256u + s * static_cast<uint32_t>(D); }
    // f32 result, A and B of the 16-bit type, A K-major, B K-major or MN-major
    __host__ __device__ static constexpr uint32_t idesc(int N, bool b_mn) {
        return (1u << 4) | (F16 ? 0u : (1u << 7) | (1u << 10)) | ((b_mn ? 1u : 0u) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
               (static_cast<uint32_t>(128 >> 4) << 24);
    }
};

// What the roles of a block need to know of one item (shared memory).
struct TileWork {
    int64_t k0;
    int q0, n, m, b, h, tok0, end;   // its tokens [tok0, end) of the sequence's
    int whole, slot;              // all its keys are here: the output is final; else the workspace slot
    int t_lo, n_u, us0, us1;      // first key tile; softmax steps of the segment, and those of each slot
    int lim_lo, lim_hi;           // keys that the first row sees, and the most that any sees
    int e_mask, mask_tile;        // tiles from e_mask on (mask_tile of the sequence) are not seen whole by some row
    int u_mask;                   // and steps from u_mask on
    int valid;                    // 0: no more items
    uint32_t any_bad, bad[4][4];  // keys with values that are not finite, by tile from mask_tile on
};

// c s - c m is one operation with c m rounded before: off by 2^-24 of c m, the same for all keys of a step,
// but not for other steps, and whole powers of two for logits of 10^7 and more, beyond fp16's
// range.  From |c m| = kFarLogit on the difference s - m is taken first (half as many operations again).
constexpr float kFarLogit = 4096.0f;

// A value that all lanes hold, in a form that the compiler knows to be the same in all of them
// (a reduction over the warp ends in a uniform register).  Operands of tcgen05.mma are uniform
// registers; from values that only happen to be equal each of them is moved there before
// every MMA, about 60 cycles an issue where the product itself takes 32 to 64.
__device__ __forceinline__ int uniform(int x) { return static_cast<int>(__reduce_or_sync(0xFFFFFFFFu, static_cast<unsigned>(x))); }

// N MMAs by one elected lane of a converged warp, the operands' start addresses (the low
// words of the descriptors) moving on by A_STEP and B_STEP 16-byte units, every fourth time
// by A_JUMP and B_JUMP more (the next 64-element chunk of a K-major operand).
template <int N, int A_STEP, int A_JUMP, int B_STEP, int B_JUMP>
__device__ __forceinline__ void mma_ss_block(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc) {
    const uint32_t a_hi = static_cast<uint32_t>(a_desc >> 32), b_hi = static_cast<uint32_t>(b_desc >> 32);
#pragma unroll
    for (int k = 0; k < N; k += 4) {
        const uint32_t a = static_cast<uint32_t>(a_desc) + (k / 4) * (4 * A_STEP + A_JUMP);
        const uint32_t b = static_cast<uint32_t>(b_desc) + (k / 4) * (4 * B_STEP + B_JUMP);
        asm volatile(
            "{\n\t.reg .pred PE, PA;\n\t.reg .b64 da, db;\n\t.reg .b32 la, lb;\n\t"
            "elect.sync _|PE, 0xffffffff;\n\t"
            "setp.ne.b32 PA, %6, 0;\n\t"
            "mov.b64 da, {%1, %2};\n\tmov.b64 db, {%3, %4};\n\t"
            "@PE tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, PA;\n\t"
            "add.u32 la, %1, %7;\n\tadd.u32 lb, %3, %8;\n\t"
            "mov.b64 da, {la, %2};\n\tmov.b64 db, {lb, %4};\n\t"
            "@PE tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, 1;\n\t"
            "add.u32 la, la, %7;\n\tadd.u32 lb, lb, %8;\n\t"
            "mov.b64 da, {la, %2};\n\tmov.b64 db, {lb, %4};\n\t"
            "@PE tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, 1;\n\t"
            "add.u32 la, la, %7;\n\tadd.u32 lb, lb, %8;\n\t"
            "mov.b64 da, {la, %2};\n\tmov.b64 db, {lb, %4};\n\t"
            "@PE tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, 1;\n\t}" ::"r"(d_tmem),
            "r"(a), "r"(a_hi), "r"(b), "r"(b_hi), "r"(idesc), "r"(k > 0 ? 1u : 0u), "n"(A_STEP), "n"(B_STEP)
            : "memory");
    }
}
// Four MMAs with A in Tensor Memory, 8 columns apart.
template <int B_STEP>
__device__ __forceinline__ void mma_ts_block4(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred PE, PA;\n\t.reg .b64 db;\n\t.reg .b32 ta, lb;\n\t"
        "elect.sync _|PE, 0xffffffff;\n\t"
        "setp.ne.b32 PA, %5, 0;\n\t"
        "mov.b64 db, {%2, %3};\n\t"
        "@PE tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, PA;\n\t"
        "add.u32 ta, %1, 8;\n\tadd.u32 lb, %2, %6;\n\tmov.b64 db, {lb, %3};\n\t"
        "@PE tcgen05.mma.cta_group::1.kind::f16 [%0], [ta], db, %4, 1;\n\t"
        "add.u32 ta, ta, 8;\n\tadd.u32 lb, lb, %6;\n\tmov.b64 db, {lb, %3};\n\t"
        "@PE tcgen05.mma.cta_group::1.kind::f16 [%0], [ta], db, %4, 1;\n\t"
        "add.u32 ta, ta, 8;\n\tadd.u32 lb, lb, %6;\n\tmov.b64 db, {lb, %3};\n\t"
        "@PE tcgen05.mma.cta_group::1.kind::f16 [%0], [ta], db, %4, 1;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "r"(static_cast<uint32_t>(b_desc)), "r"(static_cast<uint32_t>(b_desc >> 32)), "r"(idesc), "r"(accumulate), "n"(B_STEP)
        : "memory");
}

template <int D, bool F16>
__global__ void __launch_bounds__(TileCfg<D, F16>::NTHREADS, 1)
gqa_tile_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                const __grid_constant__ CUtensorMap tm_v, const TileParams p) {
    using C = TileCfg<D, F16>;
    constexpr int BN = C::BN, NST = C::NST, NSLOT = C::NSLOT, DCH = C::DCH, NWORK = C::NWORK;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[C::NBAR];
    __shared__ ScanScratch scan;
    __shared__ TileWork works[NWORK];
    __shared__ uint32_t s_abort, s_tmem;

    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const uint32_t raw_s = ptx::smem_u32(smem_raw);
    const uint32_t base_s = (raw_s + 1023u) & ~1023u;
    const uint32_t bar0 = ptx::smem_u32(bars);
    auto k_full = [&](int st) { return bar0 + 8u * st; };
    auto v_full = [&](int st) { return bar0 + 8u * (NST + st); };
    auto k_empty = [&](int st) { return bar0 + 8u * (2 * NST + st); };
    auto v_empty = [&](int st) { return bar0 + 8u * (3 * NST + st); };
    auto v_ok = [&](int st) { return bar0 + 8u * (4 * NST + st); };
    auto v_go = [&](int st) { return bar0 + 8u * (5 * NST + st); };
    auto slot_bar = [&](int kind, int s) { return bar0 + 8u * (6 * NST + kind * NSLOT + s); };
    auto q_full = [&](int s) { return slot_bar(0, s); };
    auto q_empty = [&](int s) { return slot_bar(1, s); };
    auto o_full = [&](int s) { return slot_bar(2, s); };
    auto o_empty = [&](int s) { return slot_bar(3, s); };
    auto drain = [&](int s) { return slot_bar(4, s); };
    auto s_full = [&](int s, int buf) { return slot_bar(5 + buf, s); };
    auto p_full = [&](int s, int buf) { return slot_bar(7 + buf, s); };
    auto pv_done = [&](int s, int buf) { return slot_bar(9 + buf, s); };
    auto w_full = [&](int k) { return slot_bar(11, 0) + 8u * k; };
    auto w_empty = [&](int k) { return slot_bar(11, 0) + 8u * (NWORK + k); };
    const uint32_t never = w_empty(NWORK);   // nothing arrives here

    if (threadIdx.x == 32) {
        ptx::prefetch_tmap(&tm_q);
        ptx::prefetch_tmap(&tm_k);
        ptx::prefetch_tmap(&tm_v);
    }
    if (threadIdx.x == 0) {
        for (int st = 0; st < NST; ++st) {
            ptx::mbar_init(k_full(st), 1);
            ptx::mbar_init(v_full(st), 1);
            ptx::mbar_init(k_empty(st), NSLOT);
            ptx::mbar_init(v_empty(st), NSLOT);
            ptx::mbar_init(v_ok(st), 1);
            ptx::mbar_init(v_go(st), 1);
        }
        for (int s = 0; s < NSLOT; ++s) {
            ptx::mbar_init(q_full(s), 1);
            ptx::mbar_init(q_empty(s), 1);
            ptx::mbar_init(o_full(s), 1);
            ptx::mbar_init(drain(s), 1);
            ptx::mbar_init(o_empty(s), C::SLOT_THREADS / 32);
            for (int buf = 0; buf < 2; ++buf) {
                ptx::mbar_init(s_full(s, buf), 1);
                ptx::mbar_init(pv_done(s, buf), 1);
                ptx::mbar_init(p_full(s, buf), C::SLOT_THREADS / 32);
            }
        }
        for (int k = 0; k < NWORK; ++k) {
            ptx::mbar_init(w_full(k), 1);
            ptx::mbar_init(w_empty(k), 4 + C::NSOFT);   // loads, MMA issue (2), cleaning, softmax warps
        }
        ptx::mbar_init(never, 1);
        s_abort = 0u;
        ptx::fence_barrier_init();
    }
    GqaBatch pb = p.a.b;             // what is fixed for this kernel, as constants
    pb.tile_shift = 7;
    static_assert(BN == 128);
    const WaitScope wctx{&s_abort, pb.status};
    wait_for_earlier_kernels();
    // Only now: a block that held the SM's Tensor Memory while it waits would keep blocks of the kernel in
    // front from allocating theirs, and neither would end.
    if (warp == 2) {
        ptx::tmem_alloc(ptx::smem_u32(&s_tmem), C::TMEM_COLS);
        ptx::tmem_relinquish();
    }
    const int64_t stretch = stretch_units<C::NTHREADS>(pb, gridDim.x, scan);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = uniform(*reinterpret_cast<volatile uint32_t *>(&s_tmem));
    join_may_start();    // behind the allocation too, for the same reason
    auto wait_all = [&](uint32_t bar, uint32_t par) { return wait_phase_warp(bar, par, wctx); };

    if (warp < 4) {
        ptx::regs_dec<C::REG_CTRL>();
        if (warp == 3) {
            // -------------------------------------------------------- work items
            BlockWalk walk;
            walk.start(pb, stretch, p.a.joins, lane);
            int published = 0;
            bool more = true, ok = true;
            auto publish = [&]() {     // the block's next item (or the end of them)
                more = walk.next(pb, p.a.joins, lane);
                const LineItem &it = walk.it;
                const int t0 = walk.t0, t1 = walk.t1;
                int us0 = 0, us1 = 0, v0 = 0, v1 = 0;
                const int tok0 = more ? it.i * pb.unit_tokens : 0;
                const int end = min(tok0 + pb.unit_tokens, it.s.n);     // behind the item's last token
                int lim_lo = 0;
                if (more) {
                    lim_lo = visible_keys(pb, it.s, tok0);
                    const int key_lo = t0 * BN, key_hi = min(t1 * BN, it.s.m);
                    auto steps_of = [&](int first, int &vis) {
                        const int last = min(first + p.slot_tokens, end) - 1;
                        vis = first <= last ? visible_keys(pb, it.s, last) : 0;
                        const int keys = min(vis, key_hi) - key_lo;
                        return keys > 0 ? (keys + C::BU - 1) / C::BU : 0;
                    };
                    us0 = steps_of(tok0, v0);
                    us1 = steps_of(tok0 + p.slot_tokens, v1);
                }
                const int at = published % NWORK;
                if (!(ok = wait_all(w_empty(at), ((published / NWORK) & 1) ^ 1u))) return;
                TileWork &tw = works[at];
                if (lane == 0) {
                    tw.valid = more ? 1 : 0;
                    if (more) {
                        tw.k0 = it.s.k0, tw.q0 = it.s.q0, tw.n = it.s.n, tw.m = it.s.m, tw.b = it.b, tw.h = it.h, tw.end = end;
                        tw.tok0 = tok0, tw.whole = walk.whole ? 1 : 0, tw.slot = walk.slot, tw.t_lo = t0;
                        tw.us0 = us0, tw.us1 = us1, tw.n_u = max(us0, us1);
                        tw.lim_lo = lim_lo, tw.lim_hi = max(v0, v1);
                        tw.mask_tile = lim_lo / BN, tw.e_mask = max(0, lim_lo / BN - t0);
                        tw.u_mask = max(0, lim_lo / C::BU - t0 * (BN / C::BU));
                    }
                    tw.any_bad = 0u;
#pragma unroll
                    for (int x = 0; x < 16; ++x) tw.bad[x >> 2][x & 3] = 0u;
                    ptx::mbar_arrive(w_full(at));
                }
                __syncwarp();
                ++published;
            };
            publish();
            if (more && ok) publish();
            // -------------------------------------------------------- values of masked tiles
            uint32_t go_ph = 0u;
            int kv = 0;
            for (int k = 0; ok; ++k) {     // item k + 2 is published when item k is clean
                const int at = k % NWORK;
                TileWork &tw = works[at];
                if (!tw.valid) break;
                const int n_e = (tw.n_u + 1) / 2, t_lo = tw.t_lo, lim_lo = tw.lim_lo, lim_hi = tw.lim_hi;
                for (int e = tw.e_mask; e < n_e; ++e) {
                    const int st = (kv + e) % NST, k0 = (t_lo + e) * BN;
                    if (!(ok = wait_all(v_go(st), (go_ph >> st) & 1u))) break;
                    go_ph ^= 1u << st;
                    if (!(ok = wait_all(v_full(st), ((kv + e) / NST) & 1))) break;
                    // 16-byte pieces: x = 8 key + piece, in each 64-column chunk; keys before `part` are seen
                    // by every row, those from `none` on by no row
                    uint8_t *vt = smem_raw + (base_s - raw_s) + C::V_OFF + st * C::KV_BYTES;
                    const int part = min(BN, max(0, lim_lo - k0)), none = min(BN, max(0, lim_hi - k0));
                    for (int x = none * 8 + lane; x < BN * 8; x += 32)
#pragma unroll
                        for (int c = 0; c < DCH; ++c) *reinterpret_cast<uint4 *>(vt + c * C::KV_CHUNK + x * 16) = make_uint4(0u, 0u, 0u, 0u);
                    uint32_t nan = 0u;                           // 0 * v summed: not zero where a v is not finite
#pragma unroll 4
                    for (int x = part * 8 + lane; x < none * 8; x += 32)
#pragma unroll
                        for (int c = 0; c < DCH; ++c) {
                            const uint4 v = *reinterpret_cast<const uint4 *>(vt + c * C::KV_CHUNK + x * 16);
                            nan = fma_zero16<F16>(v.x, fma_zero16<F16>(v.y, fma_zero16<F16>(v.z, fma_zero16<F16>(v.w, nan))));
                        }
                    if (__any_sync(0xFFFFFFFFu, (nan & 0x7FFF7FFFu) != 0u)) {
                        for (int x = part * 8 + lane; x < none * 8; x += 32)
#pragma unroll
                            for (int c = 0; c < DCH; ++c) {
                                uint4 *ptr = reinterpret_cast<uint4 *>(vt + c * C::KV_CHUNK + x * 16);
                                const uint4 u = *ptr;
                                uint32_t v[4] = {u.x, u.y, u.z, u.w}, any = 0u;
#pragma unroll
                                for (int w4 = 0; w4 < 4; ++w4) {
                                    const uint32_t bad = nonfinite16<F16>(v[w4]);
                                    any |= bad;
                                    v[w4] &= ~((bad >> 15) * 0xFFFFu);   // a bit per half -> 16 bits
                                }
                                if (any) {
                                    *ptr = make_uint4(v[0], v[1], v[2], v[3]);
                                    atomicOr(&tw.bad[(t_lo + e - tw.mask_tile) & 3][x >> 8], 1u << ((x >> 3) & 31));
                                    atomicOr(&tw.any_bad, 1u);
                                }
                            }
                    }
                    ptx::fence_proxy_async();   // the MMA reads what was written here
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(v_ok(st));
                }
                if (!ok) break;
                kv += n_e;
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(w_empty(at));
                if (more) publish();
            }
        } else if (warp == 0) {
            // -------------------------------------------------------- loads
            const uint32_t q_box = static_cast<uint32_t>(p.slot_tokens * pb.G) * 128u * DCH;
            uint32_t q_ph = 0u;      // bit s: parity of slot s's next wait for q_empty
            int kv = 0;              // tiles loaded so far
            bool ok = true;
            for (int k = 0; ok; ++k) {
                const int at = k % NWORK;
                if (!wait_all(w_full(at), (k / NWORK) & 1)) break;
                const TileWork &tw = works[at];
                if (!tw.valid) break;
                const int n_e = (tw.n_u + 1) / 2, us0 = tw.us0, us1 = tw.us1, t_lo = tw.t_lo, e_mask = tw.e_mask, h = tw.h;
                const int row0 = tw.q0 + tw.tok0;
                KvTiles<BN, DCH> tiles(pb, tw.k0, tw.b, h, tw.lim_hi);
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(w_empty(at));
                int pg = n_e > 0 ? tiles.page_of(t_lo, lane) : -1;
                auto load_q = [&](int s) {
                    if (!wait_all(q_empty(s), ((q_ph >> s) & 1u) ^ 1u)) return false;
                    q_ph ^= 1u << s;
                    if (ptx::elect_one()) {
                        ptx::mbar_arrive_expect_tx(q_full(s), q_box);
                        for (int c = 0; c < DCH; ++c)
                            ptx::tma_load_4d(base_s + s * C::Q_SLOT + c * C::Q_CHUNK, &tm_q, q_full(s), c * 64, h * pb.G,
                                             row0 + s * p.slot_tokens, 0);
                    }
                    __syncwarp();
                    return true;
                };
                if (us0 > 0) ok = load_q(0);
                for (int e = 0; e < n_e && ok; ++e, ++kv) {
                    const int st = kv % NST, t = t_lo + e;
                    const uint32_t ph = ((kv / NST) & 1) ^ 1u;
                    const int next = e + 1 < n_e ? tiles.page_of(t + 1, lane) : -1;
                    const uint32_t bytes = static_cast<uint32_t>(tiles.boxes(t) * tiles.box) * D * 2u;
                    if (!(ok = wait_all(k_empty(st), ph))) break;
                    ptx::mbar_arrive_expect_tx_elect(k_full(st), bytes);
                    __syncwarp();
                    tiles.load(base_s + C::K_OFF + st * C::KV_BYTES, &tm_k, k_full(st), t, lane, pg);
                    __syncwarp();
                    if (e == 0 && us1 > 0 && !(ok = load_q(1))) {
                        drain_phase(k_full(st), ph ^ 1u);
                        break;
                    }
                    if (!(ok = wait_all(v_empty(st), ph))) {
                        drain_phase(k_full(st), ph ^ 1u);
                        break;
                    }
                    ptx::mbar_arrive_expect_tx_elect(v_full(st), bytes);
                    __syncwarp();
                    tiles.load(base_s + C::V_OFF + st * C::KV_BYTES, &tm_v, v_full(st), t, lane, pg);
                    // the cleaning warp joins at tile e_mask: v_full(st) is now in this tile's phase
                    if (e >= e_mask && lane == 0) ptx::mbar_arrive(v_go(st));
                    __syncwarp();
                    pg = next;
                }
            }
            // every copy that this block started lands before it exits
#pragma unroll
            for (int s = 0; s < NSLOT; ++s)
                if ((q_ph >> s) & 1u) drain_phase(q_full(s), 0);      // an odd number of loads: the last had parity 0
                else drain_phase(q_full(s), 1);
            for (int j = max(0, kv - NST); j < kv; ++j) {
                drain_phase(k_full(j % NST), (j / NST) & 1);
                drain_phase(v_full(j % NST), (j / NST) & 1);
            }
            __syncwarp();
        } else {
            // -------------------------------------------------------- MMA issue, warp 1 + s for slot s
            const int s = warp - 1;
            constexpr uint32_t IDESC_QK = C::idesc(C::BU, false), IDESC_PV = C::idesc(D, true);
            const uint64_t dq = ptx::sdesc_sw128(base_s + s * C::Q_SLOT, 16, 1024);
            const uint64_t dk0 = ptx::sdesc_sw128(base_s + C::K_OFF, 16, 1024);
            const uint64_t dv0 = ptx::sdesc_sw128(base_s + C::V_OFF, C::KV_CHUNK, 1024);
            const uint32_t s_tm = tmem + C::s_col(s), o_tm = tmem + C::o_col(s);
            // Two streams of steps over the items: Q K^T runs two steps ahead of P V.  Step number
            // `seq` of either uses S buffer seq & 1.  Both slots count the steps (and tiles) of an item
            // alike; a slot that needs fewer passes over the rest.
            struct Item {
                int n_u, us, e_mask;
            };
            bool ok = true;
            auto fetch = [&](int &k, Item &it, bool release) {     // the next item with steps; n_u = 0: none
                it.n_u = 0;
                while (true) {
                    const int at = k % NWORK;
                    if (!wait_all(w_full(at), (k / NWORK) & 1)) {
                        ok = false;
                        return;
                    }
                    const TileWork &tw = works[at];
                    if (!uniform(tw.valid)) return;
                    it.n_u = uniform(tw.n_u), it.us = uniform(s ? tw.us1 : tw.us0), it.e_mask = uniform(tw.e_mask);
                    if (release) {
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive(w_empty(at));
                    }
                    ++k;
                    if (it.n_u > 0) return;
                }
            };
            uint32_t q_ph = 0u, p_ph = 0u, o_ph = 0u, vok_ph = 0u;   // parities of the next waits
            Item qi{}, pi{};                           // the items of the two streams
            int qk = 0, pk = 0, qu = 0, pu = 0;        // their numbers, and the steps in them
            int kt = 0, vt = 0, seq = 0;               // tiles so far of either; steps of P V
            auto qk_step = [&](int buf) {              // the next step of Q K^T, if there is one
                if (qi.n_u > 0 && qu == qi.n_u) {
                    fetch(qk, qi, false);
                    qu = 0;
                }
                if (qi.n_u == 0) return;
                const int st = kt % NST;
                if (!(qu & 1)) ok = wait_all(k_full(st), (kt / NST) & 1) && ok;
                if (qu < qi.us) {
                    if (qu == 0) {
                        ok = wait_all(q_full(s), q_ph) && ok;
                        q_ph ^= 1u;
                    }
                    ptx::tc_fence_after();
                    // S buffer = Q times 64 keys (a half of the tile)
                    if (ok)
                        mma_ss_block<D / 16, 2, (C::Q_CHUNK >> 4) - 8, 2, (C::KV_CHUNK >> 4) - 8>(
                            s_tm + buf * C::BU, dq, dk0 + ((st * C::KV_BYTES + (qu & 1) * (C::BU * 128)) >> 4), IDESC_QK);
                }
                if (qu < qi.us) ptx::mma_commit_elect(s_full(s, buf));
                if (qu + 1 == qi.us) ptx::mma_commit_elect(q_empty(s));
                if ((qu & 1) || qu + 1 == qi.n_u) {
                    ptx::mma_commit_elect(k_empty(st));
                    ++kt;
                }
                ++qu;
            };
            fetch(qk, qi, false);
            qk_step(0);
            qk_step(1);
            fetch(pk, pi, true);
            while (pi.n_u > 0) {
                const int st = vt % NST, buf = seq & 1;
                if (!(pu & 1)) {
                    ok = wait_all(v_full(st), (vt / NST) & 1) && ok;
                    if ((pu >> 1) >= pi.e_mask) {
                        ok = wait_all(v_ok(st), (vok_ph >> st) & 1u) && ok;
                        vok_ph ^= 1u << st;
                    }
                }
                if (pu < pi.us) {
                    if (pu == 0) {    // the last item's output has been read
                        ok = wait_all(o_empty(s), o_ph ^ 1u) && ok;
                        o_ph ^= 1u;
                    }
                    ok = wait_all(p_full(s, buf), (p_ph >> buf) & 1u) && ok;
                    p_ph ^= 1u << buf;
                    ptx::tc_fence_after();
                    // O += P (in the first 32 columns of its S buffer) times the same keys' values
                    if (ok)
                        mma_ts_block4<((16 * 128) >> 4)>(o_tm, s_tm + buf * C::BU,
                                                         dv0 + ((st * C::KV_BYTES + (pu & 1) * (C::BU * 128)) >> 4), IDESC_PV,
                                                         pu == 0 ? 0u : 1u);
                    ptx::mma_commit_elect(pv_done(s, buf));
                    if (pu + 1 == pi.us) ptx::mma_commit_elect(o_full(s));
                }
                qk_step(buf);
                if ((pu & 1) || pu + 1 == pi.n_u) {
                    ptx::mma_commit_elect(v_empty(st));
                    ++vt;
                }
                ++seq;
                if (++pu == pi.n_u) {
                    fetch(pk, pi, true);
                    pu = 0;
                }
            }
            ptx::mma_commit_elect(drain(s));
            drain_phase(drain(s), 0);
            __syncwarp();
        }
    } else {
        // ------------------------------------------------------------ softmax
        ptx::regs_inc<C::REG_SOFTMAX>();
        if (p.a.probe_wait && blockIdx.x == 0 && warp == 4) wait_all(never, 0);
        const int slot = warp / 4 - 1;
        const int r = (warp & 3) * 32 + lane;
        const int tl = r / pb.G, g = r - tl * pb.G;
        const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const uint32_t scol = lane_base + C::s_col(slot), ocol = lane_base + C::o_col(slot);
        const float cl2 = p.a.scale_log2;
        const float resc = fminf(8.0f / cl2, 3e38f);    // (finite: a first maximum always moves it)
        // the reference moves when the maximum rose by over 2^8 in weight
        const uint64_t c2 = ptx::f2(cl2, cl2);
        uint32_t s_ph = 0u, o_ph = 0u;   // parities: bit buf of s_ph of this buffer's next S (and P V)
        int seq = 0;
        for (int k = 0;; ++k) {
            const int at = k % NWORK;
            if (!wait_all(w_full(at), (k / NWORK) & 1)) break;
            const TileWork &tw = works[at];
            if (!tw.valid) break;
            const int steps = slot ? tw.us1 : tw.us0;
            const int u_mask = tw.u_mask, n_u = tw.n_u;
            int limit = 0;                // keys that this row sees (0 also for rows that do not exist)
            {
                const int t = tw.tok0 + slot * p.slot_tokens + tl;
                if (tl < p.slot_tokens && t < tw.end) limit = pb.causal ? max(0, tw.m - tw.n + t + 1) : tw.m;
            }
            const int mine = limit - tw.t_lo * BN;    // of them from the first tile on
            float m_ref = -INFINITY, l = 0.0f;
            bool far = false;             // the row's reference is beyond kFarLogit
            for (int u = 0; u < steps; ++u) {
                const int buf = (seq + u) & 1;
                const uint32_t sb = scol + buf * C::BU;
                const bool ok = wait_all(s_full(slot, buf), (s_ph >> buf) & 1u);
                s_ph ^= 1u << buf;
                ptx::tc_fence_after();
                uint32_t sc[2][32];
                if (ok) {
                    ptx::tmem_ld32(sb, sc[0]);
                    ptx::tmem_ld32(sb + 32, sc[1]);
                    ptx::tmem_ld_wait(sc[0]);
                    ptx::reg_tie(sc[1]);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) sc[0][i] = sc[1][i] = 0u;
                }
                if (u >= u_mask) {
                    const int left = mine - u * C::BU;
#pragma unroll
                    for (int ch = 0; ch < 2; ++ch)
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (ch * 32 + i >= left) sc[ch][i] = __float_as_uint(-INFINITY);
                }
                float mx[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) mx[j] = ptx::max3(__uint_as_float(sc[0][j]), __uint_as_float(sc[0][8 + j]), __uint_as_float(sc[0][16 + j]));
#pragma unroll
                for (int j = 0; j < 8; ++j) mx[j] = ptx::max3(mx[j], __uint_as_float(sc[0][24 + j]), __uint_as_float(sc[1][j]));
#pragma unroll
                for (int j = 0; j < 8; ++j) mx[j] = ptx::max3(mx[j], __uint_as_float(sc[1][8 + j]), __uint_as_float(sc[1][16 + j]));
#pragma unroll
                for (int j = 0; j < 8; ++j) mx[j] = fmaxf(mx[j], __uint_as_float(sc[1][24 + j]));
                const float m_loc = ptx::max3(ptx::max3(mx[0], mx[1], mx[2]), ptx::max3(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7]));
                float alpha = 1.0f;
                bool rescale = false;
                if (m_loc - m_ref > resc) {              // also the row's first finite maximum
                    rescale = m_ref != -INFINITY;        // O is zero before the first weight
                    alpha = ptx::ex2((m_ref - m_loc) * cl2);
                    l *= alpha;
                    m_ref = m_loc;
                    far = limit > 0 && fabsf(m_ref) * cl2 > kFarLogit;   // (rows that do not exist hold anything)
                }
                const float from = m_ref == -INFINITY ? 0.0f : m_ref;
                float neg = fmaf(-from, cl2, weight_bias<F16>());
                if (__any_sync(0xFFFFFFFFu, rescale || far) && ok) {
                    if (__any_sync(0xFFFFFFFFu, rescale) && u > 0) {
                        // the last step's P V may still run (this S only says that the one before it is
                        // done); the next is issued when this step's P is handed over
                        if (wait_all(pv_done(slot, buf ^ 1), ((s_ph >> (buf ^ 1)) & 1u) ^ 1u)) {
                            ptx::tc_fence_after();
                            const uint64_t a2 = ptx::f2(alpha, alpha);
#pragma unroll 1
                            for (int ch = 0; ch < D / 16; ++ch) {
                                uint32_t ov[16];
                                ptx::tmem_ld16(ocol + ch * 16, ov);
                                ptx::tmem_ld_wait16(ov);
#pragma unroll
                                for (int i = 0; i < 8; ++i) {
                                    float a, b;
                                    ptx::f2_split(ptx::mul2(ptx::f2(__uint_as_float(ov[2 * i]), __uint_as_float(ov[2 * i + 1])), a2), a, b);
                                    ov[2 * i] = __float_as_uint(a);
                                    ov[2 * i + 1] = __float_as_uint(b);
                                }
                                ptx::tmem_st16(ocol + ch * 16, ov);
                            }
                        }
                    }
                    if (__any_sync(0xFFFFFFFFu, far)) {
                        // by way of the S buffer, so that it takes few instructions (with 64 subtractions
                        // written out here all calls were 2 to 5 % slower)
#pragma unroll
                        for (int ch = 0; ch < 4; ++ch) {
                            uint32_t v[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i) v[i] = sc[ch >> 1][(ch & 1) * 16 + i];
                            ptx::tmem_st16(sb + ch * 16, v);
                        }
                        ptx::tmem_st_wait();
#pragma unroll 1
                        for (int ch = 0; ch < 4; ++ch) {
                            uint32_t v[16];
                            ptx::tmem_ld16(sb + ch * 16, v);
                            ptx::tmem_ld_wait16(v);
#pragma unroll
                            for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) - from);
                            ptx::tmem_st16(sb + ch * 16, v);
                        }
                        ptx::tmem_st_wait();
                        ptx::tmem_ld32(sb, sc[0]);
                        ptx::tmem_ld32(sb + 32, sc[1]);
                        ptx::tmem_ld_wait(sc[0]);
                        ptx::reg_tie(sc[1]);
                        neg = weight_bias<F16>();
                    }
                }
                // P = 2^(c s - c m)
                const uint64_t n2 = ptx::f2(neg, neg);
                uint64_t acc[4] = {};
                // a visible logit of +inf or NaN gives a NaN weight (inf - inf), and so a NaN sum and row
#pragma unroll
                for (int ch = 0; ch < 2; ++ch)
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float x0, x1;
                        ptx::f2_split(ptx::fma2(ptx::f2(__uint_as_float(sc[ch][2 * i]), __uint_as_float(sc[ch][2 * i + 1])), c2, n2), x0, x1);
                        sc[ch][2 * i] = __float_as_uint(x0), sc[ch][2 * i + 1] = __float_as_uint(x1);
                    }
#pragma unroll
                for (int ch = 0; ch < 2; ++ch) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) sc[ch][i] = __float_as_uint(ptx::ex2(__uint_as_float(sc[ch][i])));
                    uint32_t pk[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float p0 = __uint_as_float(sc[ch][2 * i]), p1 = __uint_as_float(sc[ch][2 * i + 1]);
                        pk[i] = pack16<F16>(p0, p1);
                        acc[i & 3] = ptx::add2(acc[i & 3], ptx::f2(p0, p1));
                    }
                    if (ok) ptx::tmem_st16(sb + ch * 16, pk);
                }
                ptx::tmem_st_wait();
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(p_full(slot, buf));
                float a0, a1;
                ptx::f2_split(ptx::add2(ptx::add2(acc[0], acc[1]), ptx::add2(acc[2], acc[3])), a0, a1);
                l += a0 + a1;
            }

            // -------------------------------------------------------- epilogue
            const int t = tw.tok0 + slot * p.slot_tokens + tl;
            const bool row_valid = tl < p.slot_tokens && t < tw.end;
            auto add_bad = [&](int ch, uint32_t (&o)[32]) {   // values that are not finite, to the rows that see them
#pragma unroll 1
                for (int x = 0; x < 512; ++x) {
                    if (!((tw.bad[x >> 7][(x >> 5) & 3] >> (x & 31)) & 1u)) continue;
                    const int key = tw.mask_tile * BN + x;
                    if (key >= limit) continue;
                    int64_t from = (tw.k0 + key) * p.v_token;
                    if (pb.mode != kKvPacked) {
                        // checked here too: it is the second look, and the table may be written meanwhile by mistake
                        const int pg = load_int(pb.table + static_cast<int64_t>(tw.b) * pb.table_w + (key >> pb.page_shift));
                        if (pg < 0 || pg >= pb.pages) {
                            atomicExch(pb.status, kStatusCheck);
                            continue;
                        }
                        from = pg * p.v_page + (key & ((1 << pb.page_shift) - 1)) * p.v_token;
                    }
                    const uint32_t *src = reinterpret_cast<const uint32_t *>(p.v + from + tw.h * p.v_head + ch * 32);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float a, b;
                        uint32_t v;
                        asm volatile("ld.global.b32 %0, [%1];" : "=r"(v) : "l"(src + i));   // one at a time: few registers
                        const uint32_t bad = nonfinite16<F16>(v);
                        unpack16<F16>(v, a, b);
                        if (bad & 0x8000u) o[2 * i] = __float_as_uint(__uint_as_float(o[2 * i]) + a);
                        if (bad & 0x80000000u) o[2 * i + 1] = __float_as_uint(__uint_as_float(o[2 * i + 1]) + b);
                    }
                }
                __syncwarp();
            };
            // Rows leave through shared memory, 64 bytes of each of the warp's 32 rows at a time: four
            // lanes write a row's 64 bytes, where a lane writing its own row 16 bytes at a time took
            // 32 cache lines per store.  Lane i holds row i's 16-byte pieces at piece ^ ((row >> 1) & 3).
            const uint32_t stage = base_s + C::OUT_OFF + (warp - 4) * C::OUT_WARP;
            const int piece = lane & 3, row_in = lane >> 2;
            const uint32_t put = stage + lane * 64, put_x = (lane >> 1) & 3, get = stage + row_in * 64 + ((piece ^ ((row_in >> 1) & 3)) << 4);
            const bool part = !tw.whole;
            const int64_t ws_at = static_cast<int64_t>(tw.slot) * 256 + slot * 128 + r;
            // byte address of this lane's row, -1: not written
            int64_t row_at = -1;
            if (row_valid)
                row_at = part ? ws_at * (D * 4)
                                  : 2 * ((static_cast<int64_t>(tw.q0) + t) * p.a.o_st + (static_cast<int64_t>(tw.h) * pb.G + g) * p.a.o_sh);
            char *const out = part ? reinterpret_cast<char *>(p.a.ws_o) : reinterpret_cast<char *>(p.a.o);
            int64_t rows[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) rows[i] = __shfl_sync(0xFFFFFFFFu, row_at, i * 8 + row_in);
            auto flush = [&](const uint32_t (&v)[16], int byte) {   // 64 bytes of every row, at this offset
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(put + ((i ^ put_x) << 4)), "r"(v[4 * i]),
                                 "r"(v[4 * i + 1]), "r"(v[4 * i + 2]), "r"(v[4 * i + 3]) : "memory");
                __syncwarp();
                uint4 u[4];   // rows i * 8 + row_in: (row >> 1) & 3 does not change with i
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(u[i].x), "=r"(u[i].y), "=r"(u[i].z), "=r"(u[i].w) : "r"(get + i * 512) : "memory");
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (rows[i] >= 0) *reinterpret_cast<uint4 *>(out + rows[i] + byte + piece * 16) = u[i];
                __syncwarp();
            };
            // a row that sees no key is zero; one whose visible logits are all -inf is 0 / 0
            const float inv = 1.0f / l;
            bool ok = true;
            if (steps > 0) {
                ok = wait_all(o_full(slot), o_ph);
                o_ph ^= 1u;
                ptx::tc_fence_after();
            }
            const bool fix = steps > 0 && *reinterpret_cast<const volatile uint32_t *>(&tw.any_bad) != 0u;
#pragma unroll 1
            for (int ch = 0; ch < D / 32; ++ch) {
                uint32_t ov[32];
                if (steps > 0 && ok) {
                    ptx::tmem_ld32(ocol + ch * 32, ov);
                    ptx::tmem_ld_wait(ov);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) ov[i] = 0u;
                }
                if (steps > 0 && ch == D / 32 - 1) {   // the next item may overwrite O
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(o_empty(slot));
                }
                if (fix) add_bad(ch, ov);
                uint32_t v[16];
                if (part) {
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) v[i] = ov[16 * hf + i];
                        flush(v, ch * 128 + hf * 64);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        v[i] = limit == 0 ? 0u : pack16<F16>(__uint_as_float(ov[2 * i]) * inv, __uint_as_float(ov[2 * i + 1]) * inv);
                    flush(v, ch * 64);
                }
            }
            if (part && row_valid) *reinterpret_cast<float2 *>(p.a.ws_ml + 2 * ws_at) = make_float2(m_ref, l);
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(w_empty(at));
            seq += n_u;
        }
    }

    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == 2) ptx::tmem_dealloc(tmem, C::TMEM_COLS);
}

}  // namespace lite
