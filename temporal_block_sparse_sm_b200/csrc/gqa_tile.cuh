// gqa_tile.cuh -- grouped-query attention of many query rows per key head (prompts, chunks
// of new tokens, video frames) on tcgen05, over packed or paged keys.
//
//   S = Q K^T (32 bits, Tensor Memory), running maximum m and sum l per row,
//   P = 2^(c S - c m) rounded to 16 bits, O += P V, o = O / l,  c = scale log2 e.
//
// A work item is 256 query rows of one key head: two slots of 128 rows, a row being one
// (token, head of the group) pair, so that the G heads of a group share every key and value
// that is loaded, and a slot covers 128 / G whole tokens (one TMA box of G heads by that many
// tokens fills it for any G; rows behind G * (128 / G) hold nothing).  Each slot owns 128
// TMEM columns of S and D of O; P is written over S and read by the MMA from TMEM.
//
// Warps: 0 loads (TMA: Q once, then 128-key tiles of K and V into rings), 1 issues MMAs,
// 2 and 3 clean the values of tiles that some row does not see whole, 4-7 and 8-11 are the
// softmax of slot 0 and 1, one thread per row with its 128 logits in registers.  While one
// slot's softmax runs, the tensor core works for the other.
//
// Per 128 x 128 x 128 slot tile the tensor core needs about 1024 cycles for both products,
// and the SM's exponential units 1024 for 16384 exponentials: a share of them runs as a
// polynomial on the FMA pipe.
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
    static constexpr int NTHREADS = 384;
    static constexpr uint32_t REG_LAUNCH = 168, REG_CTRL = 88, REG_SOFTMAX = 208;
    static_assert(128 * REG_CTRL + 256 * REG_SOFTMAX <= NTHREADS * REG_LAUNCH, "register split");
    static constexpr uint32_t Q_CHUNK = 128u * 128u, Q_SLOT = Q_CHUNK * DCH;
    static constexpr uint32_t KV_CHUNK = BN * 128u, KV_BYTES = KV_CHUNK * DCH;
    static constexpr uint32_t K_OFF = NSLOT * Q_SLOT, V_OFF = K_OFF + NST * KV_BYTES;
    static constexpr uint32_t SMEM_BYTES = V_OFF + NST * KV_BYTES + 1024u;
    static constexpr int NBAR = 2 + 6 * NST + 3 * NSLOT;
    static constexpr uint32_t TMEM_COLS = 512;
    __host__ __device__ static constexpr uint32_t s_col(int s) { return s * 128u; }
    __host__ __device__ static constexpr uint32_t o_col(int s) { return 256u + s * static_cast<uint32_t>(D); }
    // f32 result, A and B of the 16-bit type, A K-major, B K-major or MN-major
    __host__ __device__ static constexpr uint32_t idesc(int N, bool b_mn) {
        return (1u << 4) | (F16 ? 0u : (1u << 7) | (1u << 10)) | ((b_mn ? 1u : 0u) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
               (static_cast<uint32_t>(128 >> 4) << 24);
    }
    // pairs (of 16 in 32 columns) whose exponentials run on the FMA pipe
    static constexpr uint32_t POLY = 0x8888u;
};

// Maxima that keep a NaN.
__device__ __forceinline__ float max2_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// 2^x for a pair on the FMA pipe with the reduction of ptx::exp2_poly2 and a degree-5 Taylor
// polynomial of 2^f at 0: remainder (ln 2 / 2)^6 / 720 = 2.4e-6 relative.  fp16 weights are
// rounded to 2^-11, where the degree-3 polynomial's 7.5e-5 would show.
__device__ __forceinline__ void exp2_taylor2(float x0, float x1, float &y0, float &y1) {
    const uint64_t magic = ptx::f2(12582912.0f, 12582912.0f);
    const uint64_t x = ptx::f2(fmaxf(x0, -125.0f), fmaxf(x1, -125.0f));
    const uint64_t t = ptx::add2(x, magic);
    const uint64_t f = ptx::sub2(x, ptx::sub2(t, magic));
    constexpr float c1 = 0.6931471805599453f, c2 = 0.2402265069591007f, c3 = 0.05550410866482158f, c4 = 0.009618129107628477f,
                    c5 = 0.001333355814642844f;   // ln(2)^k / k!
    uint64_t q = ptx::fma2(ptx::f2(c5, c5), f, ptx::f2(c4, c4));
    q = ptx::fma2(q, f, ptx::f2(c3, c3));
    q = ptx::fma2(q, f, ptx::f2(c2, c2));
    q = ptx::fma2(q, f, ptx::f2(c1, c1));
    q = ptx::fma2(q, f, ptx::f2(1.0f, 1.0f));
    float q0, q1, t0, t1;
    ptx::f2_split(q, q0, q1);
    ptx::f2_split(t, t0, t1);
    y0 = __uint_as_float(__float_as_uint(q0) + (__float_as_uint(t0) << 23));
    y1 = __uint_as_float(__float_as_uint(q1) + (__float_as_uint(t1) << 23));
}

template <int D, bool F16>
__global__ void __launch_bounds__(TileCfg<D, F16>::NTHREADS, 1)
gqa_tile_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                const __grid_constant__ CUtensorMap tm_v, const TileParams p) {
    using C = TileCfg<D, F16>;
    constexpr int BN = C::BN, NST = C::NST, NSLOT = C::NSLOT, DCH = C::DCH;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[C::NBAR];
    __shared__ ScanScratch scan;
    __shared__ uint32_t s_abort, s_tmem, s_any_bad;
    __shared__ uint32_t s_bad[4][4];   // keys with values that are not finite, by tile from the first masked one

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t raw_s = ptx::smem_u32(smem_raw);
    const uint32_t base_s = (raw_s + 1023u) & ~1023u;
    uint8_t *base = smem_raw + (base_s - raw_s);
    const uint32_t bar0 = ptx::smem_u32(bars);
    const uint32_t q_full = bar0, drain = bar0 + 8u;
    auto k_full = [&](int st) { return bar0 + 8u * (2 + st); };
    auto v_full = [&](int st) { return bar0 + 8u * (2 + NST + st); };
    auto k_empty = [&](int st) { return bar0 + 8u * (2 + 2 * NST + st); };
    auto v_empty = [&](int st) { return bar0 + 8u * (2 + 3 * NST + st); };
    auto v_ok = [&](int st) { return bar0 + 8u * (2 + 4 * NST + st); };
    auto v_go = [&](int st) { return bar0 + 8u * (2 + 5 * NST + st); };
    auto s_full = [&](int s) { return bar0 + 8u * (2 + 6 * NST + s); };
    auto p_full = [&](int s) { return bar0 + 8u * (2 + 6 * NST + NSLOT + s); };
    auto o_full = [&](int s) { return bar0 + 8u * (2 + 6 * NST + 2 * NSLOT + s); };

    if (threadIdx.x == 0) {
        ptx::mbar_init(q_full, 1);
        ptx::mbar_init(drain, 1);
        for (int st = 0; st < NST; ++st) {
            ptx::mbar_init(k_full(st), 1);
            ptx::mbar_init(v_full(st), 1);
            ptx::mbar_init(k_empty(st), 1);
            ptx::mbar_init(v_empty(st), 1);
            ptx::mbar_init(v_ok(st), 64);
            ptx::mbar_init(v_go(st), 1);
        }
        for (int s = 0; s < NSLOT; ++s) {
            ptx::mbar_init(s_full(s), 1);
            ptx::mbar_init(p_full(s), 128);
            ptx::mbar_init(o_full(s), 1);
        }
        s_abort = 0u;
        s_any_bad = 0u;
        for (int i = 0; i < 16; ++i) s_bad[i >> 2][i & 3] = 0u;
        ptx::fence_barrier_init();
    }
    WorkItem w;
    const bool any = find_work<C::NTHREADS, true>(p.a.b, blockIdx.x, scan, w);
    __syncthreads();
    if (!any) return;
    const GqaBatch &pb = p.a.b;
    const int G = pb.G, n = w.s.n;

    // the item's tokens, the keys they see, and this segment's tiles of each slot
    const int tok0 = w.i * 2 * p.slot_tokens;
    const int lim_lo = visible_keys(pb, w.s, tok0);
    const int t_lo = w.seg * w.L;
    int lim_hi = 0, n_e = 0, ns[NSLOT];
#pragma unroll
    for (int s = 0; s < NSLOT; ++s) {
        const int first = tok0 + s * p.slot_tokens, last = min(first + p.slot_tokens, n) - 1;
        const int vis = first <= last ? visible_keys(pb, w.s, last) : 0;
        const int t_end = (vis + BN - 1) / BN;
        const int t_hi = w.L >= t_end - t_lo ? t_end : t_lo + w.L;
        ns[s] = t_hi > t_lo ? t_hi - t_lo : 0;
        lim_hi = max(lim_hi, vis);
        n_e = max(n_e, ns[s]);
    }
    if (n_e == 0 && w.segs > 1) return;                       // the join does not read it
    const int mask_tile = lim_lo / BN;                        // the first tile that some row does not see whole
    const int e_mask = max(0, mask_tile - t_lo);
    const WaitCtx wctx{&s_abort, pb.status};

    if (warp == 2) {
        ptx::tmem_alloc(ptx::smem_u32(&s_tmem), C::TMEM_COLS);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(&s_tmem);

    if (warp < 4) {
        ptx::regs_dec<C::REG_CTRL>();
        if (warp == 0) {
            // -------------------------------------------------------- loads
            KvTiles<BN, DCH> kv(pb, w, lim_hi);
            const uint32_t q_box = static_cast<uint32_t>(p.slot_tokens * G) * 128u;
            if (n_e > 0) {
                if (ptx::elect_one()) {
                    uint32_t bytes = 0;
                    for (int s = 0; s < NSLOT; ++s)
                        if (ns[s] > 0) bytes += q_box * DCH;
                    ptx::mbar_arrive_expect_tx(q_full, bytes);
                    for (int s = 0; s < NSLOT; ++s)
                        if (ns[s] > 0)
                            for (int c = 0; c < DCH; ++c)
                                ptx::tma_load_4d(base_s + s * C::Q_SLOT + c * C::Q_CHUNK, &tm_q, q_full, c * 64, w.h * G,
                                                 w.s.q0 + tok0 + s * p.slot_tokens, 0);
                }
                __syncwarp();
            }
            int pg = n_e > 0 ? kv.page_of(t_lo, lane) : -1;
            int k_issued = 0, v_issued = 0;
            for (int e = 0; e < n_e; ++e) {
                const int st = e % NST, t = t_lo + e;
                const uint32_t ph = ((e / NST) & 1) ^ 1u;
                const int next = e + 1 < n_e ? kv.page_of(t + 1, lane) : -1;
                const uint32_t bytes = static_cast<uint32_t>(kv.boxes(t) * kv.box) * D * 2u;
                if (!__all_sync(0xFFFFFFFFu, wait_bar(k_empty(st), ph, wctx))) break;
                ptx::mbar_arrive_expect_tx_elect(k_full(st), bytes);
                __syncwarp();
                kv.load(base_s + C::K_OFF + st * C::KV_BYTES, &tm_k, k_full(st), t, lane, pg);
                __syncwarp();
                k_issued = e + 1;
                if (!__all_sync(0xFFFFFFFFu, wait_bar(v_empty(st), ph, wctx))) break;
                ptx::mbar_arrive_expect_tx_elect(v_full(st), bytes);
                __syncwarp();
                kv.load(base_s + C::V_OFF + st * C::KV_BYTES, &tm_v, v_full(st), t, lane, pg);
                // the cleaning warps join at tile e_mask: v_full(st) is now in this tile's phase
                if (e >= e_mask && lane == 0) ptx::mbar_arrive(v_go(st));
                __syncwarp();
                v_issued = e + 1;
                pg = next;
            }
            // every copy that this block started lands before it exits
            if (n_e > 0) drain_wait(q_full, 0);
            for (int e = max(0, k_issued - NST); e < k_issued; ++e) drain_wait(k_full(e % NST), (e / NST) & 1);
            for (int e = max(0, v_issued - NST); e < v_issued; ++e) drain_wait(v_full(e % NST), (e / NST) & 1);
            __syncwarp();
        } else if (warp == 1) {
            // -------------------------------------------------------- MMA issue
            constexpr uint32_t IDESC_QK = C::idesc(BN, false), IDESC_PV = C::idesc(D, true);
            const uint64_t dq0 = ptx::sdesc_sw128(base_s, 16, 1024);
            const uint64_t dk0 = ptx::sdesc_sw128(base_s + C::K_OFF, 16, 1024);
            const uint64_t dv0 = ptx::sdesc_sw128(base_s + C::V_OFF, C::KV_CHUNK, 1024);
            auto wait_all = [&](uint32_t bar, uint32_t par) { return __all_sync(0xFFFFFFFFu, wait_bar(bar, par, wctx)); };
            auto issue_qk = [&](int s, int st) {
                const uint64_t qa = dq0 + ((s * C::Q_SLOT) >> 4), ka = dk0 + ((st * C::KV_BYTES) >> 4);
                if (ptx::elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        ptx::mma_ss(tmem + C::s_col(s), qa + (((kk >> 2) * C::Q_CHUNK + (kk & 3) * 32) >> 4),
                                    ka + (((kk >> 2) * C::KV_CHUNK + (kk & 3) * 32) >> 4), IDESC_QK, kk > 0 ? 1u : 0u);
                }
                __syncwarp();
            };
            auto issue_pv = [&](int s, int st, bool first) {
                const uint64_t va = dv0 + ((st * C::KV_BYTES) >> 4);
                if (ptx::elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < BN / 16; ++kk)
                        ptx::mma_ts(tmem + C::o_col(s), tmem + C::s_col(s) + kk * 8, va + ((kk * 16 * 128) >> 4), IDESC_PV,
                                    (first && kk == 0) ? 0u : 1u);
                }
                __syncwarp();
            };
            bool ok = n_e > 0 ? wait_all(q_full, 0) : true;
            if (n_e > 0) {
                ok = wait_all(k_full(0), 0) && ok;
                ptx::tc_fence_after();
                for (int s = 0; s < NSLOT; ++s)
                    if (ns[s] > 0) {
                        if (ok) issue_qk(s, 0);
                        ptx::mma_commit_elect(s_full(s));
                    }
                ptx::mma_commit_elect(k_empty(0));
            }
            for (int e = 0; e < n_e; ++e) {
                const int st = e % NST, st1 = (e + 1) % NST;
                const uint32_t ph = (e / NST) & 1, ph1 = ((e + 1) / NST) & 1;
                bool v_ready = false, k_ready = false;
                for (int s = 0; s < NSLOT; ++s) {
                    if (e < ns[s]) {
                        ok = wait_all(p_full(s), e & 1) && ok;
                        ptx::tc_fence_after();
                        if (!v_ready) {
                            ok = wait_all(v_full(st), ph) && ok;
                            if (e >= e_mask) ok = wait_all(v_ok(st), ((e - e_mask) / NST) & 1) && ok;
                            v_ready = true;
                        }
                        if (ok) issue_pv(s, st, e == 0);
                    }
                    if (e + 1 < ns[s]) {
                        if (!k_ready) {
                            ok = wait_all(k_full(st1), ph1) && ok;
                            ptx::tc_fence_after();
                            k_ready = true;
                        }
                        if (ok) issue_qk(s, st1);
                        ptx::mma_commit_elect(s_full(s));
                    }
                    if (e + 1 == ns[s]) ptx::mma_commit_elect(o_full(s));
                }
                if (e + 1 < n_e) ptx::mma_commit_elect(k_empty(st1));
                ptx::mma_commit_elect(v_empty(st));
            }
            ptx::mma_commit_elect(drain);
            drain_wait(drain, 0);
            __syncwarp();
        } else {
            // -------------------------------------------------------- values of masked tiles
            const int id = threadIdx.x - 64;
            for (int e = e_mask; e < n_e; ++e) {
                const int st = e % NST, k0 = (t_lo + e) * BN;
                if (!__all_sync(0xFFFFFFFFu, wait_bar(v_go(st), ((e - e_mask) / NST) & 1, wctx))) break;
                if (!__all_sync(0xFFFFFFFFu, wait_bar(v_full(st), (e / NST) & 1, wctx))) break;
                uint8_t *vt = base + C::V_OFF + st * C::KV_BYTES;
                for (int x = id; x < BN * DCH * 8; x += 64) {    // 16-byte pieces
                    const int key = (x >> 3) % BN;
                    uint4 *at = reinterpret_cast<uint4 *>(vt + x * 16);
                    if (k0 + key >= lim_hi) {
                        *at = make_uint4(0u, 0u, 0u, 0u);
                    } else if (k0 + key >= lim_lo) {
                        uint32_t v[4] = {at->x, at->y, at->z, at->w}, any_bad = 0u;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint32_t b = nonfinite16<F16>(v[j]);
                            any_bad |= b;
                            v[j] &= ~((b >> 15) * 0xFFFFu);      // one bit per half -> the half's 16 bits
                        }
                        if (any_bad) {
                            *at = make_uint4(v[0], v[1], v[2], v[3]);
                            atomicOr(&s_bad[(t_lo + e - mask_tile) & 3][key >> 5], 1u << (key & 31));
                            *reinterpret_cast<volatile uint32_t *>(&s_any_bad) = 1u;
                        }
                    }
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // the MMA reads what was written here
                ptx::mbar_arrive(v_ok(st));
            }
        }
    } else {
        // ------------------------------------------------------------ softmax
        ptx::regs_inc<C::REG_SOFTMAX>();
        const int slot = warp / 4 - 1;
        const int r = (warp & 3) * 32 + lane;
        const int tl = r / G, g = r - tl * G;
        const int t = tok0 + slot * p.slot_tokens + tl;
        const bool row_valid = tl < p.slot_tokens && t < n;
        const int limit = row_valid ? visible_keys(pb, w.s, t) : 0;
        const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const uint32_t scol = lane_base + C::s_col(slot), ocol = lane_base + C::o_col(slot);
        const float cl2 = p.a.scale_log2;
        const float resc = 8.0f / cl2;
        const int tiles = ns[slot];
        float m_ref = -INFINITY, l = 0.0f;
        for (int e = 0; e < tiles; ++e) {
            bool ok = __all_sync(0xFFFFFFFFu, wait_bar(s_full(slot), e & 1, wctx));
            ptx::tc_fence_after();
            uint32_t sc[4][32];
            if (ok) {
#pragma unroll
                for (int ch = 0; ch < 4; ++ch) ptx::tmem_ld32(scol + ch * 32, sc[ch]);
                ptx::tmem_ld_wait(sc[0]);
#pragma unroll
                for (int ch = 1; ch < 4; ++ch) ptx::reg_tie(sc[ch]);
            } else {
#pragma unroll
                for (int ch = 0; ch < 4; ++ch)
#pragma unroll
                    for (int i = 0; i < 32; ++i) sc[ch][i] = 0u;
            }
            if (e >= e_mask) {
                const int left = limit - (t_lo + e) * BN;
#pragma unroll
                for (int ch = 0; ch < 4; ++ch)
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (ch * 32 + i >= left) sc[ch][i] = __float_as_uint(-INFINITY);
            }
            float mx[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) mx[k] = __uint_as_float(sc[0][k]);
#pragma unroll
            for (int ch = 0; ch < 4; ++ch)
#pragma unroll
                for (int c = ch == 0 ? 8 : 0; c < 32; c += 16)
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        mx[k] = c + 8 + k < 32 ? max3_nan(mx[k], __uint_as_float(sc[ch][c + k]), __uint_as_float(sc[ch][c + 8 + k]))
                                               : max2_nan(mx[k], __uint_as_float(sc[ch][c + k]));
            const float m_loc = max3_nan(max3_nan(mx[0], mx[1], mx[2]), max3_nan(mx[3], mx[4], mx[5]), max2_nan(mx[6], mx[7]));
            float alpha = 1.0f;
            bool rescale = false;
            if (m_loc - m_ref > resc) {              // also the row's first finite maximum
                alpha = ptx::ex2((m_ref - m_loc) * cl2);
                rescale = l != 0.0f;                 // O is zero before the first weight
                l *= alpha;
                m_ref = m_loc;
            }
            // a visible logit of +inf or NaN leaves the row without a softmax (inf - inf); the
            // polynomial below would not carry that
            if (!(m_loc < INFINITY)) l = __uint_as_float(0x7FC00000u);
            if (__any_sync(0xFFFFFFFFu, rescale) && ok && e > 0) {
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
            // P = 2^(c s - c m); the sum adds the rounded weights that the product uses
            const float neg = (m_ref == -INFINITY ? 0.0f : -m_ref * cl2) + weight_bias<F16>();
            const uint64_t c2 = ptx::f2(cl2, cl2), n2 = ptx::f2(neg, neg);
            float acc[8] = {};
#pragma unroll
            for (int ch = 0; ch < 4; ++ch) {
                uint32_t pk[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    float x0, x1, p0, p1;
                    ptx::f2_split(ptx::fma2(ptx::f2(__uint_as_float(sc[ch][2 * i]), __uint_as_float(sc[ch][2 * i + 1])), c2, n2), x0, x1);
                    if ((C::POLY >> i) & 1u) {
                        if constexpr (F16) exp2_taylor2(x0, x1, p0, p1);
                        else ptx::exp2_poly2(x0, x1, p0, p1);
                    } else {
                        p0 = ptx::ex2(x0);
                        p1 = ptx::ex2(x1);
                    }
                    pk[i] = pack16<F16>(p0, p1);
                    add16x2<F16>(acc[2 * (i & 3)], acc[2 * (i & 3) + 1], pk[i]);
                }
                if (ok) ptx::tmem_st16(scol + ch * 16, pk);
            }
            l += ((acc[0] + acc[1]) + (acc[2] + acc[3])) + ((acc[4] + acc[5]) + (acc[6] + acc[7]));
            ptx::tmem_st_wait();
            ptx::tc_fence_before();
            ptx::mbar_arrive(p_full(slot));
        }

        // ------------------------------------------------------------ epilogue
        bool ok = true;
        if (tiles > 0) {
            ok = __all_sync(0xFFFFFFFFu, wait_bar(o_full(slot), 0, wctx));
            ptx::tc_fence_after();
        }
        const bool fix = tiles > 0 && *reinterpret_cast<volatile uint32_t *>(&s_any_bad) != 0u;
        const float inv = w.segs > 1 ? 1.0f : limit == 0 ? 0.0f : 1.0f / l;
        const int row = slot * 128 + r;
        const int64_t at = static_cast<int64_t>(w.slot) * 256 + row;
        uint16_t *dst = p.a.o + (static_cast<int64_t>(w.s.q0) + t) * p.a.o_st + (static_cast<int64_t>(w.h) * G + g) * p.a.o_sh;
#pragma unroll 1
        for (int ch = 0; ch < D / 32; ++ch) {
            uint32_t ov[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) ov[i] = 0u;
            if (tiles > 0 && ok) {
                ptx::tmem_ld32(ocol + ch * 32, ov);
                ptx::tmem_ld_wait(ov);
            }
            if (fix) {
#pragma unroll 1
                for (int x = 0; x < 512; ++x) {
                    if (!((s_bad[x >> 7][(x >> 5) & 3] >> (x & 31)) & 1u)) continue;
                    const int key = mask_tile * BN + x;
                    if (key >= limit) continue;
                    const int64_t from = pb.mode == kKvPacked
                        ? (w.s.k0 + key) * p.v_token
                        : __ldg(pb.table + static_cast<int64_t>(w.b) * pb.table_w + (key >> pb.page_shift)) * p.v_page +
                              (key & ((1 << pb.page_shift) - 1)) * p.v_token;
                    const uint32_t *src = reinterpret_cast<const uint32_t *>(p.v + from + w.h * p.v_head + ch * 32);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float a, b;
                        const uint32_t v = __ldg(src + i), bad = nonfinite16<F16>(v);
                        unpack16<F16>(v, a, b);
                        if (bad & 0x8000u) ov[2 * i] = __float_as_uint(__uint_as_float(ov[2 * i]) + a);
                        if (bad & 0x80000000u) ov[2 * i + 1] = __float_as_uint(__uint_as_float(ov[2 * i + 1]) + b);
                    }
                }
            }
            if (row_valid) {
                if (w.segs > 1) {
                    float4 *wo = reinterpret_cast<float4 *>(p.a.ws_o + at * D + ch * 32);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        wo[i] = make_float4(__uint_as_float(ov[4 * i]), __uint_as_float(ov[4 * i + 1]), __uint_as_float(ov[4 * i + 2]),
                                            __uint_as_float(ov[4 * i + 3]));
                } else {
                    uint32_t pk[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        pk[i] = limit == 0 ? 0u : pack16<F16>(__uint_as_float(ov[2 * i]) * inv, __uint_as_float(ov[2 * i + 1]) * inv);
                    uint4 *d4 = reinterpret_cast<uint4 *>(dst + ch * 32);
#pragma unroll
                    for (int i = 0; i < 4; ++i) d4[i] = make_uint4(pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
                }
            }
        }
        if (w.segs > 1 && row_valid) *reinterpret_cast<float2 *>(p.a.ws_ml + 2 * at) = make_float2(m_ref, l);
    }

    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == 2) ptx::tmem_dealloc(tmem, C::TMEM_COLS);
}

}  // namespace lite
