// gqa_rows.cuh -- grouped-query attention of a few query rows per key head (a decoding
// step), over paged or packed keys, split along the keys; and the kernel that joins the
// segments of split items.
//
//   o_r = sum_j 2^(c (q_r . k_j) - c m_r) v_j / sum_j 2^(c (q_r . k_j) - c m_r),
//   c = scale log2 e,  j over the keys that row r sees.
//
// A work item is 16 query rows (token t, head g of the group; flattened t * G + g) of one
// key head: all heads of a group share the keys that are read, and 16 is the M of
// mma.sync.m16n8k16.  Bound by memory: per key 4 D bytes are read for 64 D operations, far
// below what even the legacy tensor path delivers, so nothing is gained from 128-row
// tcgen05 tiles of which one row in eight would be used.
//
// A block is four computing warps and one that walks the block's items and issues TMA loads of
// 64-key tiles into a ring (three stages of 32 KB at D = 128; two blocks per SM keep up to
// 192 KB in flight).  A computing warp owns 16 keys of every tile and keeps its own running
// maximum, sum and output, so warps meet only at the ring's barriers; their states are joined at
// an item's end, while the ring already fills with the next item's keys.
//
// Measured (B200, bf16, D = 128, in a graph): 64 single tokens of 32 heads over 277,485 cached
// tokens of 8 key heads, 1138 MB, 185 us (6140 GB/s, 0.94 of a plain copy); one token over 1,000
// 12.6 us, of which walking to the first load and the join after the last part take 3 us each.  Q K^T
// in two accumulators was slower.  Up to three of two blocks' ten warps share a quarter of the SM's
// registers, 168 a thread; at D = 128 that is 20 (bf16) and 32 bytes (fp16) short, which are spilled.
//
// Values that no row sees (behind the last key, in a page's unused part) are zeroed in
// shared memory before the product, since 0 * NaN is NaN.  Where some rows see a key that
// others do not, and a value there is not finite, the product of those 16 keys is done
// with scalar code that leaves hidden keys out.
#pragma once

#include "serving_internal.cuh"

namespace lite {

struct GqaParams {
    GqaBatch b;
    const uint16_t *q;
    uint16_t *o;
    int64_t q_st, q_sh, o_st, o_sh;   // token and head strides, elements
    float scale_log2;                 // scale * log2 e
    float *ws_o;                      // workspace: [slot][rows of an item][D] unnormalised outputs
    float *ws_ml;                     // [slot][rows of an item][2]: running maximum (raw logit), sum
    JoinItem *joins;                  // [blocks]; null: no item is cut
    int probe_wait;                   // test of the timeout path: a warp of block 0 waits for what never comes
};

template <int D>
struct RowsCfg {
    static constexpr int BN = 64;               // keys of a tile
    static constexpr int ROWS = kFewRows;
    static constexpr int NWARP = 4;             // computing warps
    static constexpr int NTHREADS = 32 * (NWARP + 1);
    static constexpr int DCH = D / 64;
    static constexpr uint32_t KV_BYTES = BN * D * 2u;
    static constexpr uint32_t CHUNK_BYTES = BN * 128u;
    static constexpr int NST = D == 128 ? 3 : 6;
    static constexpr uint32_t RING_BYTES = NST * 2u * KV_BYTES;
    static constexpr uint32_t SMEM_BYTES = RING_BYTES + 1024u;
};

namespace ptx {
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t &a, uint32_t &b, uint32_t &c, uint32_t &d) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(a), "=r"(b), "=r"(c), "=r"(d) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t &a, uint32_t &b, uint32_t &c, uint32_t &d) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(a), "=r"(b), "=r"(c), "=r"(d) : "r"(addr) : "memory");
}
template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (F16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *m, uint32_t bar, int x, int y, int z, int w) {
    asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
                 : "memory");
}
}  // namespace ptx

// Where a tile's keys lie: one TMA box per page (or per tile, where a page holds it all).
// Lane `lane` of the producing warp owns box `lane` of a tile and looks its page up ahead
// of the wait for a free stage.
template <int BN, int DCH>
struct KvTiles {
    const GqaBatch &p;
    int64_t k0;   // first row of the sequence's keys (packed)
    int b, h;     // sequence and key head
    int end;      // keys that any row of the item sees; boxes behind it are not loaded
    int box;      // rows of a box
    __device__ __forceinline__ KvTiles(const GqaBatch &p_, int64_t k0_, int b_, int h_, int end_) : p(p_), k0(k0_), b(b_), h(h_), end(end_) {
        const int page = p.mode == kKvPacked ? BN : 1 << p.page_shift;
        box = page < BN ? page : BN;
    }
    __device__ __forceinline__ int boxes(int t) const {   // boxes of tile t that hold a key before `end`
        const int left = end - t * BN;
        return left >= BN ? BN / box : (left + box - 1) / box;
    }
    // the page of this lane's box of tile t (-1: the lane has none)
    __device__ __forceinline__ int page_of(int t, int lane) const {
        if (lane >= boxes(t)) return -1;
        if (p.mode == kKvPacked) return 0;
        const int pg = load_int(p.table + static_cast<int64_t>(b) * p.table_w + ((t * BN + lane * box) >> p.page_shift));
        if (pg >= 0 && pg < p.pages) return pg;
        atomicExch(p.status, kStatusCheck);
        return static_cast<int>(p.pages);   // outside the tensor map: reads as zeros
    }
    __device__ __forceinline__ void load(uint32_t dst, const CUtensorMap *m, uint32_t bar, int t, int lane, int pg) const {
        if (pg < 0) return;
        const int j = t * BN + lane * box;
        const int row = p.mode == kKvPacked ? static_cast<int>(k0) + j : j & ((1 << p.page_shift) - 1);
#pragma unroll
        for (int c = 0; c < DCH; ++c) {
            const uint32_t at = dst + c * (BN * 128u) + static_cast<uint32_t>(lane * box) * 128u;
            if (p.mode == kKvPagesBhnd) ptx::tma_load_4d(at, m, bar, c * 64, row, h, pg);
            else ptx::tma_load_4d(at, m, bar, c * 64, h, row, pg);
        }
    }
};

// The join may be launched while the kernel that writes the parts still runs.
__device__ __forceinline__ void join_may_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// What the warps of a block need to know of one item (shared memory).
struct RowsWork {
    int q0, n, m, i, h;
    int t0, t1, lim_lo, lim_hi;   // key tiles; keys that the first and the last row see
    int whole, slot, valid;
};

// Weights for the product, each as two 16-bit numbers: the weight rounded towards zero, and what that left
// over.  The kernel is bound by memory, so the second product costs next to nothing (0 to 1 %), and the
// weights' rounding, as large as the output's own, is gone.  The second number of a weight is positive where
// the first is, so that an infinite value stays infinite (0 * infinity is NaN).  What is added for that, of a
// weight p:
// bf16: at most 2^-17 p, as much as the second number's own rounding (or 2^-133, the type's least, where p is
//   below 2^-116).
// fp16: the type ends at 2^-24 and 65,504, so weights are taken relative to the largest of the 16 keys of a
//   step, at 2^15: at most 2^-39 of that one, and as much for the rounding of small weights.  The largest weights of
//   all steps are no more than the row's sum, so both stay below 16 * 2^-39 of it, however many keys there are;
//   relative to the row's largest weight they would grow with the keys (a row of 9,000 keys at 2^-40 of its largest
//   under values of 60,000 came out as 0.0014 instead of 0.0005).
constexpr float kGroupBias = 15.0f;

template <bool F16>
__device__ __forceinline__ float second_number(float p, float first) {
    if constexpr (F16) return first > 0.0f ? fmaxf(p - first, 0x1p-24f) : p;
    else return p > 0.0f ? fmaxf(p - first, fmaxf(p * 0x1p-17f, 0x1p-133f)) : 0.0f;
}
template <bool F16>
__device__ __forceinline__ void split16(float p0, float p1, uint32_t &hi, uint32_t &lo) {
    hi = pack16_down<F16>(p0, p1);
    float h0, h1;
    unpack16<F16>(hi, h0, h1);
    lo = pack16<F16>(second_number<F16>(p0, h0), second_number<F16>(p1, h1));
}

template <int D, bool F16>
__global__ void __launch_bounds__(RowsCfg<D>::NTHREADS, 2)
gqa_rows_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const GqaParams p) {
    using C = RowsCfg<D>;
    constexpr int BN = C::BN, NST = C::NST, DCH = C::DCH, NWORK = 2;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[2 * NST + 2 * NWORK + 1];
    __shared__ ScanScratch scan;
    __shared__ RowsWork works[NWORK];
    __shared__ float s_ml[C::NWARP][C::ROWS][2];
    __shared__ __align__(16) float s_o[C::NWARP][C::ROWS][36];   // 32 columns of the warps' outputs at a time
    __shared__ uint32_t s_abort;

    GqaBatch pb = p.b;               // what is fixed for this kernel, as constants
    pb.unit_tokens = 0, pb.tile_shift = 6;
    static_assert(BN == 64);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t raw_s = ptx::smem_u32(smem_raw);
    const uint32_t base_s = (raw_s + 1023u) & ~1023u;
    uint8_t *base = smem_raw + (base_s - raw_s);
    auto full = [&](int st) { return ptx::smem_u32(bars + st); };
    auto empty = [&](int st) { return ptx::smem_u32(bars + NST + st); };
    auto w_full = [&](int k) { return ptx::smem_u32(bars + 2 * NST + k); };
    auto w_empty = [&](int k) { return ptx::smem_u32(bars + 2 * NST + NWORK + k); };

    if (threadIdx.x == 0) {
        for (int st = 0; st < NST; ++st) {
            ptx::mbar_init(full(st), 1);
            ptx::mbar_init(empty(st), C::NWARP);
        }
        for (int k = 0; k < NWORK; ++k) {
            ptx::mbar_init(w_full(k), 1);
            ptx::mbar_init(w_empty(k), C::NWARP);
        }
        ptx::mbar_init(ptx::smem_u32(bars + 2 * NST + 2 * NWORK), 1);   // nothing arrives here
        s_abort = 0u;
        ptx::fence_barrier_init();
    }
    wait_for_earlier_kernels();
    const int64_t stretch = stretch_units<C::NTHREADS>(pb, gridDim.x, scan);
    __syncthreads();
    join_may_start();
    const int G = pb.G;
    const WaitScope wctx{&s_abort, pb.status};

    if (warp == C::NWARP) {
        // ------------------------------------------------------------ items and loads
        BlockWalk walk;
        walk.start(pb, stretch, p.joins, lane);
        int kv = 0;                  // tiles loaded so far
        bool ok = true;
        for (int k = 0; ok; ++k) {
            const bool more = walk.next(pb, p.joins, lane);
            const LineItem &it = walk.it;
            const int at = k % NWORK;
            if (!wait_phase_warp(w_empty(at), ((k / NWORK) & 1) ^ 1u, wctx)) break;
            if (lane == 0) {
                RowsWork &w = works[at];
                w.valid = more ? 1 : 0;
                if (more) {
                    w.q0 = it.s.q0, w.n = it.s.n, w.m = it.s.m, w.i = it.i, w.h = it.h, w.t0 = walk.t0, w.t1 = walk.t1;
                    w.lim_lo = visible_keys(pb, it.s, it.i == 0 ? 0 : static_cast<int>(quotient(static_cast<int64_t>(it.i) * C::ROWS, G)));
                    w.lim_hi = it.keys, w.whole = walk.whole ? 1 : 0, w.slot = walk.slot;
                }
                ptx::mbar_arrive(w_full(at));
            }
            __syncwarp();
            if (!more) break;
            KvTiles<BN, DCH> tiles(pb, it.s.k0, it.b, it.h, it.keys);
            int pg = walk.t0 < walk.t1 ? tiles.page_of(walk.t0, lane) : -1;
            for (int t = walk.t0; t < walk.t1; ++t, ++kv) {
                const int st = kv % NST;
                const int next = t + 1 < walk.t1 ? tiles.page_of(t + 1, lane) : -1;
                if (!(ok = wait_phase_warp(empty(st), ((kv / NST) & 1) ^ 1u, wctx))) break;
                if (lane == 0) ptx::mbar_arrive_expect_tx(full(st), tiles.boxes(t) * tiles.box * D * 4u);
                __syncwarp();
                const uint32_t dst = base_s + st * 2u * C::KV_BYTES;
                tiles.load(dst, &tm_k, full(st), t, lane, pg);
                tiles.load(dst + C::KV_BYTES, &tm_v, full(st), t, lane, pg);
                __syncwarp();
                pg = next;
            }
        }
        // every copy that this block started lands before it exits
        for (int e = max(0, kv - NST); e < kv; ++e) drain_phase(full(e % NST), (e / NST) & 1);
        return;
    }

    // ---------------------------------------------------------------- computing warps
    if (p.probe_wait && blockIdx.x == 0 && warp == 0) wait_phase_warp(ptx::smem_u32(bars + 2 * NST + 2 * NWORK), 0, wctx);
    const int gid = lane >> 2, tig = lane & 3;
    const float cl2 = p.scale_log2;
    const float resc = fminf(8.0f / cl2, 3e38f);    // (finite: a first maximum always moves it)
    // the reference moves when the maximum rose by over 2^8 in weight
    int kv = 0;
    for (int k = 0;; ++k) {
    // one decision for the four warps, so that their barriers stay balanced
    const bool known = wait_phase_warp(w_full(k % NWORK), (k / NWORK) & 1, wctx);
    if (ptx::bar_red_or(1, 32 * C::NWARP, !known)) return;
    const RowsWork w = works[k % NWORK];
    if (!w.valid) return;
    const SeqInfo seq{w.q0, w.n, w.m, 0};
    const int64_t row0 = static_cast<int64_t>(w.i) * C::ROWS;
    const int nrows = static_cast<int>(min(static_cast<int64_t>(C::ROWS), static_cast<int64_t>(w.n) * G - row0));
    const int lim_lo = w.lim_lo, lim_hi = w.lim_hi;
    // the thread's two rows (of the item's 16): gid and gid + 8
    int lim[2];
    uint32_t qf[D / 16][4];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int row = gid + 8 * r;
        const bool ok = row < nrows;
        const int t = ok ? static_cast<int>(quotient(row0 + row, G)) : 0, g = ok ? static_cast<int>(row0 + row - static_cast<int64_t>(t) * G) : 0;
        lim[r] = ok ? visible_keys(pb, seq, t) : 0;
        const uint32_t *src = reinterpret_cast<const uint32_t *>(p.q + (static_cast<int64_t>(w.q0) + t) * p.q_st +
                                                                 (static_cast<int64_t>(w.h) * G + g) * p.q_sh);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            qf[kk][r] = ok ? src[kk * 8 + tig] : 0u;
            qf[kk][2 + r] = ok ? src[kk * 8 + 4 + tig] : 0u;
        }
    }
    float m_ref[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
    float acc[D / 8][4];
#pragma unroll
    for (int n = 0; n < D / 8; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.0f;

    // ldmatrix rows of this lane: matrix lane/8, row lane%8 of it
    const int mi = lane >> 3, mr = lane & 7;
    for (int t = w.t0; t < w.t1; ++t, ++kv) {
        const int st = kv % NST;
        const bool ok = wait_phase_warp(full(st), (kv / NST) & 1, wctx);
        const int kb = t * BN + warp * 16;             // the warp's first key
        if (ok && kb < lim_hi) {
            const uint32_t kt = base_s + st * 2u * C::KV_BYTES, vt = kt + C::KV_BYTES;
            float sc[2][4] = {};
            {
                // matrices: (keys 0-7, d 0-7), (keys 0-7, d 8-15), (keys 8-15, d 0-7), (keys 8-15, d 8-15)
                const int key = warp * 16 + (mi >> 1) * 8 + mr;
                const uint32_t rowa = kt + key * 128u;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t c16 = (kk & 3) * 2 + (mi & 1);
                    uint32_t b0, b1, b2, b3;
                    ptx::ldsm4(rowa + (kk >> 2) * C::CHUNK_BYTES + ((c16 ^ (key & 7)) << 4), b0, b1, b2, b3);
                    ptx::mma16816<F16>(sc[0], qf[kk], b0, b1);
                    ptx::mma16816<F16>(sc[1], qf[kk], b2, b3);
                }
            }
            const bool masked = kb + 16 > lim_lo;       // some row does not see all of these keys
            bool scalar = false;
            if (masked) {
#pragma unroll
                for (int nb = 0; nb < 2; ++nb)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (kb + nb * 8 + 2 * tig + (j & 1) >= lim[j >> 1]) sc[nb][j] = -INFINITY;
                uint32_t bad = 0;
                for (int x = lane; x < 16 * DCH * 8; x += 32) {   // 16-byte pieces of the 16 value rows
                    const int key = x / (DCH * 8), c = (x / 8) % DCH, piece = x % 8;
                    uint4 *at = reinterpret_cast<uint4 *>(base + (vt - base_s) + c * C::CHUNK_BYTES +
                                                          (warp * 16 + key) * 128u + piece * 16u);
                    if (kb + key >= lim_hi) {
                        *at = make_uint4(0u, 0u, 0u, 0u);
                    } else if (kb + key >= lim_lo) {
                        const uint4 v = *at;
                        bad |= nonfinite16<F16>(v.x) | nonfinite16<F16>(v.y) | nonfinite16<F16>(v.z) | nonfinite16<F16>(v.w);
                    }
                }
                // the stage's next writer is TMA, by another proxy than these stores: ordered by this fence and the arrival
                ptx::fence_proxy_async();
                scalar = __any_sync(0xFFFFFFFFu, bad != 0u);
                __syncwarp();
            }
            float alpha[2], top[2];       // the largest logit of these keys
            bool moved = false;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float mx = fmaxf(fmaxf(sc[0][2 * r], sc[0][2 * r + 1]), fmaxf(sc[1][2 * r], sc[1][2 * r + 1]));
                mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
                top[r] = mx;
                alpha[r] = 1.0f;
                if (mx - m_ref[r] > resc) {             // also the row's first finite maximum
                    alpha[r] = ptx::ex2((m_ref[r] - mx) * cl2);
                    m_ref[r] = mx;
                    l[r] *= alpha[r];
                    moved = true;
                }
            }
            if (__any_sync(0xFFFFFFFFu, moved)) {
#pragma unroll
                for (int n = 0; n < D / 8; ++n) {
                    acc[n][0] *= alpha[0], acc[n][1] *= alpha[0];
                    acc[n][2] *= alpha[1], acc[n][3] *= alpha[1];
                }
            }
            // weights, in the place of the logits: of bf16 relative to the running reference; of fp16, whose range
            // is short, relative to the largest of these 16 keys (f brings the product into the frame of the sums)
            // The difference of the logits first: c s - c m with c m rounded is off by 2^-24 of c m, whole powers
            // of two for logits of 10^7 and more, which is beyond fp16's range.
            float f[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const float ref = F16 ? top[r] : m_ref[r], from = ref == -INFINITY ? 0.0f : ref;
                f[r] = !F16 ? 1.0f : ref == -INFINITY ? 0.0f : ptx::ex2(fmaf(ref - m_ref[r], cl2, -kGroupBias));
                float sum = 0.0f;
#pragma unroll
                for (int nb = 0; nb < 2; ++nb) {
#pragma unroll
                    for (int i = 2 * r; i < 2 * r + 2; ++i) sc[nb][i] = ptx::ex2(fmaf(sc[nb][i] - from, cl2, F16 ? kGroupBias : 0.0f));
                    sum += sc[nb][2 * r] + sc[nb][2 * r + 1];
                }
                l[r] = fmaf(sum, f[r], l[r]);
            }
            if (!scalar) {
                uint32_t pf[4], pl[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) split16<F16>(sc[x >> 1][2 * (x & 1)], sc[x >> 1][2 * (x & 1) + 1], pf[x], pl[x]);
                // matrices of V: (keys 0-7, d n..n+7), (keys 8-15, same d), then the next 8 d
                const int key = warp * 16 + (mi & 1) * 8 + mr;
                const uint32_t rowa = vt + key * 128u;
#pragma unroll
                for (int n = 0; n < D / 16; ++n) {
                    const uint32_t c16 = (n & 3) * 2 + (mi >> 1);
                    uint32_t b0, b1, b2, b3;
                    ptx::ldsm4t(rowa + (n >> 2) * C::CHUNK_BYTES + ((c16 ^ (key & 7)) << 4), b0, b1, b2, b3);
                    if constexpr (F16) {
                        float t0[4] = {}, t1[4] = {};
                        ptx::mma16816<F16>(t0, pf, b0, b1);
                        ptx::mma16816<F16>(t1, pf, b2, b3);
                        ptx::mma16816<F16>(t0, pl, b0, b1);
                        ptx::mma16816<F16>(t1, pl, b2, b3);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            acc[2 * n][j] = fmaf(t0[j], f[j >> 1], acc[2 * n][j]);
                            acc[2 * n + 1][j] = fmaf(t1[j], f[j >> 1], acc[2 * n + 1][j]);
                        }
                    } else {
                        ptx::mma16816<F16>(acc[2 * n], pf, b0, b1);
                        ptx::mma16816<F16>(acc[2 * n + 1], pf, b2, b3);
                        ptx::mma16816<F16>(acc[2 * n], pl, b0, b1);
                        ptx::mma16816<F16>(acc[2 * n + 1], pl, b2, b3);
                    }
                }
            } else {
#pragma unroll 1
                for (int key = 0; key < 16; ++key) {
                    const int from = (lane & ~3) | ((key & 7) >> 1);   // the lane holding this key's weights
                    float wt[2];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const float a = key < 8 ? sc[0][2 * r] : sc[1][2 * r], b = key < 8 ? sc[0][2 * r + 1] : sc[1][2 * r + 1];
                        wt[r] = f[r] * __shfl_sync(0xFFFFFFFFu, (key & 1) ? b : a, from);
                    }
                    const bool see0 = kb + key < lim[0], see1 = kb + key < lim[1];
#pragma unroll
                    for (int n = 0; n < D / 8; ++n) {
                        const uint32_t at = (n >> 3) * C::CHUNK_BYTES + (warp * 16 + key) * 128u + (((n & 7) ^ (key & 7)) << 4) + tig * 4u;
                        float v0, v1;
                        unpack16<F16>(*reinterpret_cast<const uint32_t *>(base + (vt - base_s) + at), v0, v1);
                        if (see0) acc[n][0] += wt[0] * v0, acc[n][1] += wt[0] * v1;
                        if (see1) acc[n][2] += wt[1] * v0, acc[n][3] += wt[1] * v1;
                    }
                }
            }
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(empty(st));
    }

    // ---------------------------------------------------------------- join of the four warps
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        l[r] += __shfl_xor_sync(0xFFFFFFFFu, l[r], 1);
        l[r] += __shfl_xor_sync(0xFFFFFFFFu, l[r], 2);
        if (tig == 0) {
            s_ml[warp][gid + 8 * r][0] = m_ref[r];
            s_ml[warp][gid + 8 * r][1] = l[r];
        }
    }
    ptx::bar_sync(1, 32 * C::NWARP);
    float f[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        float mx = -INFINITY;
#pragma unroll
        for (int j = 0; j < C::NWARP; ++j) mx = fmaxf(mx, s_ml[j][gid + 8 * r][0]);
        f[r] = m_ref[r] == -INFINITY ? 0.0f : ptx::ex2((m_ref[r] - mx) * cl2);
    }
    // 16 rows x 8 threads, four columns each of every 32
    const int row = threadIdx.x >> 3, col = (threadIdx.x & 7) * 4;
    float mx = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int j = 0; j < C::NWARP; ++j) mx = fmaxf(mx, s_ml[j][row][0]);
#pragma unroll
    for (int j = 0; j < C::NWARP; ++j) {
        const float mj = s_ml[j][row][0];
        sum += s_ml[j][row][1] * (mj == -INFINITY ? 0.0f : ptx::ex2((mj - mx) * cl2));   // 0 * NaN stays NaN
    }
    const int t = static_cast<int>(quotient(row0 + row, G)), g = static_cast<int>(row0 + row - static_cast<int64_t>(t) * G);
    // a row that sees no key is zero; one whose visible logits are all -inf is 0 / 0
    const float inv = visible_keys(pb, seq, t) == 0 ? 0.0f : 1.0f / sum;
    uint16_t *dst = p.o + (static_cast<int64_t>(w.q0) + t) * p.o_st + (static_cast<int64_t>(w.h) * G + g) * p.o_sh + col;
    const int64_t ws_at = static_cast<int64_t>(w.slot) * C::ROWS + row;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            float *at = &s_o[warp][gid][n * 8 + 2 * tig];
            const float (&a)[4] = acc[4 * c + n];
            *reinterpret_cast<float2 *>(at) = make_float2(a[0] * f[0], a[1] * f[0]);
            *reinterpret_cast<float2 *>(at + 8 * 36) = make_float2(a[2] * f[1], a[3] * f[1]);
        }
        ptx::bar_sync(1, 32 * C::NWARP);
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int j = 0; j < C::NWARP; ++j) {
            const float4 b = *reinterpret_cast<const float4 *>(&s_o[j][row][col]);
            v.x += b.x, v.y += b.y, v.z += b.z, v.w += b.w;
        }
        if (row < nrows) {
            if (w.whole)
                *reinterpret_cast<uint2 *>(dst + 32 * c) = make_uint2(pack16<F16>(v.x * inv, v.y * inv), pack16<F16>(v.z * inv, v.w * inv));
            else
                *reinterpret_cast<float4 *>(p.ws_o + ws_at * D + 32 * c + col) = v;
        }
        ptx::bar_sync(1, 32 * C::NWARP);
    }
    if (!w.whole && row < nrows && (threadIdx.x & 7) == 0) *reinterpret_cast<float2 *>(p.ws_ml + 2 * ws_at) = make_float2(mx, sum);
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(w_empty(k % NWORK));
    }
}

// Joins the items that reach beyond a block's stretch, from the records that the blocks left:
//   o = sum_s 2^(c (m_s - m)) O_s / sum_s 2^(c (m_s - m)) l_s  over a row's parts s.
// slot_tokens 0: items of 16 (token, head) rows; else two slots of 128 rows, slot_tokens tokens
// each.  The rows of all the items are shared out evenly over the grid, whatever few of the
// `blocks` records name an item: a warp takes a row, or, of items with many parts (up to one
// per block), 4 or 16 warps do.  (Finding the cut items again, as the blocks do, took 82 us for
// 147 of them with a block per 4 rows; reading and writing them takes 6.)
constexpr int kJoinThreads = 512, kJoinWarps = kJoinThreads / 32;

template <int D, bool F16>
__global__ void __launch_bounds__(kJoinThreads) gqa_join_kernel(const GqaParams p, int slot_tokens, int blocks) {
    constexpr int CPT = D / 32;
    __shared__ int s_sum[kJoinWarps], s_units[kJoinThreads];
    __shared__ float s_a[kJoinWarps][32][CPT + 1], s_mx[kJoinWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, G = p.b.G;
    const int rows = slot_tokens ? 256 : RowsCfg<D>::ROWS;
    auto rows_at_once = [](int parts) { return parts < 8 ? kJoinWarps : parts < 64 ? kJoinWarps / 4 : 1; };
    wait_for_earlier_kernels();
    // units (rows_at_once rows of an item) up to and with each record
    const int parts_here = threadIdx.x < blocks ? p.joins[threadIdx.x].parts : 0;
    int units = parts_here > 0 ? rows / rows_at_once(parts_here) : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int a = __shfl_up_sync(0xFFFFFFFFu, units, o);
        if (lane >= o) units += a;
    }
    if (lane == 31) s_sum[warp] = units;
    __syncthreads();
    for (int k = 0; k < warp; ++k) units += s_sum[k];
    s_units[threadIdx.x] = units;
    __syncthreads();
    const int total = s_units[kJoinThreads - 1];
    const float2 *ml = reinterpret_cast<const float2 *>(p.ws_ml);
    for (int u = blockIdx.x; u < total; u += gridDim.x) {
        int lo = 0, hi = blocks - 1;               // the first record with more than u units
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (s_units[mid] > u) hi = mid;
            else lo = mid + 1;
        }
        const JoinItem it = p.joins[lo];
        const int at_once = rows_at_once(it.parts), share = kJoinWarps / at_once;
        const int row = (u - (lo > 0 ? s_units[lo - 1] : 0)) * at_once + warp / share;
        int64_t t;
        int g;
        if (slot_tokens) {
            const int tl = (row & 127) / G;
            g = (row & 127) % G;
            t = tl < slot_tokens ? static_cast<int64_t>(it.i) * 2 * slot_tokens + (row >> 7) * slot_tokens + tl : it.n;
        } else {
            const int64_t flat = static_cast<int64_t>(it.i) * rows + row;
            t = quotient(flat, G), g = static_cast<int>(flat - t * G);
        }
        float a[CPT] = {}, sum = 0.0f, mx = -INFINITY;
        if (t < it.n) {
            // the first part may sit in its block's second slot, the others in the first one of the blocks behind
            auto part = [&](int x) { return static_cast<int64_t>(x == 0 ? it.slot0 : (it.slot0 & ~1) + 2 * x) * rows + row; };
            // the outputs of four parts are asked for before their weights are known
            constexpr int AHEAD = 4;
            for (int s0 = warp % share; s0 < it.parts; s0 += AHEAD * share) {
                float v[AHEAD][CPT];
                float2 x[AHEAD];
#pragma unroll
                for (int j = 0; j < AHEAD; ++j) {
                    const int s = s0 + j * share;
                    x[j] = make_float2(-INFINITY, 0.0f);
#pragma unroll
                    for (int c = 0; c < CPT; ++c) v[j][c] = 0.0f;
                    if (s < it.parts) {
                        const int64_t at = part(s);
                        x[j] = ml[at];
#pragma unroll
                        for (int c = 0; c < CPT; ++c) v[j][c] = p.ws_o[at * D + lane * CPT + c];
                    }
                }
                // this warp's sums to the frame of the largest maximum so far
                float top = mx;
#pragma unroll
                for (int j = 0; j < AHEAD; ++j) top = fmaxf(top, x[j].x);
                if (top != mx) {
                    const float f = ptx::ex2((mx - top) * p.scale_log2);
#pragma unroll
                    for (int c = 0; c < CPT; ++c) a[c] *= f;
                    sum *= f;
                    mx = top;
                }
#pragma unroll
                for (int j = 0; j < AHEAD; ++j) {
                    const float f = x[j].x == -INFINITY ? 0.0f : ptx::ex2((x[j].x - mx) * p.scale_log2);
#pragma unroll
                    for (int c = 0; c < CPT; ++c) a[c] += f * v[j][c];
                    sum += f * x[j].y;
                }
            }
        }
        if (share > 1) {
#pragma unroll
            for (int c = 0; c < CPT; ++c) s_a[warp][lane][c] = a[c];
            s_a[warp][lane][CPT] = sum;
            if (lane == 0) s_mx[warp] = mx;
            __syncthreads();
            if (warp % share == 0) {
                float top = mx;
                for (int j = 1; j < share; ++j) top = fmaxf(top, s_mx[warp + j]);
#pragma unroll
                for (int c = 0; c < CPT; ++c) a[c] = 0.0f;
                sum = 0.0f;
                for (int j = 0; j < share; ++j) {
                    const float f = s_mx[warp + j] == -INFINITY ? 0.0f : ptx::ex2((s_mx[warp + j] - top) * p.scale_log2);
#pragma unroll
                    for (int c = 0; c < CPT; ++c) a[c] += f * s_a[warp + j][lane][c];
                    sum += f * s_a[warp + j][lane][CPT];
                }
            }
        }
        if (t < it.n && warp % share == 0) {
            const SeqInfo seq{it.q0, it.n, it.m, 0};
            const float inv = visible_keys(p.b, seq, static_cast<int>(t)) == 0 ? 0.0f : 1.0f / sum;
            uint32_t *dst = reinterpret_cast<uint32_t *>(p.o + (static_cast<int64_t>(it.q0) + t) * p.o_st +
                                                         (static_cast<int64_t>(it.h) * G + g) * p.o_sh + lane * CPT);
#pragma unroll
            for (int c = 0; c < CPT / 2; ++c) dst[c] = pack16<F16>(a[2 * c] * inv, a[2 * c + 1] * inv);
        }
        if (share > 1) __syncthreads();
    }
}

}  // namespace lite
