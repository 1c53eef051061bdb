// rope_append.cuh -- new tokens' keys and values into a paged cache, the position rotation
// applied on the way, and the queries rotated beside them.
//
// Per token and head, for pairs (a, b) of elements below `rot` and the token's angles:
//   a' = a cos - b sin,  b' = a sin + b cos   (32 bits, rounded once),
// pairs (i, i + rot/2) or (2i, 2i + 1); the other elements and the values are copied.
//
// Bound by memory: every element is read and written once.  A thread owns 16 elements (8
// pairs) of one position inside the head, loads their angles once and walks over heads of
// its token, so the angles cost one read per `head_lanes` threads and not one per head.
// `head_lanes` threads of a token share its heads: many when there are few tokens (a
// decoding step, where only latency counts), few when there are many.
//
// Measured (B200): 20,671 tokens of 24 query and 4 key heads of 128, 341 MB, 58 us in a graph
// (5850 GB/s, 0.9 of a plain copy; the warps wait for their loads, 66% of the DRAM cycles are
// used); 64 tokens of 32 and 8 heads 4 us, a launch and two dependent loads (table, then rows).
#pragma once

#include "serving_internal.cuh"

namespace lite {

struct AppendParams {
    const uint16_t *q, *k, *v;
    uint16_t *q_out, *kc, *vc;
    int64_t q_st, q_sh, k_st, k_sh, v_st, v_sh, qo_st, qo_sh;   // token and head strides, elements
    int64_t c_sp, c_sh, c_st;                                   // cache strides: page, head, token in page
    const float *cos, *sin;                                     // [n_pos][rot / 2], or null: no rotation
    const int32_t *positions;                                   // [Tq] rows of cos and sin, or null: the cache slot
    int64_t n_pos;
    GqaBatch b;                                                 // cu_q, lens, table, pages
    int Hq, Hk, D, rot, interleaved, has_q;
    int head_lanes, tokens_per_block;
};

constexpr int kAppendThreads = 256;

struct AppendToken {
    int64_t cache;   // element offset of the token's row of head 0 in the cache, -1: none
    int pos;         // row of the angles, -1: the token is not touched
    int pad;
};

template <bool F16>
__global__ void __launch_bounds__(kAppendThreads) rope_append_kernel(const AppendParams p) {
    __shared__ AppendToken tok[kAppendThreads];
    wait_for_earlier_kernels();
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * p.tokens_per_block;
    if (threadIdx.x < p.tokens_per_block) {
        AppendToken a;
        a.cache = -1;
        a.pos = -1;
        a.pad = 0;
        const int64_t t = t0 + threadIdx.x;
        const int first = load_int(p.b.cu_q), last = load_int(p.b.cu_q + p.b.B);
        if (t < p.b.Tq && t >= first && t < last) {
            int lo = 0, hi = p.b.B;   // cu_q[lo] <= t < cu_q[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (load_int(p.b.cu_q + mid) <= t) lo = mid;
                else hi = mid;
            }
            const SeqInfo s = seq_info(p.b, lo);
            const int64_t slot = static_cast<int64_t>(s.m) - s.n + (t - s.q0);
            int pg = -1;
            if (s.n > 0 && t < s.q0 + s.n && slot >= 0)
                pg = load_int(p.b.table + static_cast<int64_t>(lo) * p.b.table_w + (slot >> p.b.page_shift));
            const int64_t pos = p.positions ? load_int(p.positions + t) : slot;
            if (pg < 0 || pg >= p.b.pages || (p.cos && (pos < 0 || pos >= p.n_pos))) {
                atomicExch(p.b.status, kStatusCheck);   // nothing of this token is written
            } else {
                a.cache = static_cast<int64_t>(pg) * p.c_sp + (slot & ((int64_t(1) << p.b.page_shift) - 1)) * p.c_st;
                a.pos = p.cos ? static_cast<int>(pos) : 0;
            }
        }
        tok[threadIdx.x] = a;
    }
    if (blockIdx.x == 0)   // sequences that no token leads to are checked as well
        for (int b = threadIdx.x; b < p.b.B; b += kAppendThreads) seq_info(p.b, b);
    __syncthreads();

    const int CH = p.D / 16;                       // threads per head
    const int chunk = threadIdx.x % CH;
    const int hl = (threadIdx.x / CH) % p.head_lanes;
    const int tl = threadIdx.x / (CH * p.head_lanes);
    if (tl >= p.tokens_per_block) return;
    const AppendToken a = tok[tl];
    if (a.pos < 0) return;
    const int64_t t = t0 + tl;
    const bool turn = p.cos != nullptr && chunk < p.rot / 16;
    // the thread's two groups of 8 elements: the two members of 8 pairs, or 16 in a row
    const int e0 = turn && !p.interleaved ? 8 * chunk : 16 * chunk;
    const int e1 = turn && !p.interleaved ? p.rot / 2 + 8 * chunk : 16 * chunk + 8;
    float c[8], s[8];
    if (turn) {
        const float4 *pc = reinterpret_cast<const float4 *>(p.cos + static_cast<int64_t>(a.pos) * (p.rot / 2) + 8 * chunk);
        const float4 *ps = reinterpret_cast<const float4 *>(p.sin + static_cast<int64_t>(a.pos) * (p.rot / 2) + 8 * chunk);
        const float4 c0 = pc[0], c1 = pc[1], s0 = ps[0], s1 = ps[1];
        c[0] = c0.x, c[1] = c0.y, c[2] = c0.z, c[3] = c0.w, c[4] = c1.x, c[5] = c1.y, c[6] = c1.z, c[7] = c1.w;
        s[0] = s0.x, s[1] = s0.y, s[2] = s0.z, s[3] = s0.w, s[4] = s1.x, s[5] = s1.y, s[6] = s1.z, s[7] = s1.w;
    }
    const int nq = p.has_q ? p.Hq : 0;
    const int heads = nq + 2 * p.Hk;
#pragma unroll 4
    for (int h = hl; h < heads; h += p.head_lanes) {
        const bool is_q = h < nq, is_v = h >= nq + p.Hk;
        const int hh = is_q ? h : is_v ? h - nq - p.Hk : h - nq;
        const uint16_t *src = is_q ? p.q + t * p.q_st + hh * p.q_sh
                              : is_v ? p.v + t * p.v_st + hh * p.v_sh : p.k + t * p.k_st + hh * p.k_sh;
        uint16_t *dst = is_q ? p.q_out + t * p.qo_st + hh * p.qo_sh : (is_v ? p.vc : p.kc) + a.cache + hh * p.c_sh;
        uint4 x = *reinterpret_cast<const uint4 *>(src + e0), y = *reinterpret_cast<const uint4 *>(src + e1);
        if (turn && !is_v) {
            uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
            if (p.interleaved) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float u, w;
                    unpack16<F16>(xs[j], u, w);
                    xs[j] = pack16<F16>(u * c[j] - w * s[j], u * s[j] + w * c[j]);
                    unpack16<F16>(ys[j], u, w);
                    ys[j] = pack16<F16>(u * c[4 + j] - w * s[4 + j], u * s[4 + j] + w * c[4 + j]);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float u0, u1, w0, w1;
                    unpack16<F16>(xs[j], u0, u1);
                    unpack16<F16>(ys[j], w0, w1);
                    xs[j] = pack16<F16>(u0 * c[2 * j] - w0 * s[2 * j], u1 * c[2 * j + 1] - w1 * s[2 * j + 1]);
                    ys[j] = pack16<F16>(u0 * s[2 * j] + w0 * c[2 * j], u1 * s[2 * j + 1] + w1 * c[2 * j + 1]);
                }
            }
            x = make_uint4(xs[0], xs[1], xs[2], xs[3]);
            y = make_uint4(ys[0], ys[1], ys[2], ys[3]);
        }
        *reinterpret_cast<uint4 *>(dst + e0) = x;
        *reinterpret_cast<uint4 *>(dst + e1) = y;
    }
}

}  // namespace lite
