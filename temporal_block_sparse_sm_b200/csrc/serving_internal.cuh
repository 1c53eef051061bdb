// serving_internal.cuh -- what the serving attention kernels share: the batch they work
// on, the division of a ragged batch into work items, and small numeric helpers.
//
// A batch is B sequences.  Sequence b has n query tokens (rows [cu_q[b], cu_q[b+1]) of q
// and o) and m keys (in pages of the cache, or rows [cu_k[b], cu_k[b+1]) of k and v).  The
// queries are the last n of the sequence's positions: query token t sees keys
// [0, m - n + t] (causal) or all m.
//
// Lengths live on the device, so that a captured graph can be replayed on other lengths;
// the host knows only upper bounds.  Every block finds its own work item by a scan over
// the sequences (a few loads per thread), and blocks behind the last item return at once.
//
// Splitting along the keys.  With few rows and long caches there are fewer (sequence, key
// head, row block) items than SMs.  Each item is then cut into segments of L key tiles,
// L = max(min_tiles, ceil(W / target)), W = all tiles of all items; the number of segments
// is at most target + items however ragged the lengths are.  A segment leaves its
// unnormalised output, running maximum and sum in the workspace, and a second kernel joins
// them.  Items of one segment write their output themselves and use no workspace; split
// items have more than L tiles, so there are at most 2 * target segments of them, which
// bounds the workspace whatever the batch.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "liteattn_internal.cuh"
#include "sm100_ptx.cuh"

namespace lite {

enum KvMode { kKvPacked = 0, kKvPagesBhnd = 1, kKvPagesBnhd = 2 };

struct GqaBatch {
    const int32_t *cu_q;   // [B + 1]
    const int32_t *cu_k;   // [B + 1] (kKvPacked)
    const int32_t *lens;   // [B] keys of each sequence (cache)
    const int32_t *table;  // [B][table_w] pages (cache)
    int64_t Tq, Tk;        // rows of q / of k and v (kKvPacked)
    int64_t pages;         // pages of the cache
    int64_t max_keys;      // table_w * page (cache)
    int32_t *status;
    int B, G, Hk, causal, mode;
    int table_w, page_shift;
    int unit_rows;         // query rows (token, head of the group) of a work item, or 0: unit_tokens tokens
    int unit_tokens;
    int tile;              // keys of a tile
    int split_target;      // 0: no splitting
    int min_tiles;
};

struct SeqInfo {
    int q0, n, m;
    int64_t k0;
};

// Sequence b, with what it says about its own rows checked against the tensors; a sequence
// that names rows or keys outside them has no work, and the plan's status says so.
__device__ __forceinline__ SeqInfo seq_info(const GqaBatch &p, int b) {
    SeqInfo s;
    s.q0 = __ldg(p.cu_q + b);
    const int q1 = __ldg(p.cu_q + b + 1);
    s.n = q1 - s.q0;
    s.k0 = 0;
    bool bad = s.q0 < 0 || q1 < s.q0 || q1 > p.Tq;
    if (p.mode == kKvPacked) {
        const int k0 = __ldg(p.cu_k + b), k1 = __ldg(p.cu_k + b + 1);
        s.k0 = k0;
        s.m = k1 - k0;
        bad = bad || k0 < 0 || k1 < k0 || k1 > p.Tk;
    } else {
        s.m = __ldg(p.lens + b);
        bad = bad || s.m < 0 || s.m > p.max_keys;
    }
    if (bad) {
        atomicExch(p.status, kStatusCheck);
        s.n = 0;
        s.m = 0;
    }
    return s;
}

__device__ __forceinline__ int seq_blocks(const GqaBatch &p, int n) {
    if (p.unit_rows) return static_cast<int>((static_cast<int64_t>(n) * p.G + p.unit_rows - 1) / p.unit_rows);
    return (n + p.unit_tokens - 1) / p.unit_tokens;
}

// One block's work: row block i of key head h of sequence b, key tiles [seg * L, (seg + 1) * L).
struct WorkItem {
    SeqInfo s;
    int b, h, i;
    int seg, segs, L;      // segs > 1: a split item
    int slot;              // its workspace slot (split items), or the slot of its first segment
    int found;
};

struct ScanScratch {
    int64_t sum[32];
    int cnt[32], spl[32];
    WorkItem w;
};

// The x-th work item of the batch (SEGMENTS: the x-th segment), found by the whole block of
// NT threads; false when there are fewer.  The order is head by head within a sequence, the
// row blocks with most keys first, so that blocks running at the same time share keys and
// the last ones are short.
template <int NT, bool SEGMENTS>
__device__ __forceinline__ bool find_work(const GqaBatch &p, int x, ScanScratch &sc, WorkItem &w) {
    constexpr int NW = NT / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int L = 1 << 30;   // no item has that many tiles: one segment each
    auto tiles_of = [&](int m) { return m > 0 ? static_cast<int>((static_cast<int64_t>(m) + p.tile - 1) / p.tile) : 1; };
    if (p.split_target > 0) {
        int64_t sum = 0;
        for (int b = p.B == 1 ? 0 : threadIdx.x; b < p.B; b += NT) {
            const SeqInfo s = seq_info(p, b);
            sum += static_cast<int64_t>(p.Hk) * seq_blocks(p, s.n) * tiles_of(s.m);
        }
        if (p.B > 1) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
            if (lane == 0) sc.sum[warp] = sum;
            __syncthreads();
            sum = 0;
#pragma unroll
            for (int k = 0; k < NW; ++k) sum += sc.sum[k];
        }
        const int64_t l = (sum + p.split_target - 1) / p.split_target;
        L = static_cast<int>(l < p.min_tiles ? p.min_tiles : l > (1 << 30) ? (1 << 30) : l);
    }
    auto fill = [&](int b, const SeqInfo &s, int y, int slot0) {
        const int nb = seq_blocks(p, s.n);
        w.segs = (tiles_of(s.m) + L - 1) / L;
        const int per = SEGMENTS ? w.segs : 1;
        w.s = s;
        w.b = b;
        w.seg = y % per;
        const int item = y / per;
        w.h = item / nb;
        w.i = nb - 1 - item % nb;
        w.L = L;
        w.slot = slot0 + item * w.segs + w.seg;
    };
    if (p.B == 1) {
        const SeqInfo s = seq_info(p, 0);
        const int items = p.Hk * seq_blocks(p, s.n);
        const int total = items * (SEGMENTS ? (tiles_of(s.m) + L - 1) / L : 1);
        if (x >= total) return false;
        fill(0, s, x, 0);
        return true;
    }
    if (threadIdx.x == 0) sc.w.found = 0;
    int base = 0, slot_base = 0;
    for (int b0 = 0; b0 < p.B; b0 += NT) {
        const int b = b0 + threadIdx.x;
        SeqInfo s = {0, 0, 0, 0};
        int cnt = 0, spl = 0;
        if (b < p.B) {
            s = seq_info(p, b);
            const int items = p.Hk * seq_blocks(p, s.n), segs = (tiles_of(s.m) + L - 1) / L;
            cnt = SEGMENTS ? items * segs : items;
            spl = segs > 1 ? items * segs : 0;
        }
        int ci = cnt, si = spl;   // inclusive scans over the warp
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int a = __shfl_up_sync(0xFFFFFFFFu, ci, o), c = __shfl_up_sync(0xFFFFFFFFu, si, o);
            if (lane >= o) ci += a, si += c;
        }
        if (lane == 31) sc.cnt[warp] = ci, sc.spl[warp] = si;
        __syncthreads();
        int before = base, sbefore = slot_base, total = 0, stotal = 0;
#pragma unroll
        for (int k = 0; k < NW; ++k) {
            if (k < warp) before += sc.cnt[k], sbefore += sc.spl[k];
            total += sc.cnt[k], stotal += sc.spl[k];
        }
        const int lo = before + ci - cnt;
        if (cnt > 0 && x >= lo && x < lo + cnt) {
            fill(b, s, x - lo, sbefore + si - spl);
            sc.w = w;
            sc.w.found = 1;
        }
        __syncthreads();
        if (x < base + total) break;
        base += total;
        slot_base += stotal;
    }
    w = sc.w;
    return w.found != 0;
}

// Keys that query token t of a sequence sees (0: none).
__device__ __forceinline__ int visible_keys(const GqaBatch &p, const SeqInfo &s, int t) {
    if (!p.causal) return s.m;
    const int v = s.m - s.n + t + 1;
    return v < 0 ? 0 : v;
}

// ---------------------------------------------------------------- 16-bit types
// Weights are 2^(x + bias): fp16 ones are scaled by 2^7, so that they lose no precision to
// subnormals until they are 2^-21 of the row's largest (which stays below 2^15).  The row's
// sum carries the same factor.
template <bool F16>
__device__ __forceinline__ constexpr float weight_bias() { return F16 ? 7.0f : 0.0f; }

template <bool F16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
    uint32_t r;
    if constexpr (F16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
template <bool F16>
__device__ __forceinline__ void unpack16(uint32_t v, float &lo, float &hi) {
    if constexpr (F16) {
        const __half2 h = *reinterpret_cast<const __half2 *>(&v);
        lo = __low2float(h);
        hi = __high2float(h);
    } else {
        lo = __uint_as_float(v << 16);
        hi = __uint_as_float(v & 0xFFFF0000u);
    }
}
// Nonzero in bit 15 (low half) / bit 31 (high half) where a half of v is an infinity or a
// NaN: its exponent bits are all ones, and one more unit in their last place carries out.
template <bool F16>
__device__ __forceinline__ uint32_t nonfinite16(uint32_t v) {
    return F16 ? ((v & 0x7C007C00u) + 0x04000400u) & 0x80008000u : ((v & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
}
// lo += low half of v, hi += high half, each exactly as an f32 (mixed-precision add).
template <bool F16>
__device__ __forceinline__ void add16x2(float &lo, float &hi, uint32_t v) {
    if constexpr (F16)
        asm("{\n\t.reg .b16 l16, h16;\n\t"
            "mov.b32 {l16, h16}, %2;\n\t"
            "add.rn.f32.f16 %0, l16, %0;\n\t"
            "add.rn.f32.f16 %1, h16, %1;\n\t}"
            : "+f"(lo), "+f"(hi)
            : "r"(v));
    else
        ptx::add_bf16x2(lo, hi, v);
}

}  // namespace lite
