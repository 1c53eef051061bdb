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

__device__ __forceinline__ int seq_tiles(const GqaBatch &p, int m) {   // a sequence without keys counts as one
    return m > 0 ? static_cast<int>((static_cast<int64_t>(m) + p.tile - 1) / p.tile) : 1;
}

// Key tiles of a segment (the whole block of NT threads; the same in every block).
template <int NT>
__device__ __forceinline__ int segment_tiles(const GqaBatch &p, ScanScratch &sc) {
    if (p.split_target <= 0) return 1 << 30;   // no item has that many tiles: one segment each
    constexpr int NW = NT / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int64_t sum = 0;
    for (int b = p.B == 1 ? 0 : threadIdx.x; b < p.B; b += NT) {
        const SeqInfo s = seq_info(p, b);
        sum += static_cast<int64_t>(p.Hk) * seq_blocks(p, s.n) * seq_tiles(p, s.m);
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
    return static_cast<int>(l < p.min_tiles ? p.min_tiles : l > (1 << 30) ? (1 << 30) : l);
}

// Work item y of sequence b, whose first segment has workspace slot `slot0`.  The order is
// by row block, those with most keys first, then by key head: blocks that run at the same
// time have about the same work, and the last ones are short.
template <bool SEGMENTS>
__device__ __forceinline__ void decode_item(const GqaBatch &p, int b, const SeqInfo &s, int L, int y, int slot0, WorkItem &w) {
    const int nb = seq_blocks(p, s.n);
    w.segs = (seq_tiles(p, s.m) + L - 1) / L;
    const int per = SEGMENTS ? w.segs : 1;
    w.s = s;
    w.b = b;
    w.seg = y % per;
    const int item = y / per;
    w.h = item % p.Hk;
    w.i = nb - 1 - item / p.Hk;
    w.L = L;
    w.slot = slot0 + item * w.segs + w.seg;
}

// The x-th work item of the batch (SEGMENTS: the x-th segment), found by the whole block of
// NT threads; false when there are fewer.
template <int NT, bool SEGMENTS>
__device__ __forceinline__ bool find_work(const GqaBatch &p, int x, ScanScratch &sc, WorkItem &w) {
    constexpr int NW = NT / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int L = segment_tiles<NT>(p, sc);
    if (p.B == 1) {
        const SeqInfo s = seq_info(p, 0);
        const int items = p.Hk * seq_blocks(p, s.n);
        if (x >= items * (SEGMENTS ? (seq_tiles(p, s.m) + L - 1) / L : 1)) return false;
        decode_item<SEGMENTS>(p, 0, s, L, x, 0, w);
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
            const int items = p.Hk * seq_blocks(p, s.n), segs = (seq_tiles(p, s.m) + L - 1) / L;
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
            decode_item<SEGMENTS>(p, b, s, L, x - lo, sbefore + si - spl, w);
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

// ---------------------------------------------------------------- division among persistent blocks
// Items of the tile kernel have very different lengths.  A batch of many items is dealt out
// whole, in order of length, back and forth over the blocks.  With few items the batch is
// laid out on a line instead, an item taking as many units as its last row sees keys, and
// kItemCost for its start and end; each block takes an equal stretch of the line, cut at the
// next tile boundary.  A block then has at most two partial items, at the ends of its stretch,
// so the workspace holds two slots per block, and at most one item per block boundary is
// joined afterwards.
constexpr int kItemCost = 256;      // measured: the turn from one item to the next costs about two tiles
constexpr int kMinStretch = 512;    // more than a tile, so that no stretch inside an item is without one
constexpr int kJoinCost = 1280;     // keys whose time partial outputs and their join cost

// Keys that the last row of block i sees.
__device__ __forceinline__ int block_keys(const GqaBatch &p, const SeqInfo &s, int i) {
    const int last = min((i + 1) * p.unit_tokens, s.n) - 1;
    return visible_keys(p, s, last);
}

// Units of the first k block groups (last rows first) of one head of a sequence.
__device__ __forceinline__ int64_t group_units(const GqaBatch &p, const SeqInfo &s, int nb, int k) {
    if (k <= 0) return 0;
    if (!p.causal) return static_cast<int64_t>(k) * (static_cast<int64_t>(s.m) + kItemCost);
    // block nb - 1 sees m keys; block x - 1 < nb - 1 sees m - n + x * unit_tokens, 0 at least
    const int64_t a = static_cast<int64_t>(s.m) - s.n, tb = p.unit_tokens;
    int64_t lo = nb - k + 1;
    const int64_t first = a > 0 ? 1 : (-a) / tb + 1;
    lo = lo < first ? first : lo;
    const int64_t hi = nb - 1;
    int64_t sum = static_cast<int64_t>(k) * kItemCost + s.m;
    if (lo <= hi) sum += (hi - lo + 1) * a + tb * ((lo + hi) * (hi - lo + 1) / 2);
    return sum;
}
// Units of a block's stretch, 0: items are dealt out whole.  The same in every block (of NT threads).
template <int NT>
__device__ __forceinline__ int64_t stretch_units(const GqaBatch &p, int blocks, ScanScratch &sc) {
    if (p.split_target <= 0) return 0;
    constexpr int NW = NT / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int64_t units = 0;
    int items = 0, longest = 0, shortest = 0;
    for (int b = p.B == 1 ? 0 : threadIdx.x; b < p.B; b += NT) {
        const SeqInfo s = seq_info(p, b);
        const int nb = seq_blocks(p, s.n);
        units += p.Hk * group_units(p, s, nb, nb);
        items += p.Hk * nb;
        if (nb > 0) longest = max(longest, s.m), shortest = block_keys(p, s, 0);
    }
    if (p.B > 1) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            units += __shfl_xor_sync(0xFFFFFFFFu, units, o);
            items += __shfl_xor_sync(0xFFFFFFFFu, items, o);
            longest = max(longest, __shfl_xor_sync(0xFFFFFFFFu, longest, o));
        }
        if (lane == 0) sc.sum[warp] = units, sc.cnt[warp] = items, sc.spl[warp] = longest;
        __syncthreads();
        units = 0, items = 0, longest = 0;
#pragma unroll
        for (int k = 0; k < NW; ++k) units += sc.sum[k], items += sc.cnt[k], longest = max(longest, sc.spl[k]);
        __syncthreads();
    }
    const int64_t even = max((units + blocks - 1) / blocks, static_cast<int64_t>(kMinStretch));
    // Dealt out whole, one sequence's items fall off in length to the shortest, and the blocks end
    // within one of those of each other; those of several sequences within about half the longest.
    const int64_t rounds = (items + blocks - 1) / blocks, most = static_cast<int64_t>(longest) + kItemCost;
    const int64_t whole = max(most, min(rounds * most, even + (p.B == 1 ? static_cast<int64_t>(shortest) : most / 2)));
    return even + kJoinCost < whole ? even : 0;
}

// An item's place: its sequence, block, head, and stretch [from, to) of the line.
struct LineItem {
    SeqInfo s;
    int b, i, h, keys;     // keys that its last row sees
    int64_t from, to;
};
__device__ __forceinline__ void line_item(const GqaBatch &p, int b, const SeqInfo &s, int64_t base, int64_t x, LineItem &it) {
    const int nb = seq_blocks(p, s.n);
    const int64_t at = x - base;
    int lo = 0, hi = nb - 1;            // the last group that starts at or before x
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.Hk * group_units(p, s, nb, mid) <= at) lo = mid;
        else hi = mid - 1;
    }
    it.s = s;
    it.b = b;
    it.i = nb - 1 - lo;
    it.keys = block_keys(p, s, it.i);
    const int64_t start = p.Hk * group_units(p, s, nb, lo), len = static_cast<int64_t>(it.keys) + kItemCost;
    it.h = static_cast<int>((at - start) / len);
    it.from = base + start + it.h * len;
    it.to = it.from + len;
}
// The tiles [t0, t1) of an item that fall to stretch q; false when there are none.  `whole`: all of them do.
__device__ __forceinline__ bool line_tiles(const GqaBatch &p, const LineItem &it, int64_t stretch, int64_t q, int &t0, int &t1, bool &whole) {
    const int nt = static_cast<int>((static_cast<int64_t>(it.keys) + p.tile - 1) / p.tile);
    auto cut = [&](int64_t x) {          // a boundary at x: the nearest tile
        const int64_t t = (x - it.from + p.tile / 2) / p.tile;
        return x <= it.from ? 0 : x >= it.to || t > nt ? nt : static_cast<int>(t);
    };
    t0 = cut(q * stretch);
    t1 = cut((q + 1) * stretch);
    whole = t0 == 0 && t1 == nt && (nt > 0 || it.from / stretch == q);
    return t1 > t0 || whole;
}
__device__ __forceinline__ int line_slot(const LineItem &it, int64_t stretch, int64_t q) {
    return static_cast<int>(2 * q) + (q * stretch > it.from ? 0 : 1);
}

// The batch walked by one warp, forwards: items by number, or by place on the line.  The lanes
// hold 32 sequences at a time.
struct WorkCursor {
    int b0;
    int64_t base, total;   // items or units before the 32 sequences, and in them
    SeqInfo s;
    int64_t lo, cnt;       // this lane's sequence: first item or unit, how many
    __device__ __forceinline__ void load(const GqaBatch &p, bool line, int lane) {
        const int b = b0 + lane;
        s = SeqInfo{0, 0, 0, 0};
        cnt = 0;
        if (b < p.B) {
            s = seq_info(p, b);
            const int nb = seq_blocks(p, s.n);
            cnt = line ? p.Hk * group_units(p, s, nb, nb) : static_cast<int64_t>(p.Hk) * nb;
        }
        int64_t ci = cnt;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t a = __shfl_up_sync(0xFFFFFFFFu, ci, o);
            if (lane >= o) ci += a;
        }
        lo = base + ci - cnt;
        total = __shfl_sync(0xFFFFFFFFu, ci, 31);
    }
    __device__ __forceinline__ void start(const GqaBatch &p, bool line, int lane) {
        b0 = 0;
        base = 0;
        load(p, line, lane);
    }
    // the sequence that holds item or unit x (not below an earlier x); false: behind the last
    __device__ __forceinline__ bool find(const GqaBatch &p, bool line, int lane, int64_t x, int &b, SeqInfo &q, int64_t &first) {
        while (x >= base + total) {
            if (b0 + 32 >= p.B) return false;
            b0 += 32;
            base += total;
            load(p, line, lane);
        }
        const int src = __ffs(__ballot_sync(0xFFFFFFFFu, x >= lo && x < lo + cnt)) - 1;
        q.q0 = __shfl_sync(0xFFFFFFFFu, s.q0, src);
        q.n = __shfl_sync(0xFFFFFFFFu, s.n, src);
        q.m = __shfl_sync(0xFFFFFFFFu, s.m, src);
        q.k0 = __shfl_sync(0xFFFFFFFFu, s.k0, src);
        first = __shfl_sync(0xFFFFFFFFu, lo, src);
        b = b0 + src;
        return true;
    }
};

// ---------------------------------------------------------------- bounded waits
// What a block's waits share: a wait that runs out makes all the others end, and the plan's
// status says so.
struct WaitScope {
    volatile uint32_t *abort_flag;
    int32_t *status;
};
// A converged warp waits for the phase of `bar` with this parity; false once the block has
// given up (after kWaitLimitNs).  All lanes poll and vote, so that the warp never splits; the
// clock is read only after some tries (reading it takes longer than most waits).
__device__ __forceinline__ bool wait_phase_warp(uint32_t bar, uint32_t parity, const WaitScope &w) {
    uint64_t t0 = 0;
    for (uint32_t it = 1;; ++it) {
        if (__all_sync(0xFFFFFFFFu, ptx::mbar_try_wait(bar, parity))) return true;
        if ((it & 63u) == 0u) {
            if (__any_sync(0xFFFFFFFFu, *w.abort_flag != 0u)) return false;
            const uint64_t t = ptx::globaltimer_ns();
            if (t0 == 0) t0 = t;
            if (__any_sync(0xFFFFFFFFu, t - t0 > kWaitLimitNs)) {
                *w.abort_flag = 1u;
                atomicExch(w.status, kStatusTimeout);
                return false;
            }
        }
    }
}
// The same while draining at the end, whether or not the block has given up.
__device__ __forceinline__ void drain_phase(uint32_t bar, uint32_t parity) {
    uint64_t t0 = 0;
    for (uint32_t it = 1;; ++it) {
        if (ptx::mbar_try_wait(bar, parity)) return;
        if ((it & 63u) == 0u) {
            const uint64_t t = ptx::globaltimer_ns();
            if (t0 == 0) t0 = t;
            if (t - t0 > kWaitLimitNs) return;
        }
    }
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
// 0 * v + acc on both halves: NaN where v is not finite.
template <bool F16>
__device__ __forceinline__ uint32_t fma_zero16(uint32_t v, uint32_t acc) {
    uint32_t d;
    if constexpr (F16) asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(v), "r"(0u), "r"(acc));
    else asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(v), "r"(0u), "r"(acc));
    return d;
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
