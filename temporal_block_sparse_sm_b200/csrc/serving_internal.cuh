// serving_internal.cuh -- what the serving attention kernels share: the batch they work
// on, the division of a ragged batch into work items, and small numeric helpers.
//
// A batch is B sequences.  Sequence b has n query tokens (rows [cu_q[b], cu_q[b+1]) of q
// and o) and m keys (in pages of the cache, or rows [cu_k[b], cu_k[b+1]) of k and v).  The
// queries are the last n of the sequence's positions: query token t sees keys
// [0, m - n + t] (causal) or all m.
//
// Lengths live on the device, so that a captured graph can be replayed on other lengths; the
// host knows only upper bounds.  The kernels' blocks are persistent, and one warp of each walks
// the batch for the block's items (BlockWalk).
//
// Division among the blocks.  A batch of many items (block of query rows, key head) is dealt
// out whole, in order of length within a sequence: of one sequence back and forth over the blocks,
// of several by a counter, to whichever block asks next (an item's result does not depend on its
// block; back and forth, counting keys, the longest block of 16 prompts of 1 to 2,048 tokens would get a
// quarter more than the mean).  With few
// items the batch is laid out on a line instead, an item taking as many units as its last row
// sees keys (half_weight eighths of that where it fills only the first of the tile kernel's two
// slots), and item_cost for its start and end; each block takes an equal stretch of the line,
// cut at the nearest tile.  A block then has at most two partial items, at the ends of its
// stretch: a partial item's unnormalised output, running maximum and sum go to one of the block's
// two workspace slots, which bounds the workspace whatever the batch, and a second kernel joins
// the at most one item per block that reaches beyond its stretch, from a record that the block
// leaves about it.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "liteattn_internal.cuh"
#include "sm100_ptx.cuh"

namespace lite {

constexpr int kFewRows = 16;   // query rows of an item of the rows kernel

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
    int unit_tokens;       // query tokens of a work item; 0: kFewRows rows (token, head of the group)
    int tile_shift;        // log2 of the keys of a tile
    int may_split;         // items may be cut
    int *next_item;        // zero before the kernel: items handed out, but for each block's first; null: back and forth
    // in keys: what an item costs beside its keys, what partial outputs and their join cost, and
    // the shortest stretch (more than a tile, so that no stretch inside an item is without one)
    int item_cost, join_cost, min_stretch;
    int half_weight;       // eighths of a key that a key costs an item of no more than half unit_tokens
};

// A length, offset, page or position.  The kernel in front may still write it when this one starts, so it is
// loaded coherently (the non-coherent path is for data that does not change during the kernel's life) and in
// program order with the wait for that kernel; and once, so that what was checked is what is used.
__device__ __forceinline__ int load_int(const int32_t *p) {
    int x;
    asm volatile("ld.global.b32 %0, [%1];" : "=r"(x) : "l"(p));
    return x;
}

struct SeqInfo {
    int q0, n, m;
    int64_t k0;
};

// Sequence b, with what it says about its own rows checked against the tensors; a sequence
// that names rows or keys outside them has no work, and the plan's status says so.
__device__ __forceinline__ SeqInfo seq_info(const GqaBatch &p, int b) {
    SeqInfo s;
    s.q0 = load_int(p.cu_q + b);
    const int q1 = load_int(p.cu_q + b + 1);
    s.n = q1 - s.q0;
    s.k0 = 0;
    bool bad = s.q0 < 0 || q1 < s.q0 || q1 > p.Tq;
    if (p.mode == kKvPacked) {
        const int k0 = load_int(p.cu_k + b), k1 = load_int(p.cu_k + b + 1);
        s.k0 = k0;
        s.m = k1 - k0;
        bad = bad || k0 < 0 || k1 < k0 || k1 > p.Tk;
    } else {
        s.m = load_int(p.lens + b);
        bad = bad || s.m < 0 || s.m > p.max_keys;
    }
    if (bad) {
        atomicExch(p.status, kStatusCheck);
        s.n = 0;
        s.m = 0;
    }
    return s;
}

// a / b for a, b >= 0; in 32 bits where they fit (a 64-bit division takes about 100 instructions).
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}

__device__ __forceinline__ int seq_blocks(const GqaBatch &p, int n) {
    return p.unit_tokens ? (n + p.unit_tokens - 1) / p.unit_tokens
                         : static_cast<int>((static_cast<int64_t>(n) * p.G + kFewRows - 1) / kFewRows);
}

// Keys that query token t of a sequence sees (0: none).
__device__ __forceinline__ int visible_keys(const GqaBatch &p, const SeqInfo &s, int t) {
    if (!p.causal) return s.m;
    const int v = s.m - s.n + t + 1;
    return v < 0 ? 0 : v;
}

// Keys that the last row of block i sees.
__device__ __forceinline__ int block_keys(const GqaBatch &p, const SeqInfo &s, int i) {
    int last;
    if (p.unit_tokens) {
        last = min((i + 1) * p.unit_tokens, s.n) - 1;
    } else {
        const int64_t end = static_cast<int64_t>(i + 1) * kFewRows;
        last = end >= static_cast<int64_t>(s.n) * p.G ? s.n - 1 : static_cast<int>(quotient(end - 1, p.G));
    }
    return visible_keys(p, s, last);
}
// Eighths of a unit that a key of block i takes; only a sequence's last block can be half empty.
__device__ __forceinline__ int block_weight(const GqaBatch &p, const SeqInfo &s, int i) {
    return p.unit_tokens && 2 * (s.n - i * p.unit_tokens) <= p.unit_tokens ? p.half_weight : 8;
}
__device__ __forceinline__ int64_t units_of(int64_t keys, int weight) { return (keys * weight + 7) >> 3; }
// Units of block i, and of the first k blocks (last rows first) of one head of a sequence.  Blocks
// of a few rows count all m keys.
__device__ __forceinline__ int64_t block_units(const GqaBatch &p, const SeqInfo &s, int i, int weight) {
    return static_cast<int64_t>(p.item_cost) + (p.unit_tokens ? units_of(block_keys(p, s, i), weight) : s.m);
}
__device__ __forceinline__ int64_t group_units(const GqaBatch &p, const SeqInfo &s, int nb, int k) {
    if (k <= 0) return 0;
    if (!p.unit_tokens) return static_cast<int64_t>(k) * (static_cast<int64_t>(s.m) + p.item_cost);
    const int64_t last = units_of(s.m, block_weight(p, s, nb - 1));
    if (!p.causal) return static_cast<int64_t>(k) * p.item_cost + static_cast<int64_t>(k - 1) * s.m + last;
    // block nb - 1 sees m keys; block x - 1 < nb - 1 sees m - n + x * unit_tokens, 0 at least
    const int64_t a = static_cast<int64_t>(s.m) - s.n, tb = p.unit_tokens;
    int64_t lo = nb - k + 1;
    const int64_t first = a > 0 ? 1 : quotient(-a, tb) + 1;
    lo = lo < first ? first : lo;
    const int64_t hi = nb - 1;
    int64_t sum = static_cast<int64_t>(k) * p.item_cost + last;
    if (lo <= hi) sum += (hi - lo + 1) * a + tb * ((lo + hi) * (hi - lo + 1) / 2);
    return sum;
}

struct ScanScratch {
    int64_t sum[32];
    int items[32], longest[32];
};

// Units that the longest item of a sequence takes, but for item_cost.
__device__ __forceinline__ int longest_of(const GqaBatch &p, const SeqInfo &s, int nb) {
    return nb == 0 ? 0 : nb > 1 ? s.m : static_cast<int>(units_of(s.m, block_weight(p, s, 0)));
}
// Units of a block's stretch, 0: items are dealt out whole.  From the batch's units, its items, and
// the units of its longest and (of a single sequence) shortest item.
__device__ __forceinline__ int64_t choose_stretch(const GqaBatch &p, int blocks, int64_t units, int items, int longest, int shortest) {
    const int64_t even = max(quotient(units + blocks - 1, blocks), static_cast<int64_t>(p.min_stretch));
    // Dealt out whole, one sequence's items fall off in length to the shortest, and the blocks end
    // within one of those of each other; those of several sequences within about half the longest.
    const int64_t rounds = (items + blocks - 1) / blocks, most = static_cast<int64_t>(longest) + p.item_cost;
    const int64_t whole = max(most, min(rounds * most, even + (p.B == 1 ? static_cast<int64_t>(shortest) : most / 2)));
    return even + p.join_cost < whole ? even : 0;
}
// The same in every block, of NT threads; batches of more than 32 sequences (a warp takes fewer by
// itself, BlockWalk).
template <int NT>
__device__ __forceinline__ int64_t stretch_units(const GqaBatch &p, int blocks, ScanScratch &sc) {
    if (!p.may_split || p.B <= 32) return 0;
    constexpr int NW = NT / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int64_t units = 0;
    int items = 0, longest = 0;
    for (int b = threadIdx.x; b < p.B; b += NT) {
        const SeqInfo s = seq_info(p, b);
        const int nb = seq_blocks(p, s.n);
        units += p.Hk * group_units(p, s, nb, nb);
        items += p.Hk * nb;
        longest = max(longest, longest_of(p, s, nb));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        units += __shfl_xor_sync(0xFFFFFFFFu, units, o);
        items += __shfl_xor_sync(0xFFFFFFFFu, items, o);
        longest = max(longest, __shfl_xor_sync(0xFFFFFFFFu, longest, o));
    }
    if (lane == 0) sc.sum[warp] = units, sc.items[warp] = items, sc.longest[warp] = longest;
    __syncthreads();
    units = 0, items = 0, longest = 0;
#pragma unroll
    for (int k = 0; k < NW; ++k) units += sc.sum[k], items += sc.items[k], longest = max(longest, sc.longest[k]);
    return choose_stretch(p, blocks, units, items, longest, 0);
}

// An item: its sequence, block of rows and head, the keys that its last row sees, and its stretch
// [from, to) of the line.
struct LineItem {
    SeqInfo s;
    int b, i, h, keys, weight;
    int64_t from, to;
};
__device__ __forceinline__ void line_item(const GqaBatch &p, int b, const SeqInfo &s, int nb, int64_t base, int64_t x, LineItem &it) {
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
    it.weight = block_weight(p, s, it.i);
    const int64_t start = p.Hk * group_units(p, s, nb, lo), len = block_units(p, s, it.i, it.weight);
    it.h = static_cast<int>(quotient(at - start, len));
    it.from = base + start + it.h * len;
    it.to = it.from + len;
}
__device__ __forceinline__ int tiles_of(const GqaBatch &p, int keys) {
    return static_cast<int>((static_cast<int64_t>(keys) + (1 << p.tile_shift) - 1) >> p.tile_shift);
}
// The tiles [t0, t1) of an item that fall to stretch q; false when there are none.  `whole`: all of them do.
__device__ __forceinline__ bool line_tiles(const GqaBatch &p, const LineItem &it, int64_t stretch, int64_t q, int &t0, int &t1, bool &whole) {
    const int nt = tiles_of(p, it.keys);
    auto cut = [&](int64_t x) {          // a boundary at x: the nearest tile
        const int64_t keys = it.weight == 8 ? x - it.from : quotient(8 * (x - it.from), it.weight);
        const int64_t t = (keys + (1 << (p.tile_shift - 1))) >> p.tile_shift;
        return x <= it.from ? 0 : x >= it.to || t > nt ? nt : static_cast<int>(t);
    };
    t0 = cut(q * stretch);
    t1 = cut((q + 1) * stretch);
    // an item without tiles belongs to the stretch that it begins in
    whole = t0 == 0 && t1 == nt && (nt > 0 || (it.from >= q * stretch && it.from < (q + 1) * stretch));
    return t1 > t0 || whole;
}
__device__ __forceinline__ int line_slot(const LineItem &it, int64_t stretch, int64_t q) {
    return static_cast<int>(2 * q) + (q * stretch > it.from ? 0 : 1);
}

// What a block leaves for the join about the item that reaches beyond its stretch.
struct JoinItem {
    int parts, slot0;      // parts 0: there is none
    int q0, n, m, i, h;    // its sequence, block of rows and head
    int pad;
};

// The batch walked by one warp, forwards: items by number, or by place on the line.  The lanes
// hold 32 sequences at a time.
struct WorkCursor {
    int b0;
    int64_t base, total;   // items or units before the 32 sequences, and in them
    SeqInfo s;
    int nb;                // this lane's sequence: its blocks,
    int64_t lo, cnt;       // first item or unit, how many
    __device__ __forceinline__ void fetch(const GqaBatch &p, int lane) {
        s = b0 + lane < p.B ? seq_info(p, b0 + lane) : SeqInfo{0, 0, 0, 0};
        nb = seq_blocks(p, s.n);
    }
    __device__ __forceinline__ void count(const GqaBatch &p, bool line) {
        const int lane = threadIdx.x & 31;
        cnt = line ? p.Hk * group_units(p, s, nb, nb) : static_cast<int64_t>(p.Hk) * nb;
        int64_t ci = cnt;
        if (p.B > 1) {
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t a = __shfl_up_sync(0xFFFFFFFFu, ci, o);
                if (lane >= o) ci += a;
            }
        }
        lo = base + ci - cnt;
        total = __shfl_sync(0xFFFFFFFFu, ci, p.B > 1 ? 31 : 0);
    }
    // `stretch`: of stretch_units for more than 32 sequences; else found here, from the one look at them
    __device__ __forceinline__ void start(const GqaBatch &p, int lane, int64_t &stretch) {
        b0 = 0;
        base = 0;
        fetch(p, lane);
        if (p.may_split && p.B <= 32) {
            int64_t units = p.Hk * group_units(p, s, nb, nb);
            int items = p.Hk * nb, longest = longest_of(p, s, nb), shortest = 0;
            if (p.B == 1) {
                if (nb > 0) shortest = min(longest, block_keys(p, s, 0));
                units = __shfl_sync(0xFFFFFFFFu, units, 0), items = __shfl_sync(0xFFFFFFFFu, items, 0);
                longest = __shfl_sync(0xFFFFFFFFu, longest, 0), shortest = __shfl_sync(0xFFFFFFFFu, shortest, 0);
            } else {
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) units += __shfl_xor_sync(0xFFFFFFFFu, units, o);
                items = __reduce_add_sync(0xFFFFFFFFu, items);
                longest = __reduce_max_sync(0xFFFFFFFFu, longest);
            }
            stretch = choose_stretch(p, static_cast<int>(gridDim.x), units, items, longest, shortest);
        }
        count(p, stretch > 0);
    }
    // the sequence that holds item or unit x (not below an earlier x); false: behind the last
    __device__ __forceinline__ bool find(const GqaBatch &p, bool line, int lane, int64_t x, int &b, SeqInfo &q, int &blocks, int64_t &first) {
        while (x >= base + total) {
            if (b0 + 32 >= p.B) return false;
            b0 += 32;
            base += total;
            fetch(p, lane);
            count(p, line);
        }
        const int src = __ffs(__ballot_sync(0xFFFFFFFFu, x >= lo && x < lo + cnt)) - 1;
        q.q0 = __shfl_sync(0xFFFFFFFFu, s.q0, src);
        q.n = __shfl_sync(0xFFFFFFFFu, s.n, src);
        q.m = __shfl_sync(0xFFFFFFFFu, s.m, src);
        q.k0 = __shfl_sync(0xFFFFFFFFu, s.k0, src);
        first = __shfl_sync(0xFFFFFFFFu, lo, src);
        blocks = __shfl_sync(0xFFFFFFFFu, nb, src);
        b = b0 + src;
        return true;
    }
};

// The items of this block in order, for one converged warp.
struct BlockWalk {
    WorkCursor cur;
    int64_t stretch, x, x_end;      // the next place on the line, or round of whole items
    LineItem it;                    // the current item
    int t0, t1, slot;               // its key tiles here; its workspace slot if they are not all
    bool whole, any;
    __device__ __forceinline__ void start(const GqaBatch &p, int64_t stretch_, JoinItem *joins, int lane) {
        stretch = stretch_;
        if (joins && lane == 0) joins[blockIdx.x] = JoinItem{};
        cur.start(p, lane, stretch);
        x = blockIdx.x * stretch;
        x_end = x + stretch;
        any = false;
    }
    // Leaves the record about the stretch's last item, if it begins here and reaches beyond.  The
    // stretches with tiles of an item are consecutive: the first is this one, or the next if the
    // nearest tile boundary is the item's start, and the last is the one that holds the middle of
    // its last tile.
    __device__ __forceinline__ void record(const GqaBatch &p, JoinItem *joins, int lane) {
        const int nt = any ? tiles_of(p, it.keys) : 0;
        if (nt == 0 || it.to <= x_end || it.from < x_end - stretch) return;
        const int64_t half = 1 << (p.tile_shift - 1);
        const int64_t q0 = blockIdx.x + (x_end < it.from + units_of(half, it.weight) ? 1 : 0);
        // (no stretch is behind the last block's, unless the lengths are written meanwhile by mistake)
        const int64_t q1 = min(quotient(it.from + units_of((static_cast<int64_t>(nt) << p.tile_shift) - half, it.weight) - 1, stretch),
                               static_cast<int64_t>(gridDim.x) - 1);
        if (q0 < q1 && lane == 0)                // else one block writes it
            joins[blockIdx.x] = JoinItem{static_cast<int>(q1 - q0) + 1, line_slot(it, stretch, q0), it.s.q0, it.s.n, it.s.m, it.i, it.h, 0};
    }
    __device__ __forceinline__ bool next(const GqaBatch &p, JoinItem *joins, int lane) {
        SeqInfo s;
        int b, nb;
        int64_t first;
        if (stretch == 0) {         // whole items, back and forth over the blocks
            const int grid = static_cast<int>(gridDim.x), blk = static_cast<int>(blockIdx.x);
            int64_t item = x * grid + ((x & 1) ? grid - 1 - blk : blk);
            if (p.next_item && x > 0) {
                const int taken = lane == 0 ? atomicAdd(p.next_item, 1) : 0;
                item = static_cast<int64_t>(grid) + __shfl_sync(0xFFFFFFFFu, taken, 0);
            }
            ++x;
            if (!cur.find(p, false, lane, item, b, s, nb, first)) return false;
            const int y = static_cast<int>(item - first);
            it.s = s, it.b = b, it.h = y % p.Hk, it.i = nb - 1 - y / p.Hk;
            it.keys = block_keys(p, s, it.i);
            t0 = 0, t1 = tiles_of(p, it.keys), slot = 0, whole = true;
            return true;
        }
        while (x < x_end && cur.find(p, true, lane, x, b, s, nb, first)) {
            line_item(p, b, s, nb, first, x, it);
            const bool mine = line_tiles(p, it, stretch, blockIdx.x, t0, t1, whole);
            slot = line_slot(it, stretch, blockIdx.x);
            x = it.to;
            any = true;
            if (mine) return true;
        }
        record(p, joins, lane);
        return false;
    }
};

namespace ptx {
// Orders this thread's ordinary accesses to shared memory before later ones of the async proxy (TMA, MMA operands).
__device__ __forceinline__ void fence_proxy_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
}  // namespace ptx

// All kernels here are launched so that they may start before the kernel in front of them on the
// stream has ended (and set up what touches no memory).  Every thread waits for that one, and for
// its writes, before its own first access, whatever its block has to do, so that a kernel's end
// says that all before it have ended.  (Prompts of 200 tokens in a row: 12.3 -> 10.3 us each; one
// token over 108,000: 49.5 -> 47.3.)
__device__ __forceinline__ void wait_for_earlier_kernels() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

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
        if (it == 1u && __any_sync(0xFFFFFFFFu, *w.abort_flag != 0u)) return false;   // once given up, quickly through the rest
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
// The tile kernel's weights are 2^(x + bias): fp16 ones are scaled by 2^7, so that they lose no
// precision to subnormals until they are 2^-21 of the row's largest (which stays below 2^15).  The
// row's sum carries the same factor.
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
__device__ __forceinline__ uint32_t pack16_down(float lo, float hi) {   // towards zero
    uint32_t r;
    if constexpr (F16) asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else asm("cvt.rz.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
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
}  // namespace lite
