// serving.cu -- host side of the serving attention calls of include/liteattn.h: the
// grouped-query plan, its argument checks, tensor maps and launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstdlib>
#include <cstring>
#include <mutex>
#include <new>

#include "liteattn.h"
#include "gqa_rows.cuh"
#include "gqa_tile.cuh"
#include "host_util.cuh"
#include "rope_append.cuh"
#include "serving_internal.cuh"

using namespace lite;

namespace {
constexpr uint32_t kGqaMagic = 0x4C414751u;  // "LAGQ"
}

struct lite_attn_gqa {
    uint32_t magic;
    int Hq, Hk, d, dtype;
    int device;
    int sms;
    int32_t *status;   // device status word (sticky)
};

namespace {

bool valid_gqa(const lite_attn_gqa *p) { return p && p->magic == kGqaMagic; }

// A [tokens][heads][d] view: what it spans, and that the kernels can address it.
bool rows_ok(const lite_attn_rows_t &r, int heads, int d, int device) {
    if (r.tokens < 0 || r.tokens >= (int64_t(1) << 31)) return false;
    if (r.tokens == 0) return true;
    if (!r.ptr || r.stride_token < d || r.stride_head < d || r.stride_token % 8 || r.stride_head % 8) return false;
    if (r.stride_token >= (int64_t(1) << 31) || r.stride_head >= (int64_t(1) << 31)) return false;
    const size_t elems = static_cast<size_t>(r.tokens - 1) * r.stride_token + static_cast<size_t>(heads - 1) * r.stride_head + d;
    return device_range_ok(r.ptr, elems * 2u, device);
}
// The kernels' factor of the logits: to the base 2, in 32 bits.
float scale_log2(float scale) { return static_cast<float>(static_cast<double>(scale) * 1.4426950408889634); }
bool scale_ok(float scale) { return scale > 0.0f && std::isfinite(scale_log2(scale)); }
// An output's rows lie apart: whole tokens behind one another, or whole heads.
bool rows_apart(const lite_attn_rows_t &r, int heads, int d) {
    return r.tokens == 0 || r.stride_token >= static_cast<int64_t>(heads - 1) * r.stride_head + d ||
           r.stride_head >= (r.tokens - 1) * r.stride_token + d;
}
size_t rows_bytes(const lite_attn_rows_t &r, int heads, int d) {
    if (r.tokens == 0) return 0;
    return 2u * (static_cast<size_t>(r.tokens - 1) * r.stride_token + static_cast<size_t>(heads - 1) * r.stride_head + d);
}
bool apart(const void *a, size_t na, const void *b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return na == 0 || nb == 0 || x + na <= y || y + nb <= x;
}
// A stretch of memory that a call reads.
struct Input {
    const void *ptr;
    size_t bytes;
};
template <int N>
bool apart_from(const void *out, size_t bytes, const Input (&in)[N]) {
    for (const Input &x : in)
        if (!apart(out, bytes, x.ptr, x.bytes)) return false;
    return true;
}
// Whether two views of the same number of tokens share an element.  Slices of one projection may lie
// between one another's rows (or heads); of other views whose ranges meet it is taken that they do.
bool share_elements(const lite_attn_rows_t &a, int heads_a, const lite_attn_rows_t &b, int heads_b, int d) {
    if (apart(a.ptr, rows_bytes(a, heads_a, d), b.ptr, rows_bytes(b, heads_b, d))) return false;
    const int64_t last = a.tokens - 1, step = a.stride_token;
    if (last > 0 && b.stride_token != step) return true;
    const int64_t base = (reinterpret_cast<intptr_t>(b.ptr) - reinterpret_cast<intptr_t>(a.ptr)) / 2;
    auto meet = [&](int64_t off) {   // rows of d elements, `off` apart in the same token: in any two tokens
        int64_t n = std::max(-last, std::min(last, -off / step));
        for (int64_t k = std::max(-last, n - 1); k <= std::min(last, n + 1); ++k)
            if (std::abs(off + k * step) < d) return true;
        return false;
    };
    if (a.stride_head == b.stride_head) {
        for (int64_t e = 1 - heads_a; e < heads_b; ++e)
            if (meet(base + e * a.stride_head)) return true;
    } else {
        for (int64_t i = 0; i < heads_a; ++i)
            for (int64_t j = 0; j < heads_b; ++j)
                if (meet(base + j * b.stride_head - i * a.stride_head)) return true;
    }
    return false;
}

struct CacheView {
    const void *k, *v;
    int64_t pages;
    int page, layout;
};
int log2_page(int page) {   // -1 unless a power of two from 16 to 65536
    for (int s = 4; s <= 16; ++s)
        if (page == 1 << s) return s;
    return -1;
}
size_t cache_bytes(const lite_attn_gqa *pl, const CacheView &c) {
    return 2u * static_cast<size_t>(c.pages) * c.page * pl->Hk * pl->d;
}
int check_cache(const lite_attn_gqa *pl, const CacheView &c) {
    if (c.layout != LITE_LAYOUT_BHND && c.layout != LITE_LAYOUT_BNHD) return LITE_ERR_INVALID_ARG;
    if (c.pages < 1 || c.pages >= (int64_t(1) << 31)) return LITE_ERR_INVALID_ARG;
    if (log2_page(c.page) < 0) return LITE_ERR_UNSUPPORTED;
    const size_t bytes = cache_bytes(pl, c);
    if (!device_range_ok(c.k, bytes, pl->device) || !device_range_ok(c.v, bytes, pl->device)) return LITE_ERR_INVALID_ARG;
    return apart(c.k, bytes, c.v, bytes) ? LITE_OK : LITE_ERR_INVALID_ARG;
}

bool ints_ok(const int32_t *p, size_t n, int device) { return device_range_ok(p, n * 4u, device, 4); }

// k or v as a 4-D tensor map of 64-element columns, 128-byte swizzle: pages as
// (d, row, head, page) or (d, head, row, page), packed rows as (d, head, row, 1).
bool encode_kv(CUtensorMap *m, const lite_attn_gqa *pl, const CacheView *c, const lite_attn_rows_t *r, int box_rows) {
    const cuuint64_t d = static_cast<cuuint64_t>(pl->d), H = static_cast<cuuint64_t>(pl->Hk);
    const cuuint32_t rows = static_cast<cuuint32_t>(box_rows);
    cuuint64_t dims[4] = {d, H, 1, 1}, strides[3];
    cuuint32_t box[4] = {64u, 1u, rows, 1u};
    const void *ptr;
    if (c) {
        const cuuint64_t P = static_cast<cuuint64_t>(c->page);
        ptr = c->k;
        dims[3] = static_cast<cuuint64_t>(c->pages);
        strides[2] = 2u * P * H * d;
        if (c->layout == LITE_LAYOUT_BHND) {
            dims[1] = P, dims[2] = H;
            strides[0] = 2u * d, strides[1] = 2u * P * d;
            box[1] = rows, box[2] = 1u;
        } else {
            dims[2] = P;
            strides[0] = 2u * d, strides[1] = 2u * H * d;
        }
    } else {
        ptr = r->ptr;
        dims[2] = static_cast<cuuint64_t>(r->tokens);
        strides[0] = 2u * static_cast<cuuint64_t>(r->stride_head);
        strides[1] = 2u * static_cast<cuuint64_t>(r->stride_token);
        strides[2] = strides[1] * dims[2];
    }
    const cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
    return driver().encode(m, pl->dtype == LITE_DTYPE_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                           const_cast<void *>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Raises a kernel's dynamic shared-memory limit once per device.
template <typename K>
int allow_smem(K kernel, std::atomic<bool> *done, int device, uint32_t bytes) {
    if (device < 0 || device >= kMaxDevices) return LITE_ERR_CUDA;
    if (done[device].load(std::memory_order_acquire)) return LITE_OK;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes)) != cudaSuccess) {
        cudaGetLastError();
        return LITE_ERR_CUDA;
    }
    done[device].store(true, std::memory_order_release);
    return LITE_OK;
}

// q as a 4-D tensor map (d, head, row, 1); a box is the heads of a group by a slot's tokens.
bool encode_q(CUtensorMap *m, const lite_attn_gqa *pl, const lite_attn_rows_t &q, int slot_tokens) {
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(pl->d), static_cast<cuuint64_t>(pl->Hq),
                                static_cast<cuuint64_t>(q.tokens), 1};
    const cuuint64_t strides[3] = {2u * static_cast<cuuint64_t>(q.stride_head), 2u * static_cast<cuuint64_t>(q.stride_token),
                                   2u * static_cast<cuuint64_t>(q.stride_token) * dims[2]};
    const cuuint32_t box[4] = {64u, static_cast<cuuint32_t>(pl->Hq / pl->Hk), static_cast<cuuint32_t>(slot_tokens), 1u};
    const cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
    return driver().encode(m, pl->dtype == LITE_DTYPE_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                           q.ptr, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// How a batch is divided among blocks: decided from what the host knows (tensor sizes and
// the bounds that the caller gives), never from the lengths on the device.
struct Division {
    bool tile;            // the tcgen05 kernel of two slots of 128 rows, or the 16-row kernel
    int rows;             // query rows of an item
    int slots;            // slots of an item (tile)
    int64_t items;        // most work items there can be
    int blocks;           // persistent blocks
    bool split;           // items may be cut
    bool by_counter;      // whole items are handed out by a counter
    size_t workspace;
};
// In keys, measured: the turn from one item to the next, what partial outputs and their join cost,
// and the shortest stretch.  Around them (26 shapes): a tile join cost of 640 made a prompt of 4,096 tokens
// 70 -> 83 us and 1,000 tokens 24 -> 27, one of 320 worse still; a rows join cost of 160 16 tokens over 300 keys
// 8.3 -> 12.5 us, one of 640 one token over 500 12.0 -> 12.7; a shortest tile stretch of 512 64 tokens
// over 8,000 keys 23.7 -> 25.7 us (300 over 2,300: 28.0 -> 27.0).
constexpr int kTileItemCost = 256, kTileJoinCost = 1280, kTileMinStretch = 256;
constexpr int kRowsItemCost = 96, kRowsJoinCost = 320, kRowsMinStretch = 128;
// Eighths of a key that a key costs an item whose second slot is empty, measured with 4, 5, 6 and 8 in turn, not
// causal.  At d = 128, 1,560 tokens over 32,760 keys of 12 heads: 412, 344, 329 and 341 us; 880 over 14,000 of 24:
// 213, 197, 193, 196; 1,100 over 20,000 of 16: 268, 230, 233, 235; 2,080 over 16,640, 24 heads on 8: 400 to 407; but
// 300 over 9,000 of 8: 41, 44, 49, 46.  At d = 64 the same five: 385, 315, 273, 272; 187, 160, 145, 148; (1,100 not
// measured); 309 all; 35, 35, 35, 37; and 11 causal chunks of up to 513 tokens over up to 16,514: 206, 174, 151, 146.
constexpr int kTileHalfWeight128 = 6, kTileHalfWeight64 = 8;
constexpr int kManyItems = 8;   // items per block from which whole items come out even within an eighth: no workspace

Division divide(const lite_attn_gqa *pl, int64_t B, int64_t tokens, int64_t max_new, int64_t max_keys) {
    const int64_t G = pl->Hq / pl->Hk;
    max_new = std::min(max_new, tokens);
    Division dv;
    // Up to one item's rows for the rows kernel, measured on both: 16 rows over 64 x 4,336 keys 60 us here, 65
    // in tiles; over 8 x 2,000 keys of 8 heads 24 and 33; 32 rows 104 and 65, 31 and 33.
    dv.tile = max_new * G > RowsCfg<128>::ROWS;
    int64_t least;        // items of a batch without padding
    int most;             // blocks that run at the same time
    dv.slots = 2;
    if (dv.tile) {
        int64_t per = 2 * (128 / G);
        dv.rows = 256;
        dv.items = pl->Hk * std::min((tokens + B * (per - 1)) / per, tokens);
        // Where there are blocks for all slots of a batch, and no item is cut, an item is one slot: alone it ends
        // before two side by side would (64 tokens over 1000 keys, 16 heads over 4: 17.9 instead of 23.1 us; a
        // prompt of 500, 32 heads over 8: 14.2 instead of 16.9; of 200: the same).
        const int64_t singles = pl->Hk * std::min((tokens + B * (per / 2 - 1)) / (per / 2), tokens);
        if (singles <= pl->sms && max_keys <= kTileJoinCost) {
            dv.slots = 1;
            dv.items = singles;
            per /= 2;
        }
        least = pl->Hk * ((tokens + per - 1) / per);
        most = pl->sms;
    } else {
        const int64_t rows = RowsCfg<128>::ROWS;
        dv.rows = RowsCfg<128>::ROWS;
        dv.items = pl->Hk * std::min((tokens * G + B * (rows - 1)) / rows, tokens * G);
        least = pl->Hk * ((tokens * G + rows - 1) / rows);
        most = 2 * pl->sms;
    }
    dv.split = least < kManyItems * most && max_keys > (dv.tile ? kTileJoinCost : kRowsJoinCost);
    // no more blocks than there can be items, unless items may be cut
    dv.blocks = dv.split ? most : static_cast<int>(std::min<int64_t>(dv.items, most));
    // By a counter, where several sequences have more items than there are blocks, against back and forth: 16
    // prompts of 1 to 2,048 tokens 276 -> 236 and 282 -> 256 us (two draws), 12 of 500 to 4,000 525 -> 512, 5 uneven
    // ones at d = 64 277 -> 260, 6 of 4,096 each 819 -> 781, 30 chunks of 300 over 1,200 keys 186 -> 177; it can cost the
    // counter's memset: 40 chunks of 100 over 600 keys 75.4 -> 76.5.  One sequence's items fall off in length evenly:
    // nothing to gain there.
    dv.by_counter = !dv.split && B > 1 && least > most;
    dv.workspace = dv.split ? static_cast<size_t>(dv.blocks) * (2 * static_cast<size_t>(dv.rows) * (pl->d + 2) * 4u + sizeof(JoinItem))
                            : dv.by_counter ? sizeof(int) : 0;
    return dv;
}

// Launches a kernel so that it may begin before the one in front of it on the stream has ended (the
// kernels wait for that one themselves, wait_for_earlier_kernels).
template <typename... P, typename... A>
int launch(void (*kernel)(P...), int64_t blocks, int threads, uint32_t smem, cudaStream_t s, const A &...args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const int rc = cuda_err(cudaLaunchKernelEx(&cfg, kernel, args...));
    if (rc != LITE_OK) cudaGetLastError();
    else g_launches.fetch_add(1);
    return rc;
}

// Joins split items, if there may be any.
template <int D, bool F16>
int launch_join(const lite_attn_gqa *pl, const GqaParams &p, const Division &dv, int slot_tokens, cudaStream_t s) {
    if (!dv.split) return LITE_OK;
    return launch(gqa_join_kernel<D, F16>, dv.tile ? 4 * pl->sms : pl->sms, kJoinThreads, 0, s, p, slot_tokens, dv.blocks);
}

template <int D, bool F16>
int launch_rows(const lite_attn_gqa *pl, const CUtensorMap &tk, const CUtensorMap &tv, const GqaParams &p, const Division &dv,
                cudaStream_t s) {
    using C = RowsCfg<D>;
    static std::atomic<bool> done[kMaxDevices];
    int rc = allow_smem(gqa_rows_kernel<D, F16>, done, pl->device, C::SMEM_BYTES);
    if (rc != LITE_OK) return rc;
    rc = launch(gqa_rows_kernel<D, F16>, dv.blocks, C::NTHREADS, C::SMEM_BYTES, s, tk, tv, p);
    return rc == LITE_OK ? launch_join<D, F16>(pl, p, dv, 0, s) : rc;
}

template <int D, bool F16>
int launch_tile(const lite_attn_gqa *pl, const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                const TileParams &p, const Division &dv, cudaStream_t s) {
    using C = TileCfg<D, F16>;
    static std::atomic<bool> done[kMaxDevices];
    if (pl->device < kMaxDevices && !done[pl->device].load(std::memory_order_acquire)) {
        // the warpgroups' register split draws on what the block is launched with
        cudaFuncAttributes attr;
        if (cudaFuncGetAttributes(&attr, gqa_tile_kernel<D, F16>) != cudaSuccess ||
            attr.numRegs * C::NTHREADS < static_cast<int>(128 * C::REG_CTRL + 256 * C::REG_SOFTMAX)) {
            cudaGetLastError();
            return LITE_ERR_CUDA;
        }
    }
    int rc = allow_smem(gqa_tile_kernel<D, F16>, done, pl->device, C::SMEM_BYTES);
    if (rc != LITE_OK) return rc;
    rc = launch(gqa_tile_kernel<D, F16>, dv.blocks, C::NTHREADS, C::SMEM_BYTES, s, tq, tk, tv, p);
    return rc == LITE_OK ? launch_join<D, F16>(pl, p.a, dv, p.slot_tokens, s) : rc;
}

// Attention of q over the cache (c) or packed rows (k, v).
int attention(lite_attn_gqa *pl, const CacheView *c, const lite_attn_rows_t *k, const lite_attn_rows_t *v,
              const lite_attn_rows_t &q, const lite_attn_rows_t &o, GqaBatch b, int64_t max_new, float scale,
              void *workspace, size_t workspace_bytes, cudaStream_t s) {
    const int G = pl->Hq / pl->Hk;
    const Division dv = divide(pl, b.B, q.tokens, max_new, c ? b.max_keys : b.Tk);
    if (dv.items >= (int64_t(1) << 31) || dv.blocks > kJoinThreads) return LITE_ERR_UNSUPPORTED;
    if (workspace_bytes < dv.workspace) return LITE_ERR_INVALID_ARG;
    if (dv.workspace && !device_range_ok(workspace, dv.workspace, pl->device)) return LITE_ERR_INVALID_ARG;
    if (dv.workspace) {    // overlaps nothing else that the call reads or writes
        const size_t kv = c ? cache_bytes(pl, *c) : 0, ints = 4u * static_cast<size_t>(b.B);
        const Input used[7] = {{o.ptr, rows_bytes(o, pl->Hq, pl->d)}, {q.ptr, rows_bytes(q, pl->Hq, pl->d)},
                               {c ? c->k : k->ptr, c ? kv : rows_bytes(*k, pl->Hk, pl->d)},
                               {c ? c->v : v->ptr, c ? kv : rows_bytes(*v, pl->Hk, pl->d)}, {b.cu_q, ints + 4u},
                               {c ? b.lens : b.cu_k, c ? ints : ints + 4u}, {b.table, c ? ints * b.table_w : 0}};
        if (!apart_from(workspace, dv.workspace, used)) return LITE_ERR_INVALID_ARG;
    }
    if (fault("launch")) return LITE_ERR_CUDA;
    b.G = G;
    b.Hk = pl->Hk;
    b.status = pl->status;
    b.unit_tokens = dv.tile ? dv.slots * (128 / G) : 0;
    const int tile = dv.tile ? 128 : RowsCfg<128>::BN;
    b.tile_shift = dv.tile ? 7 : 6;
    b.may_split = dv.split ? 1 : 0;
    b.item_cost = dv.tile ? kTileItemCost : kRowsItemCost;
    b.join_cost = dv.tile ? kTileJoinCost : kRowsJoinCost;
    b.min_stretch = dv.tile ? kTileMinStretch : kRowsMinStretch;
    b.half_weight = pl->d == 128 ? kTileHalfWeight128 : kTileHalfWeight64;
    TileParams t;
    std::memset(&t, 0, sizeof t);
    GqaParams &p = t.a;
    p.b = b;
    p.probe_wait = fault("device_wait") ? 1 : 0;
    p.q = static_cast<const uint16_t *>(q.ptr);
    p.o = static_cast<uint16_t *>(o.ptr);
    p.q_st = q.stride_token, p.q_sh = q.stride_head, p.o_st = o.stride_token, p.o_sh = o.stride_head;
    p.scale_log2 = scale_log2(scale);
    if (dv.split) {
        const size_t rows = 2 * static_cast<size_t>(dv.blocks) * dv.rows;
        p.ws_o = static_cast<float *>(workspace);
        p.ws_ml = p.ws_o + rows * pl->d;
        p.joins = reinterpret_cast<JoinItem *>(p.ws_ml + rows * 2);
    }
    if (dv.by_counter) {
        p.b.next_item = static_cast<int *>(workspace);
        const int rc = cuda_err(cudaMemsetAsync(workspace, 0, sizeof(int), s));
        if (rc != LITE_OK) return rc;
    }
    const int box = c ? std::min(c->page, tile) : tile;
    CUtensorMap tq, tk, tv;
    std::memset(&tq, 0, sizeof tq);
    std::memset(&tk, 0, sizeof tk);
    std::memset(&tv, 0, sizeof tv);
    if (c) {
        CacheView cv = *c;
        cv.k = c->v;
        if (!encode_kv(&tk, pl, c, nullptr, box) || !encode_kv(&tv, pl, &cv, nullptr, box)) return LITE_ERR_CUDA;
        t.v = static_cast<const uint16_t *>(c->v);
        t.v_page = static_cast<int64_t>(c->page) * pl->Hk * pl->d;
        t.v_head = c->layout == LITE_LAYOUT_BHND ? static_cast<int64_t>(c->page) * pl->d : pl->d;
        t.v_token = c->layout == LITE_LAYOUT_BHND ? pl->d : static_cast<int64_t>(pl->Hk) * pl->d;
    } else if (k->tokens > 0) {   // without keys nothing is loaded
        if (!encode_kv(&tk, pl, nullptr, k, box) || !encode_kv(&tv, pl, nullptr, v, box)) return LITE_ERR_CUDA;
        t.v = static_cast<const uint16_t *>(v->ptr);
        t.v_token = v->stride_token, t.v_head = v->stride_head;
    }
    const bool f16 = pl->dtype == LITE_DTYPE_FP16;
    if (!dv.tile) {
        if (pl->d == 64) return f16 ? launch_rows<64, true>(pl, tk, tv, p, dv, s) : launch_rows<64, false>(pl, tk, tv, p, dv, s);
        return f16 ? launch_rows<128, true>(pl, tk, tv, p, dv, s) : launch_rows<128, false>(pl, tk, tv, p, dv, s);
    }
    t.slot_tokens = 128 / G;
    if (!encode_q(&tq, pl, q, t.slot_tokens)) return LITE_ERR_CUDA;
    if (pl->d == 64) return f16 ? launch_tile<64, true>(pl, tq, tk, tv, t, dv, s) : launch_tile<64, false>(pl, tq, tk, tv, t, dv, s);
    return f16 ? launch_tile<128, true>(pl, tq, tk, tv, t, dv, s) : launch_tile<128, false>(pl, tq, tk, tv, t, dv, s);
}

}  // namespace

extern "C" {

int lite_attn_gqa_create(lite_attn_gqa_t *out, int Hq, int Hk, int d, int dtype) {
    if (!out) return LITE_ERR_INVALID_ARG;
    *out = nullptr;
    if (Hq < 1 || Hk < 1 || Hq % Hk || d < 1) return LITE_ERR_INVALID_ARG;
    if (dtype != LITE_DTYPE_BF16 && dtype != LITE_DTYPE_FP16) return LITE_ERR_INVALID_ARG;
    if ((d != 64 && d != 128) || Hq / Hk > 128 || Hq > 65536) return LITE_ERR_UNSUPPORTED;
    if (fault("alloc")) return LITE_ERR_ALLOC;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return LITE_ERR_CUDA;
    int major = 0, sms = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return LITE_ERR_CUDA;
    if (major != 10 || !driver().ok) return LITE_ERR_CUDA;
    lite_attn_gqa *pl = new (std::nothrow) lite_attn_gqa();
    if (!pl) return LITE_ERR_ALLOC;
    pl->Hq = Hq, pl->Hk = Hk, pl->d = d, pl->dtype = dtype, pl->device = dev, pl->sms = sms;
    if (cudaMalloc(&pl->status, 256) != cudaSuccess) {
        cudaGetLastError();
        delete pl;
        return LITE_ERR_ALLOC;
    }
    if (cudaMemset(pl->status, 0, 256) != cudaSuccess) {
        cudaFree(pl->status);
        delete pl;
        return LITE_ERR_CUDA;
    }
    pl->magic = kGqaMagic;
    *out = pl;
    return LITE_OK;
}

int lite_attn_gqa_destroy(lite_attn_gqa_t plan) {
    if (!plan) return LITE_OK;
    if (!valid_gqa(plan)) return LITE_ERR_INVALID_ARG;
    DeviceScope ds(plan->device);
    cudaDeviceSynchronize();
    cudaFree(plan->status);
    plan->magic = 0;
    delete plan;
    return LITE_OK;
}

int lite_attn_gqa_status(lite_attn_gqa_t plan, void *stream) {
    if (!valid_gqa(plan)) return LITE_ERR_INVALID_ARG;
    if (fault("status")) return LITE_ERR_DEVICE_TIMEOUT;
    DeviceScope ds(plan->device);
    if (!ds.ok) return LITE_ERR_CUDA;
    int32_t status = LITE_OK;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int rc = cuda_err(cudaMemcpyAsync(&status, plan->status, sizeof status, cudaMemcpyDeviceToHost, s));
    if (rc == LITE_OK) rc = cuda_err(cudaStreamSynchronize(s));
    if (rc != LITE_OK) return rc;
    return status == LITE_OK ? LITE_OK : status == LITE_ERR_DEVICE_CHECK ? LITE_ERR_DEVICE_CHECK : LITE_ERR_DEVICE_TIMEOUT;
}

int lite_attn_gqa_workspace(lite_attn_gqa_t plan, int B, int64_t tokens, int max_new, int64_t max_keys, size_t *bytes) {
    if (!valid_gqa(plan) || !bytes || B < 0 || tokens < 0 || max_new < 0 || max_keys < 0) return LITE_ERR_INVALID_ARG;
    *bytes = divide(plan, B, tokens, max_new, max_keys).workspace;
    return LITE_OK;
}

int lite_attn_cache_append(lite_attn_gqa_t plan, const lite_attn_append_t *a, void *stream) {
    if (!valid_gqa(plan) || !a || a->B < 0 || a->table_width < 1) return LITE_ERR_INVALID_ARG;
    const int dev = plan->device, d = plan->d;
    const bool has_q = a->q.ptr != nullptr;
    if (a->k.tokens != a->v.tokens || (has_q && (a->q.tokens != a->k.tokens || a->q_out.tokens != a->k.tokens)) ||
        (!has_q && a->q_out.ptr))
        return LITE_ERR_INVALID_ARG;
    if ((a->cos == nullptr) != (a->sin == nullptr) || (!a->cos && a->positions)) return LITE_ERR_INVALID_ARG;
    if (a->cos && (a->rot < 16 || a->rot > d || a->rot % 16 || a->angle_rows < 1 || a->angle_rows >= (int64_t(1) << 31)))
        return LITE_ERR_INVALID_ARG;
    const CacheView c{a->k_pages, a->v_pages, a->pages, a->page, a->layout};
    DeviceScope ds(dev);
    if (!ds.ok) return LITE_ERR_CUDA;
    int rc = check_cache(plan, c);
    if (rc != LITE_OK) return rc;
    if (a->k.tokens == 0 || a->B == 0) return LITE_OK;
    if (!rows_ok(a->k, plan->Hk, d, dev) || !rows_ok(a->v, plan->Hk, d, dev) ||
        (has_q && (!rows_ok(a->q, plan->Hq, d, dev) || !rows_ok(a->q_out, plan->Hq, d, dev) || !rows_apart(a->q_out, plan->Hq, d))))
        return LITE_ERR_INVALID_ARG;
    if (!ints_ok(a->cu_new, static_cast<size_t>(a->B) + 1, dev) || !ints_ok(a->lens, a->B, dev) ||
        !ints_ok(a->table, static_cast<size_t>(a->B) * a->table_width, dev) ||
        (a->positions && !ints_ok(a->positions, a->k.tokens, dev)))
        return LITE_ERR_INVALID_ARG;
    if (a->cos) {
        const size_t nb = static_cast<size_t>(a->angle_rows) * (a->rot / 2) * 4u;
        if (!device_range_ok(a->cos, nb, dev) || !device_range_ok(a->sin, nb, dev)) return LITE_ERR_INVALID_ARG;
    }
    // the outputs overlap no input and not one another; q may be rotated in place, k and v between its rows then
    const size_t cb = cache_bytes(plan, c);
    const lite_attn_rows_t *in[3] = {&a->k, &a->v, &a->q};
    const bool in_place = has_q && a->q.ptr == a->q_out.ptr && a->q.stride_token == a->q_out.stride_token &&
                          a->q.stride_head == a->q_out.stride_head;
    for (int i = 0; i < (has_q ? 3 : 2); ++i) {
        const size_t nb = rows_bytes(*in[i], i == 2 ? plan->Hq : plan->Hk, d);
        if (!apart(in[i]->ptr, nb, c.k, cb) || !apart(in[i]->ptr, nb, c.v, cb)) return LITE_ERR_INVALID_ARG;
        if (has_q && in_place && i < 2 && share_elements(a->q_out, plan->Hq, *in[i], plan->Hk, d)) return LITE_ERR_INVALID_ARG;
        if (has_q && !in_place && !apart(in[i]->ptr, nb, a->q_out.ptr, rows_bytes(a->q_out, plan->Hq, d)))
            return LITE_ERR_INVALID_ARG;
    }
    const size_t ob = has_q ? rows_bytes(a->q_out, plan->Hq, d) : 0, ints = 4u * static_cast<size_t>(a->B);
    const size_t ab = a->cos ? static_cast<size_t>(a->angle_rows) * (a->rot / 2) * 4u : 0;
    const Input fixed[6] = {{a->cos, ab}, {a->sin, ab}, {a->positions, a->positions ? 4u * static_cast<size_t>(a->k.tokens) : 0},
                            {a->cu_new, ints + 4u}, {a->lens, ints}, {a->table, ints * a->table_width}};
    if (!apart(a->q_out.ptr, ob, c.k, cb) || !apart(a->q_out.ptr, ob, c.v, cb) || !apart_from(a->q_out.ptr, ob, fixed) ||
        !apart_from(c.k, cb, fixed) || !apart_from(c.v, cb, fixed))
        return LITE_ERR_INVALID_ARG;
    if (fault("launch")) return LITE_ERR_CUDA;
    NvtxRange range("lite_attn_cache_append");

    AppendParams p;
    std::memset(&p, 0, sizeof p);
    p.q = static_cast<const uint16_t *>(a->q.ptr), p.k = static_cast<const uint16_t *>(a->k.ptr);
    p.v = static_cast<const uint16_t *>(a->v.ptr), p.q_out = static_cast<uint16_t *>(a->q_out.ptr);
    p.kc = static_cast<uint16_t *>(a->k_pages), p.vc = static_cast<uint16_t *>(a->v_pages);
    p.q_st = a->q.stride_token, p.q_sh = a->q.stride_head, p.k_st = a->k.stride_token, p.k_sh = a->k.stride_head;
    p.v_st = a->v.stride_token, p.v_sh = a->v.stride_head, p.qo_st = a->q_out.stride_token, p.qo_sh = a->q_out.stride_head;
    p.c_sp = static_cast<int64_t>(a->page) * plan->Hk * d;
    p.c_sh = a->layout == LITE_LAYOUT_BHND ? static_cast<int64_t>(a->page) * d : d;
    p.c_st = a->layout == LITE_LAYOUT_BHND ? d : static_cast<int64_t>(plan->Hk) * d;
    p.cos = a->cos, p.sin = a->sin, p.positions = a->positions, p.n_pos = a->angle_rows;
    p.Hq = plan->Hq, p.Hk = plan->Hk, p.D = d, p.rot = a->cos ? a->rot : 0, p.interleaved = a->interleaved ? 1 : 0;
    p.has_q = has_q ? 1 : 0;
    p.b.cu_q = a->cu_new, p.b.lens = a->lens, p.b.table = a->table, p.b.Tq = a->k.tokens, p.b.pages = a->pages;
    p.b.max_keys = static_cast<int64_t>(a->table_width) * a->page, p.b.status = plan->status, p.b.B = a->B;
    p.b.mode = a->layout == LITE_LAYOUT_BHND ? kKvPagesBhnd : kKvPagesBnhd;
    p.b.table_w = a->table_width, p.b.page_shift = log2_page(a->page);
    // One token per block while the tokens do not fill the GPU twice over; several then.
    const int slots = kAppendThreads / (d / 16);
    const int heads = (has_q ? plan->Hq : 0) + 2 * plan->Hk;
    int lanes = slots;
    while (lanes > 1 && lanes / 2 >= heads) lanes /= 2;      // no lane without a head
    while (lanes > 4 && a->k.tokens * lanes / slots > 4 * plan->sms) lanes /= 2;
    p.head_lanes = lanes;
    p.tokens_per_block = slots / lanes;
    const int64_t blocks = (a->k.tokens + p.tokens_per_block - 1) / p.tokens_per_block;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return launch(plan->dtype == LITE_DTYPE_FP16 ? rope_append_kernel<true> : rope_append_kernel<false>, blocks, kAppendThreads, 0, s, p);
}

int lite_attn_cache_attend(lite_attn_gqa_t plan, const lite_attn_attend_t *a, void *stream) {
    if (!valid_gqa(plan) || !a || a->B < 0 || a->table_width < 1 || a->max_new < 0)
        return LITE_ERR_INVALID_ARG;
    if (!scale_ok(a->scale) || a->q.tokens != a->o.tokens) return LITE_ERR_INVALID_ARG;
    const int dev = plan->device, d = plan->d;
    const CacheView c{a->k_pages, a->v_pages, a->pages, a->page, a->layout};
    DeviceScope ds(dev);
    if (!ds.ok) return LITE_ERR_CUDA;
    int rc = check_cache(plan, c);
    if (rc != LITE_OK) return rc;
    if (a->q.tokens == 0 || a->B == 0) return LITE_OK;
    if (a->q.tokens * plan->Hq >= (int64_t(1) << 31)) return LITE_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(a->table_width) * a->page > (int64_t(1) << 30)) return LITE_ERR_UNSUPPORTED;
    if (!rows_ok(a->q, plan->Hq, d, dev) || !rows_ok(a->o, plan->Hq, d, dev) || !rows_apart(a->o, plan->Hq, d))
        return LITE_ERR_INVALID_ARG;
    if (!ints_ok(a->cu_new, static_cast<size_t>(a->B) + 1, dev) || !ints_ok(a->lens, a->B, dev) ||
        !ints_ok(a->table, static_cast<size_t>(a->B) * a->table_width, dev))
        return LITE_ERR_INVALID_ARG;
    const size_t cb = cache_bytes(plan, c), ints = 4u * static_cast<size_t>(a->B);
    const Input in[6] = {{a->q.ptr, rows_bytes(a->q, plan->Hq, d)}, {c.k, cb}, {c.v, cb}, {a->cu_new, ints + 4u}, {a->lens, ints},
                         {a->table, ints * a->table_width}};
    if (!apart_from(a->o.ptr, rows_bytes(a->o, plan->Hq, d), in)) return LITE_ERR_INVALID_ARG;
    NvtxRange range("lite_attn_cache_attend");
    GqaBatch b;
    std::memset(&b, 0, sizeof b);
    b.cu_q = a->cu_new, b.lens = a->lens, b.table = a->table, b.Tq = a->q.tokens, b.pages = a->pages;
    b.max_keys = static_cast<int64_t>(a->table_width) * a->page, b.B = a->B, b.causal = a->causal ? 1 : 0;
    b.mode = a->layout == LITE_LAYOUT_BHND ? kKvPagesBhnd : kKvPagesBnhd;
    b.table_w = a->table_width, b.page_shift = log2_page(a->page);
    return attention(plan, &c, nullptr, nullptr, a->q, a->o, b, a->max_new, a->scale, a->workspace, a->workspace_bytes,
                     static_cast<cudaStream_t>(stream));
}

int lite_attn_prompt(lite_attn_gqa_t plan, const lite_attn_prompt_t *a, void *stream) {
    if (!valid_gqa(plan) || !a || a->B < 0) return LITE_ERR_INVALID_ARG;
    if (!scale_ok(a->scale) || a->q.tokens != a->o.tokens || a->k.tokens != a->v.tokens)
        return LITE_ERR_INVALID_ARG;
    const int dev = plan->device, d = plan->d;
    DeviceScope ds(dev);
    if (!ds.ok) return LITE_ERR_CUDA;
    if (a->q.tokens == 0 || a->B == 0) return LITE_OK;
    if (a->q.tokens * plan->Hq >= (int64_t(1) << 31) || a->k.tokens > (int64_t(1) << 30)) return LITE_ERR_UNSUPPORTED;
    if (!rows_ok(a->q, plan->Hq, d, dev) || !rows_ok(a->o, plan->Hq, d, dev) || !rows_ok(a->k, plan->Hk, d, dev) ||
        !rows_ok(a->v, plan->Hk, d, dev) || !rows_apart(a->o, plan->Hq, d))
        return LITE_ERR_INVALID_ARG;
    if (!ints_ok(a->cu_q, static_cast<size_t>(a->B) + 1, dev) || !ints_ok(a->cu_k, static_cast<size_t>(a->B) + 1, dev))
        return LITE_ERR_INVALID_ARG;
    const size_t ints = 4u * static_cast<size_t>(a->B) + 4u;
    const Input in[5] = {{a->q.ptr, rows_bytes(a->q, plan->Hq, d)}, {a->k.ptr, rows_bytes(a->k, plan->Hk, d)},
                         {a->v.ptr, rows_bytes(a->v, plan->Hk, d)}, {a->cu_q, ints}, {a->cu_k, ints}};
    if (!apart_from(a->o.ptr, rows_bytes(a->o, plan->Hq, d), in)) return LITE_ERR_INVALID_ARG;
    NvtxRange range("lite_attn_prompt");
    GqaBatch b;
    std::memset(&b, 0, sizeof b);
    b.cu_q = a->cu_q, b.cu_k = a->cu_k, b.Tq = a->q.tokens, b.Tk = a->k.tokens, b.pages = 1;
    b.B = a->B, b.causal = a->causal ? 1 : 0, b.mode = kKvPacked;
    return attention(plan, nullptr, &a->k, &a->v, a->q, a->o, b, a->q.tokens, a->scale, a->workspace, a->workspace_bytes,
                     static_cast<cudaStream_t>(stream));
}

}  // extern "C"
