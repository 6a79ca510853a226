// attention_codes.cuh -- what the attention kernels over a cache of e4m3 codes share (attention_fp8.cu,
// attention_tiles.cuh): operand layouts, two codes for a number, and the way of the codes into shared memory.
#pragma once

#include "attention.cuh"

namespace fp8bs {
namespace {

// Shared-memory matrix descriptor: `row` bytes per row, swizzled by as many (32, 64 or 128), groups of 8 rows `row` * 8
// bytes apart. K-major: a row is an M or N index; MN-major: a K index, all of M or N in one row.
__device__ __forceinline__ uint64_t smem_desc_rows(uint32_t addr, uint32_t row) {
    const uint64_t layout = row == 128 ? 2 : row == 64 ? 4 : 6;
    uint64_t d = 0;
    d |= static_cast<uint64_t>((addr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(1) << 16;
    d |= static_cast<uint64_t>((row * 8) >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= layout << 61;
    return d;
}

// Where the 16-byte piece c of a swizzled row stands.
__device__ __forceinline__ int swizzled(int row, int c, int row_bytes) {
    return row_bytes == 128 ? c ^ (row & 7) : row_bytes == 64 ? c ^ ((row >> 1) & 3) : c ^ ((row >> 2) & 1);
}

__device__ __forceinline__ float2 e4m3x2_values(uint32_t pair) {
    return __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(pair), __NV_E4M3)));
}

// Two numbers and what their e4m3 codes leave of them, as codes.
__device__ __forceinline__ void two_codes(float x, float y, uint32_t* hi, uint32_t* lo) {
    *hi = pack_e4m3x2(x, y);
    const float2 h = e4m3x2_values(*hi);
    *lo = pack_e4m3x2(x - h.x, y - h.y);
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

struct Scales {
    const float *k, *v;          // [pages, heads]
};

// The key tiles k0, k0 + BN, ... (nt of them) of an item into a ring of codes, keys or values, by TMA in boxes of
// 2^box_log2 slots (16 at least, so a tile has 8 boxes at most), one lane a box. The pages of as many boxes as whole
// tiles have in 32 lanes are looked up at once, two looks ahead, and their scales one look ahead.
// begun(st, n, first, f): called by all lanes for the n-th tile when its place st is free (of keys: and its copies are on
// their way); f holds the scales of the box of lane `first` + box.
// wait: warp_wait, or one like it.
// tail: where values of the first and last tile that do not count are to be cleared before the tile does (whatever stood
// there must not meet a probability of zero), else null.
template <int STAGES, int D, int CH, int BN, bool IS_KEYS, class It, typename Wait, typename Begun>
__device__ __forceinline__ bool bring_codes(Stream& s, const CUtensorMap* map, const fp8bs_paged_attention_args& a,
                                            const Scales& scales, const It& it, int k0, int nt, int box_log2,
                                            uint8_t* ring, uint64_t* full, uint64_t* empty, uint64_t* tail, int lane,
                                            Wait wait, Begun begun) {
    constexpr int TILE = BN * D;
    const int box = 1 << box_log2;
    const int boxes = BN >> box_log2;
    const int per_look = 32 / boxes;                     // tiles
    const int page_size = static_cast<int>(a.cache.page_size);
    const int heads = static_cast<int>(a.cache.heads);
    const int head = it.head, kv = it.kv, key_lo = it.key_lo;
    const int32_t* table = a.page_table + it.seq * a.table_stride;
    auto lookup = [&](int w) {               // look w: (page, slot) of its boxes, page -1: no keys
        const int64_t key = k0 + (static_cast<int64_t>(w) * per_look * boxes + lane) * box;
        int2 at = make_int2(-1, 0);
        if (key < kv && key + box > key_lo) {
            const int p = static_cast<int>(key) / page_size;
            at.y = static_cast<int>(key) - p * page_size;
            at.x = table[p];
            // a page outside the cache: a coordinate past the end, which reads as zeros
            if (static_cast<unsigned>(at.x) >= static_cast<unsigned>(a.cache.pages)) {
                at.x = static_cast<int>(a.cache.pages);
                if (IS_KEYS) record_error(FP8BS_DEVERR_INDEX);
            }
        }
        return at;
    };
    auto scales_of = [&](int2 at) {
        float2 f = make_float2(1.0f, 1.0f);
        if (at.x >= 0 && at.x < a.cache.pages) {
            const int64_t i = static_cast<int64_t>(at.x) * heads + head;
            if (scales.k) f.x = scales.k[i];
            if (scales.v) f.y = scales.v[i];
        }
        return f;
    };
    int2 at, next = lookup(0), after = lookup(1);
    float2 f, next_f = scales_of(next);
    int in_look = 0, look = 0;                           // tiles of the look in hand that are done, its number
    for (int j = 0; j < nt; ++j) {
        const int key0 = k0 + j * BN;
        if (in_look == 0) {
            at = next, f = next_f;
            next = after;
            next_f = scales_of(next);
            after = lookup(look + 2);
            ++look;
        }
        const int first = in_look * boxes;               // this tile's first box of the look
        if (++in_look == per_look) in_look = 0;
        // boxes [none, live) hold keys that count: those before them are past a window (their pages may have been
        // given back), those after them past the sequence
        const int live = min(boxes, (kv - key0 + box - 1) >> box_log2);
        const int none = j == 0 ? (key_lo - k0) >> box_log2 : 0;
        const int st = s.n % STAGES;
        if (!wait(&empty[st], ((s.n / STAGES) & 1) ^ 1)) return false;
        // (`tail`: values that are partly to be cleared before they count, below)
        const bool partial = tail != nullptr && (kv - key0 < BN || none > 0);
        uint64_t* bar = partial ? tail : &full[st];
        const uint32_t dst = smem_addr(ring) + st * TILE;
        if (!IS_KEYS) begun(st, s.n, first, f);
        if (lane == 0) mbar_arrive_expect_tx(bar, static_cast<uint32_t>((live - none) * box * D));
        __syncwarp();
        const int page = __shfl_sync(0xffffffffu, at.x, first + lane);
        const int slot = __shfl_sync(0xffffffffu, at.y, first + lane);
        if (lane >= none && lane < live)
#pragma unroll
            for (int c = 0; c < D / CH; ++c)
                tma_load_4d(dst + c * (BN * CH) + (lane << box_log2) * CH, map, bar, c * CH, head, slot, page);
        if (IS_KEYS) begun(st, s.n, first, f);
        __syncwarp();
        if (partial) {
            if (!wait(tail, s.tails & 1)) return false;
            ++s.tails;
            const int skip = none << box_log2;
            const int keep = min(kv - key0, BN);
            for (int i = lane; i < (BN - keep + skip) * (D / 16); i += 32) {
                const int k = i / (D / 16);
                const int key = k < skip ? k : keep + k - skip;
                *reinterpret_cast<uint4*>(ring + st * TILE + key * D + (i % (D / 16)) * 16) = make_uint4(0, 0, 0, 0);
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[st]);
        }
        ++s.n;
    }
    return true;
}

}  // namespace
}  // namespace fp8bs
