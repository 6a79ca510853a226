// attention_tiles.cuh -- the attention kernel whose query rows fill MMA tiles of 128 (attention.cu says how), over a
// cache in bf16 or of e4m3 codes (AttnCfg::CODES).
#pragma once

#include "attention_codes.cuh"

namespace fp8bs {
namespace {

constexpr float kRescale = 8.0f;

// Where a row's maximum is this large, in log2 units, binary32 holds the terms of the fused product that makes exponents
// of scores to 8 and more (a bf16 cache: 128), by which a probability would be out of the range of binary16 (bf16): a
// function of its own takes the scores relative to the maximum first (far_tiles; the chunk of 4096 over codes 318 us,
// 316 without it, 326 to 366 with the same in the loop of all rows; 192-wide heads over bf16 57.4, 56.6 without). Asked
// where a maximum grows.
template <bool CODES>
constexpr float kFar = CODES ? 67108864.0f : 1073741824.0f;

// CODES: the cache holds e4m3 codes. The keys' product then takes them as they are, and each query as the sum of two
// e4m3 numbers per channel (their products go to one S). The keys' scale joins the softmax's factor, 16 keys at a time,
// and the values' its exponent (P = exp2(c ks S + log2 vs - m), so that pages whose values differ in size share a tile);
// the row sum takes it out again. Values are widened to binary16 by four warps of their own, on the way from a ring of
// codes to the ring of values, and P is binary16 too (2^-12 of it, and 2^-23 of the largest's: the reference is up to
// four times that).
template <int DK_, int DV_, int NQ_, bool CODES_ = false>
struct AttnCfg {
    static constexpr int DK = DK_, DV = DV_, NQ = NQ_;
    static constexpr bool CODES = CODES_;
    // Keys per tile. (192-wide keys: 96, so that two tiles of values fit.)
    static constexpr int BN = NQ == 1 ? 64 : DK <= 128 ? 128 : 96;
    static constexpr int ROWS = NQ * 128;
    static constexpr int SLOTS = 4;                              // ring of work items
    static constexpr int SBUF = 2;                               // S buffers: per query tile, or 2
    static constexpr int K_TILE = BN * DK * (CODES ? 1 : 2), V_TILE = BN * DV * 2, Q_TILE = 128 * DK * 2;
    // One query tile of 64 channels: two CTAs per SM, one's softmax under the other's (a windowed mixed batch 32 ->
    // 25 us, decode of 64 sequences of 4096 keys 153 -> 109).
    static constexpr int CTAS = NQ == 1 && DK == 64 ? 2 : 1;
    static constexpr int KST =
        DK == 64 ? (NQ == 2 ? 4 : 5) : DK == 128 ? (NQ == 2 ? 3 : 6) : (NQ == 2 ? (CODES ? 3 : 2) : 4);
    static constexpr int VST = DK == 64 ? (NQ == 2 ? 4 : 5) : DK == 128 ? (NQ == 2 ? 2 : 5) : (NQ == 2 ? 2 : 4);
    static constexpr int SOFT_WARPS = 4 * NQ;
    static constexpr int KEY_WARP = SOFT_WARPS;                  // brings the keys (and hands out the items)
    static constexpr int VALUE_WARP = SOFT_WARPS + 1;
    static constexpr int MMA_WARP = SOFT_WARPS + 2;
    static constexpr int WIDEN_WARP = SOFT_WARPS + 4;            // (codes) the first of four
    // (two query tiles: a whole third warpgroup beside the softmax's, for the split of registers below)
    static constexpr int THREADS = 32 * (SOFT_WARPS + (NQ == 2 || CODES ? 4 : 3) + (CODES ? 4 : 0));
    // Codes: bytes of a key per swizzled chunk; tiles of values as codes; tiles' key scales, whose place is free when the
    // tile CST before has been read (the product that frees the place of the key tile KST before follows that P).
    static constexpr int CHK = DK % 128 == 0 ? 128 : 64;
    static constexpr int VC_TILE = CODES ? BN * DV : 0, VCST = !CODES ? 0 : DK == 64 || NQ == 1 ? 4 : 2;
    static constexpr int CST = CODES ? KST + (NQ == 2 ? 1 : 2) : 0;
    static constexpr int READERS = SOFT_WARPS + 2 + (CODES ? 4 : 0);         // warps that read a work item
    static constexpr uint32_t TMEM_COLS = tmem_cols_for(SBUF * BN + NQ * DV);
    static constexpr int BARS = 2 * KST + 2 * VST + 2 * SBUF + 3 * NQ + 3 + 2 * SLOTS + 2 * VCST + CST;
    static constexpr int SMEM = 1024 + NQ * Q_TILE + KST * K_TILE + VST * V_TILE + VCST * VC_TILE + BARS * 8 + 64;
    static_assert(SMEM <= kSmemLimit, "shared memory");
};

// D[tmem] (+)= A[smem] * B[smem]^T, bf16.
__device__ __forceinline__ void mma_bf16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                         uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Keys and values lie in shared memory as [8 keys][64 channels]: one key per 128-byte row, 128-byte swizzle, the
// blocks of 1024 bytes of the same 8 keys one after another, 8-key groups `group` bytes apart. The keys' product
// reads them K-major, the values' product MN-major (its leading offset is the step to the next 64 channels).
__device__ __forceinline__ uint64_t smem_desc_groups(uint32_t addr, uint32_t group) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((addr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(1024 >> 4) << 16;
    d |= static_cast<uint64_t>(group >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}

constexpr uint32_t kIdescBMajorMN = 1u << 16;

// The key tiles k0, k0 + BN, ... (nt of them) of an item into the ring of KEYS or values, by TMA in boxes of
// 2^box_log2 slots. The pages of 32 boxes are looked up at once, one per lane, while those before are in use, and
// each box is issued by a lane of its own (one lane for all: 64 ragged sequences with pages of 16 slots took 273
// instead of 204 us, a chunk of 4096 over 8192 keys 364 instead of 335). Values of the
// first and last tile that do not count are cleared before the tile does: whatever stood there must not meet a
// probability of zero.
// first_wait(): waited for before the first tile, under the first look at the pages.
template <class Cfg, bool KEYS, typename First>
__device__ __forceinline__ bool bring_tiles(Stream& s, const CUtensorMap* map, const fp8bs_paged_attention_args& a,
                                            const Item& it, int k0, int nt, int box_log2, int mode, uint8_t* ring,
                                            uint64_t* full, uint64_t* empty, uint64_t* tail, int2* window,
                                            int lane, First first_wait) {
    constexpr int STAGES = KEYS ? Cfg::KST : Cfg::VST;
    constexpr int TILE = KEYS ? Cfg::K_TILE : Cfg::V_TILE;
    constexpr int CH = (KEYS ? Cfg::DK : Cfg::DV) / 64;
    constexpr int BN = Cfg::BN;
    const int box = 1 << box_log2;
    const int boxes = BN >> box_log2;
    const int page_size = static_cast<int>(a.cache.page_size);
    const int heads = static_cast<int>(a.cache.heads);
    const int head = it.head, kv = it.kv, key_lo = it.key_lo;
    const int32_t* table = a.page_table + it.seq * a.table_stride;
    auto lookup = [&](int w) {               // boxes 32 w .. 32 w + 31 of the item
        const int64_t key = k0 + (static_cast<int64_t>(w) * 32 + lane) * box;
        int2 at = make_int2(0, 0);
        if (key < kv && key + box > key_lo) {
            const int p = static_cast<int>(key) / page_size;
            at.y = static_cast<int>(key) - p * page_size;
            at.x = table[p];
        }
        return at;
    };
    int window_at = 0;                       // the 32 boxes that `next` is of
    int2 next = lookup(0);
    if (s.n == 0 && !first_wait()) return false;
    for (int j = 0; j < nt; ++j) {
        const int key0 = k0 + j * BN;
        // boxes [none, live) hold keys that count: those before them are past a window (their pages may have been
        // given back), those after them past the sequence
        const int live = min(boxes, (kv - key0 + box - 1) >> box_log2);
        const int none = j == 0 ? (key_lo - k0) >> box_log2 : 0;
        const int st = s.n % STAGES;
        if (!warp_wait(&empty[st], ((s.n / STAGES) & 1) ^ 1)) return false;
        const bool partial = !KEYS && (kv - key0 < BN || none > 0);
        uint64_t* bar = partial ? tail : &full[st];
        const uint32_t dst = smem_addr(ring) + st * TILE;
        if (lane == 0) mbar_arrive_expect_tx(bar, static_cast<uint32_t>((live - none) * box * CH * 128));
        for (int b = none; b < live;) {
            const int first = j * boxes + b;
            if ((first & 31) == 0 || (j == 0 && b == none)) {
                // (the first look may begin inside a window of 32 boxes)
                while (window_at < first >> 5) {
                    next = lookup(++window_at);
                }
                // a page outside the cache: a coordinate past the end, which reads as zeros
                if (static_cast<unsigned>(next.x) >= static_cast<unsigned>(a.cache.pages)) {
                    next.x = static_cast<int>(a.cache.pages);
                    const int64_t key = k0 + (static_cast<int64_t>(window_at) * 32 + lane) * box;
                    if (KEYS && key < kv && key + box > key_lo) record_error(FP8BS_DEVERR_INDEX);
                }
                window[lane] = next;
                next = lookup(++window_at);
                __syncwarp();
            }
            const int count = min(32 - (first & 31), live - b);
            __syncwarp();
            if (lane < count) {
                const int2 at = window[(first + lane) & 31];
                const int key = (b + lane) << box_log2;           // of the tile
                if (mode == 0)
                    tma_load_5d(dst + key * (CH * 128), map, bar, 0, 0, head * CH, at.y >> 3, at.x);
                else if (mode == 1)
                    tma_load_5d(dst + key * (CH * 128), map, bar, 0, 0, 0, at.y >> 3, at.x * heads + head);
                else
                    for (int c = 0; c < CH; ++c)
                        tma_load_4d(dst + (key >> 3) * (CH * 1024) + c * 1024 + (key & 7) * 128, map, bar,
                                    c * 64, head, at.y, at.x);
            }
            __syncwarp();
            b += count;
        }
        if (partial) {
            if (!warp_wait(tail, s.tails & 1)) return false;
            ++s.tails;
            const int skip = none << box_log2;
            const int keep = min(kv - key0, BN);
            for (int i = lane; i < (BN - keep + skip) * CH * 8; i += 32) {
                const int k = i / (CH * 8);
                const int key = k < skip ? k : keep + k - skip;
                const int c = i / 8 % CH;
                *reinterpret_cast<uint4*>(ring + st * TILE + (key >> 3) * (CH * 1024) + c * 1024 +
                                          (key & 7) * 128 + (i & 7) * 16) = make_uint4(0, 0, 0, 0);
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[st]);
        }
        ++s.n;
    }
    return true;
}

// Four warps: values from codes to binary16, which holds them exactly, in the order of the key tiles; those that do not
// count become zeros (whatever stood there must not meet a probability of zero). Per 16 codes a load, eight conversions
// and two stores. (As bf16, the page's scale with them, it took 45 instructions, and 5700 cycles a tile of 128 x 128,
// twice what the products and the softmax of two query tiles take: the chunk of 4096 585 us.)
template <class Cfg>
__device__ __forceinline__ void widen_values(const Item* s_item, const uint8_t* sVC, uint8_t* sV,
                                             uint64_t* vc_full, uint64_t* vc_empty, uint64_t* v_full, uint64_t* v_empty,
                                             uint64_t* i_full, uint64_t* i_empty, int w, int lane) {
    constexpr int BN = Cfg::BN, DV = Cfg::DV, PIECES = DV / 16;      // 16 codes each, of a key
    constexpr int STEP = 128 / PIECES, ROUNDS = BN / STEP;           // keys at a time (8 of them or more: the swizzle is the
                                                                     // same for all of a thread's)
    static_assert(STEP % 8 == 0 && BN % STEP == 0, "rounds of whole groups of 8 keys");
    const int first = (w * 32 + lane) / PIECES, c = lane % PIECES;   // a thread's first key, its piece
    const int in = first * DV + (swizzled(first, c, DV) << 4);
    const int out_block = (first >> 3) * (DV / 64 * 1024) + (2 * c / 8) * 1024 + (first & 7) * 128;
    const int place0 = ((2 * c % 8) ^ (first & 7)) << 4, place1 = ((2 * c % 8 + 1) ^ (first & 7)) << 4;
    bool ok = true;
    int n = 0;
    for (int x = 0; ok; ++x) {
        ok = warp_wait(&i_full[x % Cfg::SLOTS], (x / Cfg::SLOTS) & 1);
        if (!ok) break;
        const Item& it = s_item[x % Cfg::SLOTS];
        const int seq = it.seq, kv = it.kv, key_lo = it.key_lo, key_hi = it.key_hi;
        __syncwarp();
        if (lane == 0) mbar_arrive(&i_empty[x % Cfg::SLOTS]);
        if (seq < 0) break;
        const int k0 = key_lo / BN * BN;
        const int nt = key_hi > key_lo ? (key_hi - k0 + BN - 1) / BN : 0;
        for (int j = 0; j < nt; ++j, ++n) {
            const int from = n % Cfg::VCST, to = n % Cfg::VST;
            ok = warp_wait(&vc_full[from], (n / Cfg::VCST) & 1) && warp_wait(&v_empty[to], ((n / Cfg::VST) & 1) ^ 1);
            if (!ok) break;
            const int key0 = k0 + j * BN;
            const int lo = key_lo - key0, hi = kv - key0;             // keys of the tile that count
            const uint8_t* src = sVC + from * Cfg::VC_TILE + in;
            uint8_t* dst = sV + to * Cfg::V_TILE + out_block;
            const bool part = lo > 0 || hi < BN;
#pragma unroll 4
            for (int i = 0; i < ROUNDS; ++i) {
                uint4 v = *reinterpret_cast<const uint4*>(src + i * (STEP * DV));
                if (part && (i * STEP + first < lo || i * STEP + first >= hi)) v = make_uint4(0, 0, 0, 0);
                const uint32_t words[4] = {v.x, v.y, v.z, v.w};
                uint32_t out[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const __half2 h = __half2(__nv_cvt_fp8x2_to_halfraw2(
                        static_cast<__nv_fp8x2_storage_t>(words[k / 2] >> (16 * (k & 1)) & 0xFFFFu), __NV_E4M3));
                    out[k] = *reinterpret_cast<const uint32_t*>(&h);
                }
                uint8_t* row = dst + i * (STEP / 8 * (DV / 64) * 1024);
                *reinterpret_cast<uint4*>(row + place0) = make_uint4(out[0], out[1], out[2], out[3]);
                *reinterpret_cast<uint4*>(row + place1) = make_uint4(out[4], out[5], out[6], out[7]);
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&v_full[to]);
                mbar_arrive(&vc_empty[from]);
            }
        }
    }
    if (!ok && lane == 0) record_error(FP8BS_DEVERR_PRODUCER_WAIT);
}

// A row's sums O by `keep`, in TMEM.
template <int DV>
__device__ __forceinline__ void scale_columns(uint32_t o_tmem, float keep) {
#pragma unroll 1
    for (int i = 0; i < DV / 16; ++i) {
        float o[16];
        tmem_ld_16cols(o_tmem + 16 * i, o);
        tmem_wait_ld_16(o);
#pragma unroll
        for (int k = 0; k < 16; ++k) o[k] *= keep;
        tmem_st_16cols(o_tmem + 16 * i, reinterpret_cast<const uint32_t*>(o));
    }
}

struct FarRows {
    float m, l;
    bool ok;
};

// What the softmax warps do with an item's tiles, from the j-th on, whose maximum is far in some row (kFar): 16 keys at a
// time, the reference taken from each score (codes: from the score in log2 units, rounded to binary32). row_lo, row_hi: the
// row's keys, counted from the item's first tile.
template <class Cfg>
__device__ __noinline__ FarRows far_tiles(uint32_t tmem, uint32_t o_tmem, int q, float c, const float4* scales,
                                          uint64_t* c_full, uint64_t* s_full, uint64_t* p_full, uint64_t* o_done, int n0,
                                          int j, int nt, int row_lo, int row_hi, float m, float l, int lane) {
    constexpr int BN = Cfg::BN;
    constexpr bool CODES = Cfg::CODES;
    constexpr int CST = CODES ? Cfg::CST : 1;
    bool ok = true;
#pragma unroll 1
    for (; j < nt; ++j) {
        const int n = n0 + j;
        const int buf = Cfg::NQ == 2 ? q : n & 1;
        ok = (!CODES || warp_wait(&c_full[n % CST], (n / CST) & 1)) &&
             warp_wait(&s_full[buf], Cfg::NQ == 2 ? n & 1 : (n >> 1) & 1);
        if (!ok) break;
        tc_fence_after();
        const uint32_t s_tmem_row = tmem + buf * BN;
        const int lo = row_lo - j * BN, hi = row_hi - j * BN;
        const float4* sc16 = scales + n % CST * 8;
        auto load_scores = [&](int i, float* s) {
            tmem_ld_16cols(s_tmem_row + 16 * i, s);
            tmem_wait_ld_16(s);
            float4 sc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if constexpr (CODES) sc = sc16[i];
            const float by = max_nan(c * sc.x, 1.2e-38f);
#pragma unroll
            for (int k = 0; k < 16; ++k)
                s[k] = 16 * i + k < lo || 16 * i + k >= hi ? -INFINITY : CODES ? fmaf(s[k], by, sc.y) : s[k];
        };
        float top = -INFINITY, total = 0.0f;
#pragma unroll 1
        for (int i = 0; i < BN / 16; ++i) {
            float s[16];
            load_scores(i, s);
#pragma unroll
            for (int k = 0; k < 16; ++k) top = fmaxf(top, s[k]);
        }
        const bool grow = CODES ? top > m : (top - m) * c > kRescale || (m == -INFINITY && top > m);
        const float keep = !grow ? 1.0f : CODES ? exp2_fast(m - top - 2.0f) : exp2_fast((m - top) * c);
        if (grow) m = CODES ? top + 2.0f : top;
        const float ref = m == -INFINITY ? 0.0f : m;
        // (bf16: other rows keep the rounded product that their probabilities have been taken relative to so far)
        const float rest = !CODES && fabsf(ref * c) < kFar<CODES> ? fmaf(ref, c, -(ref * c)) : 0.0f;
#pragma unroll 1
        for (int i = 0; i < BN / 16; ++i) {
            float s[16], sum = 0.0f;
            load_scores(i, s);
            uint32_t p[8];
#pragma unroll
            for (int k = 0; k < 16; ++k) sum += s[k] = exp2_fast(CODES ? s[k] - ref : fmaf(s[k] - ref, c, rest));
            if constexpr (CODES)
                total = fmaf(sum, sc16[i].z, total);
            else
                total += sum;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                p[k] = CODES ? pack_half2(s[2 * k], s[2 * k + 1]) : pack_bf16x2(s[2 * k], s[2 * k + 1]);
            tmem_st_4cols(s_tmem_row + 8 * i, p[0], p[1], p[2], p[3]);
            tmem_st_4cols(s_tmem_row + 8 * i + 4, p[4], p[5], p[6], p[7]);
        }
        if (CODES && total != total && m == -INFINITY) m = 0.0f;
        l = fmaf(l, keep, total);
        if (j > 0 && __any_sync(0xffffffffu, grow)) {
            ok = warp_wait(o_done, (n - 1) & 1);
            if (!ok) break;
            tc_fence_after();
            scale_columns<Cfg::DV>(o_tmem, keep);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[buf]);
    }
    return FarRows{m, l, ok};
}

template <class Cfg>
__global__ void __launch_bounds__(Cfg::THREADS, Cfg::CTAS)
    paged_attention_kernel(const __grid_constant__ CUtensorMap tmK,
                           const __grid_constant__ CUtensorMap tmV,
                           const __grid_constant__ fp8bs_paged_attention_args a,
                           const AttentionModes modes, const int piece_len, const int pieces, const AttnParts parts,
                           const Scales scales, const int more_rows) {
    constexpr int DK = Cfg::DK, DV = Cfg::DV, NQ = Cfg::NQ, BN = Cfg::BN;
    constexpr bool CODES = Cfg::CODES;
    extern __shared__ uint8_t smem_raw[];
    __shared__ Item s_item[Cfg::SLOTS];
    __shared__ int2 s_window[2][32];                      // (page, slot) of 32 boxes: keys', values'
    __shared__ float s_unit[CODES ? NQ * 128 : 1];        // codes: what a row's queries have been divided by
    __shared__ float4 s_scale[CODES ? Cfg::CST : 1][8];   // of 16 keys each: ks, log2 vs, 1 / vs
    __shared__ uint32_t s_tmem;
    uint8_t* smem = align_1024(smem_raw);
    uint8_t* sQ = smem;                                   // [NQ][DK/64][128 rows][128 bytes]; codes: [NQ][2][DK/CHK][..][CHK]
    uint8_t* sK = sQ + NQ * Cfg::Q_TILE;                  // [KST][BN/8][DK/64][8 keys][128 bytes]; [KST][DK/CHK][BN][CHK]
    uint8_t* sV = sK + Cfg::KST * Cfg::K_TILE;            // [VST][BN/8][DV/64][8 keys][128 bytes]
    uint8_t* sVC = sV + Cfg::VST * Cfg::V_TILE;           // [VCST][BN keys][DV bytes]
    uint64_t* k_full = reinterpret_cast<uint64_t*>(sVC + Cfg::VCST * Cfg::VC_TILE);
    uint64_t* k_empty = k_full + Cfg::KST;
    uint64_t* v_full = k_empty + Cfg::KST;
    uint64_t* v_empty = v_full + Cfg::VST;
    uint64_t* s_full = v_empty + Cfg::VST;                // [SBUF]
    uint64_t* p_full = s_full + Cfg::SBUF;                // [SBUF]
    uint64_t* q_full = p_full + Cfg::SBUF;                // [NQ] queries of an item
    uint64_t* o_done = q_full + NQ;                       // [NQ] each product with V
    uint64_t* o_last = o_done + NQ;                       // [NQ] the last one of an item
    uint64_t* v_tail = o_last + NQ;                       // an item's last, partly valid value tile
    uint64_t* i_full = v_tail + 1;                        // [SLOTS]
    uint64_t* i_empty = i_full + Cfg::SLOTS;              // [SLOTS]
    uint64_t* drain = i_empty + Cfg::SLOTS;               // all products, when given up
    uint64_t* q_first = drain + 1;                        // the first queries, once, for the value warp
    uint64_t* vc_full = q_first + 1;                      // [VCST]
    uint64_t* vc_empty = vc_full + Cfg::VCST;             // [VCST]
    uint64_t* c_full = vc_empty + Cfg::VCST;              // [CST]

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int group = static_cast<int>(a.q_heads / a.cache.heads);

    if (threadIdx.x == 0) {
        for (int i = 0; i < Cfg::KST; ++i) {
            mbar_init(&k_full[i], 1);
            mbar_init(&k_empty[i], 1);
        }
        for (int i = 0; i < Cfg::VST; ++i) {
            mbar_init(&v_full[i], CODES ? 4 : 1);
            mbar_init(&v_empty[i], 1);
        }
        for (int i = 0; i < Cfg::SBUF; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);
        }
        for (int i = 0; i < NQ; ++i) {
            mbar_init(&q_full[i], 4);
            mbar_init(&o_done[i], 1);
            mbar_init(&o_last[i], 1);
        }
        mbar_init(v_tail, 1);
        mbar_init(drain, 1);
        mbar_init(q_first, 1);
        for (int i = 0; i < Cfg::SLOTS; ++i) {
            mbar_init(&i_full[i], 1);
            mbar_init(&i_empty[i], Cfg::READERS);
        }
        for (int i = 0; i < Cfg::VCST; ++i) {
            mbar_init(&vc_full[i], 1);
            mbar_init(&vc_empty[i], 4);
        }
        for (int i = 0; i < Cfg::CST; ++i) mbar_init(&c_full[i], 1);
        fence_barrier_init();
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }
    if (warp == Cfg::MMA_WARP) tmem_alloc(&s_tmem, Cfg::TMEM_COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    grid_dependency_wait();
    grid_launch_dependents();

    // An item's key tiles start here, and are so many.
    auto first_tile = [](const Item& it) { return it.key_lo / BN * BN; };
    auto key_tiles = [&](const Item& it) {
        return it.key_hi > it.key_lo ? (it.key_hi - first_tile(it) + BN - 1) / BN : 0;
    };
    // The x-th item of this CTA (x counts from 0), for the other warps: to be waited for, and given back.
    auto item_ready = [&](int x) { return warp_wait(&i_full[x % Cfg::SLOTS], (x / Cfg::SLOTS) & 1); };
    auto item_done = [&](int x) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&i_empty[x % Cfg::SLOTS]);
    };

    // Two query tiles, registers: 168 x 384 threads at launch; the softmax's row of S needs more, the third
    // warpgroup less (208 x 256 + 80 x 128 = 63488 of 64512). Codes: 128 x 512, then 192 x 256 + 64 x 256 = 65536;
    // one query tile and two CTAs per SM 80 x 384, then 128 x 128 + 56 x 256.
    if (warp < Cfg::SOFT_WARPS) {
        if constexpr (NQ == 2)
            regs_inc<CODES ? 192 : 208>();
        else if constexpr (CODES && Cfg::CTAS == 2)
            regs_inc<128>();
        // ---- softmax warps: thread = row of query tile q
        const int q = warp >> 2;
        const int quarter = warp & 3;
        const int r = q * 128 + quarter * 32 + lane;          // row of the item's tile
        const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
        const uint32_t o_tmem = tmem + lanes + Cfg::SBUF * BN + q * DV;
        // (a scale of zero: the smallest factor keeps -inf apart from the finite scores; one that is NaN stays so.
        // Codes: their factor is only bounded where the key's scale has joined it, as a small one may belong to large
        // keys. The maximum with zero is none; without it the compiler orders the loop below otherwise, 328 us for the
        // chunk of 4096, not 321.)
        const float c_all = max_nan(fabsf(a.scale) * 1.4426950408889634f, CODES ? 0.0f : 1e-45f);
        // Queries of query tile q into shared memory (K-major, 128-byte swizzle), valid rows only (what the
        // others hold is of no consequence: rows do not meet). A negative scale turns their signs, so that
        // the row maximum is always that of the largest S.
        // Codes: each row divided by a power of two that leaves its largest channel in [224, 448), as two codes per
        // channel; a warp loads its own rows.
        auto load_queries = [&](const Item& it) {
            const uint32_t flip = a.scale < 0.0f ? 0x80008000u : 0u;
            if constexpr (CODES) {
                constexpr int LANES = DK / 8;                        // of a row, 8 channels each
                constexpr int ROWS = LANES <= 16 ? 32 / LANES : 1;   // at a time
                constexpr int BATCH = 4;
                static_assert(32 % (ROWS * BATCH) == 0, "whole batches");
                // Wide rows: a batch on its way under the one before (32 sequences of 128 rows and 2048 keys, heads of 128
                // 63.6 -> 62 us, of 192 83 -> 79). Not where the softmax comes out slower beside it: two query tiles of 128
                // channels (the chunk of 4096 334 us instead of 318), heads of 64 (the mixed batch of 8 38.2 and 37.6).
                constexpr bool AHEAD = DK > 128 || (NQ == 1 && DK == 128);
                const int piece = lane % LANES;
                const bool has = lane < ROWS * LANES;
                auto load = [&](int r0, uint4* to) {
#pragma unroll
                    for (int i = 0; i < BATCH; ++i) {
                        const int row = q * 128 + quarter * 32 + r0 + i * ROWS + lane / LANES;
                        to[i] = make_uint4(0, 0, 0, 0);
                        if (has && row < it.rows) {
                            const int pr = it.first_row + row;
                            const int tok = pr / group;
                            to[i] = __ldg(reinterpret_cast<const uint4*>(
                                              static_cast<const __nv_bfloat16*>(a.q) +
                                              (it.q0 + tok) * a.q_token_stride +
                                              (it.head * group + pr - tok * group) * a.q_head_stride) + piece);
                        }
                    }
                };
                uint4 v[BATCH], next[BATCH];
                if (AHEAD) load(0, next);
#pragma unroll 1
                for (int r0 = 0; r0 < 32; r0 += ROWS * BATCH) {
                    if constexpr (AHEAD) {
#pragma unroll
                        for (int i = 0; i < BATCH; ++i) v[i] = next[i];
                        if (r0 + ROWS * BATCH < 32) load(r0 + ROWS * BATCH, next);
                    } else {
                        load(r0, v);
                    }
#pragma unroll
                    for (int i = 0; i < BATCH; ++i) {
                        const int in_tile = quarter * 32 + r0 + i * ROWS + lane / LANES;
                        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
                        // the largest magnitude, as bf16 bits: those of infinities and NaN are larger than all numbers'
                        uint32_t top = 0;
#pragma unroll
                        for (int k = 0; k < 4; ++k) top = __vmaxu2(top, w[k] & 0x7FFF7FFFu);
                        top = max(top & 0xFFFFu, top >> 16);
                        if constexpr (ROWS == 1) {
                            top = __reduce_max_sync(0xffffffffu, top);
                        } else {
#pragma unroll
                            for (int m = LANES / 2; m > 0; m >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, m));
                        }
                        const int e = max(2, min(static_cast<int>(top >> 7) - 8 + ((top & 0x7Fu) > 0x60u ? 1 : 0), 252));
                        const float inv = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
                        uint32_t hi[4], lo[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const uint32_t x = w[k] ^ flip;
                            two_codes(bf16_lo(x) * inv, bf16_hi(x) * inv, &hi[k], &lo[k]);
                            if (top >= 0x7F80u) hi[k] = 0x7F7Fu;     // a query that is not finite: NaN
                        }
                        if (has) {
                            const int byte = 8 * piece % Cfg::CHK;
                            uint8_t* to = sQ + q * Cfg::Q_TILE + (8 * piece / Cfg::CHK) * (128 * Cfg::CHK) +
                                          in_tile * Cfg::CHK + (swizzled(in_tile, byte >> 4, Cfg::CHK) << 4) + (byte & 15);
                            *reinterpret_cast<uint2*>(to) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
                            *reinterpret_cast<uint2*>(to + 128 * DK) =
                                make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
                            if (piece == 0) s_unit[q * 128 + in_tile] = __uint_as_float(static_cast<uint32_t>(e) << 23);
                        }
                    }
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(&q_full[q]);
                return;
            }
            constexpr int PIECES = DK / 8;                           // 16-byte pieces of a row
            constexpr int BATCH = 8;
            const int here = max(0, min(128, it.rows - q * 128));
            const int tid = threadIdx.x & 127;
#pragma unroll 1
            for (int i0 = tid; i0 < here * PIECES; i0 += 128 * BATCH) {
                uint4 v[BATCH];
#pragma unroll
                for (int i = 0; i < BATCH; ++i) {
                    const int e = i0 + i * 128;
                    const int row = e / PIECES;
                    if (row < here) {
                        const int pr = it.first_row + q * 128 + row;
                        const int tok = pr / group;
                        v[i] = __ldg(reinterpret_cast<const uint4*>(
                                         static_cast<const __nv_bfloat16*>(a.q) +
                                         (it.q0 + tok) * a.q_token_stride +
                                         (it.head * group + pr - tok * group) * a.q_head_stride) +
                                     e % PIECES);
                    }
                }
#pragma unroll
                for (int i = 0; i < BATCH; ++i) {
                    const int e = i0 + i * 128;
                    const int row = e / PIECES;
                    const int ch = e % PIECES;
                    if (row < here) {
                        v[i].x ^= flip; v[i].y ^= flip; v[i].z ^= flip; v[i].w ^= flip;
                        *reinterpret_cast<uint4*>(sQ + q * Cfg::Q_TILE + (ch >> 3) * (128 * 128) +
                                                  row * 128 + (((ch & 7) ^ (row & 7)) << 4)) = v[i];
                    }
                }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(&q_full[q]);
        };
        // An item's output rows as (token, query head).
        auto out_row = [&](const Item& it, int row) {
            const int pr = it.first_row + row;
            const int tok = pr / group;
            return (it.q0 + tok) * a.q_heads + it.head * group + (pr - tok * group);
        };
        bool ok = true;
        int n0 = 0, used = 0;
        ok = item_ready(0);
        if (ok && s_item[0].seq >= 0 && key_tiles(s_item[0]) > 0) load_queries(s_item[0]);
        for (int x = 0; ok && s_item[x % Cfg::SLOTS].seq >= 0; ++x) {
            const Item& it = s_item[x % Cfg::SLOTS];
            const int nt = key_tiles(it);
            const int k0 = first_tile(it);
            const bool live = r < it.rows;
            const bool idle = q * 128 + quarter * 32 >= it.rows;     // no valid row in this warp
            const bool whole = pieces == 1 || (CODES && it.pieces == 1);     // written here
            if (CODES && live && whole && pieces > 1)
                parts.ml[out_row(it, r)] = make_float2(0.0f, kWholeRow);
            else if (live && it.piece == 0)
                // pieces that this sequence does not have are empty
                for (int p = it.pieces; p < pieces; ++p)
                    parts.ml[p * parts.rows + out_row(it, r)] = make_float2(-INFINITY, 0.0f);
            float m = -INFINITY;           // maximum in use, raw score (codes: in log2 units, its value's scale with it)
            float l = 0.0f;
            const float c = CODES ? max_nan(c_all * s_unit[r], 0.0f) : c_all;
            if (nt > 0) {
                const KeyRange kr =
                    keys_of(a, it.n, it.kv, (it.first_row + min(r, it.rows - 1)) / group);
                // tiles that need no mask for any row of this query tile
                const int last_row = min(it.rows, (q + 1) * 128) - 1;
                const int full_hi = min(it.key_hi,
                    keys_of(a, it.n, it.kv, (it.first_row + min(q * 128, it.rows - 1)) / group).hi);
                const int full_lo = max(it.key_lo,
                    keys_of(a, it.n, it.kv, (it.first_row + max(last_row, 0)) / group).lo);
                const int row_lo = max(kr.lo, it.key_lo), row_hi = min(kr.hi, it.key_hi);
                bool far = false;
                int j = 0;
                for (; j < nt; ++j) {
                    const int n = n0 + j;
                    const int buf = NQ == 2 ? q : n & 1;
                    const uint32_t sph = NQ == 2 ? n & 1 : (n >> 1) & 1;
                    if constexpr (CODES) {
                        if (!warp_wait(&c_full[n % Cfg::CST], (n / Cfg::CST) & 1)) {
                            ok = false;
                            break;
                        }
                    }
                    // (of 16 keys each, on hand before the scores are: a factor that keeps -inf apart even where the
                    // score's is next to nothing; log2 vs; 1 / vs)
                    float ck[CODES ? BN / 16 : 1], lv[CODES ? BN / 16 : 1], iv[CODES ? BN / 16 : 1];
                    if constexpr (CODES)
#pragma unroll
                        for (int g = 0; g < BN / 16; ++g) {
                            const float4 sc = s_scale[n % Cfg::CST][g];
                            ck[g] = max_nan(c * sc.x, 1.2e-38f), lv[g] = sc.y, iv[g] = sc.z;
                        }
                    if (!warp_wait(&s_full[buf], sph)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    if (!idle) {
                        const uint32_t s_tmem_row = tmem + lanes + buf * BN;
                        const int kb = k0 + j * BN;
                        const bool masked = kb < full_lo || kb + BN > full_hi;
                        uint32_t p[BN / 2];
                        float2 sum[2];
                        if constexpr (CODES) {
                            // 32 scores at a time, the next ones on their way meanwhile: with all of a row in registers
                            // the softmax warps would need more than four warpgroups leave them.
                            auto load_block = [&](int i, float* s) { tmem_ld_32cols(s_tmem_row + 32 * i, s); };
                            auto mask_block = [&](int i, float* s) {
                                if (masked) {
                                    const int lo = row_lo - kb - 32 * i, hi = row_hi - kb - 32 * i;
#pragma unroll
                                    for (int k = 0; k < 32; ++k)
                                        if (k < lo || k >= hi) s[k] = -INFINITY;
                                }
                            };
                            auto probabilities = [&]() {
                                const float ref = m == -INFINITY ? 0.0f : m;
                                float total = 0.0f, size = 0.0f;
                                float s[2][32];
                                load_block(0, s[0]);
#pragma unroll
                                for (int i = 0; i < BN / 32; ++i) {
                                    tmem_wait_ld_32(s[i & 1]);
                                    if (i + 1 < BN / 32) load_block(i + 1, s[(i + 1) & 1]);
                                    float* now = s[i & 1];
                                    mask_block(i, now);
#pragma unroll
                                    for (int g = 0; g < 2; ++g) {            // 16 keys of one scale
                                        const float off = lv[2 * i + g] - ref;
                                        const float2 c2 = make_float2(ck[2 * i + g], ck[2 * i + g]);
                                        const float2 off2 = make_float2(off, off);
                                        sum[0] = sum[1] = make_float2(0.0f, 0.0f);
#pragma unroll
                                        for (int k = 0; k < 8; ++k) {
                                            const float2 z = make_float2(now[16 * g + 2 * k], now[16 * g + 2 * k + 1]);
                                            float2 y = __ffma2_rn(z, c2, off2);
                                            y.x = exp2_fast(y.x);
                                            y.y = exp2_fast(y.y);
                                            sum[k & 1] = __fadd2_rn(sum[k & 1], y);
                                            p[16 * i + 8 * g + k] = pack_half2(y.x, y.y);
                                        }
                                        const float2 both = __fadd2_rn(sum[0], sum[1]);
                                        total = fmaf(both.x + both.y, iv[2 * i + g], total);
                                        size += both.x + both.y;
                                    }
                                }
                                sum[0] = make_float2(total, 0.0f);
                                sum[1] = make_float2(0.0f, 0.0f);
                                return size;
                            };
                            // The maximum is not looked for where it is not needed: probabilities above 1 are as good as
                            // others until their sum says that one may be past 2^15, of the 2^16 that binary16 holds. A warp
                            // looks for all of its rows, and a new reference is four times the largest so far, so that
                            // looks are few (a row at a time: the chunk of 4096 332 us instead of 317).
                            bool look = j == 0 || __any_sync(0xffffffffu, m == -INFINITY);
                            if (!look) look = __any_sync(0xffffffffu, probabilities() > 32768.0f);
                            if (look) {
                                float top = -INFINITY;
#pragma unroll 1
                                for (int i = 0; i < BN / 32; ++i) {
                                    float s[32];
                                    load_block(i, s);
                                    tmem_wait_ld_32(s);
                                    mask_block(i, s);
#pragma unroll
                                    for (int g = 0; g < 2; ++g) {
                                        float of16[2] = {s[16 * g], s[16 * g + 1]};
#pragma unroll
                                        for (int k = 2; k < 16; ++k) of16[k & 1] = fmaxf(of16[k & 1], s[16 * g + k]);
                                        const float4 sc = s_scale[n % Cfg::CST][2 * i + g];
                                        top = fmaxf(top, fmaf(fmaxf(of16[0], of16[1]), max_nan(c * sc.x, 1.2e-38f), sc.y));
                                    }
                                }
                                const bool grow = top > m;
                                const bool any_grows = __any_sync(0xffffffffu, grow);
                                if (any_grows) {
                                    far = __any_sync(0xffffffffu, grow && fabsf(top) >= kFar<true>);
                                    if (far) break;
                                }
                                const float keep = grow ? exp2_fast(m - top - 2.0f) : 1.0f;
                                if (grow) m = top + 2.0f;
                                l *= keep;
                                // (scores that are not numbers: the sum says so, any reference will do)
                                const float found = probabilities();
                                if (found != found && m == -INFINITY) m = 0.0f;
                                if (j > 0 && any_grows) {
                                    if (!warp_wait(&o_done[q], (n - 1) & 1)) {
                                        ok = false;
                                        break;
                                    }
                                    tc_fence_after();
                                    scale_columns<DV>(o_tmem, keep);
                                }
                            }
                        } else {
                            auto load_row = [&](float* s) {
#pragma unroll
                                for (int i = 0; i < BN / 32; ++i) tmem_ld_32cols(s_tmem_row + 32 * i, s + 32 * i);
#pragma unroll
                                for (int i = 0; i < BN / 32; ++i) tmem_wait_ld_32(s + 32 * i);
                                if (masked) {
                                    const int lo = row_lo - kb, hi = row_hi - kb;
#pragma unroll
                                    for (int i = 0; i < BN; ++i)
                                        if (i < lo || i >= hi) s[i] = -INFINITY;
                                }
                            };
                            // Probabilities with the maximum in use, and this tile's maximum beside them: it is only
                            // looked at afterwards, and hardly ever asks for another pass (kRescale). The first tile
                            // of a row has no maximum yet and looks before; so does the form with one query tile,
                            // whose softmax waits for the keys (64 ragged sequences: 192 us, 204 the other way; the
                            // chunk of 4096 with two tiles: 321 and 313).
                            float top = m;
                            auto probabilities = [&](const float* s) {
                                const float mc = m == -INFINITY ? 0.0f : m * c;
                                const float2 c2 = make_float2(c, c), mc2 = make_float2(-mc, -mc);
                                sum[0] = sum[1] = make_float2(0.0f, 0.0f);
                                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                                for (int k = 0; k < BN / 2; ++k) {
                                    mx[k & 3] = fmaxf(mx[k & 3], fmaxf(s[2 * k], s[2 * k + 1]));
                                    float2 y = __ffma2_rn(make_float2(s[2 * k], s[2 * k + 1]), c2, mc2);
                                    y.x = exp2_fast(y.x);
                                    y.y = exp2_fast(y.y);
                                    sum[k & 1] = __fadd2_rn(sum[k & 1], y);
                                    p[k] = pack_bf16x2(y.x, y.y);
                                }
                                top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                            };
                            bool look = NQ == 1 || j == 0 || __any_sync(0xffffffffu, m == -INFINITY);
                            if (!look) {
                                float s[BN];
                                load_row(s);
                                probabilities(s);
                                look = __any_sync(0xffffffffu, (top - m) * c > kRescale);
                            }
                            if (look) {
                                float s[BN];
                                load_row(s);
                                float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                                for (int i = 4; i < BN; ++i) mx[i & 3] = fmaxf(mx[i & 3], s[i]);
                                top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                                const bool grow = (top - m) * c > kRescale || (m == -INFINITY && top > m);
                                const bool any_grows = __any_sync(0xffffffffu, grow);
                                if (any_grows) {
                                    // (the rows behind the last hold whatever stood in memory)
                                    far = __any_sync(0xffffffffu, grow && live && fabsf(top * c) >= kFar<false>);
                                    if (far) break;
                                }
                                const float keep = grow ? exp2_fast((m - top) * c) : 1.0f;
                                if (grow) m = top;
                                l *= keep;
                                probabilities(s);
                                if (j > 0 && any_grows) {
                                    if (!warp_wait(&o_done[q], (n - 1) & 1)) {
                                        ok = false;
                                        break;
                                    }
                                    tc_fence_after();
                                    scale_columns<DV>(o_tmem, keep);
                                }
                            }
                        }
#pragma unroll
                        for (int i = 0; i < BN / 32; ++i) tmem_st_16cols(s_tmem_row + 16 * i, p + 16 * i);
                        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                        tmem_wait_st();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&p_full[buf]);
                    } else if (lane == 0) {
                        mbar_arrive(&p_full[buf]);
                    }
                }
                if (far) {
                    const FarRows f = far_tiles<Cfg>(tmem + lanes, o_tmem, q, c, s_scale[0], c_full, s_full, p_full,
                                                     &o_done[q], n0, j, nt, row_lo - k0, row_hi - k0, m, l, lane);
                    m = f.m, l = f.l, ok = f.ok;
                }
                n0 += nt;
            }
            // The next item's queries: every S of this one has been computed (this warp has seen the last),
            // so their place is free, and the next S can be computed while this O is written out.
            if (ok) ok = item_ready(x + 1);
            const Item& next = s_item[(x + 1) % Cfg::SLOTS];
            if (ok && next.seq >= 0 && key_tiles(next) > 0) load_queries(next);
            if (nt > 0) {
                if (ok && !warp_wait(&o_last[q], used & 1)) ok = false;
                ++used;
                tc_fence_after();
            }
            if (ok && !idle) {
                const int64_t row = live ? out_row(it, r) : 0;
                const float mc = m == -INFINITY ? -INFINITY : CODES ? m : m * c;
                const float inv = l == 0.0f ? 0.0f : 1.0f / l;       // (NaN stays NaN)
                if (!whole) {
                    float* dst = parts.o + (it.piece * parts.rows + row) * DV;
                    if (nt > 0)
#pragma unroll
                        for (int i = 0; i < DV / 32; ++i) {
                            float o[32];
                            tmem_ld_32cols(o_tmem + 32 * i, o);
                            tmem_wait_ld_32(o);
                            if (live)
#pragma unroll
                                for (int k = 0; k < 8; ++k)
                                    *reinterpret_cast<float4*>(dst + 32 * i + 4 * k) =
                                        make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
                        }
                    if (live) parts.ml[it.piece * parts.rows + row] = make_float2(mc, l);
                } else {
                    uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + row * DV);
#pragma unroll
                    for (int i = 0; i < DV / 32; ++i) {
                        float o[32];
                        if (nt > 0) {
                            tmem_ld_32cols(o_tmem + 32 * i, o);
                            tmem_wait_ld_32(o);
                        } else {
#pragma unroll
                            for (int k = 0; k < 32; ++k) o[k] = 0.0f;
                        }
                        if (live)
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                dst[4 * i + k] = make_uint4(
                                    pack_bf16x2(o[8 * k] * inv, o[8 * k + 1] * inv),
                                    pack_bf16x2(o[8 * k + 2] * inv, o[8 * k + 3] * inv),
                                    pack_bf16x2(o[8 * k + 4] * inv, o[8 * k + 5] * inv),
                                    pack_bf16x2(o[8 * k + 6] * inv, o[8 * k + 7] * inv));
                    }
                    if (live && a.lse)
                        a.lse[row] = l == 0.0f ? -INFINITY : (mc + log2_fast(l)) * 0.6931471805599453f;
                }
            }
            tc_fence_before();
            item_done(x);
        }
        if (!ok && lane == 0) record_error(FP8BS_DEVERR_EPILOGUE_WAIT);
    } else {
        if constexpr (NQ == 2)
            regs_dec<CODES ? 64 : 80>();
        else if constexpr (CODES && Cfg::CTAS == 2)
            regs_dec<56>();
        if (warp == Cfg::KEY_WARP) {
            // ---- hands out the items and brings their keys
            // (codes: two sequences a lane, so that the first item is on hand sooner: a mixed batch of 8 62 -> 59 us)
            ItemFinder<CODES ? 2 : 8> finder;
            finder.base = finder.before = 0;
            finder.loaded = false;
            bool ok = true;
            Stream ks = {0, 0};
            int x = 0;
            // The items are dealt out in rounds, every other one backwards: long items and short ones even out. Where
            // the last round is not whole, some CTAs have an item more than the others. Of one sequence, whose
            // items come longest first, those are dealt the short ones (a chunk of 4096 over 8192 keys: 169 key tiles
            // for the busiest CTA instead of 182, 282 us instead of 315); in a batch they may be any. (Two query
            // tiles only: few rows mean pieces of one length, and a batch of 9 us takes 0.3 more with it.)
            int ctas = gridDim.x, mine = blockIdx.x, start = 0, rounds = INT32_MAX;
            if (NQ == 2 && __builtin_expect(a.B == 1, 0)) {
                load_sequences<CODES>(finder, a, Cfg::ROWS, piece_len, lane, more_rows);
                const int items = __shfl_sync(0xffffffffu, finder.incl, 31) * static_cast<int>(a.cache.heads);
                const int whole = items / ctas, more = items % ctas;
                if (mine < ctas - more) {
                    ctas -= more;
                    rounds = whole;
                } else {
                    mine -= ctas - more;
                    start = (ctas - more) * whole;
                    ctas = more;
                    rounds = whole + 1;
                }
            }
            for (int round = 0; ok; ++round) {
                const int64_t at = round < rounds ? start + static_cast<int64_t>(round) * ctas +
                                                        (round & 1 ? ctas - 1 - mine : mine)
                                                  : int64_t{INT32_MAX};
                const Item it = find_item<CODES>(finder, a, static_cast<int>(min(at, int64_t{INT32_MAX})), Cfg::ROWS,
                                          BN, piece_len, lane, more_rows);
                if (it.seq == -2) {
                    if (lane == 0) record_error(FP8BS_DEVERR_INDEX);
                    continue;
                }
                if (!warp_wait(&i_empty[x % Cfg::SLOTS], ((x / Cfg::SLOTS) & 1) ^ 1)) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    s_item[x % Cfg::SLOTS] = it;
                    mbar_arrive(&i_full[x % Cfg::SLOTS]);
                }
                __syncwarp();
                ++x;
                if (it.seq < 0) break;
                const int nt = key_tiles(it);
                if (nt == 0) continue;
                if constexpr (CODES) {
                    ok = bring_codes<Cfg::KST, DK, Cfg::CHK, BN, true>(
                        ks, &tmK, a, scales, it, first_tile(it), nt, modes.box_log2, sK, k_full, k_empty,
                        nullptr, lane, warp_wait, [&](int, int tile, int first, float2 f) {
                            const int cs = tile % Cfg::CST;
                            const int from = (first + (lane * 16 >> modes.box_log2)) & 31;
                            const float k1 = __shfl_sync(0xffffffffu, f.x, from), v1 = __shfl_sync(0xffffffffu, f.y, from);
                            const float lv = static_cast<float>(static_cast<int>(__float_as_uint(v1) >> 23) - 127);
                            if (lane < BN / 16) s_scale[cs][lane] = make_float4(k1, lv, exp2_fast(-lv), 0.0f);
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&c_full[cs]);
                        });
                    continue;
                }
                // (the first queries come first: behind a full ring of keys they take several times as long)
                ok = bring_tiles<Cfg, true>(ks, &tmK, a, it, first_tile(it), nt, modes.box_log2, modes.k, sK,
                                            k_full, k_empty, nullptr, s_window[0], lane, [&] {
                                                for (int q = 0; q < NQ; ++q)
                                                    if (!warp_wait(&q_full[q], 0)) return false;
                                                if (lane == 0) mbar_arrive(q_first);
                                                return true;
                                            });
            }
            if (!ok && lane == 0) drain_tiles<Cfg::KST>(ks, k_full);
        } else if (warp == Cfg::VALUE_WARP) {
            // ---- brings the items' values
            bool ok = true;
            Stream vs = {0, 0};
            for (int x = 0; ok; ++x) {
                ok = item_ready(x);
                if (!ok) break;
                const Item it = s_item[x % Cfg::SLOTS];
                item_done(x);
                if (it.seq < 0) break;
                const int nt = key_tiles(it);
                if (nt == 0) continue;
                if constexpr (CODES) {
                    ok = bring_codes<Cfg::VCST, DV, DV, BN, false>(
                        vs, &tmV, a, Scales{nullptr, nullptr}, it, first_tile(it), nt, modes.box_log2, sVC, vc_full,
                        vc_empty, nullptr, lane, warp_wait, [](int, int, int, float2) {});
                    continue;
                }
                ok = bring_tiles<Cfg, false>(vs, &tmV, a, it, first_tile(it), nt, modes.box_log2, modes.v, sV,
                                             v_full, v_empty, v_tail, s_window[1], lane,
                                             [&] { return warp_wait(q_first, 0); });
            }
            if (!ok && lane == 0) {
                if constexpr (CODES) {
                    drain_tiles<Cfg::VCST>(vs, vc_full);
                } else {
                    drain_tiles<Cfg::VST>(vs, v_full);
                    mbar_wait(v_tail, vs.tails & 1, kDrainLimitNs);
                }
            }
        } else if (CODES && warp >= Cfg::WIDEN_WARP) {
            if constexpr (CODES)
                widen_values<Cfg>(s_item, sVC, sV, vc_full, vc_empty, v_full, v_empty, i_full, i_empty,
                                  warp - Cfg::WIDEN_WARP, lane);
        } else if (warp == Cfg::MMA_WARP) {
            // ---- MMA issuer. Per key tile and query tile: O += P(j) V(j), then S of the tile's next keys, which
            // takes P's place (the tensor core works in order).
            // With two query tiles one's products run under the other's softmax.
            constexpr uint32_t idesc_qk = CODES ? idesc_e4m3_f32(128, BN) : idesc_bf16_f32(128, BN);
            // (codes: P and V in binary16, whose format is the descriptor's zero)
            constexpr uint32_t idesc_pv =
                (idesc_bf16_f32(128, DV) & ~(CODES ? 1u << 7 | 1u << 10 : 0u)) | kIdescBMajorMN;
            // descriptors of the first stages; those of other stages and steps lie at constant distances (in
            // units of 16 bytes, which do not carry out of the address field)
            const uint64_t q_desc =
                CODES ? smem_desc_rows(smem_addr(sQ), Cfg::CHK) : smem_desc_k_sw128(smem_addr(sQ));
            const uint64_t k_desc = CODES ? smem_desc_rows(smem_addr(sK), Cfg::CHK)
                                          : smem_desc_groups(smem_addr(sK), DK / 64 * 1024);
            const uint64_t v_desc = smem_desc_groups(smem_addr(sV), DV / 64 * 1024);
            const uint32_t o_tmem = tmem + Cfg::SBUF * BN;
            bool ok = true;
            int n0 = 0;                        // key tiles of the items before
            int used = 0;                      // items with keys before
            // S(n): buffer q (two tiles) or n % 2, keys of tile n
            auto qk = [&](int q, int n) {
                const int st = n % Cfg::KST;
                if (q == 0) {
                    if (!warp_wait(&k_full[st], (n / Cfg::KST) & 1)) return false;
                    tc_fence_after();
                }
                const int buf = NQ == 2 ? q : n & 1;
                const uint64_t kd = k_desc + static_cast<uint32_t>(st * (Cfg::K_TILE / 16));
                if (elect_one()) {
                    if constexpr (CODES) {
#pragma unroll
                        for (int d = 0; d < DK / 16; ++d) {          // (both codes of each channel)
                            const int in = 32 * d % DK, part = 32 * d / DK;
                            mma_f8(tmem + buf * BN,
                                   q_desc + (q * Cfg::Q_TILE + part * (128 * DK) + (in / Cfg::CHK) * (128 * Cfg::CHK) +
                                             in % Cfg::CHK) / 16,
                                   kd + ((in / Cfg::CHK) * (BN * Cfg::CHK) + in % Cfg::CHK) / 16, idesc_qk, d > 0 ? 1u : 0u);
                        }
                    } else {
#pragma unroll
                        for (int d = 0; d < DK / 16; ++d)
                            mma_bf16(tmem + buf * BN,
                                     q_desc + (q * Cfg::Q_TILE + (d / 4) * (128 * 128) + (d % 4) * 32) / 16,
                                     kd + ((d / 4) * 1024 + (d % 4) * 32) / 16, idesc_qk, d > 0 ? 1u : 0u);
                    }
                    mma_commit(&s_full[buf]);
                    if (q == NQ - 1) mma_commit(&k_empty[st]);
                }
                __syncwarp();
                return true;
            };
            for (int x = 0; ok; ++x) {
                if (!item_ready(x)) {
                    ok = false;
                    break;
                }
                const int seq = s_item[x % Cfg::SLOTS].seq;
                const int nt = __shfl_sync(0xffffffffu, key_tiles(s_item[x % Cfg::SLOTS]), 0);
                item_done(x);
                if (seq < 0) break;
                if (nt == 0) continue;
                for (int q = 0; ok && q < NQ; ++q)
                    ok = warp_wait(&q_full[q], used & 1) && qk(q, n0);
                if (ok && NQ == 1 && nt > 1) ok = qk(0, n0 + 1);
                for (int j = 0; ok && j < nt; ++j) {
                    const int n = n0 + j;
                    const int st = n % Cfg::VST;
                    const uint32_t pph = NQ == 2 ? n & 1 : (n >> 1) & 1;
                    const uint64_t vd = v_desc + static_cast<uint32_t>(st * (Cfg::V_TILE / 16));
                    if (!warp_wait(&v_full[st], (n / Cfg::VST) & 1)) {
                        ok = false;
                        break;
                    }
#pragma unroll
                    for (int q = 0; q < NQ; ++q) {
                        const int buf = NQ == 2 ? q : n & 1;
                        if (!warp_wait(&p_full[buf], pph)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        if (elect_one()) {
#pragma unroll
                            for (int k = 0; k < BN / 16; ++k)
                                mma_bf16_ta(o_tmem + q * DV, tmem + buf * BN + 8 * k,
                                            vd + k * (DV / 64 * 2048 / 16), idesc_pv,
                                            j > 0 || k > 0 ? 1u : 0u);
                            mma_commit(&o_done[q]);
                            if (q == NQ - 1) mma_commit(&v_empty[st]);
                            if (j == nt - 1) mma_commit(&o_last[q]);
                        }
                        __syncwarp();
                        const int next = NQ == 2 ? j + 1 : j + 2;
                        if (next < nt) ok = qk(q, n0 + next);
                    }
                }
                n0 += nt;
                ++used;
            }
            if (!ok) {
                // abandoned: the products in flight still read shared memory; let them end
                if (lane == 0) record_error(FP8BS_DEVERR_MMA_WAIT);
                if (elect_one()) mma_commit(drain);
                __syncwarp();
                if (!warp_wait(drain, 0) && lane == 0) record_error(FP8BS_DEVERR_DRAIN_WAIT);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == Cfg::MMA_WARP) tmem_dealloc(tmem, Cfg::TMEM_COLS);
}

}  // namespace
}  // namespace fp8bs
