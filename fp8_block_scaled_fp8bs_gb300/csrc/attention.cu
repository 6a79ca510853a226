// attention.cu -- attention of new tokens over a paged cache (fp8bs_paged_attention).
//
// The query rows of one sequence that share a key head (token i, head g of the group: row i*G + g)
// are packed into tiles of 128, one MMA row and TMEM lane each, so that a single token of a grouped
// head still reads its keys once and a chunk fills the tensor core. Per key tile of BN keys:
//   S = Q K^T      tcgen05.mma, bf16, Q and K K-major in shared memory, S fp32 in TMEM
//   P = exp2(c S - m), m the running row maximum: one thread per row, S from TMEM, P as bf16 back
//                  into TMEM in place of S
//   O += P V       tcgen05.mma, P from TMEM, V from shared memory as the cache holds it (keys
//                  outermost: an MN-major operand), O fp32 in TMEM
// The maximum only moves when it has grown by more than 2^8 (kRescale): the tile's probabilities are then
// computed again and O is scaled in TMEM by its softmax warps; otherwise P is that much larger than 1 at most,
// which bf16 and fp32 hold without loss, and O is left alone. So no row waits for its maximum. The row sum is
// taken from P before its rounding to bf16, so lse is exact to binary32; the rounding of P (2^-9 on average per
// term) is of the size of the output's own.
// A row without keys is one whose sum is zero. A score that is not a number, or +infinite, makes the sum NaN (the
// maximum passes over NaN), and with it the row, in one piece or in many.
//
// Two forms (AttnCfg): NQ = 2 query tiles per CTA for chunks, whose softmax warps work on one tile
// while the tensor core works on the other; NQ = 1 with two S buffers for few rows.
//
// Chunks are bound by the tensor core and what feeds it: 4096 new tokens over 8192 keys, 32 query and 8 key heads
// of 128 channels, 412 GFLOP that count, take 282 us = 1.46 PFLOP/s (0.75 of a library product's rate; 298 us where the
// inputs come from HBM in every call). The tensor pipe is busy for 61 % of an SM's cycles and waits for the softmax the rest: a row of S is 128 exponentials, and
// the products with K, whose operands both come from shared memory, run at 80 instead of 64 cycles. Heads of 192 + 128
// channels take tiles of 96 keys (128 would leave room for one tile of values: 59 us instead of 56 for 2 chunks of
// 777 over 2500 keys, 16 heads).
// Decoding is bound by HBM: 64 ragged sequences of up to 8192 keys, 64 query and 8 key heads, 1.1 GB of keys and
// values, take 193 us = 5.7 TB/s (0.86 of a copy's rate); one sequence of 32785 keys takes 32 us for 134 MB, of
// which launch, first keys and join are 12.
//
// Keys and values come through TMA in boxes of as many slots as divide both the page and the tile, all
// channels of a box at once where the cache's strides allow it.
// Few rows and long keys: the key axis is cut into pieces (AttentionPlan), each CTA leaves its
// unnormalised O, maximum and sum, and a second kernel joins them in key order.
#include <algorithm>

#include "gemm_common.cuh"
#include "quant_math.cuh"

namespace fp8bs {

namespace {

constexpr float kRescale = 8.0f;

template <int DK_, int DV_, int NQ_>
struct AttnCfg {
    static constexpr int DK = DK_, DV = DV_, NQ = NQ_;
    // Keys per tile. (192-wide keys: 96, so that two tiles of values fit.)
    static constexpr int BN = NQ == 1 ? 64 : DK <= 128 ? 128 : 96;
    static constexpr int ROWS = NQ * 128;
    static constexpr int SLOTS = 4;                              // ring of work items
    static constexpr int SBUF = 2;                               // S buffers: per query tile, or 2
    static constexpr int K_TILE = BN * DK * 2, V_TILE = BN * DV * 2, Q_TILE = 128 * DK * 2;
    // One query tile of 64 channels: two CTAs per SM, one's softmax under the other's (a windowed mixed batch 32 ->
    // 25 us, decode of 64 sequences of 4096 keys 153 -> 109).
    static constexpr int CTAS = NQ == 1 && DK == 64 ? 2 : 1;
    static constexpr int KST = DK == 64 ? (NQ == 2 ? 4 : 5) : DK == 128 ? (NQ == 2 ? 3 : 6) : (NQ == 2 ? 2 : 4);
    static constexpr int VST = DK == 64 ? (NQ == 2 ? 4 : 5) : DK == 128 ? (NQ == 2 ? 2 : 5) : (NQ == 2 ? 2 : 4);
    static constexpr int SOFT_WARPS = 4 * NQ;
    static constexpr int KEY_WARP = SOFT_WARPS;                  // brings the keys (and hands out the items)
    static constexpr int VALUE_WARP = SOFT_WARPS + 1;
    static constexpr int MMA_WARP = SOFT_WARPS + 2;
    // (two query tiles: a whole third warpgroup beside the softmax's, for the split of registers below)
    static constexpr int THREADS = 32 * (SOFT_WARPS + (NQ == 2 ? 4 : 3));
    static constexpr uint32_t TMEM_COLS = tmem_cols_for(SBUF * BN + NQ * DV);
    static constexpr int BARS = 2 * KST + 2 * VST + 2 * SBUF + 3 * NQ + 3 + 2 * SLOTS;
    static constexpr int SMEM = 1024 + NQ * Q_TILE + KST * K_TILE + VST * V_TILE + BARS * 8 + 64;
    static_assert(SMEM <= kSmemLimit, "shared memory");
};

// A work item: a tile of packed rows (i * G + g) of one sequence and key head, and one piece of its keys.
struct Item {
    int seq;               // -1: no more items; -2: a sequence out of bounds, to be passed over
    int n, q0, kv;         // its new tokens, first query token and keys
    int first_row, rows;   // first packed row and valid rows of the tile
    int head, piece, pieces;   // key head; piece of the keys, of so many
    int key_lo, key_hi;    // keys of the piece that any row attends
};

// Keys [lo, hi) that the i-th new token attends.
struct KeyRange {
    int lo, hi;
};

__device__ __forceinline__ KeyRange keys_of(const fp8bs_paged_attention_args& a, int n, int kv, int i) {
    const int64_t last = static_cast<int64_t>(kv) - n + i;
    KeyRange r;
    r.hi = a.causal ? static_cast<int>(min(static_cast<int64_t>(kv), max(last + 1, int64_t{0}))) : kv;
    r.lo = a.window > 0 ? static_cast<int>(min(static_cast<int64_t>(kv), max(last - a.window + 1, int64_t{0}))) : 0;
    return r;
}

// Most keys that the rows of one tile attend, counted from the start of a key tile: what the pieces of a
// sequence with n new tokens and kv keys are cut from. It grows with n and kv, so that the host's bounds give
// a bound of it.
__host__ __device__ inline int64_t key_span(const fp8bs_paged_attention_args& a, int rows, int64_t n,
                                            int64_t kv) {
    if (a.window == 0) return kv;
    const int64_t tokens = rows / (a.q_heads / a.cache.heads) + 2;
    const int64_t span = a.window + (a.causal && tokens < n ? tokens : n) + 128;
    return span < kv ? span : kv;
}

// The work items in order, for one warp: sequences in order, in each the row tiles from the last (whose keys
// are the most) to the first, for each tile its pieces, for each piece the key heads (which read the same
// slots). Calls ask for rising items; the sequences are read 256 at a time, eight per lane.
struct ItemFinder {
    int base, before;       // first sequence of the chunk in hand, units (items / heads) before it
    int start[9], kv[8];    // lane's sequences: first query tokens (and the next one's), keys
    int units[8];           // of each
    int incl, sum;          // of the chunk up to and with this lane, of this lane
    bool loaded;
};

struct Cut {
    int tiles, pieces;
};

__device__ __forceinline__ Cut cut_of(const fp8bs_paged_attention_args& a, int rows, int piece_len, int n, int kv,
                                      int group) {
    Cut c;
    c.tiles = (n * group + rows - 1) / rows;
    const unsigned span = static_cast<unsigned>(key_span(a, rows, n, max(kv, 0)));
    c.pieces = span > piece_len ? static_cast<int>((span + piece_len - 1) / piece_len) : 1;
    return c;
}

__device__ __forceinline__ void load_sequences(ItemFinder& f, const fp8bs_paged_attention_args& a, int rows,
                                               int piece_len, int lane) {
    const int group = static_cast<int>(a.q_heads / a.cache.heads);
    f.sum = 0;
#pragma unroll
    for (int i = 0; i < 9; ++i) {
        const int64_t b = f.base + 8 * lane + i;
        f.start[i] = a.q_start[b < a.B ? b : a.B];
        if (i < 8) f.kv[i] = b < a.B ? a.kv_len[b] : 0;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int n = f.start[i + 1] - f.start[i];
        f.units[i] = 0;
        if (n > a.max_q_len || f.kv[i] > a.max_kv_len) {
            f.units[i] = 1;      // out of bounds: handed out once, to be reported
        } else if (n > 0) {
            const Cut c = cut_of(a, rows, piece_len, n, f.kv[i], group);
            f.units[i] = c.tiles * c.pieces;
        }
        f.sum += f.units[i];
    }
    f.incl = f.sum;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, f.incl, m);
        if (lane >= m) f.incl += o;
    }
    f.loaded = true;
}

__device__ __forceinline__ Item find_item(ItemFinder& f, const fp8bs_paged_attention_args& a, int item, int rows,
                                          int bn, int piece_len, int lane) {
    Item it;
    it.seq = -1;
    const int heads = static_cast<int>(a.cache.heads);
    const int group = static_cast<int>(a.q_heads / a.cache.heads);
    const int unit = item / heads;
    it.head = item - unit * heads;
    while (f.base < a.B) {
        if (!f.loaded) load_sequences(f, a, rows, piece_len, lane);
        const unsigned hit = __ballot_sync(0xffffffffu, f.before + f.incl > unit);
        if (hit) {
            const int src = __ffs(hit) - 1;
            int seq = 0, n = 0, q0 = 0, kv = 0, tile = 0, piece = 0, pieces = 1;
            if (lane == src) {
                int left = unit - f.before - (f.incl - f.sum);
                int mine = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (left >= 0 && left < f.units[i]) {
                        seq = f.base + 8 * lane + i;
                        n = f.start[i + 1] - f.start[i];
                        q0 = f.start[i];
                        kv = f.kv[i];
                        mine = left;
                    }
                    left -= f.units[i];
                }
                const Cut c = cut_of(a, rows, piece_len, n, kv, group);
                pieces = c.pieces;
                tile = c.tiles - 1 - mine / c.pieces;
                piece = mine % c.pieces;
            }
            it.seq = __shfl_sync(0xffffffffu, seq, src);
            it.n = __shfl_sync(0xffffffffu, n, src);
            it.q0 = __shfl_sync(0xffffffffu, q0, src);
            it.kv = __shfl_sync(0xffffffffu, kv, src);
            it.first_row = __shfl_sync(0xffffffffu, tile, src) * rows;
            it.piece = __shfl_sync(0xffffffffu, piece, src);
            it.pieces = __shfl_sync(0xffffffffu, pieces, src);
            if (it.n > a.max_q_len || it.kv > a.max_kv_len || it.kv < 0 || it.q0 < 0 ||
                it.q0 + static_cast<int64_t>(it.n) > a.T) {
                it.seq = -2;
                return it;
            }
            it.rows = min(rows, it.n * group - it.first_row);
            const int lo = keys_of(a, it.n, it.kv, it.first_row / group).lo;
            const int hi = keys_of(a, it.n, it.kv, (it.first_row + it.rows - 1) / group).hi;
            const int64_t p0 = lo / bn * bn + static_cast<int64_t>(it.piece) * piece_len;
            it.key_lo = static_cast<int>(max(static_cast<int64_t>(lo), p0));
            it.key_hi = static_cast<int>(min(static_cast<int64_t>(hi), p0 + piece_len));
            return it;
        }
        f.before += __shfl_sync(0xffffffffu, f.incl, 31);
        f.base += 256;
        f.loaded = false;
    }
    return it;
}

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float log2_fast(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The larger one, or NaN if either is. (The same by comparison and selection cost the chunk of 4096 1.3 %.)
__device__ __forceinline__ float max_nan(float x, float y) {
    float z;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(z) : "f"(x), "f"(y));
    return z;
}

__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ void tma_load_4d(uint32_t smem_dst, const CUtensorMap* map, uint64_t* bar,
                                            int32_t c0, int32_t c1, int32_t c2, int32_t c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_addr(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
}

__device__ __forceinline__ void tma_load_5d(uint32_t smem_dst, const CUtensorMap* map, uint64_t* bar,
                                            int32_t c0, int32_t c1, int32_t c2, int32_t c3, int32_t c4) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(smem_dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_addr(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
        : "memory");
}

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

struct AttnParts {
    float* o;      // [piece][T * q_heads][DV], unnormalised
    float2* ml;    // [piece][T * q_heads]: (maximum in log2 units, sum); a sum of zero: no keys, o not written
    int64_t rows;  // T * q_heads
};

// One warp's state in bringing keys or values.
struct Stream {
    int n;         // tiles so far, over all items
    int tails;     // partly valid value tiles so far
};

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

// After a wait that ran out: the copies of the ring's last tiles, so that none is still writing shared memory
// when the CTA ends.
template <int STAGES>
__device__ __forceinline__ void drain_tiles(const Stream& s, uint64_t* full) {
    record_error(FP8BS_DEVERR_PRODUCER_WAIT);
    for (int i = max(0, s.n - STAGES); i < s.n; ++i)
        if (!mbar_wait(&full[i % STAGES], (i / STAGES) & 1, kDrainLimitNs)) record_error(FP8BS_DEVERR_DRAIN_WAIT);
}

template <class Cfg>
__global__ void __launch_bounds__(Cfg::THREADS, Cfg::CTAS)
    paged_attention_kernel(const __grid_constant__ CUtensorMap tmK,
                           const __grid_constant__ CUtensorMap tmV,
                           const __grid_constant__ fp8bs_paged_attention_args a,
                           const AttentionModes modes, const int piece_len, const int pieces, const AttnParts parts) {
    constexpr int DK = Cfg::DK, DV = Cfg::DV, NQ = Cfg::NQ, BN = Cfg::BN;
    extern __shared__ uint8_t smem_raw[];
    __shared__ Item s_item[Cfg::SLOTS];
    __shared__ int2 s_window[2][32];                      // (page, slot) of 32 boxes: keys', values'
    __shared__ uint32_t s_tmem;
    uint8_t* smem = align_1024(smem_raw);
    uint8_t* sQ = smem;                                   // [NQ][DK/64][128 rows][128 bytes]
    uint8_t* sK = sQ + NQ * Cfg::Q_TILE;                  // [KST][BN/8][DK/64][8 keys][128 bytes]
    uint8_t* sV = sK + Cfg::KST * Cfg::K_TILE;            // [VST][BN/8][DV/64][8 keys][128 bytes]
    uint64_t* k_full = reinterpret_cast<uint64_t*>(sV + Cfg::VST * Cfg::V_TILE);
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

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int group = static_cast<int>(a.q_heads / a.cache.heads);

    if (threadIdx.x == 0) {
        for (int i = 0; i < Cfg::KST; ++i) {
            mbar_init(&k_full[i], 1);
            mbar_init(&k_empty[i], 1);
        }
        for (int i = 0; i < Cfg::VST; ++i) {
            mbar_init(&v_full[i], 1);
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
            mbar_init(&i_empty[i], Cfg::SOFT_WARPS + 2);
        }
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
    // warpgroup less (208 x 256 + 80 x 128 = 63488 of 64512).
    if (warp < Cfg::SOFT_WARPS) {
        if constexpr (NQ == 2) regs_inc<208>();
        // ---- softmax warps: thread = row of query tile q
        const int q = warp >> 2;
        const int quarter = warp & 3;
        const int r = q * 128 + quarter * 32 + lane;          // row of the item's tile
        const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
        const uint32_t o_tmem = tmem + lanes + Cfg::SBUF * BN + q * DV;
        // (a scale of zero: any tiny factor keeps -inf apart from the finite scores; one that is NaN stays so)
        const float c = max_nan(fabsf(a.scale) * 1.4426950408889634f, 1e-30f);
        // Queries of query tile q into shared memory (K-major, 128-byte swizzle), valid rows only (what the
        // others hold is of no consequence: rows do not meet). A negative scale turns their signs, so that
        // the row maximum is always that of the largest S.
        auto load_queries = [&](const Item& it) {
            const uint32_t flip = a.scale < 0.0f ? 0x80008000u : 0u;
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
            if (live && it.piece == 0)
                // pieces that this sequence does not have are empty
                for (int p = it.pieces; p < pieces; ++p)
                    parts.ml[p * parts.rows + out_row(it, r)] = make_float2(-INFINITY, 0.0f);
            float m = -INFINITY;           // maximum in use, raw score
            float l = 0.0f;
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
                for (int j = 0; j < nt; ++j) {
                    const int n = n0 + j;
                    const int buf = NQ == 2 ? q : n & 1;
                    const uint32_t sph = NQ == 2 ? n & 1 : (n >> 1) & 1;
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
                            const float keep = grow ? exp2_fast((m - top) * c) : 1.0f;
                            if (grow) m = top;
                            l *= keep;
                            probabilities(s);
                            if (j > 0 && __any_sync(0xffffffffu, grow)) {
                                if (!warp_wait(&o_done[q], (n - 1) & 1)) {
                                    ok = false;
                                    break;
                                }
                                tc_fence_after();
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
                const float mc = m == -INFINITY ? -INFINITY : m * c;
                const float inv = l == 0.0f ? 0.0f : 1.0f / l;       // (NaN stays NaN)
                if (pieces > 1) {
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
        if constexpr (NQ == 2) regs_dec<80>();
        if (warp == Cfg::KEY_WARP) {
            // ---- hands out the items and brings their keys
            ItemFinder finder;
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
                load_sequences(finder, a, Cfg::ROWS, piece_len, lane);
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
                const Item it = find_item(finder, a, static_cast<int>(min(at, int64_t{INT32_MAX})), Cfg::ROWS,
                                          BN, piece_len, lane);
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
                ok = bring_tiles<Cfg, false>(vs, &tmV, a, it, first_tile(it), nt, modes.box_log2, modes.v, sV,
                                             v_full, v_empty, v_tail, s_window[1], lane,
                                             [&] { return warp_wait(q_first, 0); });
            }
            if (!ok && lane == 0) {
                drain_tiles<Cfg::VST>(vs, v_full);
                mbar_wait(v_tail, vs.tails & 1, kDrainLimitNs);
            }
        } else if (warp == Cfg::MMA_WARP) {
            // ---- MMA issuer. Per key tile and query tile: O += P(j) V(j), then S of the tile's next keys, which
            // takes P's place (the tensor core works in order).
            // With two query tiles one's products run under the other's softmax.
            constexpr uint32_t idesc_qk = idesc_bf16_f32(128, BN);
            constexpr uint32_t idesc_pv = idesc_bf16_f32(128, DV) | kIdescBMajorMN;
            // descriptors of the first stages; those of other stages and steps lie at constant distances (in
            // units of 16 bytes, which do not carry out of the address field)
            const uint64_t q_desc = smem_desc_k_sw128(smem_addr(sQ));
            const uint64_t k_desc = smem_desc_groups(smem_addr(sK), DK / 64 * 1024);
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
#pragma unroll
                    for (int d = 0; d < DK / 16; ++d)
                        mma_bf16(tmem + buf * BN,
                                 q_desc + (q * Cfg::Q_TILE + (d / 4) * (128 * 128) + (d % 4) * 32) / 16,
                                 kd + ((d / 4) * 1024 + (d % 4) * 32) / 16, idesc_qk, d > 0 ? 1u : 0u);
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

// Join the pieces of a row: WPR warps per row, warp w of them the pieces w, w + WPR, ... in key order, DV / 32
// channels per lane; the warps' sums are added in warp order. Bound by latency when the rows are few: the pieces'
// maxima and sums are read by all lanes at once, and no piece's load waits for another's.
template <int DV, int WPR>
__global__ void __launch_bounds__(128) attention_join_kernel(const AttnParts parts, int pieces,
                                                             __nv_bfloat16* out, float* lse) {
    constexpr int PER = DV / 32;
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int warp = (threadIdx.x >> 5) % WPR;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (4 / WPR) + (threadIdx.x >> 5) / WPR;
    if (row >= parts.rows) return;               // (whole blocks where a row's warps meet)
    // lane i: piece i * WPR + warp and, of more than 32 WPR pieces, every 32 WPR-th after it
    float top = -INFINITY;
    for (int p = lane; p < pieces; p += 32) top = fmaxf(top, parts.ml[p * parts.rows + row].x);
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
    float o[PER] = {}, l = 0.0f;
    for (int base = 0; base < pieces; base += 32 * WPR) {
        const int mine = base + WPR * lane + warp;
        float w = 0.0f;
        if (mine < pieces) {
            const float2 ml = parts.ml[mine * parts.rows + row];
            if (ml.y != 0.0f) {                      // (a sum that is NaN makes the row's NaN, whatever w is)
                w = exp2_fast(ml.x - top);
                l = fmaf(w, ml.y, l);
            }
        }
        const int count = min(32, (pieces - base - warp + WPR - 1) / WPR);
#pragma unroll 8
        for (int i = 0; i < count; ++i) {
            const float wi = __shfl_sync(0xffffffffu, w, i);
            if (wi != 0.0f) {                    // (an empty piece's O has not been written)
                const float* src = parts.o + ((base + WPR * i + warp) * parts.rows + row) * DV + PER * lane;
#pragma unroll
                for (int k = 0; k < PER; k += 2) {
                    const float2 f = *reinterpret_cast<const float2*>(src + k);
                    o[k] = fmaf(wi, f.x, o[k]);
                    o[k + 1] = fmaf(wi, f.y, o[k + 1]);
                }
            }
        }
    }
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) l += __shfl_xor_sync(0xffffffffu, l, i);
    if constexpr (WPR > 1) {
        __shared__ float s_o[WPR][DV];
        __shared__ float s_l[WPR];
#pragma unroll
        for (int k = 0; k < PER; ++k) s_o[warp][PER * lane + k] = o[k];
        if (lane == 0) s_l[warp] = l;
        __syncthreads();
        if (warp > 0) return;
        for (int w = 1; w < WPR; ++w) {
            l += s_l[w];
#pragma unroll
            for (int k = 0; k < PER; ++k) o[k] += s_o[w][PER * lane + k];
        }
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    uint32_t* dst = reinterpret_cast<uint32_t*>(out + row * DV) + PER / 2 * lane;
#pragma unroll
    for (int i = 0; i < PER / 2; ++i) dst[i] = pack_bf16x2(o[2 * i] * inv, o[2 * i + 1] * inv);
    if (lse && lane == 0)
        lse[row] = l == 0.0f ? -INFINITY : (top + log2_fast(l)) * 0.6931471805599453f;
}

int64_t tile_bound(const fp8bs_paged_attention_args& a, int rows) {
    // sum over sequences of ceil(n G / rows) <= T G / rows + min(B, T) (a sequence without queries
    // has no tile)
    const int64_t group = a.q_heads / a.cache.heads;
    return a.T * group / rows + (a.B < a.T ? a.B : a.T);
}

// Whether the two-tile form is used: where the average sequence has more rows than one tile holds. (32 sequences of
// 2048 keys, 8 heads of 128 channels, one tile and two: 128 rows 62 and 76 us, 160 rows 122 and 80, 512 rows 268 and
// 148; heads of 64 35 and 54, 82 and 61; of 192 75 and 94, 148 and 96. 4 sequences of 8192 keys, 4 heads: 128 rows 25
// and 33, 160 to 256 rows even.)
bool two_tiles(const fp8bs_paged_attention_args& a) {
    const int64_t group = a.q_heads / a.cache.heads;
    return a.T * group > 128 * a.B;
}

AttnParts attention_parts(const fp8bs_paged_attention_args& a, const AttentionPlan& plan) {
    AttnParts p = {};
    p.rows = a.T * a.q_heads;
    if (plan.pieces > 1) {
        p.o = static_cast<float*>(a.workspace);
        p.ml = reinterpret_cast<float2*>(p.o + plan.pieces * p.rows * a.cache.dv);
    }
    return p;
}

template <class Cfg>
cudaError_t launch_attention(const CUtensorMap& tmK, const CUtensorMap& tmV,
                             const fp8bs_paged_attention_args& a, const AttentionModes& modes,
                             const AttentionPlan& plan, int num_sms, cudaStream_t stream) {
    auto kernel = paged_attention_kernel<Cfg>;
    cudaError_t e = set_smem(kernel, Cfg::SMEM);
    if (e != cudaSuccess) return e;
    const AttnParts parts = attention_parts(a, plan);
    const int64_t items = tile_bound(a, Cfg::ROWS) * a.cache.heads * plan.pieces;
    if (items >= INT32_MAX) return cudaErrorInvalidValue;
    const int64_t resident = static_cast<int64_t>(num_sms) * Cfg::CTAS;
    const unsigned grid = static_cast<unsigned>(items < resident ? items : resident);
    e = launch_pdl(kernel, grid, Cfg::THREADS, Cfg::SMEM, stream, tmK, tmV, a, modes, plan.piece_len,
                   plan.pieces, parts);
    if (e != cudaSuccess || plan.pieces == 1) return e;
    // Many pieces of few rows: four warps a row; else a warp each (more blocks than the GPU holds at once would
    // keep the next kernel from starting: 4096 rows of 8 pieces took 30 us with four warps each, none to be seen
    // with one).
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out);
    if (parts.rows <= 1024)
        return launch_pdl(attention_join_kernel<Cfg::DV, 4>, static_cast<unsigned>(parts.rows), 128, 0, stream,
                          parts, plan.pieces, out, a.lse);
    return launch_pdl(attention_join_kernel<Cfg::DV, 1>, static_cast<unsigned>((parts.rows + 3) / 4), 128, 0,
                      stream, parts, plan.pieces, out, a.lse);
}

}  // namespace

namespace {

// Bytes that one piece of the keys leaves for the join: every row's O, maximum and sum.
int64_t part_bytes(const fp8bs_paged_attention_args& a) { return a.T * a.q_heads * (a.cache.dv * 4 + 8); }

// Most bytes that all pieces leave (a single one leaves none). 64 sequences of 64 heads of 128 channels: 245 pieces,
// so that a table of 250,000 keys still gives the pieces of 1024 that ragged batches want.
constexpr int64_t kMaxPartBytes = int64_t{1} << 29;

}  // namespace

AttentionPlan attention_plan(const fp8bs_paged_attention_args& a, int num_sms) {
    const bool two = two_tiles(a);
    const int64_t rows = two ? 256 : 128;
    const int64_t group = a.q_heads / a.cache.heads;
    // (sequences of one length, as in decoding, are counted exactly)
    const int64_t items = a.cache.heads * (a.T == a.B * a.max_q_len ? a.B * ((a.max_q_len * group + rows - 1) / rows)
                                                                    : tile_bound(a, rows));
    int64_t keys = key_span(a, rows, a.max_q_len, a.max_kv_len);
    if (keys < 1) keys = 1;
    const int64_t unit = two && a.cache.dk > 128 ? 192 : 128;       // whole key tiles
    int64_t len = keys;
    if (two) {
        // chunks that do not fill the GPU: the number of pieces with the lowest time, in keys, of the busiest
        // CTA, where a piece costs as much as 512 keys more (queries, output, its part of the join)
        int64_t best = keys;
        for (int64_t p = 2; items < num_sms && p <= 16 && keys / p >= 256; ++p) {
            const int64_t l = ((keys + p - 1) / p + unit - 1) / unit * unit;
            const int64_t time = (items * p + num_sms - 1) / num_sms * (l + 512);
            if (time < best) {
                best = time;
                len = l;
            }
        }
    } else if (items * keys < int64_t{4096} * num_sms) {
        // few rows and keys: as above, where a piece costs as much as 128 keys more, and joining p of them as much as
        // 128 + 32 p. (Cutting by one CTA's share of all keys instead, in 128 keys or more: 43.8 us instead of 30.3
        // for 14 sequences of 3183 keys, 57 instead of 43 for 5 of 9411, and around 12 instead of 9 where
        // sequences of 100 to 300 keys need no second kernel.)
        int64_t best = 0;
        for (int64_t p = 1; p <= 64 && (p == 1 || keys / p >= 64); ++p) {
            const int64_t step = p == 1 ? 64 : 128;
            const int64_t l = ((keys + p - 1) / p + step - 1) / step * step;
            const int64_t time = (items * p + num_sms - 1) / num_sms * (l + 128) + (p > 1 ? 128 + 32 * p : 0);
            if (p == 1 || time < best) {
                best = time;
                len = l;
            }
        }
    } else if (items < 8 * num_sms) {
        // many shares' worth of keys: pieces of 1024 at most, so that the longest sequence of a ragged batch does
        // not finish last on its own
        len = 1024;
    }
    // The bounds may be far above the sequences (a page table's whole width): no more pieces than kMaxPartBytes hold.
    const int64_t most = std::max<int64_t>(1, kMaxPartBytes / std::max<int64_t>(1, part_bytes(a)));
    if (len * most < keys) len = (keys + most - 1) / most;
    len = std::min<int64_t>((len + unit - 1) / unit * unit, int64_t{1} << 30);
    AttentionPlan p;
    p.piece_len = static_cast<int>(len);
    p.pieces = static_cast<int>((keys + len - 1) / len);
    return p;
}

size_t attention_workspace(const fp8bs_paged_attention_args& a, const AttentionPlan& plan) {
    if (plan.pieces == 1) return 0;
    return static_cast<size_t>(plan.pieces) * static_cast<size_t>(part_bytes(a));
}

cudaError_t launch_paged_attention(const CUtensorMap& tmK, const CUtensorMap& tmV,
                                   const fp8bs_paged_attention_args& a, const AttentionModes& modes,
                                   const AttentionPlan& plan, int num_sms, cudaStream_t stream) {
    const bool two = two_tiles(a);
    switch (a.cache.dk) {
        case 64:
            return two ? launch_attention<AttnCfg<64, 64, 2>>(tmK, tmV, a, modes, plan, num_sms, stream)
                       : launch_attention<AttnCfg<64, 64, 1>>(tmK, tmV, a, modes, plan, num_sms, stream);
        case 128:
            return two ? launch_attention<AttnCfg<128, 128, 2>>(tmK, tmV, a, modes, plan, num_sms, stream)
                       : launch_attention<AttnCfg<128, 128, 1>>(tmK, tmV, a, modes, plan, num_sms, stream);
        default:
            return two ? launch_attention<AttnCfg<192, 128, 2>>(tmK, tmV, a, modes, plan, num_sms, stream)
                       : launch_attention<AttnCfg<192, 128, 1>>(tmK, tmV, a, modes, plan, num_sms, stream);
    }
}

namespace {

// How a cache's rows of `d` channels can be fetched (AttentionModes).
int fetch_mode(const fp8bs_kv_cache& c, int64_t d, int64_t head_stride, int64_t page_stride) {
    if (c.page_size % 8 != 0) return 2;
    if (c.heads == 1 || head_stride == d) return 0;
    if (c.pages == 1 || page_stride == c.heads * head_stride)
        return c.pages * c.heads < (int64_t{1} << 31) ? 1 : 2;
    return 2;
}

}  // namespace

AttentionModes attention_modes(const fp8bs_kv_cache& c) {
    AttentionModes m;
    m.k = fetch_mode(c, c.dk, c.k_head_stride, c.k_page_stride);
    m.v = fetch_mode(c, c.dv, c.v_head_stride, c.v_page_stride);
    // slots per box: the largest power of two that divides the page and the key tiles (64 and 128, or 64 and 96)
    const int most = m.k == 2 || m.v == 2 ? 3 : c.dk > 128 ? 5 : 6;
    m.box_log2 = 0;
    while (m.box_log2 < most && c.page_size % (int64_t{2} << m.box_log2) == 0) ++m.box_log2;
    return m;
}

cudaError_t read_error_attention(unsigned int* out, bool clear, cudaStream_t stream) {
    return read_tu_error(out, clear, stream);
}

}  // namespace fp8bs
