// attention.cuh -- what the attention kernels share (attention.cu over a bf16 cache, attention_fp8.cu over one of e4m3
// codes): the work items and how they are found, the pieces of the key axis and their join.
#pragma once

#include <algorithm>

#include "gemm_common.cuh"
#include "quant_math.cuh"

namespace fp8bs {
namespace {

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
// slots). Calls ask for rising items; the sequences are read 32 PER at a time, PER per lane.
template <int PER>
struct ItemFinder {
    int base, before;       // first sequence of the chunk in hand, units (items / heads) before it
    int start[PER + 1], kv[PER];   // lane's sequences: first query tokens (and the next one's), keys
    int units[PER];         // of each
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

// SOME: sequences of more_rows rows or fewer have no items.
template <bool SOME, int PER>
__device__ __forceinline__ void load_sequences(ItemFinder<PER>& f, const fp8bs_paged_attention_args& a, int rows,
                                               int piece_len, int lane, int more_rows) {
    const int group = static_cast<int>(a.q_heads / a.cache.heads);
    f.sum = 0;
#pragma unroll
    for (int i = 0; i < PER + 1; ++i) {
        const int64_t b = f.base + PER * lane + i;
        f.start[i] = a.q_start[b < a.B ? b : a.B];
        if (i < PER) f.kv[i] = b < a.B ? a.kv_len[b] : 0;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int n = f.start[i + 1] - f.start[i];
        f.units[i] = 0;
        if (n > a.max_q_len || f.kv[i] > a.max_kv_len) {
            f.units[i] = 1;      // out of bounds: handed out once, to be reported
        } else if (n > 0 && (!SOME || static_cast<int64_t>(n) * group > more_rows)) {
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

template <bool SOME, int PER>
__device__ __forceinline__ Item find_item(ItemFinder<PER>& f, const fp8bs_paged_attention_args& a, int item, int rows,
                                          int bn, int piece_len, int lane, int more_rows) {
    Item it;
    it.seq = -1;
    const int heads = static_cast<int>(a.cache.heads);
    const int group = static_cast<int>(a.q_heads / a.cache.heads);
    const int unit = item / heads;
    it.head = item - unit * heads;
    while (f.base < a.B) {
        if (!f.loaded) load_sequences<SOME>(f, a, rows, piece_len, lane, more_rows);
        const unsigned hit = __ballot_sync(0xffffffffu, f.before + f.incl > unit);
        if (hit) {
            const int src = __ffs(hit) - 1;
            int seq = 0, n = 0, q0 = 0, kv = 0, tile = 0, piece = 0, pieces = 1;
            if (lane == src) {
                int left = unit - f.before - (f.incl - f.sum);
                int mine = 0;
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    if (left >= 0 && left < f.units[i]) {
                        seq = f.base + PER * lane + i;
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
        f.base += 32 * PER;
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

// After a wait that ran out: the copies of the ring's last tiles, so that none is still writing shared memory
// when the CTA ends.
template <int STAGES>
__device__ __forceinline__ void drain_tiles(const Stream& s, uint64_t* full) {
    record_error(FP8BS_DEVERR_PRODUCER_WAIT);
    for (int i = max(0, s.n - STAGES); i < s.n; ++i)
        if (!mbar_wait(&full[i % STAGES], (i / STAGES) & 1, kDrainLimitNs)) record_error(FP8BS_DEVERR_DRAIN_WAIT);
}

// Join the pieces of a row: WPR warps per row, warp w of them the pieces w, w + WPR, ... in key order, DV / 32
// channels per lane; the warps' sums are added in warp order. Bound by latency when the rows are few: the pieces'
// maxima and sums are read by all lanes at once, and no piece's load waits for another's. WHOLE: rows that were
// computed in one piece have been written already, which their first piece's sum says (kWholeRow).
constexpr float kWholeRow = -1.0f;

template <int DV, int WPR, bool WHOLE = false>
__global__ void __launch_bounds__(128) attention_join_kernel(const AttnParts parts, int pieces,
                                                             __nv_bfloat16* out, float* lse) {
    constexpr int PER = DV / 32;
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int warp = (threadIdx.x >> 5) % WPR;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (4 / WPR) + (threadIdx.x >> 5) / WPR;
    if (row >= parts.rows) return;               // (whole blocks where a row's warps meet)
    if (WHOLE && parts.ml[row].y == kWholeRow) return;
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

inline int64_t tile_bound(const fp8bs_paged_attention_args& a, int rows) {
    // sum over sequences of ceil(n G / rows) <= T G / rows + min(B, T) (a sequence without queries
    // has no tile)
    const int64_t group = a.q_heads / a.cache.heads;
    return a.T * group / rows + (a.B < a.T ? a.B : a.T);
}

// Bytes that one piece of the keys leaves for the join: every row's O, maximum and sum.
inline int64_t part_bytes(const fp8bs_paged_attention_args& a) { return a.T * a.q_heads * (a.cache.dv * 4 + 8); }

// Most bytes that all pieces leave (a single one leaves none). 64 sequences of 64 heads of 128 channels: 245 pieces,
// so that a table of 250,000 keys still gives the pieces of 1024 that ragged batches want.
constexpr int64_t kMaxPartBytes = int64_t{1} << 29;

}  // namespace
}  // namespace fp8bs
