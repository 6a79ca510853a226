// attention_fp8.cu -- attention of new tokens over a paged cache of e4m3 codes with one scale per page and head
// (fp8bs_paged_attention_fp8).
//
// The codes go from HBM to the tensor core as they are: nothing is widened on the way. With 128 keys per tile as the
// MMA's M side and the R query rows of a work item (token i, head g of the group: row i*G + g) on its N side,
//   S^T = K Q^T    e4m3 x e4m3: each row of Q as the sum of two e4m3 numbers per channel (columns r and R + r) in a unit
//                  that leaves its largest in [224, 448): exact for channels of 0.25 units and more (2^-9 of the
//                  largest), else off by 2^-10 units at most; K as the cache holds it, S^T fp32 in TMEM
//   P = exp2(c ks S + log2 vs - m), one thread per key, m the row's running maximum of that: probability and
//                  value scale in one, so that pages whose values differ in size share a tile
//   O^T = V^T P    e4m3 x e4m3: P as p + p'/32, two e4m3 numbers again (2^-8 of it, and 2^-23 of the row's largest);
//                  V as the cache holds it (keys outermost: an MN-major operand), one fp32 tile in TMEM per key tile,
//                  which the threads (one per channel) add to their sums in registers
// The sum of a row is taken from P in binary32 before its rounding, each term divided by its value's scale (a power of
// two): lse is as good as binary32 holds the exponentials, as long as a term does not vanish under the value scale of
// another page 2^80 times as large, and 2^8 over the smallest scale is a number (the range that the header states). Two
// or three groups of four warps take steps of one or two key tiles in turn, one's softmax under the others' products;
// the query warp puts their sums of an item together, in a fixed order. A row without keys is one whose sum is zero. A
// score that is not a number, or +infinite, makes the sum NaN.
//
// The work is cut into equal chunks of key tiles for each key head (RowsPlan), whatever the sequences' lengths: a chunk
// is the end of one sequence, some whole ones and the beginning of another. Parts of a sequence are joined in key order
// by a second kernel.
//
// Measured: 64 sequences of up to 8192 keys, 64 / 8 heads of 128, 556 MB: 108 us (0.77 of a copy's rate; the bf16 cache of
// twice the bytes 195); one sequence of 32785 keys 23.7 us; 24 sequences of up to 5000 keys, three tokens each, 16 heads of
// 192 / 128: 64 us for 322 MB. What bounds it then is a step's chain, not memory: S^T read, maxima over four warps,
// probabilities as codes, the product, of which three groups cover most; short sequences are bound by what starts and ends
// an item (queries into codes, sums of the groups): 128 sequences of up to 300 keys 38 us.
#include "attention_codes.cuh"
#include "attention_join.h"

namespace fp8bs {

namespace {

constexpr int KEYS = 128;             // keys per tile

template <int DK_, int DV_, int R_>
struct RowsCfg {
    static constexpr int DK = DK_, DV = DV_, R = R_;
    static constexpr int CHK = DK % 128 == 0 ? 128 : 64;         // bytes of a key per swizzled chunk
    static constexpr int N1 = 2 * R;                             // columns of S^T
    static constexpr int NP = R < 16 ? 32 : 2 * R;               // bytes of P per key (columns of O^T)
    static constexpr int K_TILE = KEYS * DK, V_TILE = KEYS * DV;
    static constexpr int Q_TILE = N1 * DK;
    // Tiles that a group takes at a time: two where the registers hold their scores, so that the ways between the warps
    // (maxima, P, products) are gone half as often.
    static constexpr int TPS = R <= 16 ? 2 : 1;
    // Groups: three where the registers allow it.
    static constexpr int NG = R == 8 ? 3 : 2;
    static constexpr int KST = DK == 64 ? 9 : DK == 128 ? (R == 32 ? 4 : 5) : (R == 32 ? 3 : 4);
    static constexpr int VST = DK == 64 ? 9 : DK == 128 ? (R == 32 ? 4 : 5) : 4;
    static constexpr int SBUF = NG + 1;                          // S^T of steps ahead
    static constexpr int CST = KST + SBUF * TPS;                 // tiles' scales
    static constexpr int P_STEP = TPS * KEYS * NP;
    static constexpr int SLOTS = 4;                              // ring of work items
    static constexpr int KEY_WARP = 4 * NG, VALUE_WARP = 4 * NG + 1, MMA_WARP = 4 * NG + 2, QUERY_WARP = 4 * NG + 3;
    static constexpr int THREADS = 32 * (4 * NG + 4);
    static constexpr uint32_t O_COL = SBUF * TPS * N1;
    static constexpr uint32_t TMEM_COLS = tmem_cols_for(O_COL + NG * NP);
    static constexpr int BARS = 2 * KST + 2 * VST + CST + SBUF + 3 * NG + 8 + 2 * SLOTS;
    // keys, values, P, queries (two items'), the groups' sums of an item, scales
    static constexpr int SMEM = 1024 + KST * K_TILE + VST * V_TILE + NG * P_STEP + 2 * Q_TILE + NG * R * DV * 4 +
                                CST * KEYS * 8 + BARS * 8;
    static_assert(SMEM <= kSmemLimit - 5120 - 160 * R, "shared memory");
};

// How the work is cut: for each key head into `chunks` equal ranges of positions, where a sequence counts its key tiles
// and kItemTiles more (whole: one, so that chunks hold whole sequences).
struct RowsPlan {
    int chunks;
    bool whole;
};

// What starting an item costs, in key tiles.
constexpr int kItemTiles = 2;

// Parts of sequences, for the join: of each (chunk, key head) the one that a chunk begins with (slot 0) and the one that
// it ends with (slot 1), and, where the part that it begins with ends its sequence, what is to be joined (JoinHead).
struct RowsParts {
    float2* mark;          // null, or where the other kernel's join is told which rows are none of its own
    float* o;              // [chunk][head][2][R][DV], unnormalised
    float2* ml;            // [chunk][head][2][R]: (reference in log2 units, sum)
    JoinHead* head;        // [chunk][head]
};

// A work item: the rows of a sequence that share a key head, and a range of its keys.
struct RowItem {
    int seq;               // -1: no more items
    int n, q0, kv, rows, head;
    int key_lo, key_hi;    // keys of the item that any row attends
    int slot;              // -1: the sequence's only item; else where its part goes, in slots
};

// mbar_wait and warp_wait with all but the first look out of line: the kernels here have many waits, and code that does
// not fit the instruction cache is fetched again for every work item.
__device__ __noinline__ bool long_wait(uint64_t* bar, uint32_t parity) { return mbar_wait(bar, parity); }

__device__ __forceinline__ bool thread_wait(uint64_t* bar, uint32_t parity) {
    return mbar_try_wait(smem_addr(bar), parity) || long_wait(bar, parity);
}

__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, thread_wait(bar, parity));
}

// Whether the phase has completed, asked once.
__device__ __forceinline__ bool thread_test(uint64_t* bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    return done != 0;
}

constexpr uint32_t kIdescBothMN = 1u << 15 | 1u << 16;       // A and B MN-major

// Probabilities (up to 256) as two codes, what the first leaves 32 times. By way of binary16, whose 11 bits hold a
// probability to 2^-12 of it and the difference from its code exactly.
__device__ __forceinline__ void two_codes_p(float x, float y, uint32_t* hi, uint32_t* lo) {
    const __half2 e = __floats2half2_rn(x, y);
    const __half2_raw er = static_cast<__half2_raw>(e);
    const __nv_fp8x2_storage_t c = __nv_cvt_halfraw2_to_fp8x2(er, __NV_SATFINITE, __NV_E4M3);
    const __half2 h = __half2(__nv_cvt_fp8x2_to_halfraw2(c, __NV_E4M3));
    const __half2 rest = __hmul2(__hsub2(e, h), __float2half2_rn(32.0f));
    *hi = c;
    *lo = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(rest), __NV_SATFINITE, __NV_E4M3);
}

// A reference that no key has set yet: the lowest number, below any score but itself, and finite, so that a difference from
// it is never NaN.
constexpr float kNoReference = -3.402823466e38f;

// Each of the R values summed over the warp's lanes, R a power of two: halves change hands until every lane holds one
// value's sum over some lanes, in l[0], then those. Returns which value it is.
template <int R>
__device__ __forceinline__ int sum_rows(float* l, int lane) {
    int row = 0, m = 16;
#pragma unroll
    for (int w = R / 2; w > 0; w /= 2, m /= 2) {
        const bool upper = lane & m;
#pragma unroll
        for (int k = 0; k < w; ++k) {
            const float got = __shfl_xor_sync(0xffffffffu, upper ? l[k] : l[k + w], m);
            l[k] = (upper ? l[k + w] : l[k]) + got;
        }
        row += upper ? w : 0;
    }
#pragma unroll
    for (; m > 0; m /= 2) l[0] += __shfl_xor_sync(0xffffffffu, l[0], m);
    return row;
}

// Likewise their maxima, NaN passed over.
template <int R>
__device__ __forceinline__ int max_rows(float* v, int lane) {
    int row = 0, m = 16;
#pragma unroll
    for (int w = R / 2; w > 0; w /= 2, m /= 2) {
        const bool upper = lane & m;
#pragma unroll
        for (int k = 0; k < w; ++k) {
            const float got = __shfl_xor_sync(0xffffffffu, upper ? v[k] : v[k + w], m);
            v[k] = fmaxf(upper ? v[k + w] : v[k], got);
        }
        row += upper ? w : 0;
    }
#pragma unroll
    for (; m > 0; m /= 2) v[0] = fmaxf(v[0], __shfl_xor_sync(0xffffffffu, v[0], m));
    return row;
}

// out[0..1] = a * b + c.
__device__ __forceinline__ void fma2_to(float* out, float2 a, float2 b, float2 c) {
    const float2 z = __ffma2_rn(a, b, c);
    out[0] = z.x;
    out[1] = z.y;
}

// 256 sequences of a call: their first tokens, keys, and the positions before each (and before the one after the last),
// counted from the first of them.
struct SequenceLook {
    int64_t at[257];
    int start[257], kv[256];
};

struct TileRange {
    int lo, hi, first, tiles;    // keys that any row attends; their first tile's first key and how many tiles
};

__device__ __forceinline__ TileRange tiles_of_rows(const fp8bs_paged_attention_args& a, int n, int kv) {
    TileRange t;
    t.lo = keys_of(a, n, kv, 0).lo;
    t.hi = keys_of(a, n, kv, n - 1).hi;
    t.first = t.lo / KEYS * KEYS;
    t.tiles = t.hi > t.lo ? (t.hi - t.first + KEYS - 1) / KEYS : 0;
    return t;
}

// Whether a sequence stays within what the caller said.
__device__ __forceinline__ bool in_bounds(const fp8bs_paged_attention_args& a, int q0, int n, int kv) {
    return n <= a.max_q_len && kv <= a.max_kv_len && kv >= 0 && q0 >= 0 && q0 + static_cast<int64_t>(n) <= a.T;
}

// Fills `f` with the sequences from `base` on (one warp) and returns the positions that they count.
__device__ __forceinline__ int64_t look_at(SequenceLook& f, int base, const fp8bs_paged_attention_args& a, bool whole,
                                           int rows, int lane) {
    const int group = static_cast<int>(a.q_heads / a.cache.heads);
    const int count = static_cast<int>(min(int64_t{256}, a.B - base));
    int64_t before = 0;
    auto load = [&](int b) {                                 // first token, the next one's, keys
        return b < count ? make_int3(a.q_start[base + b], a.q_start[base + b + 1], a.kv_len[base + b])
                         : make_int3(0, 0, 0);
    };
    int3 next = load(lane);
    __syncwarp();
#pragma unroll 1
    for (int i = 0; i < count; i += 32) {
        const int b = i + lane;
        const int3 seq = next;
        next = load(b + 32);
        int cost = 0;                                        // (2^24 tiles at most)
        if (b < count) {
            const int q0 = seq.x, n = seq.y - q0, kv = seq.z;
            f.start[b] = q0;
            f.kv[b] = kv;
            if (b == count - 1) f.start[b + 1] = q0 + n;
            if (whole)
                cost = 1;
            else if (n > 0 && !in_bounds(a, q0, n, kv))
                cost = 1;                    // out of bounds: met once, to be reported
            else if (n > 0 && static_cast<int64_t>(n) * group <= rows)
                cost = tiles_of_rows(a, n, kv).tiles + kItemTiles;
        }
        int incl = cost;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, incl, m);
            if (lane >= m) incl += o;
        }
        if (b < count) f.at[b] = before + incl - cost;
        before += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) f.at[count] = before;
    __syncwarp();
    return before;
}

// x * y / z of numbers that are not negative; in 32 bits, if they fit, which takes a fraction of the time.
__device__ __forceinline__ int64_t part_of(int64_t x, int64_t y, int64_t z) {
    const int64_t xy = x * y;
    return (xy | z) >> 32 == 0 ? static_cast<int64_t>(static_cast<uint32_t>(xy) / static_cast<uint32_t>(z)) : xy / z;
}

// The sequence of a look that holds position `at` (one that counts something): the last that begins at or before it.
__device__ __forceinline__ int sequence_at(const SequenceLook& f, int count, int64_t at, int lane) {
    // the eight that hold it, then the one
    const unsigned far = __ballot_sync(0xffffffffu, 8 * lane < count && f.at[8 * lane] <= at);
    const int eight = 8 * (31 - __clz(far));
    const unsigned near = __ballot_sync(0xffffffffu, lane < 8 && eight + lane < count && f.at[eight + lane] <= at);
    return eight + 31 - __clz(near);
}

template <class Cfg>
__global__ void __launch_bounds__(Cfg::THREADS, 1)
    attention_rows_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                          const __grid_constant__ fp8bs_paged_attention_args a, const Scales scales, const int box_log2,
                          const RowsPlan plan, const RowsParts parts, const bool early) {
    constexpr int DK = Cfg::DK, DV = Cfg::DV, R = Cfg::R, N1 = Cfg::N1, NP = Cfg::NP, TPS = Cfg::TPS, NG = Cfg::NG;
    extern __shared__ uint8_t smem_raw[];
    __shared__ RowItem s_item[Cfg::SLOTS];
    __shared__ SequenceLook s_look;
    __shared__ __align__(16) float s_factor[2][R];       // of each row of an item: what turns S into log2 units, but ks
    __shared__ int2 s_range[2][R];                       // its keys
    __shared__ __align__(16) float s_max[NG][2][4][R];   // group, step, warp: largest P's exponents
    __shared__ __align__(16) float s_m[NG][R];           // group: an item's references
    __shared__ float s_l[NG][4][R];                      // group, warp: its sums of probabilities
    __shared__ uint32_t s_tmem;
    uint8_t* smem = align_1024(smem_raw);
    uint8_t* sK = smem;                                  // [KST][DK/CHK][128 keys][CHK]
    uint8_t* sV = sK + Cfg::KST * Cfg::K_TILE;           // [VST][128 keys][DV]
    uint8_t* sP = sV + Cfg::VST * Cfg::V_TILE;           // [group][TPS * 128 keys][NP]
    uint8_t* sQ = sP + NG * Cfg::P_STEP;                 // [2][DK/CHK][N1 rows][CHK]
    float* sO = reinterpret_cast<float*>(sQ + 2 * Cfg::Q_TILE);          // [group][R][DV]
    float2* s_scale = reinterpret_cast<float2*>(sO + NG * R * DV);       // [CST][128]
    uint64_t* k_full = reinterpret_cast<uint64_t*>(s_scale + Cfg::CST * KEYS);
    uint64_t* k_empty = k_full + Cfg::KST;
    uint64_t* v_full = k_empty + Cfg::KST;
    uint64_t* v_empty = v_full + Cfg::VST;
    uint64_t* c_full = v_empty + Cfg::VST;               // [CST]
    uint64_t* s_full = c_full + Cfg::CST;                // [SBUF]
    uint64_t* x_full = s_full + Cfg::SBUF;               // [group] its warps' maxima
    uint64_t* p_full = x_full + NG;                      // [group]
    uint64_t* o_full = p_full + NG;                      // [group]
    uint64_t* q_full = o_full + NG;                      // [2]
    uint64_t* q_empty = q_full + 2;                      // [2]
    uint64_t* j_full = q_empty + 2;                      // the groups' sums of an item
    uint64_t* j_empty = j_full + 1;
    uint64_t* v_tail = j_empty + 1;
    uint64_t* drain = v_tail + 1;
    uint64_t* i_full = drain + 1;                        // [SLOTS]
    uint64_t* i_empty = i_full + Cfg::SLOTS;             // [SLOTS]

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
        for (int i = 0; i < Cfg::CST; ++i) mbar_init(&c_full[i], 1);
        for (int i = 0; i < Cfg::SBUF; ++i) mbar_init(&s_full[i], 1);
        for (int i = 0; i < NG; ++i) {
            mbar_init(&x_full[i], 4);
            mbar_init(&p_full[i], 4);
            mbar_init(&o_full[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&q_full[i], 1);
            mbar_init(&q_empty[i], 4 * NG);
        }
        mbar_init(j_full, 4 * NG);
        mbar_init(j_empty, 1);
        mbar_init(v_tail, 1);
        mbar_init(drain, 1);
        for (int i = 0; i < Cfg::SLOTS; ++i) {
            mbar_init(&i_full[i], 1);
            mbar_init(&i_empty[i], 4 * NG + 3);
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
    // (early: the launch before is the other kernel of the same call, which has waited for those before it; nothing here
    // reads what it writes, and this one ends after it)
    if (!early) grid_dependency_wait();
    grid_launch_dependents();

    auto first_tile = [](const RowItem& it) { return it.key_lo / KEYS * KEYS; };
    auto key_tiles = [&](const RowItem& it) {
        return it.key_hi > it.key_lo ? (it.key_hi - first_tile(it) + KEYS - 1) / KEYS : 0;
    };
    // The x-th item of this CTA (x counts from 0): to be waited for, and given back.
    auto item_ready = [&](int x) { return wait_all(&i_full[x % Cfg::SLOTS], (x / Cfg::SLOTS) & 1); };
    auto item_done = [&](int x) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&i_empty[x % Cfg::SLOTS]);
    };

    if (warp < 4 * NG) {
        // ---- groups of four warps: thread = key of the group's tiles for S and P, channel for O
        const int g = warp >> 2;
        const int tid = threadIdx.x & 127;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t o_addr = tmem + lanes + Cfg::O_COL + g * NP;
        // (64 channels: an MMA of 64 rows, whose results stand in the first 16 lanes of each warp)
        const bool has_channel = DV == 128 || lane < 16;
        const int channel = DV == 128 ? tid : (warp & 3) * 16 + (lane & 15);
        bool ok = true;
        int n0 = 0, s0 = 0, used = 0;              // key tiles, steps and items with keys before
        for (int x = 0; ok; ++x) {
            if (!item_ready(x)) {
                ok = false;
                break;
            }
            const RowItem& it = s_item[x % Cfg::SLOTS];
            if (it.seq < 0) break;
            const int nt = key_tiles(it);
            const int k0 = first_tile(it);
            const int ns = (nt + TPS - 1) / TPS;
            float m[R], l[R], acc[R];
#pragma unroll
            for (int r = 0; r < R; ++r) m[r] = kNoReference, l[r] = 0.0f, acc[r] = 0.0f;
            float m_lane = kNoReference;                                 // m[lane % R]
            // O^T of this group's step before (the i-th of the group's steps) onto the sums
            auto add_o = [&](int i) {
                if (!wait_all(&o_full[g], i & 1)) return false;
                tc_fence_after();
                float o[2 * R];
#pragma unroll
                for (int h = 0; h < 2 * R; h += 16) tmem_ld_16cols(o_addr + h, o + h);
#pragma unroll
                for (int h = 0; h < 2 * R; h += 16) tmem_wait_ld_16(o + h);
#pragma unroll
                for (int r = 0; r < R; r += 2) {
                    const float2 sum = __fadd2_rn(make_float2(acc[r], acc[r + 1]), make_float2(o[r], o[r + 1]));
                    fma2_to(acc + r, make_float2(o[R + r], o[R + r + 1]), make_float2(1.0f / 32.0f, 1.0f / 32.0f), sum);
                }
                return true;
            };
            int last = -1;                                               // the group's step before, in this item
            if (nt > 0) {
                const int b = used & 1;
                if (!wait_all(&q_full[b], (used >> 1) & 1)) {           // (factors and ranges)
                    ok = false;
                    break;
                }
                // tiles that need no mask for any row
                const int full_hi = s_range[b][0].y, full_lo = s_range[b][it.rows - 1].x;
                for (int u = (g + NG - s0 % NG) % NG; u < ns; u += NG) {
                    const int s = s0 + u;
                    const int i = s / NG;                                // of the group's steps
                    const int j = u * TPS, n = n0 + j;                   // first tile
                    const bool both = TPS == 2 && j + 1 < nt;
                    ok = wait_all(&c_full[n % Cfg::CST], (n / Cfg::CST) & 1);
                    if (ok && both) ok = wait_all(&c_full[(n + 1) % Cfg::CST], ((n + 1) / Cfg::CST) & 1);
                    if (ok) ok = wait_all(&s_full[s % Cfg::SBUF], (s / Cfg::SBUF) & 1);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t s_addr = tmem + lanes + (s % Cfg::SBUF) * (TPS * N1);
                    float t[TPS][R], inv_vs[TPS];
#pragma unroll
                    for (int h = 0; h < TPS; ++h) {
                        if (h == 1 && !both) {
                            inv_vs[h] = 0.0f;
#pragma unroll
                            for (int r = 0; r < R; ++r) t[h][r] = -INFINITY;
                            break;
                        }
                        const float2 sc = s_scale[((n + h) % Cfg::CST) * KEYS + tid];
                        inv_vs[h] = exp2_fast(-sc.y);
                        float y[2 * R];
#pragma unroll
                        for (int k = 0; k < 2 * R; k += 16) tmem_ld_16cols(s_addr + h * N1 + k, y + k);
#pragma unroll
                        for (int k = 0; k < 2 * R; k += 16) tmem_wait_ld_16(y + k);
#pragma unroll
                        for (int r = 0; r < R; r += 2) {
                            const float2 f = *reinterpret_cast<const float2*>(&s_factor[b][r]);
                            // (the factors first: large scales and small queries meet before either is out of range)
                            const float2 z = __fadd2_rn(make_float2(y[r], y[r + 1]), make_float2(y[R + r], y[R + r + 1]));
                            fma2_to(&t[h][r], z, __fmul2_rn(f, make_float2(sc.x, sc.x)), make_float2(sc.y, sc.y));
                        }
                        const int kb = k0 + (j + h) * KEYS;
                        if (kb < full_lo || kb + KEYS > full_hi) {
#pragma unroll
                            for (int r = 0; r < R; ++r) {
                                const int2 range = s_range[b][r];
                                if (kb + tid < range.x || kb + tid >= range.y) t[h][r] = -INFINITY;
                            }
                        }
                    }
                    // the rows' maxima over the step's keys
                    float (*tops)[R] = s_max[g][i & 1];
                    {
                        float v[R];
#pragma unroll
                        for (int r = 0; r < R; ++r) v[r] = TPS == 2 ? fmaxf(t[0][r], t[TPS - 1][r]) : t[0][r];
                        const int row = max_rows<R>(v, lane);
                        if ((lane & (32 / R - 1)) == 0) tops[warp & 3][row] = v[0];
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&x_full[g]);
                    if (last >= 0 && !add_o(last)) {
                        ok = false;
                        break;
                    }
                    if (!wait_all(&x_full[g], i & 1)) {
                        ok = false;
                        break;
                    }
                    // P's reference: 2^8 below the largest so far, so that P uses e4m3's range up to 256. Every warp of
                    // the group finds the same; it hardly ever moves. (From 2^24 on binary32 does not hold every such
                    // difference: where it comes out larger, the largest itself is the reference, and P at most 1.)
                    const float most = fmaxf(fmaxf(tops[0][lane % R], tops[1][lane % R]),
                                             fmaxf(tops[2][lane % R], tops[3][lane % R]));
                    const bool move = most - m_lane > 8.0f;
                    if (__any_sync(0xffffffffu, move)) {
                        if (move) {
                            const float ref = most - 8.0f;
                            m_lane = most - ref > 8.0f ? most : ref;
                        }
#pragma unroll
                        for (int r = 0; r < R; ++r) {
                            const float ref = __shfl_sync(0xffffffffu, m_lane, r);
                            if (ref > m[r]) {
                                const float keep = exp2_fast(m[r] - ref);
                                m[r] = ref;
                                l[r] *= keep;
                                acc[r] *= keep;
                            }
                        }
                    }
#pragma unroll
                    for (int h = 0; h < TPS; ++h) {
                        if (h == 1 && !both) break;
                        uint32_t p[R / 4], p2[R / 4];
#pragma unroll
                        for (int r = 0; r < R; r += 4) {
                            float e[4];
                            uint32_t h0, h1, l0, l1;
#pragma unroll
                            for (int k = 0; k < 4; k += 2) {
                                const float2 z = __fadd2_rn(make_float2(t[h][r + k], t[h][r + k + 1]),
                                                            make_float2(-m[r + k], -m[r + k + 1]));
                                e[k] = exp2_fast(z.x);
                                e[k + 1] = exp2_fast(z.y);
                                fma2_to(&l[r + k], make_float2(e[k], e[k + 1]), make_float2(inv_vs[h], inv_vs[h]),
                                        make_float2(l[r + k], l[r + k + 1]));
                            }
                            two_codes_p(e[0], e[1], &h0, &l0);
                            two_codes_p(e[2], e[3], &h1, &l1);
                            p[r / 4] = h0 | h1 << 16;
                            p2[r / 4] = l0 | l1 << 16;
                        }
                        uint8_t* row = sP + g * Cfg::P_STEP + (h * KEYS + tid) * NP;
                        if constexpr (R == 8) {
                            *reinterpret_cast<uint4*>(row + (swizzled(tid, 0, NP) << 4)) =
                                make_uint4(p[0], p[1], p2[0], p2[1]);
                        } else {
#pragma unroll
                            for (int c = 0; c < R / 16; ++c) {
                                *reinterpret_cast<uint4*>(row + (swizzled(tid, c, NP) << 4)) =
                                    make_uint4(p[4 * c], p[4 * c + 1], p[4 * c + 2], p[4 * c + 3]);
                                *reinterpret_cast<uint4*>(row + (swizzled(tid, R / 16 + c, NP) << 4)) =
                                    make_uint4(p2[4 * c], p2[4 * c + 1], p2[4 * c + 2], p2[4 * c + 3]);
                            }
                        }
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&p_full[g]);
                    last = i;
                }
                n0 += nt;
                s0 += ns;
                ++used;
            }
            if (!ok) break;
            if (last >= 0 && !add_o(last)) {
                ok = false;
                break;
            }
            tc_fence_before();
            // What the group found, for the query warp, which puts the groups' sums together
            if (!wait_all(j_empty, (x & 1) ^ 1)) {
                ok = false;
                break;
            }
            const int sum_row = sum_rows<R>(l, lane);
            if ((lane & (32 / R - 1)) == 0) s_l[g][warp & 3][sum_row] = l[0];
            if (tid == 0)
#pragma unroll
                for (int r = 0; r < R; r += 4)
                    *reinterpret_cast<float4*>(&s_m[g][r]) = make_float4(m[r], m[r + 1], m[r + 2], m[r + 3]);
            if (has_channel)
#pragma unroll
                for (int r = 0; r < R; ++r) sO[(g * R + r) * DV + channel] = acc[r];
            __syncwarp();
            if (lane == 0) mbar_arrive(j_full);
            if (nt > 0 && lane == 0) mbar_arrive(&q_empty[(used - 1) & 1]);
            item_done(x);
        }
        if (!ok && lane == 0) record_error(FP8BS_DEVERR_EPILOGUE_WAIT);
    } else if (warp == Cfg::KEY_WARP) {
        // ---- finds the items of the CTA's chunks and brings their keys
        bool ok = true;
        Stream ks = {0, 0};
        int x = 0;
        auto publish = [&](const RowItem& it) {
            if (!wait_all(&i_empty[x % Cfg::SLOTS], ((x / Cfg::SLOTS) & 1) ^ 1)) return false;
            if (lane == 0) {
                s_item[x % Cfg::SLOTS] = it;
                mbar_arrive(&i_full[x % Cfg::SLOTS]);
            }
            __syncwarp();
            ++x;
            return true;
        };
        const int heads = static_cast<int>(a.cache.heads);
        const int B = static_cast<int>(a.B);
        SequenceLook& f = s_look;
        // all positions
        int64_t all = 0, now = 0;                  // (now: those of the look in hand)
        for (int base = 0; base < B; base += 256) {
            now = look_at(f, base, a, plan.whole, R, lane);
            all += now;
        }
        int base = 0;                              // the look in hand: from this sequence on,
        int64_t before = 0;                        // after so many positions
        if (B > 256) now = look_at(f, 0, a, plan.whole, R, lane);
        const int64_t chunks = min(static_cast<int64_t>(plan.chunks), max(all, int64_t{1}));
        // (after a wait that ran out the rest of the ids get heads without parts: the join follows all of them)
        for (int64_t id = blockIdx.x; id < static_cast<int64_t>(plan.chunks) * heads; id += gridDim.x) {
            const int64_t chunk = part_of(id, 1, heads);
            const int head = static_cast<int>(id - chunk * heads);
            JoinHead join = {0, 0, 0, 0};
            if (ok && chunk < chunks) {
                // positions [at, end)
                int64_t at = part_of(chunk, all, chunks);
                const int64_t end = part_of(chunk + 1, all, chunks);
                while (ok && at < end) {
                    // the look that holds `at` (chunks of a CTA rise)
                    while (at >= before + now) {
                        before += now;
                        base += 256;
                        now = look_at(f, base, a, plan.whole, R, lane);
                    }
                    const int b = sequence_at(f, min(256, B - base), at - before, lane);
                    const int64_t first = before + f.at[b];              // the sequence's first position
                    const int cost = static_cast<int>(f.at[b + 1] - f.at[b]);
                    RowItem it;
                    it.seq = base + b;
                    it.q0 = f.start[b];
                    it.n = f.start[b + 1] - it.q0;
                    it.kv = f.kv[b];
                    const int64_t here = at;
                    at = min(end, first + cost);
                    if (it.n <= 0) continue;
                    if (!in_bounds(a, it.q0, it.n, it.kv)) {
                        if (lane == 0) record_error(FP8BS_DEVERR_INDEX);
                        continue;
                    }
                    if (static_cast<int64_t>(it.n) * group > R) continue;         // (whole sequences: not ours)
                    it.head = head;
                    it.rows = it.n * group;
                    const TileRange t = tiles_of_rows(a, it.n, it.kv);
                    int lo = 0, hi = t.tiles;                            // tiles of this item
                    if (!plan.whole) {
                        lo = static_cast<int>(max(here - first - kItemTiles, int64_t{0}));
                        hi = static_cast<int>(max(at - first - kItemTiles, int64_t{0}));
                        if (lo == hi && (t.tiles > 0 || here > first)) continue;
                    }
                    it.key_lo = lo == 0 ? t.lo : t.first + lo * KEYS;
                    it.key_hi = hi == t.tiles ? t.hi : t.first + hi * KEYS;
                    if (t.tiles == 0) it.key_lo = it.key_hi = 0;
                    it.slot = -1;
                    if (lo > 0) {
                        // (a part that is not the first: the chunk begins with it)
                        it.slot = static_cast<int>(2 * id);
                        if (hi == t.tiles)
                            // chunk that holds the sequence's first tile: the last to begin at or before it
                            join.first = static_cast<int>(part_of((first + kItemTiles + 1) * chunks - 1, 1, all)),
                            join.parts = static_cast<int>(chunk) - join.first + 1, join.q0 = it.q0, join.rows = it.rows;
                    } else if (hi < t.tiles) {
                        it.slot = static_cast<int>(2 * id + 1);
                    }
                    ok = publish(it);
                    if (!ok) break;
                    const int nt = key_tiles(it);
                    if (nt > 0)
                        ok = bring_codes<Cfg::KST, DK, Cfg::CHK, KEYS, true>(
                            ks, &tmK, a, scales, it, first_tile(it), nt, box_log2, sK, k_full, k_empty, nullptr, lane,
                            wait_all, [&](int, int tile, int first, float2 f) {
                                // (ks, log2 vs) of each key
                                const int cs = tile % Cfg::CST;
#pragma unroll
                                for (int i = 0; i < KEYS / 32; ++i) {
                                    const int key = lane + 32 * i;
                                    const float k1 = __shfl_sync(0xffffffffu, f.x, first + (key >> box_log2));
                                    const float v1 = __shfl_sync(0xffffffffu, f.y, first + (key >> box_log2));
                                    s_scale[cs * KEYS + key] =
                                        make_float2(k1, static_cast<float>(static_cast<int>(__float_as_uint(v1) >> 23) - 127));
                                }
                                __syncwarp();
                                if (lane == 0) mbar_arrive(&c_full[cs]);
                            });
                }
            }
            if (!plan.whole && lane == 0) parts.head[id] = ok ? join : JoinHead{0, 0, 0, 0};
        }
        if (ok) {
            RowItem none = {};
            none.seq = -1;
            ok = publish(none);
        }
        if (!ok && lane == 0) drain_tiles<Cfg::KST>(ks, k_full);
    } else if (warp == Cfg::VALUE_WARP) {
        // ---- brings the items' values
        bool ok = true;
        Stream vs = {0, 0};
        for (int x = 0; ok; ++x) {
            ok = item_ready(x);
            if (!ok) break;
            const RowItem it = s_item[x % Cfg::SLOTS];
            item_done(x);
            if (it.seq < 0) break;
            const int nt = key_tiles(it);
            if (nt == 0) continue;
            ok = bring_codes<Cfg::VST, DV, DV, KEYS, false>(vs, &tmV, a, Scales{nullptr, nullptr}, it, first_tile(it), nt,
                                                            box_log2, sV, v_full, v_empty, v_tail, lane, wait_all,
                                                            [](int, int, int, float2) {});
        }
        if (!ok && lane == 0) {
            drain_tiles<Cfg::VST>(vs, v_full);
            mbar_wait(v_tail, vs.tails & 1, kDrainLimitNs);
        }
    } else if (warp == Cfg::QUERY_WARP) {
        // ---- brings the items' queries and writes their results
        // An item's queries into buffer b: each row divided by a power of two that leaves its largest channel in
        // [224, 448), then as two codes per channel; missing rows as zeros. A lane has PER neighbouring channels of each
        // CHK of a row, and the addresses, factors and keys of row `lane`.
        constexpr int PER = DK == 128 ? 4 : 2, PARTS = DK / (32 * PER);
        auto load_queries = [&](const RowItem& it, int b) {
            uint8_t* dst = sQ + b * Cfg::Q_TILE;
            const int mine = min(lane, it.rows - 1);                         // (a missing row: the last one's address)
            const int tok = mine / group;
            const int64_t at = (it.q0 + tok) * a.q_token_stride +
                               (it.head * group + mine - tok * group) * a.q_head_stride;
            int my_e = 2;
            constexpr int BATCH = R == 32 ? 8 : 4;                           // rows on their way at once
#pragma unroll 1
            for (int r0 = 0; r0 < R; r0 += BATCH) {
                uint32_t v[BATCH][PARTS][PER / 2];
#pragma unroll
                for (int i = 0; i < BATCH; ++i) {
                    const __nv_bfloat16* src =
                        static_cast<const __nv_bfloat16*>(a.q) + __shfl_sync(0xffffffffu, at, r0 + i) + PER * lane;
#pragma unroll
                    for (int c = 0; c < PARTS; ++c) {
                        if constexpr (PER == 4)
                            *reinterpret_cast<uint2*>(v[i][c]) = __ldg(reinterpret_cast<const uint2*>(src + 32 * PER * c));
                        else
                            v[i][c][0] = __ldg(reinterpret_cast<const uint32_t*>(src + 32 * PER * c));
                    }
                }
                // the largest magnitude, as bf16 bits: those of infinities and NaN are larger than all numbers'
                uint32_t top[BATCH];
#pragma unroll
                for (int i = 0; i < BATCH; ++i) {
                    uint32_t t = 0;
#pragma unroll
                    for (int c = 0; c < PARTS; ++c)
#pragma unroll
                        for (int k = 0; k < PER / 2; ++k) {
                            if (r0 + i >= it.rows) v[i][c][k] = 0;
                            t = __vmaxu2(t, v[i][c][k] & 0x7FFF7FFFu);
                        }
                    top[i] = __reduce_max_sync(0xffffffffu, max(t & 0xFFFFu, t >> 16));
                }
#pragma unroll
                for (int i = 0; i < BATCH; ++i) {
                    const int r = r0 + i;
                    // amax / 448, up to a power of two: 448 is 1.75 * 2^8 (between 2^-125 and 2^125, for its reciprocal)
                    const int e = max(2, min(static_cast<int>(top[i] >> 7) - 8 + ((top[i] & 0x7Fu) > 0x60u ? 1 : 0), 252));
                    if (lane == r) my_e = e;
                    const float inv = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
#pragma unroll
                    for (int c = 0; c < PARTS; ++c) {
                        uint32_t hi[PER / 2], lo[PER / 2];
#pragma unroll
                        for (int k = 0; k < PER / 2; ++k) {
                            two_codes(bf16_lo(v[i][c][k]) * inv, bf16_hi(v[i][c][k]) * inv, &hi[k], &lo[k]);
                            if (top[i] >= 0x7F80u) hi[k] = 0x7F7Fu;          // a query that is not finite: NaN
                        }
                        const int channel = 32 * PER * c + PER * lane, byte = channel % Cfg::CHK;
                        uint8_t* chunk = dst + (channel / Cfg::CHK) * (N1 * Cfg::CHK);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int row = h * R + r;
                            uint8_t* to = chunk + row * Cfg::CHK + (swizzled(row, byte >> 4, Cfg::CHK) << 4) + (byte & 15);
                            const uint32_t* from = h == 0 ? hi : lo;
                            if constexpr (PER == 4)
                                *reinterpret_cast<uint32_t*>(to) = from[0] | from[1] << 16;
                            else
                                *reinterpret_cast<uint16_t*>(to) = static_cast<uint16_t>(from[0]);
                        }
                    }
                }
            }
            if (lane < R) {
                s_factor[b][lane] =
                    a.scale * 1.4426950408889634f * __uint_as_float(static_cast<uint32_t>(my_e) << 23);
                KeyRange kr = {0, 0};
                if (lane < it.rows) kr = keys_of(a, it.n, it.kv, tok);
                s_range[b][lane] = make_int2(max(kr.lo, it.key_lo), min(kr.hi, it.key_hi));
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(&q_full[b]);
        };
        // The groups' sums of item x put together, in the groups' order, and written out: the sequence's rows, or a part of
        // them for the join. A lane has DV / 32 channels.
        auto finish = [&](const RowItem& it, int x) {
            if (!wait_all(j_full, x & 1)) return false;
            // lane r: row r. A group without keys has a sum of zero and no reference; one whose scores are all not
            // numbers has no reference either, but its sum says so.
            float top = kNoReference, sum = 0.0f, factor[NG];
            const int mine = lane % R;
#pragma unroll
            for (int k = 0; k < NG; ++k) top = fmaxf(top, s_m[k][mine]);
#pragma unroll
            for (int k = 0; k < NG; ++k) {
                const float mk = s_m[k][mine];
                factor[k] = mk == kNoReference ? 0.0f : exp2_fast(mk - top);
                const float lk = (s_l[k][0][mine] + s_l[k][1][mine]) + (s_l[k][2][mine] + s_l[k][3][mine]);
                sum += mk == kNoReference ? lk : lk * factor[k];
            }
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;               // (NaN stays NaN)
            const int tok = mine / group;
            const int64_t my_row = (it.q0 + tok) * a.q_heads + it.head * group + (mine - tok * group);
            constexpr int OUT = DV / 32;
            // where row `lane` goes, in channels
            const int64_t to = (it.slot < 0 ? my_row : static_cast<int64_t>(it.slot) * R + mine) * DV;
#pragma unroll 1
            for (int r0 = 0; r0 < it.rows; r0 += 2) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int r = r0 + i;
                    float o[OUT] = {};
#pragma unroll
                    for (int k = 0; k < NG; ++k) {
                        const float f = __shfl_sync(0xffffffffu, factor[k], r);
                        const float* src = sO + (k * R + r) * DV + OUT * lane;
                        float v[OUT];
                        if constexpr (OUT == 4)
                            *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(src);
                        else
                            *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(src);
#pragma unroll
                        for (int c = 0; c < OUT; ++c) o[c] = fmaf(f == 0.0f ? 0.0f : v[c], f, o[c]);
                    }
                    const int64_t where = __shfl_sync(0xffffffffu, to, r) + OUT * lane;
                    const float scale = __shfl_sync(0xffffffffu, inv, r);
                    if (r < it.rows) {
                        if (it.slot < 0) {
                            uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.out) + where);
                            if constexpr (OUT == 4)
                                *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(o[0] * scale, o[1] * scale),
                                                                            pack_bf16x2(o[2] * scale, o[3] * scale));
                            else
                                *dst = pack_bf16x2(o[0] * scale, o[1] * scale);
                        } else if constexpr (OUT == 4) {
                            *reinterpret_cast<float4*>(parts.o + where) = make_float4(o[0], o[1], o[2], o[3]);
                        } else {
                            *reinterpret_cast<float2*>(parts.o + where) = make_float2(o[0], o[1]);
                        }
                    }
                }
            }
            if (lane < it.rows) {
                if (parts.mark) parts.mark[my_row] = make_float2(0.0f, kWholeRow);
                if (it.slot >= 0)
                    parts.ml[static_cast<int64_t>(it.slot) * R + lane] = make_float2(top, sum);
                else if (a.lse)
                    a.lse[my_row] = sum == 0.0f ? -INFINITY : (top + log2_fast(sum)) * 0.6931471805599453f;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(j_empty);
            return true;
        };
        bool ok = true;
        int used = 0;                              // items with keys before
        RowItem before = {};
        for (int x = 0; ok; ++x) {
            ok = item_ready(x);
            if (!ok) break;
            const RowItem it = s_item[x % Cfg::SLOTS];
            item_done(x);
            if (it.seq >= 0 && key_tiles(it) > 0) {
                ok = wait_all(&q_empty[used & 1], ((used >> 1) & 1) ^ 1);
                if (!ok) break;
                load_queries(it, used & 1);
                ++used;
            }
            if (x > 0) ok = finish(before, x - 1);
            if (it.seq < 0) break;
            before = it;
        }
        if (!ok && lane == 0) record_error(FP8BS_DEVERR_PRODUCER_WAIT);
    } else {
        // ---- MMA issuer. S^T goes ahead of O^T by up to SBUF steps (P's arrival shows that a step's S^T has been read);
        // whichever has its operands is issued, so that neither waits for the other's. Descriptors are those of the
        // rings' first places and constant distances (in units of 16 bytes, which do not carry out of the address field),
        // places are counted on. (By an elected thread of a converged warp: four MMAs and two commits take 163 cycles,
        // by a lane of its own 269.)
        constexpr uint32_t idesc_s = idesc_e4m3_f32(KEYS, N1);
        constexpr uint32_t idesc_o = idesc_e4m3_f32(DV, NP) | kIdescBothMN;
        const uint64_t k_desc = smem_desc_rows(smem_addr(sK), Cfg::CHK), q_desc = smem_desc_rows(smem_addr(sQ), Cfg::CHK);
        const uint64_t v_desc = smem_desc_rows(smem_addr(sV), DV), p_desc = smem_desc_rows(smem_addr(sP), NP);
        auto ready = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, thread_test(bar, parity)); };
        bool ok = true;
        int used = 0;
        int ks = 0, vs = 0, ss = 0, g = 0;                     // places: keys, values, S^T's step, O^T's group
        uint32_t kp = 0, vp = 0, pp = 0;                       // phases of keys, values, P
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
            ok = wait_all(&q_full[used & 1], (used >> 1) & 1);
            const uint64_t qd = q_desc + static_cast<uint32_t>((used & 1) * (Cfg::Q_TILE / 16));
            int js = 0, jo = 0;                                // tiles whose S^T, O^T has been issued
            int ahead = 0;                                     // steps whose S^T has been begun and whose P has not arrived
            bool arrived = false;                              // P of the step of tile jo
            uint64_t since = 0;                                // since when nothing could be issued
            while (ok && jo < nt) {
                bool issued = false;
                if (jo < js) {
                    if (!arrived && ready(&p_full[g], pp)) {
                        arrived = true;
                        --ahead;
                    }
                    if (arrived && ready(&v_full[vs], vp)) {
                        tc_fence_after();
                        const int h = jo % TPS;
                        const bool last = h == TPS - 1 || jo == nt - 1;
                        const uint64_t vd = v_desc + static_cast<uint32_t>(vs * (Cfg::V_TILE / 16));
                        const uint64_t pd = p_desc + static_cast<uint32_t>(g * (Cfg::P_STEP / 16) + h * (KEYS * NP / 16));
                        if (elect_one()) {
#pragma unroll
                            for (int k = 0; k < KEYS / 32; ++k)
                                mma_f8(tmem + Cfg::O_COL + g * NP, vd + 32 * k * DV / 16, pd + 32 * k * NP / 16, idesc_o,
                                       h > 0 || k > 0 ? 1u : 0u);
                            mma_commit(&v_empty[vs]);
                            if (last) mma_commit(&o_full[g]);
                        }
                        __syncwarp();
                        if (++vs == Cfg::VST) vs = 0, vp ^= 1;
                        ++jo;
                        if (last) {
                            arrived = false;
                            if (++g == NG) g = 0, pp ^= 1;
                        }
                        issued = true;
                    }
                }
                // (a step's S^T stands where that of SBUF steps before stood, whose P has arrived)
                if (js < nt && (js % TPS != 0 || ahead < Cfg::SBUF) && ready(&k_full[ks], kp)) {
                    tc_fence_after();
                    const int h = js % TPS;
                    const bool last = h == TPS - 1 || js == nt - 1;
                    if (h == 0) ++ahead;
                    const uint64_t kd = k_desc + static_cast<uint32_t>(ks * (Cfg::K_TILE / 16));
                    if (elect_one()) {
#pragma unroll
                        for (int d = 0; d < DK / 32; ++d) {
                            const int c = 32 * d / Cfg::CHK, in = 32 * d % Cfg::CHK;
                            mma_f8(tmem + (ss * TPS + h) * N1, kd + (c * (KEYS * Cfg::CHK) + in) / 16,
                                   qd + (c * (N1 * Cfg::CHK) + in) / 16, idesc_s, d > 0 ? 1u : 0u);
                        }
                        mma_commit(&k_empty[ks]);
                        if (last) mma_commit(&s_full[ss]);
                    }
                    __syncwarp();
                    if (++ks == Cfg::KST) ks = 0, kp ^= 1;
                    ++js;
                    if (last && ++ss == Cfg::SBUF) ss = 0;
                    issued = true;
                }
                if (issued) {
                    since = 0;
                } else {
                    const uint64_t t = global_timer_ns();
                    if (since == 0) since = t;
                    ok = __all_sync(0xffffffffu, t - since <= kWaitLimitNs);
                }
            }
            ++used;
        }
        if (!ok) {
            // abandoned: the products in flight still read shared memory; let them end
            if (lane == 0) record_error(FP8BS_DEVERR_MMA_WAIT);
            if (elect_one()) mma_commit(drain);
            __syncwarp();
            if (!wait_all(drain, 0) && lane == 0) record_error(FP8BS_DEVERR_DRAIN_WAIT);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == Cfg::MMA_WARP) tmem_dealloc(tmem, Cfg::TMEM_COLS);
    if (early) grid_dependency_wait();
}

// Joins the parts of the sequence that ends in the part that a chunk begins with: block (chunk and key head, group of
// rows), one thread per channel, the parts in key order.
template <int DV, int R>
__global__ void __launch_bounds__(DV) attention_rows_join_kernel(const __grid_constant__ fp8bs_paged_attention_args a,
                                                                 const RowsParts parts, const int chunks) {
    __shared__ float2 s_ml[DV];
    const int heads = static_cast<int>(a.cache.heads);
    const int group = static_cast<int>(static_cast<unsigned>(a.q_heads) / static_cast<unsigned>(heads));
    const int head = static_cast<int>(blockIdx.x % static_cast<unsigned>(heads));
    grid_dependency_wait();
    grid_launch_dependents();
    const JoinHead j = parts.head[blockIdx.x];
    if (!join_in_reach(j, chunks, R, group, static_cast<uint32_t>(a.T))) return;
    // where the i-th part stands: at the end of its chunk for the first, at the beginning for the others
    auto slot = [&](int i) { return (2 * (static_cast<int64_t>(j.first + i) * heads + head) + (i == 0 ? 1 : 0)) * R; };
    for (int r = blockIdx.y; r < j.rows; r += gridDim.y) {
        float top = kNoReference, l = 0.0f, o = 0.0f;
        for (int i0 = 0; i0 < j.parts; i0 += DV) {
            // (references and sums of as many parts as there are threads, one each)
            const int count = min(DV, j.parts - i0);
            __syncthreads();
            if (static_cast<int>(threadIdx.x) < count) s_ml[threadIdx.x] = parts.ml[slot(i0 + threadIdx.x) + r];
            __syncthreads();
            const float before = top;
#pragma unroll 8
            for (int i = 0; i < count; ++i) top = fmaxf(top, s_ml[i].x);
            if (i0 > 0) {
                const float keep = before == kNoReference ? 1.0f : exp2_fast(before - top);
                l *= keep, o *= keep;
            }
#pragma unroll 8
            for (int i = 0; i < count; ++i) {
                const float2 ml = s_ml[i];
                const float part = parts.o[(slot(i0 + i) + r) * DV + threadIdx.x];
                // (no reference: no keys, or scores that are not numbers, which the sum says)
                const float w = ml.x == kNoReference ? 0.0f : exp2_fast(ml.x - top);
                l += ml.x == kNoReference ? ml.y : ml.y * w;
                o = fmaf(w == 0.0f ? 0.0f : part, w, o);
            }
        }
        const int tok = r / group;
        const int64_t row = (j.q0 + tok) * a.q_heads + head * group + (r - tok * group);
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        static_cast<__nv_bfloat16*>(a.out)[row * DV + threadIdx.x] = __float2bfloat16_rn(o * inv);
        if (a.lse && threadIdx.x == 0)
            a.lse[row] = l == 0.0f ? -INFINITY : (top + log2_fast(l)) * 0.6931471805599453f;
    }
}

// Rows per item: the smallest form that holds the longest sequence's; where those of many rows go to the other kernel,
// that holds a single token's, and all longer ones go there (a chunk of 256 beside 200 single tokens, groups of 4 heads:
// 140 us; with the form of 32 rows for them 240).
int row_form(const fp8bs_paged_attention_args& a) {
    const int64_t group = a.q_heads / a.cache.heads;
    const int64_t rows = a.max_q_len * group <= kFewRows ? a.max_q_len * group : group;
    return rows <= 8 ? 8 : rows <= 16 ? 16 : kFewRows;
}

RowsPlan rows_plan(const fp8bs_paged_attention_args& a, int num_sms) {
    const int64_t heads = a.cache.heads;
    const int64_t B = a.B < a.T ? a.B : a.T;                  // (sequences with queries)
    const int64_t keys = key_span(a, kFewRows, a.max_q_len, a.max_kv_len);
    const int64_t tiles = std::max<int64_t>(1, (keys + KEYS - 1) / KEYS);
    // In key tiles of the busiest CTA: whole sequences; or equal chunks, of which each CTA gets the same number, and a
    // join, which costs as much as 10.
    int64_t best = (a.B * heads + num_sms - 1) / num_sms * (tiles + 3);
    RowsPlan p = {static_cast<int>(a.B), true};
    for (int64_t k = 1; k <= 8; ++k) {
        const int64_t chunks = std::min<int64_t>(k * num_sms / heads, B * tiles);
        if (chunks < 1) continue;
        const int64_t each = (chunks * heads + num_sms - 1) / num_sms;
        const int64_t time = each * ((B * (tiles + kItemTiles) + chunks - 1) / chunks + 3) + 10;
        if (time < best) {
            best = time;
            p = {static_cast<int>(chunks), false};
        }
    }
    return p;
}

// Where the parts stand, from `base` on, and their size.
size_t rows_parts(const fp8bs_paged_attention_args& a, const RowsPlan& plan, int R, uint8_t* base, RowsParts* parts) {
    *parts = RowsParts{};
    if (plan.whole) return 0;
    const size_t ids = static_cast<size_t>(plan.chunks) * static_cast<size_t>(a.cache.heads);
    const size_t o = ids * 2 * R * a.cache.dv * 4, ml = ids * 2 * R * 8;
    parts->o = reinterpret_cast<float*>(base);
    parts->ml = reinterpret_cast<float2*>(base + o);
    parts->head = reinterpret_cast<JoinHead*>(base + o + ml);
    return o + ml + ids * sizeof(JoinHead);
}

template <class Cfg>
cudaError_t launch_rows(const AttentionMapsFp8& maps, const fp8bs_paged_attention_args& a, const Scales& scales,
                        const RowsPlan& plan, const RowsParts& parts, bool early, int num_sms, cudaStream_t stream) {
    auto kernel = attention_rows_kernel<Cfg>;
    cudaError_t e = set_smem(kernel, Cfg::SMEM);
    if (e != cudaSuccess) return e;
    const int64_t ids = plan.chunks * a.cache.heads;
    const unsigned grid = static_cast<unsigned>(ids < num_sms ? ids : num_sms);
    e = launch_pdl(kernel, grid, Cfg::THREADS, Cfg::SMEM, stream, maps.k, maps.v, a, scales, maps.box_log2, plan, parts,
                   early);
    if (e != cudaSuccess || plan.whole) return e;
    const unsigned rows = static_cast<unsigned>(std::min<int64_t>(Cfg::R, a.max_q_len * (a.q_heads / a.cache.heads)));
    return launch_pdl(attention_rows_join_kernel<Cfg::DV, Cfg::R>, dim3(static_cast<unsigned>(ids), rows), Cfg::DV, 0,
                      stream, a, parts, plan.chunks);
}

template <int DK, int DV>
cudaError_t launch_rows(const AttentionMapsFp8& maps, const fp8bs_paged_attention_args& a, const Scales& scales,
                        const RowsPlan& plan, const RowsParts& parts, bool early, int num_sms, cudaStream_t stream) {
    switch (row_form(a)) {
        case 8: return launch_rows<RowsCfg<DK, DV, 8>>(maps, a, scales, plan, parts, early, num_sms, stream);
        case 16: return launch_rows<RowsCfg<DK, DV, 16>>(maps, a, scales, plan, parts, early, num_sms, stream);
        default: return launch_rows<RowsCfg<DK, DV, kFewRows>>(maps, a, scales, plan, parts, early, num_sms, stream);
    }
}

// Which kernels a call runs, and what they leave for their joins: of the tiles first, then of the few rows.
struct Fp8Plan {
    bool tiles, few;
    bool two;              // query tiles per CTA
    AttentionPlan of_tiles;
    RowsPlan of_rows;
    size_t tile_bytes, bytes;
    RowsParts parts;
};

// Whether the other kernel's CTAs take two query tiles: where the average sequence has more rows than one tile holds, or
// the longest has many. (32 sequences of 2048 keys, 8 heads of 128 channels, one tile and two: 128 rows 63 and 80 us,
// 160 rows 149 and 82; heads of 64 44 and 65, 116 and 66; of 192 84 and 107, 205 and 109. Beside 63 single tokens a
// sequence of 2048 rows 165 and 142; beside 32 one of 528 rows 47 and 65, beside 200 one of 1024 rows 133 and 138.)
bool two_tiles(const fp8bs_paged_attention_args& a) {
    const int64_t group = a.q_heads / a.cache.heads;
    return a.T * group > 128 * a.B || a.max_q_len * group > 1024;
}

Fp8Plan fp8_plan(const fp8bs_paged_attention_args& a, int num_sms) {
    Fp8Plan p = {};
    const int64_t rows = a.max_q_len * (a.q_heads / a.cache.heads);
    p.tiles = rows > kFewRows;
    // (both: unless all sequences are alike, or a single token has too many rows)
    p.few = !p.tiles || (a.T != a.B * a.max_q_len && a.q_heads / a.cache.heads <= kFewRows);
    if (p.tiles) {
        p.two = two_tiles(a);
        p.of_tiles = attention_plan(a, num_sms, p.two);
        if (p.of_tiles.pieces > 1) p.tile_bytes = (p.of_tiles.pieces * part_bytes(a) + 255) / 256 * 256;
    }
    p.bytes = p.tile_bytes;
    if (p.few) {
        p.of_rows = rows_plan(a, num_sms);
        p.bytes += rows_parts(a, p.of_rows, row_form(a), static_cast<uint8_t*>(a.workspace) + p.tile_bytes, &p.parts);
        if (p.tile_bytes > 0)
            p.parts.mark = reinterpret_cast<float2*>(static_cast<float*>(a.workspace) +
                                                     p.of_tiles.pieces * a.T * a.q_heads * a.cache.dv);
    }
    return p;
}

}  // namespace

int attention_fp8_box_log2(const fp8bs_kv_cache& c) {
    // the largest power of two that divides the page and the key tiles (64 and 128, or 64 and 96)
    const int most = c.dk > 128 ? 5 : 6;
    int b = 4;
    while (b < most && c.page_size % (int64_t{2} << b) == 0) ++b;
    return b;
}

int attention_fp8_key_chunk(int64_t dk) { return dk % 128 == 0 ? 128 : 64; }

size_t attention_fp8_workspace(const fp8bs_paged_attention_args& a, int num_sms) { return fp8_plan(a, num_sms).bytes; }

cudaError_t launch_paged_attention_fp8(const AttentionMapsFp8& maps, const fp8bs_paged_attention_args& a,
                                       const float* k_scale, const float* v_scale, int num_sms, cudaStream_t stream) {
    const Scales scales = {k_scale, v_scale};
    const Fp8Plan p = fp8_plan(a, num_sms);
    cudaError_t e = cudaSuccess;
    if (p.tiles)
        e = launch_attention_fp8_tiles(maps, a, k_scale, v_scale, p.of_tiles, p.two, p.few ? row_form(a) : 0, num_sms, stream);
    if (e == cudaSuccess && p.few) {
        const bool early = p.tiles;
        switch (a.cache.dk) {
            case 64: e = launch_rows<64, 64>(maps, a, scales, p.of_rows, p.parts, early, num_sms, stream); break;
            case 128: e = launch_rows<128, 128>(maps, a, scales, p.of_rows, p.parts, early, num_sms, stream); break;
            default: e = launch_rows<192, 128>(maps, a, scales, p.of_rows, p.parts, early, num_sms, stream);
        }
    }
    if (e == cudaSuccess && p.tiles && p.of_tiles.pieces > 1) e = launch_attention_fp8_tiles_join(a, p.of_tiles, stream);
    return e;
}

cudaError_t read_error_attention_fp8(unsigned int* out, bool clear, cudaStream_t stream) {
    return read_tu_error(out, clear, stream);
}

}  // namespace fp8bs
