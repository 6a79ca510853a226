// attention_fp8.cu -- attention of new tokens over a paged cache of e4m3 codes with one scale per page and head
// (fp8bs_paged_attention_fp8).
//
// The codes go from HBM to the tensor core as they are: nothing is widened on the way. With 128 keys per tile as the
// MMA's M side and the R query rows of a work item (token i, head g of the group: row i*G + g) on its N side,
//   S^T = K Q^T    e4m3 x e4m3: each row of Q as the sum of two e4m3 numbers per channel (columns r and R + r), exact
//                  but for channels 2^-17 below the row's largest; K as the cache holds it, S^T fp32 in TMEM
//   P = exp2(c ks S + log2 vs - m), one thread per key, m the row's running maximum of that: probability and
//                  value scale in one, so that pages whose values differ in size share a tile
//   O^T = V^T P    e4m3 x e4m3: P as p + p'/32, two e4m3 numbers again (2^-8 of it, and 2^-23 of the row's largest);
//                  V as the cache holds it (keys outermost: an MN-major operand), one fp32 tile in TMEM per key tile,
//                  which the threads (one per channel) add to their sums in registers
// The sum of a row is taken from P in binary32 before its rounding, each term divided by its value's scale (a power of
// two), so lse is exact to binary32. Two groups of four warps take every other key tile, one's softmax under the
// other's products; their sums meet at the end of an item, in a fixed order.
// A row without keys is one whose sum is zero. A score that is not a number, or +infinite, makes the sum NaN.
//
// Few rows and long keys: the key axis is cut into pieces, whose results a second kernel joins in key order
// (attention.cuh); rows of a single piece are written here.
#include "attention.cuh"

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
    static constexpr int Q_TILE = N1 * DK, P_TILE = KEYS * NP;
    static constexpr int KST = DK == 64 ? 10 : DK == 128 ? (R == 32 ? 5 : 6) : 4;
    static constexpr int VST = DK == 64 ? 10 : DK == 128 ? (R == 32 ? 5 : 6) : (R == 32 ? 4 : 5);
    static constexpr int CST = KST + 2;                          // tiles' scales
    static constexpr int SLOTS = 4;                              // ring of work items
    static constexpr int KEY_WARP = 8, VALUE_WARP = 9, MMA_WARP = 10;
    static constexpr int THREADS = 32 * 11;
    static constexpr uint32_t O_COL = 2 * N1;
    static constexpr uint32_t TMEM_COLS = tmem_cols_for(2 * N1 + 2 * NP);
    static constexpr int BARS = 2 * KST + 2 * VST + CST + 16 + 2 * SLOTS;
    // keys, values, queries (two items'), P (and, when an item's products have ended, the second group's sums), scales
    static constexpr int SMEM = 1024 + KST * K_TILE + VST * V_TILE + 2 * Q_TILE + 2 * P_TILE + CST * KEYS * 8 + BARS * 8;
    static_assert(R * DV * 4 <= 2 * P_TILE, "the second group's sums");
    static_assert(SMEM <= kSmemLimit - 512 - 140 * R, "shared memory");
};

__device__ __forceinline__ float warp_max(float x) {
    float m;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(x));
    return m;
}

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

constexpr uint32_t kIdescBothMN = 1u << 15 | 1u << 16;       // A and B MN-major

// Where the 16-byte piece c of a swizzled row stands.
__device__ __forceinline__ int swizzled(int row, int c, int row_bytes) {
    return row_bytes == 128 ? c ^ (row & 7) : row_bytes == 64 ? c ^ ((row >> 1) & 3) : c ^ ((row >> 2) & 1);
}

__device__ __forceinline__ float2 e4m3x2_values(uint32_t pair) {
    return __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(pair), __NV_E4M3)));
}

// x and what its e4m3 code leaves of it, 2^SHIFT times, as codes.
template <int SHIFT>
__device__ __forceinline__ void two_codes(float x, float y, uint32_t* hi, uint32_t* lo) {
    *hi = pack_e4m3x2(x, y);
    const float2 h = e4m3x2_values(*hi);
    constexpr float up = static_cast<float>(1 << SHIFT);
    *lo = pack_e4m3x2((x - h.x) * up, (y - h.y) * up);
}

struct Scales {
    const float *k, *v;          // [pages, heads]
};

// The key tiles k0, k0 + KEYS, ... (nt of them) of an item into the ring of KEYS or values, by TMA in boxes of
// 2^box_log2 slots (16 at least, so a tile has 8 boxes at most), one lane a box. The pages of 32 boxes are looked up at
// once, one per lane, two looks ahead, and their scales one look ahead. With the keys goes (ks, log2 vs) of each key.
// Values of the first and last tile that do not count are cleared before the tile does: whatever stood there must not
// meet a probability of zero.
template <class Cfg, bool IS_KEYS>
__device__ __forceinline__ bool bring_codes(Stream& s, const CUtensorMap* map, const fp8bs_paged_attention_args& a,
                                            const Scales& scales, const Item& it, int k0, int nt, int box_log2,
                                            uint8_t* ring, uint64_t* full, uint64_t* empty, uint64_t* tail,
                                            float2* s_scale, uint64_t* c_full, int lane) {
    constexpr int STAGES = IS_KEYS ? Cfg::KST : Cfg::VST;
    constexpr int D = IS_KEYS ? Cfg::DK : Cfg::DV;
    constexpr int CH = IS_KEYS ? Cfg::CHK : D;
    constexpr int TILE = KEYS * D;
    const int box = 1 << box_log2;
    const int boxes = KEYS >> box_log2;
    const int page_size = static_cast<int>(a.cache.page_size);
    const int heads = static_cast<int>(a.cache.heads);
    const int head = it.head, kv = it.kv, key_lo = it.key_lo;
    const int32_t* table = a.page_table + it.seq * a.table_stride;
    auto lookup = [&](int w) {               // boxes 32 w .. 32 w + 31 of the item: (page, slot), page -1: no keys
        const int64_t key = k0 + (static_cast<int64_t>(w) * 32 + lane) * box;
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
        if (IS_KEYS && at.x >= 0 && at.x < a.cache.pages) {
            const int64_t i = static_cast<int64_t>(at.x) * heads + head;
            f = make_float2(scales.k[i], scales.v[i]);
        }
        return f;
    };
    int2 at, next = lookup(0), after = lookup(1);
    float2 f, next_f = scales_of(next);
    for (int j = 0; j < nt; ++j) {
        const int key0 = k0 + j * KEYS;
        const int first = (j * boxes) & 31;              // this tile's first box of the look
        if (first == 0) {
            at = next, f = next_f;
            next = after;
            next_f = scales_of(next);
            after = lookup(((j * boxes) >> 5) + 2);
        }
        // boxes [none, live) hold keys that count: those before them are past a window (their pages may have been
        // given back), those after them past the sequence
        const int live = min(boxes, (kv - key0 + box - 1) >> box_log2);
        const int none = j == 0 ? (key_lo - k0) >> box_log2 : 0;
        const int st = s.n % STAGES;
        if (!warp_wait(&empty[st], ((s.n / STAGES) & 1) ^ 1)) return false;
        const bool partial = !IS_KEYS && (kv - key0 < KEYS || none > 0);
        uint64_t* bar = partial ? tail : &full[st];
        const uint32_t dst = smem_addr(ring) + st * TILE;
        if (lane == 0) mbar_arrive_expect_tx(bar, static_cast<uint32_t>((live - none) * box * D));
        __syncwarp();
        const int page = __shfl_sync(0xffffffffu, at.x, first + lane);
        const int slot = __shfl_sync(0xffffffffu, at.y, first + lane);
        if (lane >= none && lane < live)
#pragma unroll
            for (int c = 0; c < D / CH; ++c)
                tma_load_4d(dst + c * (KEYS * CH) + (lane << box_log2) * CH, map, bar, c * CH, head, slot, page);
        if constexpr (IS_KEYS) {
            const int cs = s.n % Cfg::CST;
#pragma unroll
            for (int i = 0; i < KEYS / 32; ++i) {
                const int key = lane + 32 * i;
                const float ks = __shfl_sync(0xffffffffu, f.x, first + (key >> box_log2));
                const float vs = __shfl_sync(0xffffffffu, f.y, first + (key >> box_log2));
                s_scale[cs * KEYS + key] =
                    make_float2(ks, static_cast<float>(static_cast<int>(__float_as_uint(vs) >> 23) - 127));
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&c_full[cs]);
        }
        __syncwarp();
        if (partial) {
            if (!warp_wait(tail, s.tails & 1)) return false;
            ++s.tails;
            const int skip = none << box_log2;
            const int keep = min(kv - key0, KEYS);
            for (int i = lane; i < (KEYS - keep + skip) * (D / 16); i += 32) {
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

template <class Cfg>
__global__ void __launch_bounds__(Cfg::THREADS, 1)
    attention_rows_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                          const __grid_constant__ fp8bs_paged_attention_args a, const Scales scales, const int box_log2,
                          const int piece_len, const int pieces, const AttnParts parts) {
    constexpr int DK = Cfg::DK, DV = Cfg::DV, R = Cfg::R, N1 = Cfg::N1, NP = Cfg::NP;
    extern __shared__ uint8_t smem_raw[];
    __shared__ Item s_item[Cfg::SLOTS];
    __shared__ __align__(16) float s_factor[2][R];       // of each row of an item: what turns S into log2 units, but ks
    __shared__ int2 s_range[2][R];                       // its keys
    __shared__ __align__(16) float s_max[2][2][4][R];    // group, tile, warp: largest P's exponents
    __shared__ float s_m[2][R], s_l[2][4][R];            // group: reference; warps' sums
    __shared__ uint32_t s_tmem;
    uint8_t* smem = align_1024(smem_raw);
    uint8_t* sK = smem;                                  // [KST][DK/CHK][128 keys][CHK]
    uint8_t* sV = sK + Cfg::KST * Cfg::K_TILE;           // [VST][128 keys][DV]
    uint8_t* sP = sV + Cfg::VST * Cfg::V_TILE;           // [group][128 keys][NP]
    uint8_t* sQ = sP + 2 * Cfg::P_TILE;                  // [2][DK/CHK][N1 rows][CHK]
    float* sO = reinterpret_cast<float*>(sP);            // [R][DV]
    float2* s_scale = reinterpret_cast<float2*>(sQ + 2 * Cfg::Q_TILE);   // [CST][128]
    uint64_t* k_full = reinterpret_cast<uint64_t*>(s_scale + Cfg::CST * KEYS);
    uint64_t* k_empty = k_full + Cfg::KST;
    uint64_t* v_full = k_empty + Cfg::KST;
    uint64_t* v_empty = v_full + Cfg::VST;
    uint64_t* c_full = v_empty + Cfg::VST;               // [CST]
    uint64_t* s_full = c_full + Cfg::CST;                // [group]
    uint64_t* x_full = s_full + 2;                       // [group] its warps' maxima
    uint64_t* p_full = x_full + 2;                       // [group]
    uint64_t* o_full = p_full + 2;                       // [group]
    uint64_t* q_full = o_full + 2;                       // [2]
    uint64_t* j_bar = q_full + 2;                        // [3] the groups' meeting at an item's end
    uint64_t* v_tail = j_bar + 3;
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
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&x_full[i], 4);
            mbar_init(&p_full[i], 4);
            mbar_init(&o_full[i], 1);
            mbar_init(&q_full[i], 8);
        }
        for (int i = 0; i < 3; ++i) mbar_init(&j_bar[i], 8);
        mbar_init(v_tail, 1);
        mbar_init(drain, 1);
        for (int i = 0; i < Cfg::SLOTS; ++i) {
            mbar_init(&i_full[i], 1);
            mbar_init(&i_empty[i], 10);
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

    auto first_tile = [](const Item& it) { return it.key_lo / KEYS * KEYS; };
    auto key_tiles = [&](const Item& it) {
        return it.key_hi > it.key_lo ? (it.key_hi - first_tile(it) + KEYS - 1) / KEYS : 0;
    };
    // The x-th item of this CTA (x counts from 0): to be waited for, and given back.
    auto item_ready = [&](int x) { return warp_wait(&i_full[x % Cfg::SLOTS], (x / Cfg::SLOTS) & 1); };
    auto item_done = [&](int x) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&i_empty[x % Cfg::SLOTS]);
    };

    if (warp < 8) {
        // ---- two groups of four warps: thread = key of the group's tiles for S and P, channel for O
        const int g = warp >> 2;
        const int tid = threadIdx.x & 127;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t s_addr = tmem + lanes + g * N1;
        const uint32_t o_addr = tmem + lanes + Cfg::O_COL + g * NP;
        // (64 channels: an MMA of 64 rows, whose results stand in the first 16 lanes of each warp)
        const bool has_channel = DV == 128 || lane < 16;
        const int channel = DV == 128 ? tid : (warp & 3) * 16 + (lane & 15);
        // An item's queries into buffer b: each row divided by a power of two that leaves its largest channel in
        // [224, 448), then as two codes per channel; missing rows as zeros.
        auto load_queries = [&](const Item& it, int b) {
            uint8_t* dst = sQ + b * Cfg::Q_TILE;
#pragma unroll
            for (int i = 0; i < R / 8; ++i) {
                const int r = warp + 8 * i;
                uint32_t v[DK / 64];
                float amax = 0.0f;
                bool finite = true;
                int tok = 0;
                if (r < it.rows) {
                    const int pr = it.first_row + r;
                    tok = pr / group;
                    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.q) +
                                               (it.q0 + tok) * a.q_token_stride +
                                               (it.head * group + pr - tok * group) * a.q_head_stride;
#pragma unroll
                    for (int c = 0; c < DK / 64; ++c)
                        v[c] = __ldg(reinterpret_cast<const uint32_t*>(src) + 32 * c + lane);
                } else {
#pragma unroll
                    for (int c = 0; c < DK / 64; ++c) v[c] = 0;
                }
#pragma unroll
                for (int c = 0; c < DK / 64; ++c) {
                    const float x = fabsf(bf16_lo(v[c])), y = fabsf(bf16_hi(v[c]));
                    finite = finite && x <= 3.4e38f && y <= 3.4e38f;
                    amax = fmaxf(amax, fmaxf(x, y));
                }
                amax = warp_max(amax);
                // amax / 448, up to a power of two: 448 is 1.75 * 2^8 (and 2^126 at most, for its reciprocal)
                const uint32_t bits = __float_as_uint(amax);
                int e = static_cast<int>(bits >> 23) - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
                e = max(2, min(e, 252));
                const float unit = __uint_as_float(static_cast<uint32_t>(e) << 23);
                const float inv = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
                const bool whole = __all_sync(0xffffffffu, finite);
#pragma unroll
                for (int c = 0; c < DK / 64; ++c) {
                    uint32_t hi, lo;
                    two_codes<0>(bf16_lo(v[c]) * inv, bf16_hi(v[c]) * inv, &hi, &lo);
                    if (!whole) hi = 0x7F7Fu;             // a query that is not finite: NaN
                    const int byte = (64 * c + 2 * lane) % Cfg::CHK;
                    uint8_t* chunk = dst + (64 * c / Cfg::CHK) * (N1 * Cfg::CHK);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int row = h * R + r;
                        *reinterpret_cast<uint16_t*>(chunk + row * Cfg::CHK +
                                                     (swizzled(row, byte >> 4, Cfg::CHK) << 4) + (byte & 15)) =
                            static_cast<uint16_t>(h == 0 ? hi : lo);
                    }
                }
                if (lane == 0) {
                    s_factor[b][r] = a.scale * 1.4426950408889634f * unit;
                    KeyRange kr = {0, 0};
                    if (r < it.rows) kr = keys_of(a, it.n, it.kv, tok);
                    s_range[b][r] = make_int2(max(kr.lo, it.key_lo), min(kr.hi, it.key_hi));
                }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(&q_full[b]);
        };
        auto out_row = [&](const Item& it, int row) {
            const int pr = it.first_row + row;
            const int tok = pr / group;
            return (it.q0 + tok) * a.q_heads + it.head * group + (pr - tok * group);
        };
        bool ok = true;
        int n0 = 0, used = 0, met = 0;             // key tiles, items with keys and items before
        ok = item_ready(0);
        if (ok && s_item[0].seq >= 0 && key_tiles(s_item[0]) > 0) load_queries(s_item[0], 0);
        for (int x = 0; ok && s_item[x % Cfg::SLOTS].seq >= 0; ++x) {
            const Item& it = s_item[x % Cfg::SLOTS];
            const int nt = key_tiles(it);
            const int k0 = first_tile(it);
            float m[R], l[R], acc[R];
#pragma unroll
            for (int r = 0; r < R; ++r) m[r] = -INFINITY, l[r] = 0.0f, acc[r] = 0.0f;
            // O^T of this group's last tile (in the order of the group's tiles: the i-th) onto the sums
            auto add_o = [&](int i) {
                if (!warp_wait(&o_full[g], i & 1)) return false;
                tc_fence_after();
#pragma unroll
                for (int h = 0; h < 2 * R; h += 16) {
                    float o[16];
                    tmem_ld_16cols(o_addr + h, o);
                    tmem_wait_ld_16(o);
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const int c = h + k;
                        acc[c % R] = fmaf(o[k], c < R ? 1.0f : 1.0f / 32.0f, acc[c % R]);
                    }
                }
                return true;
            };
            bool any = false;
            if (nt > 0) {
                const int b = used & 1;
                if (!warp_wait(&q_full[b], (used >> 1) & 1)) {           // (factors and ranges)
                    ok = false;
                    break;
                }
                // tiles that need no mask for any row
                const int full_hi = s_range[b][0].y, full_lo = s_range[b][it.rows - 1].x;
                for (int j = (n0 & 1) ^ g; j < nt; j += 2) {
                    const int n = n0 + j;
                    const int i = n >> 1;                                // of the group's tiles
                    if (!warp_wait(&c_full[n % Cfg::CST], (n / Cfg::CST) & 1) || !warp_wait(&s_full[g], i & 1)) {
                        ok = false;
                        break;
                    }
                    const float2 sc = s_scale[(n % Cfg::CST) * KEYS + tid];
                    tc_fence_after();
                    float t[2 * R];
#pragma unroll
                    for (int h = 0; h < 2 * R; h += 16) tmem_ld_16cols(s_addr + h, t + h);
#pragma unroll
                    for (int h = 0; h < 2 * R; h += 16) tmem_wait_ld_16(t + h);
#pragma unroll
                    for (int r = 0; r < R; r += 4) {
                        const float4 f = *reinterpret_cast<const float4*>(&s_factor[b][r]);
                        t[r] = fmaf((t[r] + t[R + r]) * sc.x, f.x, sc.y);
                        t[r + 1] = fmaf((t[r + 1] + t[R + r + 1]) * sc.x, f.y, sc.y);
                        t[r + 2] = fmaf((t[r + 2] + t[R + r + 2]) * sc.x, f.z, sc.y);
                        t[r + 3] = fmaf((t[r + 3] + t[R + r + 3]) * sc.x, f.w, sc.y);
                    }
                    const int kb = k0 + j * KEYS;
                    if (kb < full_lo || kb + KEYS > full_hi) {
#pragma unroll
                        for (int r = 0; r < R; ++r) {
                            const int2 range = s_range[b][r];
                            if (kb + tid < range.x || kb + tid >= range.y) t[r] = -INFINITY;
                        }
                    }
                    // the rows' maxima over the tile's keys
                    float (*mine)[R] = s_max[g][i & 1];
#pragma unroll
                    for (int r = 0; r < R; r += 4) {
                        const float4 top = make_float4(warp_max(t[r]), warp_max(t[r + 1]), warp_max(t[r + 2]),
                                                       warp_max(t[r + 3]));
                        if (lane == 0) *reinterpret_cast<float4*>(&mine[warp & 3][r]) = top;
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&x_full[g]);
                    if (any && !add_o(i - 1)) {
                        ok = false;
                        break;
                    }
                    if (!warp_wait(&x_full[g], i & 1)) {
                        ok = false;
                        break;
                    }
                    // P's reference: 2^8 below the largest so far, so that P uses e4m3's range up to 256
                    float now[R];
                    bool grows = false;
#pragma unroll
                    for (int r = 0; r < R; r += 4) {
                        float4 top = *reinterpret_cast<const float4*>(&mine[0][r]);
#pragma unroll
                        for (int w = 1; w < 4; ++w) {
                            const float4 y = *reinterpret_cast<const float4*>(&mine[w][r]);
                            top = make_float4(fmaxf(top.x, y.x), fmaxf(top.y, y.y), fmaxf(top.z, y.z),
                                              fmaxf(top.w, y.w));
                        }
                        now[r] = top.x - 8.0f, now[r + 1] = top.y - 8.0f;
                        now[r + 2] = top.z - 8.0f, now[r + 3] = top.w - 8.0f;
                    }
#pragma unroll
                    for (int r = 0; r < R; ++r) grows = grows || now[r] > m[r];
                    if (grows) {                                         // (the same in all threads of the group)
#pragma unroll
                        for (int r = 0; r < R; ++r) {
                            if (now[r] > m[r]) {
                                const float keep = exp2_fast(m[r] - now[r]);
                                m[r] = now[r];
                                l[r] *= keep;
                                acc[r] *= keep;
                            }
                        }
                    }
                    const float inv_vs = exp2_fast(-sc.y);
                    uint32_t p[R / 4], p2[R / 4];
#pragma unroll
                    for (int r = 0; r < R; r += 4) {
                        float e[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            e[k] = exp2_fast(t[r + k] - (m[r + k] == -INFINITY ? 0.0f : m[r + k]));
                            l[r + k] = fmaf(e[k], inv_vs, l[r + k]);
                        }
                        uint32_t h0, h1, l0, l1;
                        two_codes<5>(e[0], e[1], &h0, &l0);
                        two_codes<5>(e[2], e[3], &h1, &l1);
                        p[r / 4] = h0 | h1 << 16;
                        p2[r / 4] = l0 | l1 << 16;
                    }
                    uint8_t* row = sP + g * Cfg::P_TILE + tid * NP;
                    if constexpr (R == 8) {
                        *reinterpret_cast<uint4*>(row + (swizzled(tid, 0, NP) << 4)) = make_uint4(p[0], p[1], p2[0], p2[1]);
                    } else {
#pragma unroll
                        for (int c = 0; c < R / 16; ++c) {
                            *reinterpret_cast<uint4*>(row + (swizzled(tid, c, NP) << 4)) =
                                make_uint4(p[4 * c], p[4 * c + 1], p[4 * c + 2], p[4 * c + 3]);
                            *reinterpret_cast<uint4*>(row + (swizzled(tid, R / 16 + c, NP) << 4)) =
                                make_uint4(p2[4 * c], p2[4 * c + 1], p2[4 * c + 2], p2[4 * c + 3]);
                        }
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&p_full[g]);
                    any = true;
                }
                n0 += nt;
                ++used;
            }
            if (!ok) break;
            // The next item's queries. Their buffer held those of the item before this one, whose products have all
            // ended (the groups have met since).
            if (!item_ready(x + 1)) {
                ok = false;
                break;
            }
            const Item& next = s_item[(x + 1) % Cfg::SLOTS];
            if (next.seq >= 0 && key_tiles(next) > 0) load_queries(next, used & 1);
            // the group's last tile so far is number (n0 - 1 - ((n0 - 1 - g) & 1)) / 2 of its tiles
            if (any && !add_o((n0 - 1 - ((n0 - 1 - g) & 1)) >> 1)) {
                ok = false;
                break;
            }
            tc_fence_before();
            // The groups' sums meet.
#pragma unroll
            for (int r = 0; r < R; ++r) {
#pragma unroll
                for (int i = 16; i > 0; i >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], i);
                if (lane == 0) s_l[g][warp & 3][r] = l[r];
                if (tid == 0) s_m[g][r] = m[r];
            }
            auto meet = [&](int i) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&j_bar[i]);
                return warp_wait(&j_bar[i], met & 1);
            };
            if (!meet(0)) {
                ok = false;
                break;
            }
            if (g == 1) {
                // (group 1 brings its sums, group 0 writes the item)
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float top = fmaxf(s_m[0][r], s_m[1][r]);
                    const float f = m[r] == -INFINITY ? 0.0f : exp2_fast(m[r] - top);
                    if (has_channel) sO[r * DV + channel] = m[r] == -INFINITY ? 0.0f : acc[r] * f;
                }
            }
            if (!meet(1)) {
                ok = false;
                break;
            }
            if (g == 0) {
                const bool whole = it.pieces == 1;
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    if (r >= it.rows) break;
                    const float m1 = s_m[1][r];
                    const float top = fmaxf(m[r], m1);
                    const float f0 = m[r] == -INFINITY ? 0.0f : exp2_fast(m[r] - top);
                    const float f1 = m1 == -INFINITY ? 0.0f : exp2_fast(m1 - top);
                    const float l0 = (s_l[0][0][r] + s_l[0][1][r]) + (s_l[0][2][r] + s_l[0][3][r]);
                    const float l1 = (s_l[1][0][r] + s_l[1][1][r]) + (s_l[1][2][r] + s_l[1][3][r]);
                    // (a group without keys has a sum of zero; one whose scores are not numbers has no reference)
                    float sum = m[r] == -INFINITY ? l0 : l0 * f0;
                    sum += m1 == -INFINITY ? l1 : l1 * f1;
                    const float o = (m[r] == -INFINITY ? 0.0f : acc[r] * f0) + (has_channel ? sO[r * DV + channel] : 0.0f);
                    const int64_t row = out_row(it, r);
                    if (whole) {
                        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;           // (NaN stays NaN)
                        if (has_channel)
                            static_cast<__nv_bfloat16*>(a.out)[row * DV + channel] = __float2bfloat16_rn(o * inv);
                        if (tid == 0) {
                            if (a.lse)
                                a.lse[row] = sum == 0.0f ? -INFINITY : (top + log2_fast(sum)) * 0.6931471805599453f;
                            if (pieces > 1) parts.ml[row] = make_float2(0.0f, kWholeRow);
                        }
                    } else {
                        if (has_channel && nt > 0) parts.o[(it.piece * parts.rows + row) * DV + channel] = o;
                        if (tid == 0) {
                            parts.ml[it.piece * parts.rows + row] = make_float2(top, sum);
                            // pieces that this sequence does not have are empty
                            if (it.piece == 0)
                                for (int q = it.pieces; q < pieces; ++q)
                                    parts.ml[q * parts.rows + row] = make_float2(-INFINITY, 0.0f);
                        }
                    }
                }
            }
            // (the meeting place is free again)
            if (!meet(2)) {
                ok = false;
                break;
            }
            ++met;
            item_done(x);
        }
        if (!ok && lane == 0) record_error(FP8BS_DEVERR_EPILOGUE_WAIT);
    } else if (warp == Cfg::KEY_WARP) {
        // ---- hands out the items (in rounds, every other one backwards) and brings their keys
        ItemFinder finder;
        finder.base = finder.before = 0;
        finder.loaded = false;
        bool ok = true;
        Stream ks = {0, 0};
        int x = 0;
        const int ctas = gridDim.x, mine = blockIdx.x;
        for (int round = 0; ok; ++round) {
            const int64_t at = static_cast<int64_t>(round) * ctas + (round & 1 ? ctas - 1 - mine : mine);
            const Item it = find_item(finder, a, static_cast<int>(min(at, int64_t{INT32_MAX})), R, KEYS, piece_len, lane);
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
            ok = bring_codes<Cfg, true>(ks, &tmK, a, scales, it, first_tile(it), nt, box_log2, sK, k_full, k_empty,
                                        nullptr, s_scale, c_full, lane);
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
            ok = bring_codes<Cfg, false>(vs, &tmV, a, scales, it, first_tile(it), nt, box_log2, sV, v_full, v_empty,
                                         v_tail, nullptr, nullptr, lane);
        }
        if (!ok && lane == 0) {
            drain_tiles<Cfg::VST>(vs, v_full);
            mbar_wait(v_tail, vs.tails & 1, kDrainLimitNs);
        }
    } else {
        // ---- MMA issuer: S^T of the first two tiles, then per tile O^T and S^T of the tile after next, whose place
        // P's arrival has shown to be free
        constexpr uint32_t idesc_s = idesc_e4m3_f32(KEYS, N1);
        constexpr uint32_t idesc_o = idesc_e4m3_f32(DV, NP) | kIdescBothMN;
        bool ok = true;
        int n0 = 0, used = 0;
        auto product_s = [&](int n, int b) {
            const int st = n % Cfg::KST;
            if (!warp_wait(&k_full[st], (n / Cfg::KST) & 1)) return false;
            tc_fence_after();
            if (elect_one()) {
                const uint32_t ka = smem_addr(sK) + st * Cfg::K_TILE, qa = smem_addr(sQ) + b * Cfg::Q_TILE;
#pragma unroll
                for (int d = 0; d < DK / 32; ++d) {
                    const int c = 32 * d / Cfg::CHK, in = 32 * d % Cfg::CHK;
                    mma_f8(tmem + (n & 1) * N1, smem_desc_rows(ka + c * (KEYS * Cfg::CHK) + in, Cfg::CHK),
                           smem_desc_rows(qa + c * (N1 * Cfg::CHK) + in, Cfg::CHK), idesc_s, d > 0 ? 1u : 0u);
                }
                mma_commit(&s_full[n & 1]);
                mma_commit(&k_empty[st]);
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
            const int b = used & 1;
            ok = warp_wait(&q_full[b], (used >> 1) & 1) && product_s(n0, b) && (nt == 1 || product_s(n0 + 1, b));
            for (int j = 0; ok && j < nt; ++j) {
                const int n = n0 + j;
                const int st = n % Cfg::VST;
                if (!warp_wait(&v_full[st], (n / Cfg::VST) & 1) || !warp_wait(&p_full[n & 1], (n >> 1) & 1)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t va = smem_addr(sV) + st * Cfg::V_TILE, pa = smem_addr(sP) + (n & 1) * Cfg::P_TILE;
#pragma unroll
                    for (int k = 0; k < KEYS / 32; ++k)
                        mma_f8(tmem + Cfg::O_COL + (n & 1) * NP, smem_desc_rows(va + 32 * k * DV, DV),
                               smem_desc_rows(pa + 32 * k * NP, NP), idesc_o, k > 0 ? 1u : 0u);
                    mma_commit(&o_full[n & 1]);
                    mma_commit(&v_empty[st]);
                }
                __syncwarp();
                if (j + 2 < nt) ok = product_s(n + 2, b);
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
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == Cfg::MMA_WARP) tmem_dealloc(tmem, Cfg::TMEM_COLS);
}

// Rows per item: the smallest form that holds the longest sequence's.
int row_form(const fp8bs_paged_attention_args& a) {
    const int64_t rows = a.max_q_len * (a.q_heads / a.cache.heads);
    return rows <= 8 ? 8 : rows <= 16 ? 16 : 32;
}

AttnParts parts_of(const fp8bs_paged_attention_args& a, const AttentionPlan& plan) {
    AttnParts p = {};
    p.rows = a.T * a.q_heads;
    if (plan.pieces > 1) {
        p.o = static_cast<float*>(a.workspace);
        p.ml = reinterpret_cast<float2*>(p.o + plan.pieces * p.rows * a.cache.dv);
    }
    return p;
}

template <class Cfg>
cudaError_t launch_rows(const AttentionMapsFp8& maps, const fp8bs_paged_attention_args& a, const Scales& scales,
                        const AttentionPlan& plan, int num_sms, cudaStream_t stream) {
    auto kernel = attention_rows_kernel<Cfg>;
    cudaError_t e = set_smem(kernel, Cfg::SMEM);
    if (e != cudaSuccess) return e;
    const AttnParts parts = parts_of(a, plan);
    const int64_t items = tile_bound(a, Cfg::R) * a.cache.heads * plan.pieces;
    if (items >= INT32_MAX) return cudaErrorInvalidValue;
    const unsigned grid = static_cast<unsigned>(items < num_sms ? items : num_sms);
    e = launch_pdl(kernel, grid, Cfg::THREADS, Cfg::SMEM, stream, maps.k, maps.v, a, scales, maps.box_log2,
                   plan.piece_len, plan.pieces, parts);
    if (e != cudaSuccess || plan.pieces == 1) return e;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out);
    if (parts.rows <= 1024)
        return launch_pdl(attention_join_kernel<Cfg::DV, 4, true>, static_cast<unsigned>(parts.rows), 128, 0, stream,
                          parts, plan.pieces, out, a.lse);
    return launch_pdl(attention_join_kernel<Cfg::DV, 1, true>, static_cast<unsigned>((parts.rows + 3) / 4), 128, 0,
                      stream, parts, plan.pieces, out, a.lse);
}

template <int DK, int DV>
cudaError_t launch_rows(const AttentionMapsFp8& maps, const fp8bs_paged_attention_args& a, const Scales& scales,
                        const AttentionPlan& plan, int num_sms, cudaStream_t stream) {
    switch (row_form(a)) {
        case 8: return launch_rows<RowsCfg<DK, DV, 8>>(maps, a, scales, plan, num_sms, stream);
        case 16: return launch_rows<RowsCfg<DK, DV, 16>>(maps, a, scales, plan, num_sms, stream);
        default: return launch_rows<RowsCfg<DK, DV, 32>>(maps, a, scales, plan, num_sms, stream);
    }
}

}  // namespace

int attention_fp8_box_log2(const fp8bs_kv_cache& c) {
    // the largest power of two that divides the page, up to a tile
    int b = 4;
    while (b < 7 && c.page_size % (int64_t{2} << b) == 0) ++b;
    return b;
}

int attention_fp8_key_chunk(int64_t dk) { return dk % 128 == 0 ? 128 : 64; }

AttentionPlan attention_fp8_plan(const fp8bs_paged_attention_args& a, int num_sms) {
    const int64_t rows = row_form(a);
    const int64_t group = a.q_heads / a.cache.heads;
    // (sequences of one length, as in decoding, are counted exactly)
    const int64_t items = a.cache.heads * (a.T == a.B * a.max_q_len ? a.B * ((a.max_q_len * group + rows - 1) / rows)
                                                                    : tile_bound(a, static_cast<int>(rows)));
    int64_t keys = key_span(a, static_cast<int>(rows), a.max_q_len, a.max_kv_len);
    if (keys < 1) keys = 1;
    int64_t len = keys;
    if (items * keys < int64_t{8192} * num_sms) {
        // few rows and keys: the number of pieces with the lowest time, in keys, of the busiest CTA, where a piece costs
        // as much as 256 keys more, and joining p of them as much as 256 + 64 p
        int64_t best = 0;
        for (int64_t p = 1; p <= 64 && (p == 1 || keys / p >= 128); ++p) {
            const int64_t l = ((keys + p - 1) / p + KEYS - 1) / KEYS * KEYS;
            const int64_t time = (items * p + num_sms - 1) / num_sms * (l + 256) + (p > 1 ? 256 + 64 * p : 0);
            if (p == 1 || time < best) {
                best = time;
                len = l;
            }
        }
    } else if (items < 8 * num_sms) {
        // many shares' worth of keys: so that the longest sequence of a ragged batch does not finish last on its own
        len = 2048;
    }
    const int64_t most = std::max<int64_t>(1, kMaxPartBytes / std::max<int64_t>(1, part_bytes(a)));
    if (len * most < keys) len = (keys + most - 1) / most;
    len = std::min<int64_t>((len + KEYS - 1) / KEYS * KEYS, int64_t{1} << 30);
    AttentionPlan p;
    p.piece_len = static_cast<int>(len);
    p.pieces = static_cast<int>((keys + len - 1) / len);
    return p;
}

size_t attention_fp8_workspace(const fp8bs_paged_attention_args& a, const AttentionPlan& plan) {
    if (plan.pieces == 1) return 0;
    return static_cast<size_t>(plan.pieces) * static_cast<size_t>(part_bytes(a));
}

cudaError_t launch_paged_attention_fp8(const AttentionMapsFp8& maps, const fp8bs_paged_attention_args& a,
                                       const float* k_scale, const float* v_scale, const AttentionPlan& plan,
                                       int num_sms, cudaStream_t stream) {
    const Scales scales = {k_scale, v_scale};
    switch (a.cache.dk) {
        case 64: return launch_rows<64, 64>(maps, a, scales, plan, num_sms, stream);
        case 128: return launch_rows<128, 128>(maps, a, scales, plan, num_sms, stream);
        default: return launch_rows<192, 128>(maps, a, scales, plan, num_sms, stream);
    }
}

cudaError_t read_error_attention_fp8(unsigned int* out, bool clear, cudaStream_t stream) {
    return read_tu_error(out, clear, stream);
}

}  // namespace fp8bs
