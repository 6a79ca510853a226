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
// The maximum only moves when it has grown by more than 2^8 (kRescale): O is then scaled in TMEM by
// its softmax warps; otherwise P is that much larger than 1 at most, which bf16 and fp32 hold without
// loss, and O is left alone. The row sum is taken from P before its rounding to bf16, so lse is exact
// to binary32; the rounding of P (2^-9 on average per term) is of the size of the output's own.
//
// Two forms (AttnCfg): NQ = 2 query tiles per CTA for chunks, whose softmax warps work on one tile
// while the tensor core works on the other; NQ = 1 with two S buffers for few rows, two CTAs per SM.
// Keys and values come through TMA in boxes of as many slots as divide both the page and the tile.
// Few rows and long keys: the key axis is cut into pieces (AttentionPlan), each CTA leaves its
// unnormalised O, maximum and sum, and a second kernel joins them in key order.
#include "gemm_common.cuh"
#include "quant_math.cuh"

namespace fp8bs {

namespace {

constexpr float kRescale = 8.0f;

template <int DK_, int DV_, int NQ_>
struct AttnCfg {
    static constexpr int DK = DK_, DV = DV_, NQ = NQ_;
    static constexpr int BN = NQ == 2 && DK <= 128 ? 128 : 64;   // keys per tile
    static constexpr int ROWS = NQ * 128;
    static constexpr int SBUF = 2;                               // S buffers: per query tile, or 2
    static constexpr int K_TILE = BN * DK * 2, V_TILE = BN * DV * 2, Q_TILE = 128 * DK * 2;
    static constexpr int KST = DK == 64 ? 4 : DK == 128 ? (NQ == 2 ? 3 : 2) : (NQ == 2 ? 3 : 4);
    static constexpr int VST = DK == 64 ? 4 : DK == 128 ? 2 : (NQ == 2 ? 3 : 4);
    static constexpr int SOFT_WARPS = 4 * NQ;
    static constexpr int LOAD_WARP = SOFT_WARPS;
    static constexpr int MMA_WARP = SOFT_WARPS + 1;
    static constexpr int THREADS = 32 * (SOFT_WARPS + 2);
    static constexpr int CTAS = NQ == 1 && DK <= 128 ? 2 : 1;    // per SM
    static constexpr uint32_t TMEM_COLS = tmem_cols_for(SBUF * BN + NQ * DV);
    static constexpr int BARS = 2 * KST + 2 * VST + 3 * SBUF + 2 * NQ + 1;
    static constexpr int SMEM = 1024 + NQ * Q_TILE + KST * K_TILE + VST * V_TILE + BARS * 8 + 64;
    static_assert(SMEM <= kSmemLimit, "shared memory");
};

// A row tile of one sequence.
struct RowTile {
    int seq, first_row;    // first packed row (i * G + g) of the tile
    int n;                 // new tokens of the sequence
    int q0;                // its first query token
    int kv;                // its keys
};

// The tile'th run of `rows` packed rows, counted over the sequences in order; seq = -1 past the last.
// One warp: eight sequences per lane and step.
__device__ __forceinline__ RowTile find_row_tile(const fp8bs_paged_attention_args& a, int64_t tile,
                                                 int group, int rows, int lane) {
    RowTile t = {-1, 0, 0, 0, 0};
    if (a.max_q_len == 1 && group <= rows && tile < a.B) {
        // single tokens everywhere before it: the tile is its own sequence
        const int q0 = a.q_start[tile], q1 = a.q_start[tile + 1];
        if (q0 == tile && q1 == tile + 1)
            return RowTile{static_cast<int>(tile), 0, 1, q0, a.kv_len[tile]};
    }
    for (int64_t base = 0; base < a.B; base += 256) {
        int start[9], sum = 0;
#pragma unroll
        for (int i = 0; i < 9; ++i) {
            const int64_t b = base + 8 * lane + i;
            start[i] = a.q_start[b < a.B ? b : a.B];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            sum += (max(start[i + 1] - start[i], 0) * group + rows - 1) / rows;
        int incl = sum;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, incl, m);
            if (lane >= m) incl += o;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, incl > tile);
        if (hit) {
            const int src = __ffs(hit) - 1;
            if (lane == src) {
                int64_t left = tile - (incl - sum);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int n = max(start[i + 1] - start[i], 0);
                    const int tiles = (n * group + rows - 1) / rows;
                    if (t.seq < 0 && left < tiles)
                        t = RowTile{static_cast<int>(base) + 8 * lane + i,
                                    static_cast<int>(left) * rows, n, start[i], 0};
                    left -= tiles;
                }
                t.kv = a.kv_len[t.seq];
            }
            t.seq = __shfl_sync(0xffffffffu, t.seq, src);
            t.first_row = __shfl_sync(0xffffffffu, t.first_row, src);
            t.n = __shfl_sync(0xffffffffu, t.n, src);
            t.q0 = __shfl_sync(0xffffffffu, t.q0, src);
            t.kv = __shfl_sync(0xffffffffu, t.kv, src);
            return t;
        }
        tile -= __shfl_sync(0xffffffffu, incl, 31);
    }
    return t;
}

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

__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}

// TMA load of one box {64 channels, 1 head, slots, 1 page} of a cache.
__device__ __forceinline__ void tma_load_4d(uint32_t smem_dst, const CUtensorMap* map, uint64_t* bar,
                                            int32_t c0, int32_t c1, int32_t c2, int32_t c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_addr(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
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

// Descriptor of an MN-major operand with 128-byte swizzle: blocks of 64 channels x all keys, `block`
// bytes apart; within a block one key per 128-byte row, 8-key swizzle atoms 1024 bytes apart.
__device__ __forceinline__ uint64_t smem_desc_mn_sw128(uint32_t addr, uint32_t block) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((addr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(block >> 4) << 16;         // leading byte offset: next 64 channels
    d |= static_cast<uint64_t>(1024 >> 4) << 32;          // stride byte offset: next 8 keys
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}

constexpr uint32_t kIdescBMajorMN = 1u << 16;

struct AttnParts {
    float* o;      // [piece][T * q_heads][DV], unnormalised
    float2* ml;    // [piece][T * q_heads]: (maximum in log2 units, sum)
    int64_t rows;  // T * q_heads
};

template <class Cfg>
__global__ void __launch_bounds__(Cfg::THREADS, Cfg::CTAS)
    paged_attention_kernel(const __grid_constant__ CUtensorMap tmK,
                           const __grid_constant__ CUtensorMap tmV,
                           const __grid_constant__ fp8bs_paged_attention_args a, const int box_log2,
                           const int piece_len, const int pieces, const AttnParts parts) {
    constexpr int DK = Cfg::DK, DV = Cfg::DV, NQ = Cfg::NQ, BN = Cfg::BN;
    extern __shared__ uint8_t smem_raw[];
    __shared__ RowTile s_tile;
    __shared__ uint32_t s_tmem;
    uint8_t* smem = align_1024(smem_raw);
    uint8_t* sQ = smem;                                   // [NQ][DK/64][128 rows][128 bytes]
    uint8_t* sK = sQ + NQ * Cfg::Q_TILE;                  // [KST][DK/64][BN][128 bytes]
    uint8_t* sV = sK + Cfg::KST * Cfg::K_TILE;            // [VST][DV/64][BN][128 bytes]
    uint64_t* k_full = reinterpret_cast<uint64_t*>(sV + Cfg::VST * Cfg::V_TILE);
    uint64_t* k_empty = k_full + Cfg::KST;
    uint64_t* v_full = k_empty + Cfg::KST;
    uint64_t* v_empty = v_full + Cfg::VST;
    uint64_t* s_full = v_empty + Cfg::VST;                // [SBUF]
    uint64_t* p_full = s_full + Cfg::SBUF;                // [SBUF][2 halves]
    uint64_t* o_done = p_full + 2 * Cfg::SBUF;            // [NQ]
    uint64_t* drain = o_done + NQ;                        // [NQ]
    uint64_t* v_tail = drain + NQ;                        // the last, partly valid value tile

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int heads = static_cast<int>(a.cache.heads);
    const int group = static_cast<int>(a.q_heads / a.cache.heads);
    // heads fastest: neighbouring CTAs read the same slots; later tiles (longer keys) first
    const int64_t tiles = gridDim.x / heads;
    const int64_t tile = tiles - 1 - blockIdx.x / heads;
    const int head = blockIdx.x % heads;
    const int piece = blockIdx.y;

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
            mbar_init(&p_full[2 * i], 4);
            mbar_init(&p_full[2 * i + 1], 4);
        }
        for (int i = 0; i < NQ; ++i) {
            mbar_init(&o_done[i], 1);
            mbar_init(&drain[i], 1);
        }
        mbar_init(v_tail, 1);
        fence_barrier_init();
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }
    grid_dependency_wait();
    grid_launch_dependents();
    if (warp == 0) {
        const RowTile t = find_row_tile(a, tile, group, Cfg::ROWS, lane);
        if (lane == 0) {
            s_tile = t;
            if (t.seq >= 0 && (t.n > a.max_q_len || t.kv > a.max_kv_len || t.kv < 0 ||
                               t.q0 < 0 || t.q0 + static_cast<int64_t>(t.n) > a.T)) {
                record_error(FP8BS_DEVERR_INDEX);
                s_tile.seq = -1;
            }
        }
    }
    if (warp == Cfg::MMA_WARP) tmem_alloc(&s_tmem, Cfg::TMEM_COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    const RowTile rt = s_tile;

    // Keys of the tile: [key_lo, key_hi) over all its rows, cut to this piece, in whole key tiles.
    const int rows_all = rt.n * group;
    const int rows = min(Cfg::ROWS, rows_all - rt.first_row);       // valid rows of this CTA
    int key_lo = 0, key_hi = 0;
    if (rt.seq >= 0) {
        key_lo = keys_of(a, rt.n, rt.kv, rt.first_row / group).lo;
        key_hi = keys_of(a, rt.n, rt.kv, (rt.first_row + rows - 1) / group).hi;
        const int64_t p0 = static_cast<int64_t>(piece) * piece_len;
        key_lo = static_cast<int>(max(static_cast<int64_t>(key_lo), p0));
        key_hi = static_cast<int>(min(static_cast<int64_t>(key_hi), p0 + piece_len));
    }
    const int k0 = key_lo / BN * BN;
    const int nt = key_hi > key_lo ? (key_hi - k0 + BN - 1) / BN : 0;

    if (rt.seq >= 0 && nt == 0) {
        // No key for any row: zeros (or, of several pieces, an empty part).
        for (int r = threadIdx.x; r < rows; r += Cfg::THREADS) {
            const int pr = rt.first_row + r;
            const int64_t row =
                (rt.q0 + pr / group) * a.q_heads + head * group + pr % group;
            if (pieces > 1) {
                parts.ml[piece * parts.rows + row] = make_float2(-INFINITY, 0.0f);
            } else {
                uint4* o = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + row * DV);
                for (int c = 0; c < DV / 8; ++c) o[c] = make_uint4(0, 0, 0, 0);
                if (a.lse) a.lse[row] = -INFINITY;
            }
        }
    } else if (rt.seq >= 0) {
        // Queries into shared memory (K-major, 128-byte swizzle); a negative scale turns their signs,
        // so that the row maximum is always that of the largest S.
        const uint32_t flip = a.scale < 0.0f ? 0x80008000u : 0u;
        for (int i = threadIdx.x; i < Cfg::ROWS * (DK / 8); i += Cfg::THREADS) {
            const int r = i / (DK / 8);
            const int c = i - r * (DK / 8);
            uint4 v = make_uint4(0, 0, 0, 0);
            if (r < rows) {
                const int pr = rt.first_row + r;
                const int tok = pr / group;
                v = __ldg(reinterpret_cast<const uint4*>(
                              static_cast<const __nv_bfloat16*>(a.q) +
                              (rt.q0 + tok) * a.q_token_stride +
                              (head * group + pr - tok * group) * a.q_head_stride) + c);
                v.x ^= flip; v.y ^= flip; v.z ^= flip; v.w ^= flip;
            }
            *reinterpret_cast<uint4*>(sQ + (r >> 7) * Cfg::Q_TILE + (c >> 3) * (128 * 128) +
                                      (r & 127) * 128 + (((c & 7) ^ (r & 7)) << 4)) = v;
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncthreads();

        if (warp == Cfg::LOAD_WARP) {
            // ---- TMA producer: all lanes issue, lane l the boxes l, l + 32, ... of a tile.
            const int box = 1 << box_log2;
            const int boxes = BN >> box_log2;
            const int page_size = static_cast<int>(a.cache.page_size);
            const int32_t* table = a.page_table + rt.seq * a.table_stride;
            const int per_lane = (boxes + 31) / 32;
            constexpr int MAXB = BN / 32;
            int page[MAXB], slot[MAXB];
            auto lookup = [&](int j) {
#pragma unroll
                for (int i = 0; i < MAXB; ++i) {
                    const int b = lane + 32 * i;
                    const int key = k0 + j * BN + b * box;
                    page[i] = -1;
                    slot[i] = 0;
                    if (i < per_lane && b < boxes && key < rt.kv) {
                        const int pg = key / page_size;
                        slot[i] = key - pg * page_size;
                        page[i] = table[pg];
                    }
                }
            };
            bool ok = true;
            int kst = 0, vst = 0;
            uint32_t kph = 0, vph = 0;
            int k_issued = 0, v_issued = 0;
            bool tail_issued = false;
            lookup(0);
            for (int j = 0; ok && j < nt; ++j) {
                int pg[MAXB], sl[MAXB];
                const int key0 = k0 + j * BN;
                const int live = min(boxes, (rt.kv - key0 + box - 1) >> box_log2);
                bool bad = false;
#pragma unroll
                for (int i = 0; i < MAXB; ++i) {
                    pg[i] = page[i];
                    sl[i] = slot[i];
                    const int b = lane + 32 * i;
                    // out of the cache: a coordinate past the end, which reads as zeros
                    if (i < per_lane && b < live && (pg[i] < 0 || pg[i] >= a.cache.pages)) {
                        bad = true;
                        pg[i] = static_cast<int>(a.cache.pages);
                    }
                }
                if (bad) record_error(FP8BS_DEVERR_INDEX);
                if (j + 1 < nt) lookup(j + 1);
                // keys
                if (!warp_wait(&k_empty[kst], kph ^ 1)) { ok = false; break; }
                if (lane == 0) mbar_arrive_expect_tx(&k_full[kst], static_cast<uint32_t>(live * box * DK * 2));
                __syncwarp();
#pragma unroll
                for (int i = 0; i < MAXB; ++i) {
                    const int b = lane + 32 * i;
                    if (i < per_lane && b < live)
#pragma unroll
                        for (int d = 0; d < DK / 64; ++d)
                            tma_load_4d(smem_addr(sK) + kst * Cfg::K_TILE + d * (BN * 128) + b * box * 128,
                                        &tmK, &k_full[kst], d * 64, head, sl[i], pg[i]);
                }
                ++k_issued;
                if (++kst == Cfg::KST) { kst = 0; kph ^= 1; }
                // values; those of the last tile are cleared past the sequence's end before they count
                if (!warp_wait(&v_empty[vst], vph ^ 1)) { ok = false; break; }
                const bool partial = rt.kv - key0 < BN;
                uint64_t* bar = partial ? v_tail : &v_full[vst];
                if (lane == 0) mbar_arrive_expect_tx(bar, static_cast<uint32_t>(live * box * DV * 2));
                __syncwarp();
#pragma unroll
                for (int i = 0; i < MAXB; ++i) {
                    const int b = lane + 32 * i;
                    if (i < per_lane && b < live)
#pragma unroll
                        for (int d = 0; d < DV / 64; ++d)
                            tma_load_4d(smem_addr(sV) + vst * Cfg::V_TILE + d * (BN * 128) + b * box * 128,
                                        &tmV, bar, d * 64, head, sl[i], pg[i]);
                }
                if (partial) {
                    tail_issued = true;
                    if (!warp_wait(v_tail, 0)) { ok = false; break; }
                    const int keep = rt.kv - key0;
                    for (int i = lane; i < (BN - keep) * 8 * (DV / 64); i += 32) {
                        const int d = i / ((BN - keep) * 8);
                        const int rem = i - d * (BN - keep) * 8;
                        *reinterpret_cast<uint4*>(sV + vst * Cfg::V_TILE + d * (BN * 128) +
                                                  keep * 128 + rem * 16) = make_uint4(0, 0, 0, 0);
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&v_full[vst]);
                } else {
                    ++v_issued;
                }
                if (++vst == Cfg::VST) { vst = 0; vph ^= 1; }
            }
            if (!ok) {
                // drain what is in flight before the CTA gives up its shared memory
                if (lane == 0) {
                    record_error(FP8BS_DEVERR_PRODUCER_WAIT);
                    for (int i = max(0, k_issued - Cfg::KST); i < k_issued; ++i)
                        if (!mbar_wait(&k_full[i % Cfg::KST], (i / Cfg::KST) & 1, kDrainLimitNs))
                            record_error(FP8BS_DEVERR_DRAIN_WAIT);
                    for (int i = max(0, v_issued - Cfg::VST); i < v_issued; ++i)
                        if (!mbar_wait(&v_full[i % Cfg::VST], (i / Cfg::VST) & 1, kDrainLimitNs))
                            record_error(FP8BS_DEVERR_DRAIN_WAIT);
                    if (tail_issued && !mbar_wait(v_tail, 0, kDrainLimitNs))
                        record_error(FP8BS_DEVERR_DRAIN_WAIT);
                }
            }
        } else if (warp == Cfg::MMA_WARP) {
            // ---- MMA issuer. Per key tile and query tile: O += P(j) V(j) in two halves as the softmax
            // hands them over, then S of the tile's next keys, which takes P's place (the tensor core
            // works in order). With two query tiles one's products run under the other's softmax.
            constexpr uint32_t idesc_qk = idesc_bf16_f32(128, BN);
            constexpr uint32_t idesc_pv = idesc_bf16_f32(128, DV) | kIdescBMajorMN;
            const uint32_t q_addr = smem_addr(sQ);
            const uint32_t o_tmem = tmem + Cfg::SBUF * BN;
            bool ok = true;
            int ended = 0;                 // query tiles whose last product has been committed
            auto qk = [&](int q, int j) {  // S(j): buffer q (two tiles) or j % 2
                const int st = j % Cfg::KST;
                if (q == 0) {
                    if (!warp_wait(&k_full[st], (j / Cfg::KST) & 1)) return false;
                    tc_fence_after();
                }
                const int buf = NQ == 2 ? q : j & 1;
                const uint32_t k_addr = smem_addr(sK) + st * Cfg::K_TILE;
                if (elect_one()) {
#pragma unroll
                    for (int d = 0; d < DK / 16; ++d)
                        mma_bf16(tmem + buf * BN,
                                 smem_desc_k_sw128(q_addr + q * Cfg::Q_TILE + (d / 4) * (128 * 128) +
                                                   (d % 4) * 32),
                                 smem_desc_k_sw128(k_addr + (d / 4) * (BN * 128) + (d % 4) * 32),
                                 idesc_qk, d > 0 ? 1u : 0u);
                    mma_commit(&s_full[buf]);
                    if (q == NQ - 1) mma_commit(&k_empty[st]);
                }
                __syncwarp();
                return true;
            };
            for (int q = 0; ok && q < NQ; ++q) ok = qk(q, 0);
            if (ok && NQ == 1 && nt > 1) ok = qk(0, 1);
            for (int j = 0; ok && j < nt; ++j) {
                const int st = j % Cfg::VST;
                const uint32_t pph = NQ == 2 ? j & 1 : (j >> 1) & 1;
                const uint32_t v_addr = smem_addr(sV) + st * Cfg::V_TILE;
                if (!warp_wait(&v_full[st], (j / Cfg::VST) & 1)) {
                    ok = false;
                    break;
                }
#pragma unroll
                for (int q = 0; q < NQ; ++q) {
                    const int buf = NQ == 2 ? q : j & 1;
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        if (!ok || !warp_wait(&p_full[2 * buf + half], pph)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        if (elect_one()) {
#pragma unroll
                            for (int k = half * (BN / 32); k < (half + 1) * (BN / 32); ++k)
                                mma_bf16_ta(o_tmem + q * DV, tmem + buf * BN + 8 * k,
                                            smem_desc_mn_sw128(v_addr + k * 2048, BN * 128), idesc_pv,
                                            j > 0 || k > 0 ? 1u : 0u);
                            if (half == 1) {
                                mma_commit(&o_done[q]);
                                if (q == NQ - 1) mma_commit(&v_empty[st]);
                                if (j == nt - 1) mma_commit(&drain[q]);
                            }
                        }
                        __syncwarp();
                    }
                    if (!ok) break;
                    if (j == nt - 1) ++ended;
                    const int next = NQ == 2 ? j + 1 : j + 2;
                    if (next < nt) ok = qk(q, next);
                }
            }
            if (!ok && lane == 0) record_error(FP8BS_DEVERR_MMA_WAIT);
            if (elect_one())
                for (int q = ended; q < NQ; ++q) mma_commit(&drain[q]);
            __syncwarp();
            for (int q = 0; q < NQ; ++q)
                if (!warp_wait(&drain[q], 0) && lane == 0) record_error(FP8BS_DEVERR_DRAIN_WAIT);
        } else {
            // ---- softmax warps: thread = row
            const int q = warp >> 2;
            const int quarter = warp & 3;
            const int r = q * 128 + quarter * 32 + lane;          // row of the CTA
            const bool idle = q * 128 + quarter * 32 >= rows;     // no valid row in this warp
            const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
            const uint32_t o_tmem = tmem + lanes + Cfg::SBUF * BN + q * DV;
            // (a scale of zero: any tiny factor keeps -inf apart from the finite scores)
            const float c = fmaxf(fabsf(a.scale) * 1.4426950408889634f, 1e-30f);
            const int pr = rt.first_row + min(r, rows - 1);
            const KeyRange kr = keys_of(a, rt.n, rt.kv, pr / group);
            // tiles that need no mask for any row of this warp's query tile
            const int last_row = min(rows, (q + 1) * 128) - 1;
            const int full_hi = keys_of(a, rt.n, rt.kv, (rt.first_row + min(q * 128, rows - 1)) / group).hi;
            const int full_lo = keys_of(a, rt.n, rt.kv, (rt.first_row + max(last_row, 0)) / group).lo;
            const int row_lo = max(kr.lo, key_lo), row_hi = min(kr.hi, key_hi);
            float m = -INFINITY;           // maximum in use, raw score
            float l = 0.0f;
            bool ok = true;
            for (int j = 0; j < nt; ++j) {
                const int buf = NQ == 2 ? q : j & 1;
                const uint32_t sph = NQ == 2 ? j & 1 : (j >> 1) & 1;
                if (!warp_wait(&s_full[buf], sph)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (!idle) {
                    const uint32_t s_tmem_row = tmem + lanes + buf * BN;
                    float s[BN];
#pragma unroll
                    for (int i = 0; i < BN / 32; ++i) tmem_ld_32cols(s_tmem_row + 32 * i, s + 32 * i);
#pragma unroll
                    for (int i = 0; i < BN / 32; ++i) tmem_wait_ld_32(s + 32 * i);
                    const int kb = k0 + j * BN;
                    if (kb < full_lo || kb < key_lo || kb + BN > full_hi || kb + BN > key_hi) {
                        const int lo = row_lo - kb, hi = row_hi - kb;
#pragma unroll
                        for (int i = 0; i < BN; ++i)
                            if (i < lo || i >= hi) s[i] = -INFINITY;
                    }
                    float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                    for (int i = 4; i < BN; i += 4) {
                        mx[0] = fmaxf(mx[0], s[i]);
                        mx[1] = fmaxf(mx[1], s[i + 1]);
                        mx[2] = fmaxf(mx[2], s[i + 2]);
                        mx[3] = fmaxf(mx[3], s[i + 3]);
                    }
                    const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                    const bool grow = (top - m) * c > kRescale || (m == -INFINITY && top > m);
                    if (__any_sync(0xffffffffu, grow)) {
                        const float keep = grow ? exp2_fast((m - top) * c) : 1.0f;
                        if (grow) m = top;
                        l *= keep;
                        if (j > 0) {
                            if (!warp_wait(&o_done[q], (j - 1) & 1)) {
                                ok = false;
                                break;
                            }
                            tc_fence_after();
#pragma unroll 1
                            for (int i = 0; i < DV / 32; ++i) {
                                float o[32];
                                tmem_ld_32cols(o_tmem + 32 * i, o);
                                tmem_wait_ld_32(o);
#pragma unroll
                                for (int k = 0; k < 32; ++k) o[k] *= keep;
                                tmem_st_32cols(o_tmem + 32 * i, reinterpret_cast<const uint32_t*>(o));
                            }
                        }
                    }
                    const float mc = m == -INFINITY ? 0.0f : m * c;
                    float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
                    const float2 c2 = make_float2(c, c), mc2 = make_float2(-mc, -mc);
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        constexpr int H = BN / 2;
#pragma unroll
                        for (int i = 0; i < H / 32; ++i) {
                            uint32_t p[16];
#pragma unroll
                            for (int k = 0; k < 16; ++k) {
                                const int e = half * H + 32 * i + 2 * k;
                                float2 x = __ffma2_rn(make_float2(s[e], s[e + 1]), c2, mc2);
                                x.x = exp2_fast(x.x);
                                x.y = exp2_fast(x.y);
                                sum[k & 1] = __fadd2_rn(sum[k & 1], x);
                                p[k] = pack_bf16x2(x.x, x.y);
                            }
                            tmem_st_16cols(s_tmem_row + half * (H / 2) + 16 * i, p);
                        }
                        tmem_wait_st();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&p_full[2 * buf + half]);
                    }
                    l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                } else if (lane == 0) {
                    mbar_arrive(&p_full[2 * buf]);
                    mbar_arrive(&p_full[2 * buf + 1]);
                }
            }
            // every product of this query tile is done (o_done's parity would not tell: with two S
            // buffers the last two products may complete before this warp looks)
            if (ok && !warp_wait(&drain[q], 0)) ok = false;
            if (!ok && lane == 0) record_error(FP8BS_DEVERR_EPILOGUE_WAIT);
            tc_fence_after();
            if (ok && !idle) {
                const int64_t row = (rt.q0 + pr / group) * a.q_heads + head * group + pr % group;
                const bool live = r < rows;
                const float mc = m == -INFINITY ? -INFINITY : m * c;
                if (pieces > 1) {
                    float* dst = parts.o + (piece * parts.rows + row) * DV;
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
                    if (live) parts.ml[piece * parts.rows + row] = make_float2(mc, l);
                } else {
                    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
                    uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + row * DV);
#pragma unroll
                    for (int i = 0; i < DV / 32; ++i) {
                        float o[32];
                        tmem_ld_32cols(o_tmem + 32 * i, o);
                        tmem_wait_ld_32(o);
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
                        a.lse[row] = l > 0.0f ? (mc + log2_fast(l)) * 0.6931471805599453f : -INFINITY;
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == Cfg::MMA_WARP) tmem_dealloc(tmem, Cfg::TMEM_COLS);
}

// Join the pieces of a row in key order: one warp per row, the pieces' maxima and sums across lanes,
// then DV / 32 channels per lane.
template <int DV>
__global__ void __launch_bounds__(128) attention_join_kernel(const AttnParts parts, int pieces,
                                                             __nv_bfloat16* out, float* lse) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    if (row >= parts.rows) return;
    float top = -INFINITY;
    for (int p = lane; p < pieces; p += 32) top = fmaxf(top, parts.ml[p * parts.rows + row].x);
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
    constexpr int PER = DV / 32;
    float o[PER] = {}, l = 0.0f;
    if (top > -INFINITY) {
        for (int p = 0; p < pieces; ++p) {
            const float2 ml = parts.ml[p * parts.rows + row];
            if (ml.x == -INFINITY) continue;
            const float w = exp2_fast(ml.x - top);
            l = fmaf(w, ml.y, l);
            const float* src = parts.o + (p * parts.rows + row) * DV + PER * lane;
#pragma unroll
            for (int i = 0; i < PER; i += 2) {
                const float2 v = *reinterpret_cast<const float2*>(src + i);
                o[i] = fmaf(w, v.x, o[i]);
                o[i + 1] = fmaf(w, v.y, o[i + 1]);
            }
        }
    }
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
    uint32_t* dst = reinterpret_cast<uint32_t*>(out + row * DV) + PER / 2 * lane;
#pragma unroll
    for (int i = 0; i < PER / 2; ++i) dst[i] = pack_bf16x2(o[2 * i] * inv, o[2 * i + 1] * inv);
    if (lse && lane == 0)
        lse[row] = l > 0.0f ? (top + log2_fast(l)) * 0.6931471805599453f : -INFINITY;
}

int64_t tile_bound(const fp8bs_paged_attention_args& a, int rows) {
    // sum over sequences of ceil(n G / rows) <= T G / rows + min(B, T) (a sequence without queries
    // has no tile)
    const int64_t group = a.q_heads / a.cache.heads;
    return a.T * group / rows + (a.B < a.T ? a.B : a.T);
}

// Whether the two-tile form is used: its 256 rows have to be filled by the average sequence.
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
                             const fp8bs_paged_attention_args& a, int box_log2,
                             const AttentionPlan& plan, cudaStream_t stream) {
    auto kernel = paged_attention_kernel<Cfg>;
    cudaError_t e = set_smem(kernel, Cfg::SMEM);
    if (e != cudaSuccess) return e;
    const AttnParts parts = attention_parts(a, plan);
    const dim3 grid(static_cast<unsigned>(tile_bound(a, Cfg::ROWS) * a.cache.heads),
                    static_cast<unsigned>(plan.pieces));
    e = launch_pdl(kernel, grid, Cfg::THREADS, Cfg::SMEM, stream, tmK, tmV, a, box_log2, plan.piece_len,
                   plan.pieces, parts);
    if (e != cudaSuccess || plan.pieces == 1) return e;
    return launch_pdl(attention_join_kernel<Cfg::DV>, static_cast<unsigned>((parts.rows + 3) / 4), 128, 0,
                      stream, parts, plan.pieces, static_cast<__nv_bfloat16*>(a.out), a.lse);
}

}  // namespace

AttentionPlan attention_plan(const fp8bs_paged_attention_args& a, int num_sms) {
    const bool two = two_tiles(a);
    const int64_t items = tile_bound(a, two ? 256 : 128) * a.cache.heads;
    const int64_t slots = static_cast<int64_t>(num_sms) * (!two && a.cache.dk <= 128 ? 2 : 1);
    const int64_t keys = a.max_kv_len > 0 ? a.max_kv_len : 1;
    AttentionPlan p;
    int64_t len;
    if (two) {
        // chunks: only to fill the GPU, in pieces long enough to pay for the joining
        const int64_t want = items >= slots ? 1 : slots / items;
        len = (keys + want - 1) / want;
        if (len < 512) len = 512;
    } else {
        // few rows: as many pieces as fill the GPU once, and none so long that the longest sequence
        // of a ragged batch finishes last on its own
        len = (items * keys + slots - 1) / slots;
        if (len > 1024) len = 1024;
        if (len < 128) len = 128;
        if (items >= 8 * slots) len = keys;
    }
    len = (len + 127) / 128 * 128;
    if (len > (int64_t{1} << 30)) len = int64_t{1} << 30;
    p.piece_len = static_cast<int>(len);
    p.pieces = static_cast<int>((keys + len - 1) / len);
    if (p.pieces > 65535) {
        p.piece_len = static_cast<int>(((keys + 65534) / 65535 + 127) / 128 * 128);
        p.pieces = static_cast<int>((keys + p.piece_len - 1) / p.piece_len);
    }
    return p;
}

size_t attention_workspace(const fp8bs_paged_attention_args& a, const AttentionPlan& plan) {
    if (plan.pieces == 1) return 0;
    return static_cast<size_t>(plan.pieces) * static_cast<size_t>(a.T * a.q_heads) *
           (static_cast<size_t>(a.cache.dv) * 4 + 8);
}

cudaError_t launch_paged_attention(const CUtensorMap& tmK, const CUtensorMap& tmV,
                                   const fp8bs_paged_attention_args& a, int box_log2,
                                   const AttentionPlan& plan, cudaStream_t stream) {
    const bool two = two_tiles(a);
    switch (a.cache.dk) {
        case 64:
            return two ? launch_attention<AttnCfg<64, 64, 2>>(tmK, tmV, a, box_log2, plan, stream)
                       : launch_attention<AttnCfg<64, 64, 1>>(tmK, tmV, a, box_log2, plan, stream);
        case 128:
            return two ? launch_attention<AttnCfg<128, 128, 2>>(tmK, tmV, a, box_log2, plan, stream)
                       : launch_attention<AttnCfg<128, 128, 1>>(tmK, tmV, a, box_log2, plan, stream);
        default:
            return two ? launch_attention<AttnCfg<192, 128, 2>>(tmK, tmV, a, box_log2, plan, stream)
                       : launch_attention<AttnCfg<192, 128, 1>>(tmK, tmV, a, box_log2, plan, stream);
    }
}

int attention_box_log2(int64_t page_size) {
    // slots per TMA box: the largest power of two that divides the page and the key tiles (64 or 128)
    int l = 0;
    while (l < 6 && page_size % (int64_t{2} << l) == 0) ++l;
    return l;
}

cudaError_t read_error_attention(unsigned int* out, bool clear, cudaStream_t stream) {
    return read_tu_error(out, clear, stream);
}

}  // namespace fp8bs
