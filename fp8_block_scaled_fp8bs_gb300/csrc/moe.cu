// moe.cu -- the experts of a mixture-of-experts layer for a few tokens (fp8bs_moe_experts), two
// kernels ("DeepSeek-V3 Administrator & Developer Guide", §6.4 MoE expert routing; the products as in
// §8.5.3 fp8_gemm_kernel):
//   moe_up_kernel    h = silu(Wg x) * (Wu x) of every active expert, quantised per 128 channels
//   moe_down_kernel  y[t] = sum over active experts of weight[t, e] * W2 h, in binary32, bf16 once
//
// Bound by the weights' bytes: 3 D I per active expert, read once, while the tokens (64 at most) are few.
// So 128 rows of weights take the MMA's M side and the tokens its N side. The up kernel takes up to 16
// tokens whole, of more it gathers those that chose the expert (TMA, four rows at a time); the down kernel takes
// all. The partial of each K block is scaled and added to binary32 registers by the promotion warps, as in
// gemm_swapab.cu.
//
// The choices meet the products in the factors: the up kernel writes zero codes and a zero factor for a
// token that did not choose the expert, and otherwise the factor (block scale of h) * (weight of the
// expert), so that the down kernel's accumulators run over all experts without a break: one sum per output,
// in expert and channel order, the same bits every time.
//
// Measured for 32 experts of 2048 channels, D = 7168, 8 chosen per token (1.4 GB of weights when all are met):
// 64 tokens 255 us for the layer (up, down and router overlap), 5.5 TB/s (0.83 of a copy's rate);
// 7 tokens 186 us for 1.2 GB (0.98); one token 67 us for 353 MB (0.79): the router comes first,
// and the grids are 128 and 112 CTAs for 152 SMs. At 64 tokens the down kernel's 112 CTAs have 64 columns to scale
// per K block, 87 us where its weights take 70.
#include "gemm_common.cuh"
#include "quant_math.cuh"

namespace fp8bs {

namespace {

// Warps of both kernels: 0 brings the stages' weights and 11 their activations, 1 and 10 issue the MMAs of the first and
// second weight tile of a stage, 2..5 promote the first, 6..9 the second (TMEM lanes: warp % 4). (One warp for weights
// and activations: issuing a stage's copies one after another took longer than its weights do, 64 tokens 265 us
// instead of 255; two tokens 14.7 instead of 15.0.)
constexpr int MOE_PROMOTE_WARP0 = 2;
constexpr int MOE_PROMOTE_WARPS = 8;
constexpr int MOE_ISSUER2 = MOE_PROMOTE_WARP0 + MOE_PROMOTE_WARPS;
constexpr int MOE_LOADER2 = MOE_ISSUER2 + 1;
constexpr int MOE_THREADS = (MOE_LOADER2 + 1) * 32;
constexpr int MOE_NBUF = 4;                           // TMEM buffers (K blocks in flight)
constexpr int kMaxExperts = 512;

// Which experts have tokens, and which tokens: built by every CTA from the ids.
struct Routing {
    unsigned long long mask[kMaxExperts];             // bit t: token t chose the expert
    uint16_t active[kMaxExperts];                     // the experts with tokens, in order
    int n;
};

// Dynamic shared memory of both kernels, at most: what Routing and the TMEM address leave.
constexpr int kMoeSmem = kSmemLimit - 6144;
static_assert(sizeof(Routing) + 64 <= 6144, "static shared memory");

// All threads of the CTA: before the ids are there, and when they are (`first`: this thread's own; a block barrier
// between the two, and one at the end).
__device__ __forceinline__ void clear_routing(Routing& r, const MoeArgs& a) {
    for (int e = threadIdx.x; e < a.E; e += MOE_THREADS) r.mask[e] = 0;
}

__device__ __forceinline__ int first_id(const MoeArgs& a) {
    return threadIdx.x < a.T * a.top_k ? a.ids[threadIdx.x] : -1;
}

__device__ __forceinline__ void build_routing(Routing& r, const MoeArgs& a, int first, bool report) {
    for (int s = threadIdx.x; s < a.T * a.top_k; s += MOE_THREADS) {
        const int e = s == threadIdx.x ? first : a.ids[s];
        if (e >= 0 && e < a.E)
            atomicOr(&r.mask[e], 1ull << (s / a.top_k));
        else if (e != -1 && report)
            record_error(FP8BS_DEVERR_INDEX);
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        int n = 0;
        for (int base = 0; base < a.E; base += 32) {
            const bool on = base + lane < a.E && r.mask[base + lane] != 0;
            const unsigned b = __ballot_sync(0xffffffffu, on);
            if (on) r.active[n + __popc(b & ((1u << lane) - 1))] = static_cast<uint16_t>(base + lane);
            n += __popc(b);
        }
        if (lane == 0) r.n = n;
    }
    __syncthreads();
}

// Barriers of a CTA.
struct MoeBars {
    uint64_t *full, *empty, *tfull, *tempty, *drain;
};

__device__ __forceinline__ MoeBars carve_bars(uint8_t* p, int stages) {
    MoeBars b;
    b.full = reinterpret_cast<uint64_t*>(p);
    b.empty = b.full + stages;
    b.tfull = b.empty + stages;
    b.tempty = b.tfull + MOE_NBUF;
    b.drain = b.tempty + MOE_NBUF;
    return b;
}

constexpr int moe_bar_bytes(int stages) { return (2 * stages + 2 * MOE_NBUF + 1) * 8; }

// Position of the i-th set bit (counting from 0); there are more than i.
__device__ __forceinline__ int nth_bit(unsigned long long mask, int i) {
    for (; i > 0; --i) mask &= mask - 1;
    return __ffsll(mask) - 1;
}

// Rows r0 .. r3 of a map with boxes of one row, one after another at dst.
__device__ __forceinline__ void tma_gather4(void* smem_dst, const CUtensorMap* map, uint64_t* bar, int32_t col,
                                            int32_t r0, int32_t r1, int32_t r2, int32_t r3) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(smem_addr(smem_dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_addr(bar)), "r"(col), "r"(r0), "r"(r1), "r"(r2), "r"(r3)
        : "memory");
}

// Scales of the weights along a CTA's sequence of K blocks: lane l of a warp holds those of blocks
// 32 c + l of chunk c, the next chunk's already on their way.
template <typename Load>
struct ScaleStream {
    float cur, next;
    __device__ __forceinline__ ScaleStream(int lane, const Load& load) : next(load(lane)) { cur = 0.0f; }
    __device__ __forceinline__ float at(int n, int lane, const Load& load) {
        if ((n & 31) == 0) {
            cur = next;
            next = load(n + 32 + lane);
        }
        return __shfl_sync(0xffffffffu, cur, n & 31);
    }
};

// A named barrier of `THREADS` promotion threads, and whether any of their threads failed: all of them learn of it
// together, so that none is left waiting.
template <int THREADS>
__device__ __forceinline__ bool promotion_any(int barrier, bool failed) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "bar.red.or.pred p, %2, %3, q;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"(failed ? 1 : 0), "r"(barrier), "n"(THREADS)
        : "memory");
    return r != 0;
}

// v[i] * x[i] * s added to acc, two at a time.
template <int MT>
__device__ __forceinline__ void promote(float* acc, const float* v, const float* xs, float s) {
#pragma unroll
    for (int i = 0; i < MT; i += 4) {
        const float4 f = *reinterpret_cast<const float4*>(xs + i);
        const float2 f0 = __fmul2_rn(make_float2(f.x, f.y), make_float2(s, s));
        const float2 f1 = __fmul2_rn(make_float2(f.z, f.w), make_float2(s, s));
        fma2_into(acc + i, v[i], v[i + 1], f0.x, f0.y);
        fma2_into(acc + i + 2, v[i + 2], v[i + 3], f1.x, f1.y);
    }
}

// A stage of both kernels: two weight tiles and the activations they share.
template <int MT>
struct MoeCfg {
    static constexpr int X_TILE = MT * BK;
    static constexpr int STAGE = 2 * A_TILE + X_TILE;
    static constexpr int F_BYTES = MT * 4;                   // (down) factors of the tokens
    static constexpr uint32_t TMEM_COLS = tmem_cols_for(MOE_NBUF * 2 * MT);
    // shared memory beside the stages
    // More than 16 tokens: the up kernel gathers the rows of those that chose the expert.
    static constexpr bool GATHER = MT > 16;
    static constexpr int up_fixed(int nkb) {
        return 1024 + nkb * MT * 4 * (GATHER ? 2 : 1) + 7 * MT * 4 + MT * BM * 4 + moe_bar_bytes(kMaxStages);
    }
    static constexpr int down_fixed() { return 1024 + kMaxStages * F_BYTES + moe_bar_bytes(kMaxStages); }
    static int stages(int fixed) {
        const int s = (kMoeSmem - fixed) / STAGE;
        return s < kMaxStages ? s : kMaxStages;
    }
};

// After a wait that ran out: the copies of the last stages, so that none is still writing shared memory when the
// CTA ends.
__device__ __forceinline__ void drain_stages(const MoeBars& bar, int stages, int n) {
    record_error(FP8BS_DEVERR_PRODUCER_WAIT);
    for (int i = max(0, n - stages); i < n; ++i)
        if (!mbar_wait(&bar.full[i % stages], (i / stages) & 1, kDrainLimitNs)) record_error(FP8BS_DEVERR_DRAIN_WAIT);
}

// The MMAs of one weight tile (half 0 or 1) of every stage; rows_of(m): rows of activations, a multiple of 16, of
// the m-th run of `per` stages.
template <int MT, typename Rows>
__device__ __forceinline__ void issue_half(int half, int total, int per, int stages, const uint8_t* sW,
                                           const uint8_t* sX, uint32_t tmem, const MoeBars& bar, Rows rows_of) {
    uint32_t idesc = 0;
    int left = 0, run = 0;
    const uint64_t w0 = smem_desc_k_sw128(smem_addr(sW) + half * A_TILE);
    const uint64_t x0 = smem_desc_k_sw128(smem_addr(sX));
    int st = 0;
    uint32_t phase = 0;
    for (int n = 0; n < total; ++n) {
        const int buf = n % MOE_NBUF;
        if (!mbar_wait(&bar.tempty[buf], ((n / MOE_NBUF) & 1) ^ 1) || !mbar_wait(&bar.full[st], phase)) {
            record_error(FP8BS_DEVERR_MMA_WAIT);
            break;
        }
        tc_fence_after();
        if (left == 0) {
            idesc = idesc_e4m3_f32(BM, rows_of(run++));
            left = per;
        }
        --left;
        const uint64_t w = w0 + static_cast<uint32_t>(st * (2 * A_TILE / 16));
        const uint64_t x = x0 + static_cast<uint32_t>(st * (MT * BK / 16));
        const uint32_t d = tmem + static_cast<uint32_t>((2 * buf + half) * MT);
#pragma unroll
        for (int j = 0; j < BK / MMA_K; ++j)
            mma_f8(d, w + j * MMA_K / 16, x + j * MMA_K / 16, idesc, j > 0 ? 1u : 0u);
        mma_commit(&bar.empty[st]);
        mma_commit(&bar.tfull[buf]);
        if (++st == stages) {
            st = 0;
            phase ^= 1;
        }
    }
    mma_commit(bar.drain);
    if (!mbar_wait(bar.drain, 0, kDrainLimitNs)) record_error(FP8BS_DEVERR_DRAIN_WAIT);
}

// One K block's partial of this thread's row, taken from TMEM (MT columns at t0), the buffer handed back, scaled
// and added to acc.
template <int MT>
__device__ __forceinline__ void promote_block(float* acc, uint32_t t0, const float* xs, float s, uint64_t* tempty,
                                              int lane) {
    float v[MT];
    if constexpr (MT == 16) {
        tmem_ld_16cols(t0, v);
        tmem_wait_ld_16(v);
    } else {
#pragma unroll
        for (int c = 0; c < MT / 32; ++c) tmem_ld_32cols(t0 + 32 * c, v + 32 * c);
#pragma unroll
        for (int c = 0; c < MT / 32; ++c) tmem_wait_ld_32(v + 32 * c);
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(tempty);
    promote<MT>(acc, v, xs, s);
}

// SPLIT: with few items (experts and blocks of 128 channels) for the SMs, clusters of 2^log2s CTAs share an item's channels
// of x: each computes its part of the K blocks, rank 0 adds the sums in rank order and goes on with them. (One token of
// 6400 channels, 4 experts of 256: 33 -> 21 us for the layer. A form of its own: with the split decided at run time the
// others took 0.5 to 0.9 us more.)
template <int MT, bool SPLIT>
__global__ void __launch_bounds__(MOE_THREADS, 1)
    moe_up_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                  const MoeArgs a, const float* xs, uint8_t* h8, float* hs, const int stages, const int log2s) {
    using Cfg = MoeCfg<MT>;
    constexpr bool GATHER = Cfg::GATHER;
    extern __shared__ uint8_t smem_raw[];
    __shared__ Routing rt;
    __shared__ uint32_t s_tmem;
    uint8_t* smem = align_1024(smem_raw);
    const int nkb = a.D / BK;
    uint8_t* sW = smem;                                      // [stages][gate, up][128 x 128]
    uint8_t* sX = sW + stages * 2 * A_TILE;                  // [stages][MT x 128]
    float* sXs = reinterpret_cast<float*>(sX + stages * Cfg::X_TILE);   // [nkb][MT] scales of x
    float* sGs = sXs + nkb * MT;                             // (GATHER) [nkb][MT] those of the item's rows
    float* sMax = sGs + (GATHER ? nkb * MT : 0);             // [4][MT]
    float2* sScale = reinterpret_cast<float2*>(sMax + 4 * MT);   // [MT] scale of a column's block, its reciprocal
    int* sTok = reinterpret_cast<int*>(sScale + MT);         // [MT] its token, or -1
    float* sU = reinterpret_cast<float*>(sTok + MT);                                 // [MT][128] products for the other half's warps
    const MoeBars bar = carve_bars(reinterpret_cast<uint8_t*>(sU + MT * BM), stages);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < stages; ++i) {
            mbar_init(&bar.full[i], 1);
            mbar_init(&bar.empty[i], 2);
        }
        for (int i = 0; i < MOE_NBUF; ++i) {
            mbar_init(&bar.tfull[i], 2);
            mbar_init(&bar.tempty[i], MOE_PROMOTE_WARPS);
        }
        mbar_init(bar.drain, 2);
        fence_barrier_init();
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmX);
    }
    if (warp == 1) tmem_alloc(&s_tmem, Cfg::TMEM_COLS);
    clear_routing(rt, a);
    tc_fence_before();
    __syncthreads();
    grid_dependency_wait();
    grid_launch_dependents();
    const int first = first_id(a);                           // (on its way while the scales are)
    for (int i = threadIdx.x; i < nkb * MT; i += MOE_THREADS) {
        const int t = i % MT;
        sXs[i] = t < a.T ? xs[(i / MT) * kMoeMaxTokens + t] : 0.0f;
    }
    build_routing(rt, a, first, blockIdx.x == 0);
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    const int iblocks = a.I / BK;
    const int items = rt.n * iblocks;
    // this cluster's items: first, first + clusters, ...; K blocks [k0, k0 + nk) of each, counted on through them
    const int first_item = SPLIT ? blockIdx.x >> log2s : blockIdx.x;
    const int clusters = SPLIT ? gridDim.x >> log2s : gridDim.x;
    const int rank = SPLIT ? blockIdx.x & ((1 << log2s) - 1) : 0;
    const int k0 = SPLIT ? rank * nkb >> log2s : 0;
    const int nk = SPLIT ? ((rank + 1) * nkb >> log2s) - k0 : nkb;
    const int mine = first_item < items ? (items - 1 - first_item) / clusters + 1 : 0;
    const int total = mine * nk;

    if (warp == 0 || warp == MOE_LOADER2) {
        // Lanes 0 and 1 of the first loader bring the weight tiles, lane 0 of the second the activations; GATHER: lane
        // i rows 4i .. 4i + 3 of those that chose the expert (a row past them: any).
        const bool weights = warp == 0;
        const uint64_t policy = weights ? l2_policy_evict_first() : l2_policy_evict_last();
        int n = 0;
        bool ok = true;
        for (int m = 0; ok && m < mine; ++m) {
            const int item = first_item + m * clusters;
            const int act = item / iblocks;
            const int e = rt.active[act];
            const int row = e * 2 * a.I + (item - act * iblocks) * BM + (lane == 1 ? a.I : 0);
            int tok[4] = {0, 0, 0, 0};
            int gathers = 0;
            if constexpr (GATHER) {
                unsigned long long mask = rt.mask[e];
                gathers = (__popcll(mask) + 3) / 4;
                if (lane < gathers) {
                    for (int i = 0; i < 4 * lane; ++i) mask &= mask - 1;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        tok[i] = mask ? __ffsll(mask) - 1 : tok[0];
                        mask &= mask - 1;
                    }
                }
            }
            const uint32_t bytes = 2 * A_TILE + (GATHER ? gathers * 4 * BK : Cfg::X_TILE);
            for (int kb = k0; kb < k0 + nk; ++kb, ++n) {
                const int st = n % stages;
                if (!warp_wait(&bar.empty[st], ((n / stages) & 1) ^ 1)) {
                    ok = false;
                    break;
                }
                if (weights) {
                    if (lane == 0) mbar_arrive_expect_tx(&bar.full[st], bytes);
                    __syncwarp();
                    if (lane < 2)
                        tma_load_2d_hint(sW + (2 * st + lane) * A_TILE, &tmW, &bar.full[st], kb * BK, row, policy);
                } else if (GATHER) {
                    if (lane < gathers)
                        tma_gather4(sX + st * Cfg::X_TILE + lane * 4 * BK, &tmX, &bar.full[st], kb * BK, tok[0],
                                    tok[1], tok[2], tok[3]);
                } else if (lane == 0) {
                    tma_load_2d_hint(sX + st * Cfg::X_TILE, &tmX, &bar.full[st], kb * BK, 0, policy);
                }
            }
        }
        if (!ok && lane == 0) drain_stages(bar, stages, n);
    } else if (warp == 1 || warp == MOE_ISSUER2) {
        if (lane == 0)
            issue_half<MT>(warp == 1 ? 0 : 1, total, nk, stages, sW, sX, tmem, bar, [&](int m) {
                if (!GATHER) return MT;
                const int act = (first_item + m * clusters) / iblocks;
                return (__popcll(rt.mask[rt.active[act]]) + 15) / 16 * 16;
            });
    } else {
        const int half = (warp - MOE_PROMOTE_WARP0) >> 2;    // gate or up
        const int quarter = warp & 3;
        const int r = quarter * 32 + lane;                   // row of the tile = channel of the block
        const uint32_t t0 = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(half * MT);
        auto scale_of = [&](int n) {
            if (n >= total) return 0.0f;
            const int m = n / nk;
            const int item = first_item + m * clusters;
            const int act = item / iblocks;
            const int64_t block = static_cast<int64_t>(rt.active[act]) * 2 * iblocks + half * iblocks +
                                  (item - act * iblocks);
            return __ldg(a.s13 + block * nkb + k0 + (n - m * nk));
        };
        ScaleStream<decltype(scale_of)> ws(lane, scale_of);
        bool ok = true;
        int n = 0;
        for (int m = 0; m < mine; ++m) {
            float g[MT];
#pragma unroll
            for (int i = 0; i < MT; ++i) g[i] = 0.0f;
            const int item = first_item + m * clusters;
            const int act = item / iblocks;
            const int ib = item - act * iblocks;
            const int e = rt.active[act];
            const unsigned long long mask = rt.mask[e];
            // the item's columns: its rows of x, or all tokens
            const int cols = GATHER ? __popcll(mask) : a.T;
            const int tid = threadIdx.x - MOE_PROMOTE_WARP0 * 32;
            float route_w = 0.0f;              // thread tid: the expert's weight for column tid's token
            if (tid < cols) {
                const int t = GATHER ? nth_bit(mask, tid) : tid;
#pragma unroll 8
                for (int j = 0; j < a.top_k; ++j) {
                    const int id = a.ids[t * a.top_k + j];
                    const float w = a.weights[t * a.top_k + j];
                    route_w += id == e ? w : 0.0f;
                }
            }
            const float* scales = sXs;
            if constexpr (GATHER) {
                // the scales of the item's rows, side by side (barrier 1: no warp reads the last item's any more)
                const int i = tid % MT;
                if (i < cols) {
                    const int t = nth_bit(mask, i);
                    for (int kb = tid / MT; kb < nkb; kb += 256 / MT) sGs[kb * MT + i] = sXs[kb * MT + t];
                }
                asm volatile("bar.sync 4, 256;" ::: "memory");
                scales = sGs;
            }
            for (int kb = k0; ok && kb < k0 + nk; ++kb, ++n) {
                const float s = ws.at(n, lane, scale_of);
                const int buf = n % MOE_NBUF;
                if (!warp_wait(&bar.tfull[buf], (n / MOE_NBUF) & 1)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t at = t0 + static_cast<uint32_t>(2 * buf * MT);
                if (GATHER && cols <= 16)
                    promote_block<16>(g, at, scales + kb * MT, s, &bar.tempty[buf], lane);
                else if (MT > 32 && cols <= 32)
                    promote_block<32>(g, at, scales + kb * MT, s, &bar.tempty[buf], lane);
                else
                    promote_block<MT>(g, at, scales + kb * MT, s, &bar.tempty[buf], lane);
            }
            // h = silu(gate) * up. The gate's warps take the first half of the columns, the up product's warps the
            // others, four at a time (one after another, they are all latency: 41000 cycles for 16 tokens, half as
            // much as the item's weights take); each side hands the other what it needs through shared memory.
            if constexpr (SPLIT) {
                // [rank - 1][column][256 rows], where rank 0's stages were
                cluster_sync();                                  // every CTA is done with its stages
                if (rank > 0) {
                    const uint32_t recv = mapa_shared(smem_addr(smem), 0) +
                                          static_cast<uint32_t>(((rank - 1) * MT * 2 * BM + half * BM + r) * 4);
#pragma unroll
                    for (int i = 0; i < MT; ++i)
                        if (i < cols) st_shared_cluster_f32(recv + static_cast<uint32_t>(i * 2 * BM * 4), g[i]);
                }
                cluster_sync();
                if (rank > 0) break;
                const float* got = reinterpret_cast<const float*>(smem) + half * BM + r;
                for (int q = 0; q < (1 << log2s) - 1; ++q)
#pragma unroll
                    for (int i = 0; i < MT; ++i)
                        if (i < cols) g[i] += got[(q * MT + i) * 2 * BM];
            }
            const int mid = (cols + 7) / 8 * 4;
            auto here = [&](int c) { return (4 * c < mid) == (half == 0); };
#pragma unroll
            for (int c = 0; c < MT / 4; ++c)
                if (4 * c < cols && !here(c))
#pragma unroll
                    for (int i = 4 * c; i < 4 * c + 4; ++i) sU[i * BM + r] = g[i];
            if (promotion_any<256>(1, !ok)) {
                ok = false;
                break;
            }
#pragma unroll
            for (int c = 0; c < MT / 4; ++c)
                if (4 * c < cols && here(c)) {
#pragma unroll
                    for (int i = 4 * c; i < 4 * c + 4; ++i) {
                        const float other = sU[i * BM + r];
                        const float gate = half == 0 ? g[i] : other;
                        g[i] = __fdividef(gate, 1.0f + __expf(-gate)) * (half == 0 ? other : g[i]);
                        const float mag = fmaxf(fabsf(g[i]), 0.0f);          // (NaN counts as nothing)
                        const unsigned top = __reduce_max_sync(0xffffffffu, __float_as_uint(mag));
                        if (lane == 0) sMax[quarter * MT + i] = __uint_as_float(top);
                    }
                }
            asm volatile("bar.sync 2, 256;" ::: "memory");
            // One thread per column: the block's scale, its reciprocal, and the factor of the down product. The
            // factors of the tokens that did not choose the expert are zero, and their codes.
            const int64_t out0 = static_cast<int64_t>(act) * a.T * a.I + ib * BK;
            if (tid < MT) {
                float* factor = hs + (static_cast<int64_t>(act) * iblocks + ib) * kMoeMaxTokens;
                if (tid < cols) {
                    const float sc = block_scale(fmaxf(fmaxf(sMax[tid], sMax[MT + tid]),
                                                       fmaxf(sMax[2 * MT + tid], sMax[3 * MT + tid])), a.ue8m0);
                    const int t = GATHER ? nth_bit(mask, tid) : tid;
                    sScale[tid] = make_float2(sc, __frcp_rn(sc));
                    sTok[tid] = (mask >> t) & 1 ? t : -1;
                    if ((mask >> t) & 1) factor[t] = route_w * sc;
                }
                if (tid >= a.T || !((mask >> tid) & 1)) factor[tid] = 0.0f;
            } else {
                for (int i = tid - MT; i < a.T * (BK / 16); i += 256 - MT) {
                    const int t = i / (BK / 16);
                    if (!((mask >> t) & 1))
                        *reinterpret_cast<uint4*>(h8 + out0 + static_cast<int64_t>(t) * a.I + i % (BK / 16) * 16) =
                            make_uint4(0, 0, 0, 0);
                }
            }
            asm volatile("bar.sync 3, 256;" ::: "memory");
#pragma unroll
            for (int c = 0; c < MT / 4; ++c)
                if (4 * c < cols && here(c)) {
                    const int4 t4 = *reinterpret_cast<const int4*>(sTok + 4 * c);
                    const int tok[4] = {t4.x, t4.y, t4.z, t4.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 sc = sScale[4 * c + i];
                        const uint8_t code = static_cast<uint8_t>(
                            pack_e4m3x2(div_by_scale(g[4 * c + i], sc.x, sc.y), 0.0f));
                        if (4 * c + i < cols && tok[i] >= 0)
                            h8[out0 + static_cast<int64_t>(tok[i]) * a.I + r] = code;
                    }
                }
        }
        if (SPLIT && mine == 0) {
            cluster_sync();
            cluster_sync();
        }
        if (!ok && lane == 0) record_error(FP8BS_DEVERR_EPILOGUE_WAIT);
    }
    if (SPLIT && !(warp >= MOE_PROMOTE_WARP0 && warp < MOE_PROMOTE_WARP0 + MOE_PROMOTE_WARPS)) {
        cluster_sync();
        cluster_sync();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, Cfg::TMEM_COLS);
}

// One cluster per 256 output channels (two tiles of 128 rows, which share the activations); its C CTAs share the
// (expert, K block) units evenly and add their sums in rank order.
template <int MT>
__global__ void __launch_bounds__(MOE_THREADS, 1)
    moe_down_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmH,
                    const MoeArgs a, const float* hs, const int C, const int stages) {
    using Cfg = MoeCfg<MT>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ Routing rt;
    __shared__ uint32_t s_tmem;
    uint8_t* smem = align_1024(smem_raw);
    uint8_t* sW = smem;                                      // [stages][2][128 x 128]
    uint8_t* sX = sW + stages * 2 * A_TILE;                  // [stages][MT x 128]
    float* sF = reinterpret_cast<float*>(sX + stages * Cfg::X_TILE);   // [stages][MT]
    const MoeBars bar = carve_bars(reinterpret_cast<uint8_t*>(sF + stages * MT), stages);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int pair = blockIdx.x / C;
    const int rank = blockIdx.x - pair * C;

    if (threadIdx.x == 0) {
        for (int i = 0; i < stages; ++i) {
            mbar_init(&bar.full[i], 1);
            mbar_init(&bar.empty[i], 2 + MOE_PROMOTE_WARPS);
        }
        for (int i = 0; i < MOE_NBUF; ++i) {
            mbar_init(&bar.tfull[i], 2);
            mbar_init(&bar.tempty[i], MOE_PROMOTE_WARPS);
        }
        mbar_init(bar.drain, 2);
        fence_barrier_init();
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmH);
    }
    if (warp == 1) tmem_alloc(&s_tmem, Cfg::TMEM_COLS);
    clear_routing(rt, a);
    tc_fence_before();
    __syncthreads();
    // The ids and weights were complete before the up kernel let this one start (it does so after its own
    // wait), so the experts are known and the weights' ring fills while the up kernel is still running.
    build_routing(rt, a, first_id(a), false);
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    const int nkb = a.I / BK;
    const int units = rt.n * nkb;
    const int u0 = static_cast<int>(static_cast<int64_t>(rank) * units / C);
    const int total = static_cast<int>(static_cast<int64_t>(rank + 1) * units / C) - u0;

    if (warp == 0 || warp == MOE_LOADER2) {
        // One lane for each of a stage's four copies: the two weight tiles by the first loader, h and the factors by the
        // second. (The second tile of the last pair may lie past D: it reads the next expert's rows, or zeros past the
        // last one's, and is not stored.)
        const bool weights = warp == 0;
        const uint64_t policy = weights ? l2_policy_evict_first() : l2_policy_evict_last();
        auto load = [&](int n) {
            const int st = n % stages;
            const int act = (u0 + n) / nkb;
            const int kb = u0 + n - act * nkb;
            if (weights) {
                if (lane == 0) mbar_arrive_expect_tx(&bar.full[st], Cfg::STAGE + Cfg::F_BYTES);
                __syncwarp();
                if (lane < 2)
                    tma_load_2d_hint(sW + (2 * st + lane) * A_TILE, &tmW, &bar.full[st], kb * BK,
                                     rt.active[act] * a.D + (2 * pair + lane) * BM, policy);
            } else if (lane == 0) {
                tma_load_2d_hint(sX + st * Cfg::X_TILE, &tmH, &bar.full[st], kb * BK, act * a.T, policy);
            } else if (lane == 1) {
                bulk_load(sF + st * MT, hs + (static_cast<int64_t>(act) * nkb + kb) * kMoeMaxTokens,
                          Cfg::F_BYTES, &bar.full[st]);
            }
        };
        if (!weights) grid_dependency_wait();
        int n = 0;
        for (; n < min(stages, total); ++n) load(n);
        if (weights) grid_dependency_wait();
        grid_launch_dependents();
        for (; n < total; ++n) {
            if (!warp_wait(&bar.empty[n % stages], ((n / stages) & 1) ^ 1)) {
                if (lane == 0) drain_stages(bar, stages, n);
                break;
            }
            load(n);
        }
    } else if (warp == 1 || warp == MOE_ISSUER2) {
        grid_dependency_wait();
        if (lane == 0) issue_half<MT>(warp == 1 ? 0 : 1, total, total, stages, sW, sX, tmem, bar, [](int) { return MT; });
    } else {
        grid_dependency_wait();
        const int half = (warp - MOE_PROMOTE_WARP0) >> 2;
        const int quarter = warp & 3;
        const int r = quarter * 32 + lane;
        const int slab = 2 * pair + half;                    // this thread's output channel: slab * 128 + r
        const bool inside = slab * BM < a.D;
        const uint32_t t0 = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(half * MT);
        auto scale_of = [&](int n) {
            if (n >= total || !inside) return 0.0f;
            const int act = (u0 + n) / nkb;
            const int kb = u0 + n - act * nkb;
            return __ldg(a.s2 + (static_cast<int64_t>(rt.active[act]) * (a.D / BK) + slab) * nkb + kb);
        };
        ScaleStream<decltype(scale_of)> ss(lane, scale_of);
        float acc[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i) acc[i] = 0.0f;
        bool ok = true;
        int st = 0;
        uint32_t phase = 0;
        for (int n = 0; n < total; ++n) {
            const float s = ss.at(n, lane, scale_of);
            const int buf = n % MOE_NBUF;
            // (the products are done, so the stage has landed; its barrier orders the factors' copy)
            if (!warp_wait(&bar.tfull[buf], (n / MOE_NBUF) & 1) || !warp_wait(&bar.full[st], phase)) {
                ok = false;
                break;
            }
            tc_fence_after();
            promote_block<MT>(acc, t0 + static_cast<uint32_t>(2 * buf * MT), sF + st * MT, s, &bar.tempty[buf],
                              lane);
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.empty[st]);
            if (++st == stages) {
                st = 0;
                phase ^= 1;
            }
        }
        if (!ok && lane == 0) record_error(FP8BS_DEVERR_EPILOGUE_WAIT);
        __nv_bfloat16* y = static_cast<__nv_bfloat16*>(a.y) + slab * BM + r;
        if (C == 1) {
            if (inside)
#pragma unroll
                for (int t = 0; t < MT; ++t)
                    if (t < a.T) y[static_cast<int64_t>(t) * a.D] = __float2bfloat16_rn(acc[t]);
        } else {
            // CTA q of the cluster adds up tokens q * per .. of every rank's sums: [rank][token][256 channels]
            const int per = (MT + C - 1) / C;
            const int col = half * BM + r;
            const uint32_t recv = smem_addr(smem);
            cluster_sync();                                  // every CTA is done with its stages
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                const int q = t / per;
                st_shared_cluster_f32(
                    mapa_shared(recv + static_cast<uint32_t>(((rank * per + t - q * per) * 2 * BM + col) * 4),
                                static_cast<uint32_t>(q)),
                    acc[t]);
            }
            cluster_sync();
            const float* got = reinterpret_cast<const float*>(smem);
            for (int i = 0; i < per; ++i) {
                const int t = rank * per + i;
                if (t >= a.T) break;
                float v = got[i * 2 * BM + col];
                for (int q = 1; q < C; ++q) v += got[(q * per + i) * 2 * BM + col];
                if (inside) y[static_cast<int64_t>(t) * a.D] = __float2bfloat16_rn(v);
            }
        }
    }
    if (C > 1 && !(warp >= MOE_PROMOTE_WARP0 && warp < MOE_PROMOTE_WARP0 + MOE_PROMOTE_WARPS)) {
        cluster_sync();
        cluster_sync();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, Cfg::TMEM_COLS);
}

template <int MT>
cudaError_t launch_experts(const MoeMaps& m, const MoeArgs& a, const MoeWorkspace& w, int num_sms,
                           cudaStream_t stream) {
    using Cfg = MoeCfg<MT>;
    const int nkb = a.D / BK;
    const int up_stages = Cfg::stages(Cfg::up_fixed(nkb));
    const int down_stages = Cfg::stages(Cfg::down_fixed());
    if (up_stages < 2 || down_stages < 2) return cudaErrorInvalidValue;
    const int up_smem = Cfg::up_fixed(nkb) + up_stages * Cfg::STAGE;
    const int down_smem = Cfg::down_fixed() + down_stages * Cfg::STAGE;
    // (The limit belongs to the kernel, for all threads of the process: it is the same whatever D is.)
    cudaError_t e = set_smem(moe_up_kernel<MT, false>, kMoeSmem);
    if (e == cudaSuccess) e = set_smem(moe_up_kernel<MT, true>, kMoeSmem);
    if (e == cudaSuccess) e = set_smem(moe_down_kernel<MT>, kMoeSmem);
    if (e != cudaSuccess) return e;
    const int most_active = a.E < a.T * a.top_k ? a.E : a.T * a.top_k;
    const int64_t items = static_cast<int64_t>(most_active) * (a.I / BK);
    // Few items: clusters of as many CTAs as fit the GPU at once, 4 K blocks or more each.
    int log2s = 3;
    static_assert(kMaxSplit == 8, "log2s");
    while (log2s > 0 &&
           (items << log2s > num_sms || nkb < 4 << log2s ||
            ((1 << log2s) - 1) * MT * 2 * BM * 4 > up_stages * Cfg::STAGE ||
            max_active_clusters(reinterpret_cast<const void*>(moe_up_kernel<MT, true>), MOE_THREADS, up_smem,
                                1 << log2s) < items))
        --log2s;
    const int grid = static_cast<int>(items << log2s < num_sms ? items << log2s : num_sms);
    const float* xs = reinterpret_cast<const float*>(a.ws + w.xs);
    float* hs = reinterpret_cast<float*>(a.ws + w.hs);
    e = launch_pdl_cluster(log2s ? moe_up_kernel<MT, true> : moe_up_kernel<MT, false>, dim3(grid), MOE_THREADS, up_smem,
                           stream, 1 << log2s, false, m.w13, m.x8, a, xs, a.ws + w.h8, hs, up_stages, log2s);
    if (e != cudaSuccess) return e;
    // The most CTAs per pair of slabs that leave every cluster of the grid its own SMs and each CTA work.
    const int pairs = (a.D / BM + 1) / 2;
    // (Powers of two: five CTAs instead of four for 28 pairs took 324 instead of 303 us at 64 tokens.)
    int C = kMaxSplit;
    while (C > 1 && (static_cast<int64_t>(pairs) * C > num_sms || items < 2 * C ||
                     max_active_clusters(reinterpret_cast<const void*>(moe_down_kernel<MT>), MOE_THREADS,
                                         down_smem, C) < pairs))
        C /= 2;
    return launch_pdl_cluster(moe_down_kernel<MT>, dim3(pairs * C), MOE_THREADS, down_smem, stream, C, false,
                              m.w2, m.h8, a, hs, C, down_stages);
}

}  // namespace

MoeWorkspace moe_workspace(int64_t T, int64_t D, int64_t I, int64_t E, int64_t top_k) {
    size_t at = 0;
    auto take = [&](int64_t bytes) {
        const size_t here = at;
        at += (static_cast<size_t>(bytes) + 255) / 256 * 256;
        return here;
    };
    MoeWorkspace w = {};
    const int64_t slots = T * top_k;
    w.active = E < slots ? E : slots;
    w.x8 = take(T * D);
    w.xs = take(D / BK * kMoeMaxTokens * 4);
    w.h8 = take(w.active * T * I);
    w.hs = take(w.active * (I / BK) * kMoeMaxTokens * 4);
    w.weights = take(slots * 4);
    w.ids = take(slots * 4);
    w.total = at;
    return w;
}

int moe_token_rows(int64_t T) { return T <= 16 ? 16 : T <= 32 ? 32 : 64; }

cudaError_t launch_moe_experts(const MoeMaps& m, const MoeArgs& a, const MoeWorkspace& w, int num_sms,
                               cudaStream_t stream) {
    switch (moe_token_rows(a.T)) {
        case 16: return launch_experts<16>(m, a, w, num_sms, stream);
        case 32: return launch_experts<32>(m, a, w, num_sms, stream);
        default: return launch_experts<64>(m, a, w, num_sms, stream);
    }
}

cudaError_t read_error_moe(unsigned int* out, bool clear, cudaStream_t stream) {
    return read_tu_error(out, clear, stream);
}

}  // namespace fp8bs
