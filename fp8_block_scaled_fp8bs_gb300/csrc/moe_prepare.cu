// moe_prepare.cu -- the router of a mixture-of-experts layer and the quantisation of its input, one
// kernel ("DeepSeek-V3 Administrator & Developer Guide", §6.4 MoE expert routing and §8.5.1
// act_quant_kernel).
//
// A cluster of 8 CTAs serves PREP_TOKENS tokens: CTA r takes every 8th part of the channels, quantises
// them and computes its part of all logits, so that the router's weights (2 bytes x experts x D, from
// L2 after their first reader) are spread over 8 SMs even for a single token. The partial logits meet
// in CTA 0 through distributed shared memory, are added in rank order (the same bits every time) and
// one warp per token makes the choice. Bound by latency: a single token's 32 x 7168 router is
// 0.46 MB: 4.2 us for the choice alone, 7.7 for 64 tokens (16 clusters, 128 CTAs).
#include "gemm_common.cuh"
#include "quant_math.cuh"

namespace fp8bs {

namespace {

constexpr int PREP_CLUSTER = 8;
constexpr int PREP_TOKENS = 4;
constexpr int PREP_THREADS = 256;
constexpr int PREP_EXPERTS = 4;     // experts a warp computes at once
constexpr int PREP_AHEAD = 4;       // 16-byte pieces of each of their rows a lane has in flight
constexpr int kMaxExperts = 512;
constexpr int kMaxChannels = 16384;

// Dynamic shared memory: x of a CTA's blocks of channels, and with a router the partial logits and the choices.
constexpr int64_t prep_smem_bytes(int64_t D, int64_t E, bool router) {
    const int64_t blocks = (D / BK + PREP_CLUSTER - 1) / PREP_CLUSTER;
    return PREP_TOKENS * blocks * BK * 2 + (router ? (PREP_CLUSTER + 1) * PREP_TOKENS * E * 4 : 0);
}

struct PrepArgs {
    const uint4* x;
    const uint4* router_w;    // null: no routing
    const float* bias;
    float* weights;
    int32_t* ids;
    uint4* x8;                // null: no quantisation
    float* xs;
    int64_t T;
    int D, E, top_k, groups, topk_groups, score, normalise, ue8m0;
    float route_scale;
};

// Unsigned integers in the order of the floats.
__device__ __forceinline__ uint32_t order_of(float v) {
    const uint32_t b = __float_as_uint(v);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// Larger key = better choice: the value's order, then the lower index.
__device__ __forceinline__ uint64_t choice_key(float v, int e) {
    return (static_cast<uint64_t>(order_of(v)) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(e));
}

// The choice for one token by one warp: logits in sc[0..E), biases in ch[0..E) (shared memory). Lane l holds the
// scores of experts l, l + 32, ...: J of them at most.
template <int J>
__device__ __forceinline__ void choose(const PrepArgs& a, const float* sc, float* ch, int64_t t, int lane) {
    const int E = a.E;
    float score[J];
#pragma unroll
    for (int i = 0; i < J; ++i) score[i] = lane + 32 * i < E ? sc[lane + 32 * i] : -INFINITY;
    if (a.score == FP8BS_SCORE_SIGMOID) {
#pragma unroll
        for (int i = 0; i < J; ++i) score[i] = 1.0f / (1.0f + expf(-score[i]));
    } else {
        float m = score[0];
#pragma unroll
        for (int i = 1; i < J; ++i) m = fmaxf(m, score[i]);
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < J; ++i) {
            score[i] = expf(score[i] - m);
            sum += score[i];
        }
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
#pragma unroll
        for (int i = 0; i < J; ++i) score[i] /= sum;
    }
    float choice[J];
#pragma unroll
    for (int i = 0; i < J; ++i) choice[i] = a.bias && lane + 32 * i < E ? score[i] + ch[lane + 32 * i] : score[i];
    unsigned keep = 0xFFFFFFFFu;       // bit g: group g stays
    const int per = E / a.groups;
    if (a.groups > 1) {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < J; ++i)
            if (lane + 32 * i < E) ch[lane + 32 * i] = choice[i];
        __syncwarp();
        float m1 = -INFINITY, m2 = -INFINITY;      // lane g: the two highest of group g
        if (lane < a.groups) {
#pragma unroll 4
            for (int i = 0; i < per; ++i) {
                const float v = ch[lane * per + i];
                m2 = fmaxf(m2, fminf(m1, v));
                m1 = fmaxf(m1, v);
            }
        }
        const uint64_t key = choice_key(a.bias && per > 1 ? m1 + m2 : m1, lane);
        int better = 0;
#pragma unroll 4
        for (int g = 0; g < a.groups; ++g) better += __shfl_sync(0xffffffffu, key, g) > key ? 1 : 0;
        keep = __ballot_sync(0xffffffffu, lane < a.groups && better < a.topk_groups);
    }
    // Keys in the order of the choices; 0: not to be had (no expert, a group that is out, taken).
    uint32_t key[J];
#pragma unroll
    for (int i = 0; i < J; ++i) {
        const int e = lane + 32 * i;
        key[i] = e < E && (a.groups == 1 || (keep >> (e / per)) & 1u) ? max(order_of(choice[i]), 1u) : 0u;
    }
    // top_k rounds of the highest key, of equal ones the lowest index
    float mine_score = 0.0f;           // lane j keeps the j-th choice
    int mine = 0;
    for (int j = 0; j < a.top_k; ++j) {
        uint32_t best = key[0];
        int at = 0;
#pragma unroll
        for (int i = 1; i < J; ++i)
            if (key[i] > best) {
                best = key[i];
                at = i;
            }
        const uint32_t top = __reduce_max_sync(0xffffffffu, best);
        const int e = static_cast<int>(
            __reduce_min_sync(0xffffffffu, best == top ? static_cast<unsigned>(lane + 32 * at) : 0xFFFFFFFFu));
        float s = score[0];
#pragma unroll
        for (int i = 0; i < J; ++i)
            if (e == lane + 32 * i) {
                key[i] = 0;
                s = score[i];
            }
        s = __shfl_sync(0xffffffffu, s, e & 31);
        if (lane == j) {
            mine = e;
            mine_score = s;
        }
    }
    float total = mine_score;          // (lanes past top_k hold 0)
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) total += __shfl_xor_sync(0xffffffffu, total, k);
    if (lane < a.top_k) {
        a.ids[t * a.top_k + lane] = mine;
        a.weights[t * a.top_k + lane] = (a.normalise ? mine_score / total : mine_score) * a.route_scale;
    }
}

__global__ void __launch_bounds__(PREP_THREADS) moe_prepare_kernel(const PrepArgs a) {
    extern __shared__ __align__(16) uint8_t prep_smem[];
    const int rank = static_cast<int>(cluster_ctarank());
    const int64_t t0 = static_cast<int64_t>(blockIdx.x / PREP_CLUSTER) * PREP_TOKENS;
    const int nt = static_cast<int>(min(static_cast<int64_t>(PREP_TOKENS), a.T - t0));
    const int nb = a.D / BK;
    const int b0 = rank * nb / PREP_CLUSTER;
    const int nbr = (rank + 1) * nb / PREP_CLUSTER - b0;      // this CTA's blocks of 128 channels
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    // [tokens][blocks of this CTA, most of any][16 pieces of 16 bytes]
    const int nb_max = (nb + PREP_CLUSTER - 1) / PREP_CLUSTER;
    uint4* sx = reinterpret_cast<uint4*>(prep_smem);
    const int pitch = nb_max * (BK / 8);
    float* part = reinterpret_cast<float*>(sx + PREP_TOKENS * pitch);  // CTA 0: [rank][tokens][E]
    float* choice = part + PREP_CLUSTER * PREP_TOKENS * a.E;             // CTA 0: [tokens][E]

    if (a.router_w) asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    grid_dependency_wait();
    grid_launch_dependents();
    // The router's weights of the warp's first experts are on their way before x.
    const int pieces = nbr * (BK / 8);               // 16-byte pieces of this CTA's channels
    uint4 wv[PREP_EXPERTS][PREP_AHEAD];
    auto load_weights = [&](int e0, int c0) {
#pragma unroll
        for (int i = 0; i < PREP_EXPERTS; ++i) {
            const uint4* row = a.router_w + (static_cast<int64_t>(min(e0 + i, a.E - 1)) * a.D + b0 * BK) / 8;
#pragma unroll
            for (int k = 0; k < PREP_AHEAD; ++k) {
                const int c = c0 + 32 * k + lane;
                wv[i][k] = c < pieces ? __ldg(row + c) : make_uint4(0, 0, 0, 0);
            }
        }
    };
    if (a.router_w && warp * PREP_EXPERTS < a.E) load_weights(warp * PREP_EXPERTS, 0);
    // x into shared memory and its codes and scales out: 8 lanes per block of 128.
    const int tasks = PREP_TOKENS * nbr;
    for (int base = warp * 4; base < tasks; base += PREP_THREADS / 8) {
        const int task = base + (lane >> 3);
        const int tok = nbr ? task / nbr : 0;
        const int blk = task - tok * nbr;
        const int chunk = lane & 7;
        uint4 v0 = make_uint4(0, 0, 0, 0), v1 = v0;
        const bool live = task < tasks && tok < nt;
        if (live) {
            const uint4* src = a.x + ((t0 + tok) * a.D + (b0 + blk) * BK) / 8 + 2 * chunk;
            v0 = __ldg(src);
            v1 = __ldg(src + 1);
        }
        if (task < tasks) {
            sx[tok * pitch + blk * (BK / 8) + 2 * chunk] = v0;
            sx[tok * pitch + blk * (BK / 8) + 2 * chunk + 1] = v1;
        }
        if (a.x8) {
            const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
            uint32_t out[4];
            const float sc = a.ue8m0 ? quant_block16<true>(w, out) : quant_block16<false>(w, out);
            if (live) {
                a.x8[((t0 + tok) * a.D + (b0 + blk) * BK) / 16 + chunk] =
                    make_uint4(out[0], out[1], out[2], out[3]);
                if (chunk == 0) a.xs[(b0 + blk) * kMoeMaxTokens + t0 + tok] = sc;
            }
        }
    }
    if (!a.router_w) return;       // uniform over the grid
    __syncthreads();               // x staged
    // CTA 0 gets the biases where the choice will look for them.
    if (rank == 0 && a.bias && warp < nt)
        for (int e = lane; e < a.E; e += 32) choice[warp * a.E + e] = __ldg(a.bias + e);
    // Partial logits: a warp takes PREP_EXPERTS experts at a time, its lanes the channels.
    const uint32_t part0 = mapa_shared(smem_addr(part), 0);
    constexpr int VALUES = PREP_EXPERTS * PREP_TOKENS;
    static_assert(VALUES == 16, "the reduction below hands each pair of lanes one value");
    for (int e0 = warp * PREP_EXPERTS; e0 < a.E; e0 += PREP_THREADS / 32 * PREP_EXPERTS) {
        float acc[VALUES] = {};                      // [expert][token]
        for (int c0 = 0; c0 < pieces; c0 += 32 * PREP_AHEAD) {
            if (c0 > 0 || e0 > warp * PREP_EXPERTS) load_weights(e0, c0);
#pragma unroll
            for (int h = 0; h < PREP_AHEAD; ++h) {
                const int c = min(c0 + 32 * h + lane, pieces - 1);       // (past the end the weights are zero)
                if (c0 + 32 * h >= pieces) break;
#pragma unroll
                for (int k = 0; k < PREP_TOKENS; ++k) {
                    const uint4 xv = sx[k * pitch + c];
                    const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
                    for (int i = 0; i < PREP_EXPERTS; ++i) {
                        const uint32_t ww[4] = {wv[i][h].x, wv[i][h].y, wv[i][h].z, wv[i][h].w};
                        float& t = acc[i * PREP_TOKENS + k];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            t = fmaf(bf16_lo(xw[j]), bf16_lo(ww[j]), t);
                            t = fmaf(bf16_hi(xw[j]), bf16_hi(ww[j]), t);
                        }
                    }
                }
            }
        }
        // 16 values over 32 lanes: in each step a lane keeps one half of them and hands its partner the other, so
        // that lanes 2v and 2v + 1 end with value v.
#pragma unroll
        for (int half = 8; half > 0; half >>= 1) {
            const bool upper = lane & (2 * half);
#pragma unroll
            for (int i = 0; i < half; ++i) {
                const float send = upper ? acc[i] : acc[i + half];
                const float keep = upper ? acc[i + half] : acc[i];
                acc[i] = keep + __shfl_xor_sync(0xffffffffu, send, 2 * half);
            }
        }
        // (every CTA of the cluster has to be running before the first store into another's memory)
        if (e0 == warp * PREP_EXPERTS) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
        const float v = acc[0] + __shfl_xor_sync(0xffffffffu, acc[0], 1);
        const int value = lane >> 1;
        const int e = e0 + value / PREP_TOKENS;
        if ((lane & 1) == 0 && e < a.E)
            st_shared_cluster_f32(
                part0 + static_cast<uint32_t>(((rank * PREP_TOKENS + value % PREP_TOKENS) * a.E + e) * 4), v);
    }
    if (warp * PREP_EXPERTS >= a.E) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    cluster_sync();
    if (rank != 0) return;
    for (int i = threadIdx.x; i < PREP_TOKENS * a.E; i += PREP_THREADS) {
        float v = part[i];
        for (int r = 1; r < PREP_CLUSTER; ++r) v += part[r * PREP_TOKENS * a.E + i];
        part[i] = v;               // slot of rank 0: logits [tokens][E]
    }
    __syncthreads();
    if (warp >= nt) return;
    const float* logits = part + warp * a.E;
    float* mine = choice + warp * a.E;
    if (a.E <= 32)
        choose<1>(a, logits, mine, t0 + warp, lane);
    else if (a.E <= 64)
        choose<2>(a, logits, mine, t0 + warp, lane);
    else if (a.E <= 256)
        choose<8>(a, logits, mine, t0 + warp, lane);
    else
        choose<16>(a, logits, mine, t0 + warp, lane);
}

}  // namespace

cudaError_t launch_moe_prepare(const void* x, const fp8bs_moe_routing* routing, float* weights,
                               int32_t* ids, void* x8, float* xs, int64_t T, int64_t D, int64_t E,
                               bool ue8m0, cudaStream_t stream) {
    PrepArgs a = {};
    a.x = static_cast<const uint4*>(x);
    a.x8 = static_cast<uint4*>(x8);
    a.xs = xs;
    a.T = T;
    a.D = static_cast<int>(D);
    a.E = static_cast<int>(E);
    a.ue8m0 = ue8m0 ? 1 : 0;
    if (routing) {
        a.router_w = static_cast<const uint4*>(routing->router_w);
        a.bias = routing->bias;
        a.weights = weights;
        a.ids = ids;
        a.top_k = static_cast<int>(routing->top_k);
        a.groups = static_cast<int>(routing->groups);
        a.topk_groups = static_cast<int>(routing->topk_groups);
        a.score = routing->score;
        a.normalise = routing->normalise;
        a.route_scale = routing->route_scale;
    }
    const int64_t smem = prep_smem_bytes(D, E, routing != nullptr);
    // (The limit belongs to the kernel, for all threads of the process: it is the same whatever D and E are.)
    cudaError_t e = set_smem(moe_prepare_kernel, static_cast<int>(prep_smem_bytes(kMaxChannels, kMaxExperts, true)));
    if (e != cudaSuccess) return e;
    const int64_t clusters = (T + PREP_TOKENS - 1) / PREP_TOKENS;
    return launch_pdl_cluster(moe_prepare_kernel, dim3(static_cast<unsigned>(clusters * PREP_CLUSTER)),
                              PREP_THREADS, smem, stream, PREP_CLUSTER, false, a);
}

}  // namespace fp8bs
