// norm_rope.cu -- RMS norm of queries and keys per head, rotation by position and the write of
// keys and values into a paged cache, in one pass (fp8bs_qk_norm_rope).
//
// Bound by memory: every element is read and written once, 4 bytes per element of q, k and v. One
// CTA per token; LPR lanes share a row (one head of the token), each lane taking two chunks of 8
// channels (16-byte loads and stores). The two chunks are the two halves of the same rotation
// pairs, so the rotation needs no exchange between lanes, and the norm one reduction over LPR
// lanes. The token's cosines and sines are read once into registers and serve all its heads.
//
// Measured: 8192 tokens of 32 + 8 + 8 heads of 128 channels, norm and rotation, keys and values into the cache,
// 34 us for 205 MB = 6.0 TB/s (0.90 of a copy's rate), 37 us on inputs that change from call to call; 1000 tokens of 16
// heads of 192 channels 6.7 us, 9.1 where they come from HBM; five tokens 2.7 us, a launch and two dependent loads.
#include "gemm_common.cuh"
#include "quant_math.cuh"

namespace fp8bs {

namespace {

constexpr int NR_BATCH = 2;      // query rows a lane group loads before it computes either

// A lane's 16 channels of a row as 8 pairs (the rotation's partners lie 8 apart: pair i of the first chunk with
// pair i of the second).
struct Chunk16 {
    uint4 a, b;
};

__device__ __forceinline__ Chunk16 zero16() {
    return Chunk16{make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
}

__device__ __forceinline__ void unpack16(const Chunk16& v, float2* f) {
    const uint32_t w[8] = {v.a.x, v.a.y, v.a.z, v.a.w, v.b.x, v.b.y, v.b.z, v.b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = make_float2(bf16_lo(w[i]), bf16_hi(w[i]));
}

__device__ __forceinline__ Chunk16 pack16(const float2* f) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = pack_bf16x2(f[i].x, f[i].y);
    return Chunk16{make_uint4(w[0], w[1], w[2], w[3]), make_uint4(w[4], w[5], w[6], w[7])};
}

// What the rows of a token share.
template <int LPR, bool INTERLEAVED>
struct TokenRows {
    float2 cs[4], sn[4];       // cosines and sines of the lane's 8 pairs
    bool rotates, has;         // rotated chunks; any chunk of a q or k row
    float eps, inv_d;

    // Norm (w: the lane's weights, or null) and rotation of one row's chunks; every lane of the warp calls it.
    __device__ __forceinline__ Chunk16 row(const Chunk16& x, const float2* w, bool norm) const {
        float2 f[8];
        unpack16(x, f);
        if (norm) {
            float2 s2 = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < 8; ++i) s2 = __ffma2_rn(f[i], f[i], s2);
            float ss = s2.x + s2.y;
#pragma unroll
            for (int m = LPR / 2; m > 0; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
            const float inv = rsqrtf(fmaf(ss, inv_d, eps));
            const float2 i2 = make_float2(inv, inv);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = __fmul2_rn(__fmul2_rn(f[i], i2), w[i]);
        }
        if (rotates) {
            if constexpr (INTERLEAVED) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float c = i & 1 ? cs[i / 2].y : cs[i / 2].x;
                    const float s = i & 1 ? sn[i / 2].y : sn[i / 2].x;
                    f[i] = make_float2(f[i].x * c - f[i].y * s, f[i].x * s + f[i].y * c);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 u = f[i], y = f[4 + i];
                    const float2 ns = make_float2(-sn[i].x, -sn[i].y);
                    f[i] = __ffma2_rn(y, ns, __fmul2_rn(u, cs[i]));
                    f[4 + i] = __ffma2_rn(u, sn[i], __fmul2_rn(y, cs[i]));
                }
            }
        }
        return pack16(f);
    }
};

// MANY tokens (more than stay in L2 on their way to the attention): two warps per token, and the stream is marked
// as not to be kept; else four warps, for the latency of the single token.
template <int LPR, bool INTERLEAVED, bool MANY>
__global__ void __launch_bounds__(MANY ? 64 : 128, (INTERLEAVED ? 5 : 6) * (MANY ? 2 : 1)) qk_norm_rope_kernel(
    const __grid_constant__ fp8bs_qk_norm_rope_args a) {
    constexpr int GROUPS = (MANY ? 64 : 128) / LPR;
    auto load = [](const uint4* from) { return MANY ? __ldcs(from) : __ldg(from); };
    const int64_t t = blockIdx.x;
    const int p = threadIdx.x % LPR;
    const int grp = threadIdx.x / LPR;
    const int dk = static_cast<int>(a.cache.dk);
    const int hq = static_cast<int>(a.q_heads);
    const int hk = static_cast<int>(a.cache.heads);
    const int kv_rows = hk + (a.v ? hk : 0);

    // This lane's chunks of a q or k row: rotated chunks come as pairs (the chunk, the one half the rotated range
    // further on), the others in order.
    const int r0 = static_cast<int>(a.rot_start) / 8;
    const int nr = static_cast<int>(a.rot_dim) / 8;
    TokenRows<LPR, INTERLEAVED> rows;
    rows.rotates = p < nr / 2;
    int c0, c1;
    if (rows.rotates) {
        c0 = r0 + p;
        c1 = c0 + nr / 2;
    } else {
        const int i = 2 * (p - nr / 2);
        c0 = i < r0 ? i : i + nr;
        c1 = i + 1 < r0 ? i + 1 : i + 1 + nr;
    }
    rows.has = p < dk / 16;
    rows.eps = a.eps;
    rows.inv_d = 1.0f / static_cast<float>(dk);
    const bool has_v = p < static_cast<int>(a.cache.dv) / 16;

    grid_dependency_wait();
    grid_launch_dependents();

    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + t * a.q_token_stride;
    const __nv_bfloat16* k = static_cast<const __nv_bfloat16*>(a.k) + t * a.k_token_stride;
    const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(a.v) + (a.v ? t * a.v_token_stride : 0);
    auto load_q = [&](int r) {
        if (r >= hq || !rows.has) return zero16();
        const uint4* src = reinterpret_cast<const uint4*>(q + r * a.q_head_stride);
        return Chunk16{load(src + c0), load(src + c1)};
    };
    auto load_kv = [&](int r) {
        if (r < hk) {
            if (!rows.has) return zero16();
            const uint4* src = reinterpret_cast<const uint4*>(k + r * a.k_head_stride);
            return Chunk16{load(src + c0), load(src + c1)};
        }
        if (r >= kv_rows || !has_v) return zero16();
        const uint4* src = reinterpret_cast<const uint4*>(v + (r - hk) * a.v_head_stride);
        return Chunk16{load(src + 2 * p), load(src + 2 * p + 1)};
    };

    // The first rows are on their way before the position is known, from which the cosines come.
    Chunk16 xq[NR_BATCH];
#pragma unroll
    for (int b = 0; b < NR_BATCH; ++b) xq[b] = load_q(b * GROUPS + grp);
    Chunk16 xk = load_kv(grp);
    const int pos = a.positions[t];
    int64_t slot = a.slots ? a.slots[t] : t;
    const bool pos_ok = pos >= 0 && pos < a.max_positions;
    const bool slot_past = slot >= a.cache.pages * a.cache.page_size;
    if ((!pos_ok || slot_past) && threadIdx.x == 0) record_error(FP8BS_DEVERR_INDEX);
    const bool store_kv = pos_ok && slot >= 0 && !slot_past;
    if (!store_kv) slot = 0;
    rows.rotates = rows.rotates && pos_ok;
    if (rows.rotates) {
        // pair 8p + i (halves), or the 4 pairs of each of the two chunks (interleaved)
        const float* ct = a.cos + static_cast<int64_t>(pos) * (a.rot_dim / 2);
        const float* st = a.sin + static_cast<int64_t>(pos) * (a.rot_dim / 2);
        const int i0 = INTERLEAVED ? 4 * p : 8 * p;
        const int i1 = INTERLEAVED ? 4 * (p + nr / 2) : 8 * p + 4;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            rows.cs[i] = make_float2(__ldg(ct + i0 + 2 * i), __ldg(ct + i0 + 2 * i + 1));
            rows.sn[i] = make_float2(__ldg(st + i0 + 2 * i), __ldg(st + i0 + 2 * i + 1));
            rows.cs[2 + i] = make_float2(__ldg(ct + i1 + 2 * i), __ldg(ct + i1 + 2 * i + 1));
            rows.sn[2 + i] = make_float2(__ldg(st + i1 + 2 * i), __ldg(st + i1 + 2 * i + 1));
        }
    }
    float2 w[8];
    auto load_weight = [&](const void* from) {
        Chunk16 v16 = zero16();
        if (from && rows.has) {
            const uint4* src = static_cast<const uint4*>(from);
            v16 = Chunk16{__ldg(src + c0), __ldg(src + c1)};
        }
        unpack16(v16, w);
    };

    // Queries. Row loops are uniform over the CTA: the norm's reduction shuffles across whole warps.
    load_weight(a.q_weight);
    __nv_bfloat16* qo = static_cast<__nv_bfloat16*>(a.q_out) + t * hq * dk;
    for (int base = 0; base < hq; base += GROUPS * NR_BATCH) {
#pragma unroll
        for (int b = 0; b < NR_BATCH; ++b) {
            const int r = base + b * GROUPS + grp;
            if (base + b * GROUPS >= hq) break;
            Chunk16 y = rows.row(xq[b], w, a.q_weight != nullptr);
            if (!pos_ok) y = zero16();
            if (r < hq && rows.has) {
                uint4* dst = reinterpret_cast<uint4*>(qo + r * dk);
                if (MANY) {
                    __stcs(dst + c0, y.a);
                    __stcs(dst + c1, y.b);
                } else {
                    dst[c0] = y.a;
                    dst[c1] = y.b;
                }
            }
            xq[b] = load_q(r + GROUPS * NR_BATCH);
        }
    }
    // Keys, and values as they are.
    load_weight(a.k_weight);
    const int64_t page = slot / a.cache.page_size;
    const int64_t off = slot - page * a.cache.page_size;
    __nv_bfloat16* ko = static_cast<__nv_bfloat16*>(a.cache.k) + page * a.cache.k_page_stride +
                        off * a.cache.k_slot_stride;
    __nv_bfloat16* vo = static_cast<__nv_bfloat16*>(a.cache.v) + page * a.cache.v_page_stride +
                        off * a.cache.v_slot_stride;
    for (int base = 0; base < kv_rows; base += GROUPS) {
        const int r = base + grp;
        const Chunk16 x = xk;
        xk = load_kv(r + GROUPS);
        Chunk16 y = x;
        if (base < hk) y = rows.row(x, w, a.k_weight != nullptr);   // (rows of v beside rows of k: not used)
        if (r < hk) {
            if (rows.has && store_kv) {
                uint4* dst = reinterpret_cast<uint4*>(ko + r * a.cache.k_head_stride);
                dst[c0] = y.a;
                dst[c1] = y.b;
            }
        } else if (r < kv_rows && has_v && store_kv) {
            uint4* dst = reinterpret_cast<uint4*>(vo + (r - hk) * a.cache.v_head_stride);
            dst[2 * p] = x.a;
            dst[2 * p + 1] = x.b;
        }
    }
}

template <int LPR, bool INTERLEAVED>
cudaError_t launch_norm_rope(const fp8bs_qk_norm_rope_args& a, cudaStream_t stream) {
    // 8192 tokens of 32 + 8 heads of 128: 34.3 us with two warps (0.90 of HBM), 38.1 with four, 57.9 with eight;
    // 5 tokens: 3.4, 2.6 and 2.6 us.
    const unsigned grid = static_cast<unsigned>(a.T);
    if (a.T >= 2048)
        return launch_pdl(qk_norm_rope_kernel<LPR, INTERLEAVED, true>, grid, 64, 0, stream, a);
    return launch_pdl(qk_norm_rope_kernel<LPR, INTERLEAVED, false>, grid, 128, 0, stream, a);
}

template <int LPR>
cudaError_t launch_norm_rope(const fp8bs_qk_norm_rope_args& a, cudaStream_t stream) {
    return a.interleaved ? launch_norm_rope<LPR, true>(a, stream) : launch_norm_rope<LPR, false>(a, stream);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const fp8bs_qk_norm_rope_args& a, cudaStream_t stream) {
    const int64_t d = a.v && a.cache.dv > a.cache.dk ? a.cache.dv : a.cache.dk;
    if (d <= 64) return launch_norm_rope<4>(a, stream);
    if (d <= 128) return launch_norm_rope<8>(a, stream);
    return launch_norm_rope<16>(a, stream);
}

cudaError_t read_error_norm_rope(unsigned int* out, bool clear, cudaStream_t stream) {
    return read_tu_error(out, clear, stream);
}

}  // namespace fp8bs
