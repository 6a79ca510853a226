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
#include "norm_rows.cuh"

namespace fp8bs {

namespace {

constexpr int NR_BATCH = 2;      // query rows a lane group loads before it computes either

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

    const int r0 = static_cast<int>(a.rot_start) / 8;
    const int nr = static_cast<int>(a.rot_dim) / 8;
    TokenRows<LPR, INTERLEAVED> rows;
    rows.rotates = p < nr / 2;
    int c0, c1;
    lane_chunks(p, r0, nr, &c0, &c1);
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
    if (rows.rotates) rows.load_turn(a, pos, p, nr);
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
