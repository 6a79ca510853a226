// norm_rope_fp8.cu -- RMS norm of queries and keys per head, rotation by position and the write of keys and values
// into a paged cache of e4m3 codes with one power-of-two scale per page and head (fp8bs_qk_norm_rope_fp8).
//
// Two kinds of CTAs in one launch. Queries: one CTA per token, as in norm_rope.cu. Keys and values: one CTA per run
// (the tokens of the call that go to one page, one after another) and head. It passes over the run's rows twice, for
// the largest magnitude and, with the page's new scale known, for the codes; the second pass reads from L1 or L2. No
// other CTA touches that page and head, so nothing is atomic and the same call gives the same bits. A page that grows
// keeps the larger of its scale and what the run asks for; where that is more than before, its codes are rounded again
// by the ratio, a power of two (exact but for codes that become subnormal).
#include "norm_rows.cuh"

namespace fp8bs {

namespace {

constexpr int NR_THREADS = 128;

// A page's slot is given to a token of the call: its position and slot are valid.
struct TokenSlot {
    int64_t slot;
    bool ok;
};

__device__ __forceinline__ TokenSlot token_slot(const fp8bs_qk_norm_rope_args& a, int64_t t) {
    TokenSlot s = {-1, false};
    if (t >= 0 && t < a.T) {
        s.slot = a.slots[t];
        const int pos = a.positions[t];
        s.ok = s.slot >= 0 && s.slot < a.cache.pages * a.cache.page_size && pos >= 0 && pos < a.max_positions;
    }
    return s;
}

// Whether token t continues the run of the token before it: the next slot of the same page.
__device__ __forceinline__ bool continues(const fp8bs_qk_norm_rope_args& a, const TokenSlot& before, const TokenSlot& s) {
    return before.ok && s.ok && s.slot == before.slot + 1 && s.slot % a.cache.page_size != 0;
}

// Codes of 16 values, by a scale's reciprocal (a power of two: the products are exact but for subnormals of binary32,
// whose codes are zero).
__device__ __forceinline__ uint2 codes8(const float2* f, float rs) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        w[i] = static_cast<uint32_t>(pack_e4m3x2(f[2 * i].x * rs, f[2 * i].y * rs)) |
               static_cast<uint32_t>(pack_e4m3x2(f[2 * i + 1].x * rs, f[2 * i + 1].y * rs)) << 16;
    return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ uint32_t rescaled(uint32_t codes, float ratio) {
    uint32_t out = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const __nv_fp8x2_storage_t pair = static_cast<__nv_fp8x2_storage_t>((codes >> (16 * h)) & 0xFFFFu);
        const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(pair, __NV_E4M3)));
        out |= static_cast<uint32_t>(pack_e4m3x2(f.x * ratio, f.y * ratio)) << (16 * h);
    }
    return out;
}

// The scale of values up to amax, a power of two; an infinite amax gets the one of the largest bf16 number.
__device__ __forceinline__ float page_scale(float amax) { return fminf(block_scale(amax, true), 0x1p120f); }

// A page's scale after a run that asks for `need` and begins at slot `off`; a page that holds nothing yet has a scale
// that is not a positive number.
__device__ __forceinline__ float grown_scale(float old, float need, int64_t off) {
    return off > 0 && old > need && old <= 0x1p127f ? old : need;
}

template <int LPR, bool INTERLEAVED>
__global__ void __launch_bounds__(NR_THREADS) qk_norm_rope_fp8_kernel(
    const __grid_constant__ fp8bs_qk_norm_rope_args a, float* k_scale, float* v_scale, const int window,
    const unsigned windows) {
    constexpr int GROUPS = NR_THREADS / LPR;
    __shared__ float s_max[2][NR_THREADS / 32];
    __shared__ unsigned s_starts[NR_THREADS / 32];
    const int tid = threadIdx.x;
    const int p = tid % LPR;
    const int grp = tid / LPR;
    const int dk = static_cast<int>(a.cache.dk), dv = static_cast<int>(a.cache.dv);
    const int hk = static_cast<int>(a.cache.heads);
    const int r0 = static_cast<int>(a.rot_start) / 8;
    const int nr = static_cast<int>(a.rot_dim) / 8;
    TokenRows<LPR, INTERLEAVED> rows;
    int c0, c1;
    lane_chunks(p, r0, nr, &c0, &c1);
    rows.has = p < dk / 16;
    rows.eps = a.eps;
    rows.inv_d = 1.0f / static_cast<float>(dk);
    float2 w[8];
    auto load_weight = [&](const void* from) {
        Chunk16 v16 = zero16();
        if (from && rows.has) {
            const uint4* src = static_cast<const uint4*>(from);
            v16 = Chunk16{__ldg(src + c0), __ldg(src + c1)};
        }
        unpack16(v16, w);
    };

    grid_dependency_wait();
    grid_launch_dependents();

    if (blockIdx.x >= windows * static_cast<unsigned>(hk)) {
        // ---- the queries of a token
        const int64_t t = blockIdx.x - windows * static_cast<unsigned>(hk);
        const int hq = static_cast<int>(a.q_heads);
        const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + t * a.q_token_stride;
        auto load_q = [&](int r) {
            if (r >= hq || !rows.has) return zero16();
            const uint4* src = reinterpret_cast<const uint4*>(q + r * a.q_head_stride);
            return Chunk16{__ldg(src + c0), __ldg(src + c1)};
        };
        Chunk16 x = load_q(grp);
        const int pos = a.positions[t];
        const bool pos_ok = pos >= 0 && pos < a.max_positions;
        if ((!pos_ok || a.slots[t] >= a.cache.pages * a.cache.page_size) && tid == 0) record_error(FP8BS_DEVERR_INDEX);
        rows.rotates = p < nr / 2 && pos_ok;
        if (rows.rotates) rows.load_turn(a, pos, p, nr);
        load_weight(a.q_weight);
        __nv_bfloat16* qo = static_cast<__nv_bfloat16*>(a.q_out) + t * hq * dk;
        for (int base = 0; base < hq; base += GROUPS) {
            const int r = base + grp;
            const Chunk16 next = load_q(r + GROUPS);
            Chunk16 y = rows.row(x, w, a.q_weight != nullptr);
            if (!pos_ok) y = zero16();
            if (r < hq && rows.has) {
                uint4* dst = reinterpret_cast<uint4*>(qo + static_cast<int64_t>(r) * dk);
                dst[c0] = y.a;
                dst[c1] = y.b;
            }
            x = next;
        }
        return;
    }

    // ---- the runs that begin among `window` tokens, of one key head
    const int head = static_cast<int>(blockIdx.x % static_cast<unsigned>(hk));
    const int64_t t0 = static_cast<int64_t>(blockIdx.x / static_cast<unsigned>(hk)) * window;
    const int64_t page_size = a.cache.page_size;
    {
        // (window <= NR_THREADS: one token a thread)
        const TokenSlot s = token_slot(a, t0 + tid);
        const bool starts = tid < window && s.ok && !continues(a, token_slot(a, t0 + tid - 1), s);
        const unsigned mask = __ballot_sync(0xffffffffu, starts);
        if ((tid & 31) == 0) s_starts[tid >> 5] = mask;
        __syncthreads();
    }
    load_weight(a.k_weight);
    const bool has_v = p < dv / 16;
    for (int at = 0; at < window; ++at) {
        if (!(s_starts[at >> 5] >> (at & 31) & 1u)) continue;            // (uniform over the CTA)
        const int64_t t = t0 + at;
        const int64_t slot = a.slots[t];
        const int64_t page = slot / page_size, off = slot - page * page_size;
        // the run's length: tokens t + 1, t + 2, ... that continue it
        int64_t n = 1;
        while (true) {
            const TokenSlot s = token_slot(a, t + n + tid);
            const bool more = continues(a, token_slot(a, t + n + tid - 1), s);
            const unsigned mask = __ballot_sync(0xffffffffu, more);
            __syncthreads();
            if ((tid & 31) == 0) s_max[0][tid >> 5] = __uint_as_float(mask);
            __syncthreads();
            int got = 0;
#pragma unroll
            for (int i = 0; i < NR_THREADS / 32; ++i) {
                const unsigned m = ~__float_as_uint(s_max[0][i]);
                if (got == 32 * i) got += m ? __ffs(m) - 1 : 32;
            }
            n += got;
            if (got < NR_THREADS) break;
        }
        // the rows' values: keys (after norm and rotation), values
        auto key_values = [&](int64_t r, float2* f) {
            Chunk16 x = zero16();
            rows.rotates = false;
            if (r < n) {
                if (rows.has) {
                    const uint4* src = reinterpret_cast<const uint4*>(
                        static_cast<const __nv_bfloat16*>(a.k) + (t + r) * a.k_token_stride + head * a.k_head_stride);
                    x = Chunk16{__ldg(src + c0), __ldg(src + c1)};
                }
                rows.rotates = p < nr / 2;
                if (rows.rotates) rows.load_turn(a, a.positions[t + r], p, nr);
            }
            rows.values(x, w, a.k_weight != nullptr, f);
        };
        auto value_values = [&](int64_t r, float2* f) {
            Chunk16 x = zero16();
            if (r < n && has_v) {
                const uint4* src = reinterpret_cast<const uint4*>(
                    static_cast<const __nv_bfloat16*>(a.v) + (t + r) * a.v_token_stride + head * a.v_head_stride);
                x = Chunk16{__ldg(src + 2 * p), __ldg(src + 2 * p + 1)};
            }
            unpack16(x, f);
        };
        float amax[2] = {0.0f, 0.0f};
        for (int64_t base = 0; base < n; base += GROUPS) {
            float2 f[8];
            key_values(base + grp, f);
#pragma unroll
            for (int i = 0; i < 8; ++i) amax[0] = fmaxf(amax[0], fmaxf(fabsf(f[i].x), fabsf(f[i].y)));
            value_values(base + grp, f);
#pragma unroll
            for (int i = 0; i < 8; ++i) amax[1] = fmaxf(amax[1], fmaxf(fabsf(f[i].x), fabsf(f[i].y)));
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int m = 16; m > 0; m >>= 1) amax[i] = fmaxf(amax[i], __shfl_xor_sync(0xffffffffu, amax[i], m));
            if ((tid & 31) == 0) s_max[i][tid >> 5] = amax[i];
        }
        const int64_t si = page * hk + head;
        const float old_k = k_scale[si], old_v = v_scale[si];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 2; ++i)
            amax[i] = fmaxf(fmaxf(s_max[i][0], s_max[i][1]), fmaxf(s_max[i][2], s_max[i][3]));
        const float sk = grown_scale(old_k, page_scale(amax[0]), off);
        const float sv = grown_scale(old_v, page_scale(amax[1]), off);
        uint8_t* kc = static_cast<uint8_t*>(a.cache.k) + page * a.cache.k_page_stride + head * a.cache.k_head_stride;
        uint8_t* vc = static_cast<uint8_t*>(a.cache.v) + page * a.cache.v_page_stride + head * a.cache.v_head_stride;
        // codes that the page holds already, by a scale that has grown
        auto rescale = [&](uint8_t* codes, int64_t slot_stride, int d, float old, float now) {
            if (off == 0 || !(old > 0.0f) || !(old < now)) return;
            const float ratio = old / now;
            const int pieces = d / 16;
            for (int64_t i = tid; i < page_size * pieces; i += NR_THREADS) {
                const int64_t o = i / pieces;
                if (o >= off && o < off + n) continue;
                uint4* at16 = reinterpret_cast<uint4*>(codes + o * slot_stride) + i % pieces;
                const uint4 c = *at16;
                *at16 = make_uint4(rescaled(c.x, ratio), rescaled(c.y, ratio), rescaled(c.z, ratio),
                                   rescaled(c.w, ratio));
            }
        };
        rescale(kc, a.cache.k_slot_stride, dk, old_k, sk);
        rescale(vc, a.cache.v_slot_stride, dv, old_v, sv);
        if (tid == 0) {
            k_scale[si] = sk;
            v_scale[si] = sv;
        }
        const float rk = 1.0f / sk, rv = 1.0f / sv;
        for (int64_t base = 0; base < n; base += GROUPS) {
            const int64_t r = base + grp;
            float2 f[8];
            key_values(r, f);
            if (r < n && rows.has) {
                uint2* dst = reinterpret_cast<uint2*>(kc + (off + r) * a.cache.k_slot_stride);
                dst[c0] = codes8(f, rk);
                dst[c1] = codes8(f + 4, rk);
            }
            value_values(r, f);
            if (r < n && has_v) {
                const uint2 lo = codes8(f, rv), hi = codes8(f + 4, rv);
                reinterpret_cast<uint4*>(vc + (off + r) * a.cache.v_slot_stride)[p] =
                    make_uint4(lo.x, lo.y, hi.x, hi.y);
            }
        }
        __syncthreads();                                     // (s_max is written again)
    }
}

template <int LPR>
cudaError_t launch_fp8(const fp8bs_qk_norm_rope_args& a, float* k_scale, float* v_scale, cudaStream_t stream) {
    const int window = a.T >= 2048 ? 64 : 1;
    const unsigned windows = static_cast<unsigned>((a.T + window - 1) / window);
    const unsigned grid = windows * static_cast<unsigned>(a.cache.heads) +
                          (a.q_heads > 0 ? static_cast<unsigned>(a.T) : 0u);
    auto kernel = a.interleaved ? qk_norm_rope_fp8_kernel<LPR, true> : qk_norm_rope_fp8_kernel<LPR, false>;
    return launch_pdl(kernel, grid, NR_THREADS, 0, stream, a, k_scale, v_scale, window, windows);
}

}  // namespace

cudaError_t launch_qk_norm_rope_fp8(const fp8bs_qk_norm_rope_args& a, float* k_scale, float* v_scale,
                                    cudaStream_t stream) {
    const int64_t d = a.cache.dv > a.cache.dk ? a.cache.dv : a.cache.dk;
    if (d <= 64) return launch_fp8<4>(a, k_scale, v_scale, stream);
    if (d <= 128) return launch_fp8<8>(a, k_scale, v_scale, stream);
    return launch_fp8<16>(a, k_scale, v_scale, stream);
}

cudaError_t read_error_norm_rope_fp8(unsigned int* out, bool clear, cudaStream_t stream) {
    return read_tu_error(out, clear, stream);
}

}  // namespace fp8bs
