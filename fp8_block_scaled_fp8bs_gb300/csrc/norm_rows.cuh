// norm_rows.cuh -- norm and rotation of one head's row (a token's query or key), as the kernels that write a cache
// share them (norm_rope.cu, norm_rope_fp8.cu): LPR lanes hold a row, each two chunks of 8 channels, the two halves
// of the same rotation pairs.
#pragma once

#include "gemm_common.cuh"
#include "quant_math.cuh"

namespace fp8bs {
namespace {

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

    // Norm (w: the lane's weights) and rotation of one row's chunks, in binary32; every lane of the warp calls it.
    // REFINE: the reciprocal root with a step of Newton's method, to about half its last bit (codes have borders).
    template <bool REFINE = false>
    __device__ __forceinline__ void values(const Chunk16& x, const float2* w, bool norm, float2* f) const {
        unpack16(x, f);
        if (norm) {
            float2 s2 = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < 8; ++i) s2 = __ffma2_rn(f[i], f[i], s2);
            float ss = s2.x + s2.y;
#pragma unroll
            for (int m = LPR / 2; m > 0; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
            const float mean = fmaf(ss, inv_d, eps);
            float inv = rsqrtf(mean);
            if constexpr (REFINE) {
                const float better = fmaf(0.5f * inv, fmaf(-mean * inv, inv, 1.0f), inv);
                if (better == better) inv = better;              // (a mean of 0 or infinity: the root stands)
            }
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
    }

    __device__ __forceinline__ Chunk16 row(const Chunk16& x, const float2* w, bool norm) const {
        float2 f[8];
        values(x, w, norm, f);
        return pack16(f);
    }

    // The cosines and sines of a token at `pos`: pair 8p + i (halves), or the 4 pairs of each of the lane's two
    // chunks (interleaved), nr rotated chunks in all.
    __device__ __forceinline__ void load_turn(const fp8bs_qk_norm_rope_args& a, int pos, int p, int nr) {
        const float* ct = a.cos + static_cast<int64_t>(pos) * (a.rot_dim / 2);
        const float* st = a.sin + static_cast<int64_t>(pos) * (a.rot_dim / 2);
        const int i0 = INTERLEAVED ? 4 * p : 8 * p;
        const int i1 = INTERLEAVED ? 4 * (p + nr / 2) : 8 * p + 4;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            cs[i] = make_float2(__ldg(ct + i0 + 2 * i), __ldg(ct + i0 + 2 * i + 1));
            sn[i] = make_float2(__ldg(st + i0 + 2 * i), __ldg(st + i0 + 2 * i + 1));
            cs[2 + i] = make_float2(__ldg(ct + i1 + 2 * i), __ldg(ct + i1 + 2 * i + 1));
            sn[2 + i] = make_float2(__ldg(st + i1 + 2 * i), __ldg(st + i1 + 2 * i + 1));
        }
    }
};

// This lane's chunks (8 channels each) of a q or k row: rotated chunks come as pairs (the chunk, the one half the
// rotated range further on), the others in order. r0: first rotated chunk, nr: how many.
__device__ __forceinline__ void lane_chunks(int p, int r0, int nr, int* c0, int* c1) {
    if (p < nr / 2) {
        *c0 = r0 + p;
        *c1 = *c0 + nr / 2;
    } else {
        const int i = 2 * (p - nr / 2);
        *c0 = i < r0 ? i : i + nr;
        *c1 = i + 1 < r0 ? i + 1 : i + 1 + nr;
    }
}

}  // namespace
}  // namespace fp8bs
