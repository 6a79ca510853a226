// norm_rope.cu -- RMS norm of queries and keys per head, rotation by position and the write of
// keys and values into a paged cache, in one pass (fp8bs_qk_norm_rope).
//
// Bound by memory: every element is read and written once, 4 bytes per element of q, k and v. One
// CTA per token; LPR lanes share a row (one head of the token), each lane taking two chunks of 8
// channels (16-byte loads and stores). The two chunks are the two halves of the same rotation
// pairs, so the rotation needs no exchange between lanes, and the norm one reduction over LPR
// lanes. The token's cosines and sines are read once into registers and serve all its heads.
#include "gemm_common.cuh"
#include "quant_math.cuh"

namespace fp8bs {

namespace {

constexpr int NR_THREADS = 128;
constexpr int NR_BATCH = 4;      // rows a lane group loads before it computes any

__device__ __forceinline__ void unpack8(const uint4& v, float* f) {
    f[0] = bf16_lo(v.x); f[1] = bf16_hi(v.x); f[2] = bf16_lo(v.y); f[3] = bf16_hi(v.y);
    f[4] = bf16_lo(v.z); f[5] = bf16_hi(v.z); f[6] = bf16_lo(v.w); f[7] = bf16_hi(v.w);
}

__device__ __forceinline__ uint4 pack8(const float* f) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}

template <int LPR>
__global__ void __launch_bounds__(NR_THREADS) qk_norm_rope_kernel(
    const __grid_constant__ fp8bs_qk_norm_rope_args a) {
    constexpr int GROUPS = NR_THREADS / LPR;
    const int64_t t = blockIdx.x;
    const int p = threadIdx.x % LPR;
    const int grp = threadIdx.x / LPR;
    const int dk = static_cast<int>(a.cache.dk);
    const int dv = static_cast<int>(a.cache.dv);
    const int hq = static_cast<int>(a.q_heads);
    const int hk = static_cast<int>(a.cache.heads);
    const int rows = hq + hk + (a.v ? hk : 0);

    // This lane's chunks of a q or k row: rotated chunks come as pairs (the chunk, the one half
    // the rotated range further on), the others in order.
    const int r0 = static_cast<int>(a.rot_start) / 8;
    const int nr = static_cast<int>(a.rot_dim) / 8;
    const bool rotates = p < nr / 2;
    int c0, c1;
    if (rotates) {
        c0 = r0 + p;
        c1 = c0 + nr / 2;
    } else {
        const int i = 2 * (p - nr / 2);
        c0 = i < r0 ? i : i + nr;
        c1 = i + 1 < r0 ? i + 1 : i + 1 + nr;
    }
    const bool has_k = p < dk / 16;
    const bool has_v = p < dv / 16;

    grid_dependency_wait();
    grid_launch_dependents();

    const int pos = a.positions[t];
    const bool pos_ok = pos >= 0 && pos < a.max_positions;
    int64_t slot = a.slots ? a.slots[t] : t;
    const bool slot_past = slot >= a.cache.pages * a.cache.page_size;
    if ((!pos_ok || slot_past) && threadIdx.x == 0) record_error(FP8BS_DEVERR_INDEX);
    const bool store_kv = pos_ok && slot >= 0 && !slot_past;
    if (!store_kv) slot = 0;
    const int64_t page = slot / a.cache.page_size;
    const int64_t off = slot - page * a.cache.page_size;

    // cosines and sines of this lane's 8 pairs: pair 8p + i (halves), or the 4 pairs of each of
    // its two chunks (interleaved)
    float cs[8], sn[8];
    if (rotates && pos_ok) {
        const float* ct = a.cos + static_cast<int64_t>(pos) * (a.rot_dim / 2);
        const float* st = a.sin + static_cast<int64_t>(pos) * (a.rot_dim / 2);
        const int i0 = a.interleaved ? 4 * p : 8 * p;
        const int i1 = a.interleaved ? 4 * (p + nr / 2) : 8 * p + 4;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            cs[i] = __ldg(ct + i0 + i);
            sn[i] = __ldg(st + i0 + i);
            cs[4 + i] = __ldg(ct + i1 + i);
            sn[4 + i] = __ldg(st + i1 + i);
        }
    }

    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + t * a.q_token_stride;
    const __nv_bfloat16* k = static_cast<const __nv_bfloat16*>(a.k) + t * a.k_token_stride;
    const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(a.v) + (a.v ? t * a.v_token_stride : 0);
    __nv_bfloat16* qo = static_cast<__nv_bfloat16*>(a.q_out) + t * hq * dk;
    __nv_bfloat16* ko = static_cast<__nv_bfloat16*>(a.cache.k) + page * a.cache.k_page_stride +
                        off * a.cache.k_slot_stride;
    __nv_bfloat16* vo = static_cast<__nv_bfloat16*>(a.cache.v) + page * a.cache.v_page_stride +
                        off * a.cache.v_slot_stride;

    // Row loops are uniform over the CTA: the norm's reduction shuffles across whole warps.
    for (int base = 0; base < rows; base += GROUPS * NR_BATCH) {
        uint4 x0[NR_BATCH], x1[NR_BATCH];
#pragma unroll
        for (int b = 0; b < NR_BATCH; ++b) {
            const int r = base + b * GROUPS + grp;
            x0[b] = x1[b] = make_uint4(0, 0, 0, 0);
            if (r >= rows) continue;
            if (r < hq + hk) {
                if (!has_k) continue;
                const uint4* src = reinterpret_cast<const uint4*>(
                    r < hq ? q + r * a.q_head_stride : k + (r - hq) * a.k_head_stride);
                x0[b] = __ldg(src + c0);
                x1[b] = __ldg(src + c1);
            } else if (has_v) {
                const uint4* src =
                    reinterpret_cast<const uint4*>(v + (r - hq - hk) * a.v_head_stride);
                x0[b] = __ldg(src + 2 * p);
                x1[b] = __ldg(src + 2 * p + 1);
            }
        }
#pragma unroll
        for (int b = 0; b < NR_BATCH; ++b) {
            const int r = base + b * GROUPS + grp;
            if (base + b * GROUPS >= rows) break;
            if (base + b * GROUPS < hq + hk) {
                // (rows of v beside rows of k in a warp take part in the reduction only)
                float f[16];
                unpack8(x0[b], f);
                unpack8(x1[b], f + 8);
                const void* w = r < hq ? a.q_weight : a.k_weight;
                float ss = 0.0f;
#pragma unroll
                for (int i = 0; i < 16; ++i) ss = fmaf(f[i], f[i], ss);
#pragma unroll
                for (int m = LPR / 2; m > 0; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
                if (r < hq + hk && has_k) {
                    if (w) {
                        const float inv = 1.0f / sqrtf(ss / static_cast<float>(dk) + a.eps);
                        float wf[16];
                        unpack8(__ldg(static_cast<const uint4*>(w) + c0), wf);
                        unpack8(__ldg(static_cast<const uint4*>(w) + c1), wf + 8);
#pragma unroll
                        for (int i = 0; i < 16; ++i) f[i] = f[i] * inv * wf[i];
                    }
                    if (rotates && pos_ok) {
                        if (a.interleaved) {
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const float u = f[2 * i], y = f[2 * i + 1];
                                f[2 * i] = u * cs[i] - y * sn[i];
                                f[2 * i + 1] = u * sn[i] + y * cs[i];
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const float u = f[i], y = f[8 + i];
                                f[i] = u * cs[i] - y * sn[i];
                                f[8 + i] = u * sn[i] + y * cs[i];
                            }
                        }
                    }
                    const uint4 zero = make_uint4(0, 0, 0, 0);
                    const uint4 o0 = pos_ok ? pack8(f) : zero;
                    const uint4 o1 = pos_ok ? pack8(f + 8) : zero;
                    if (r < hq) {
                        uint4* dst = reinterpret_cast<uint4*>(qo + r * dk);
                        dst[c0] = o0;
                        dst[c1] = o1;
                    } else if (store_kv) {
                        uint4* dst =
                            reinterpret_cast<uint4*>(ko + (r - hq) * a.cache.k_head_stride);
                        dst[c0] = o0;
                        dst[c1] = o1;
                    }
                }
            }
            if (r >= hq + hk && r < rows && has_v && store_kv) {
                uint4* dst = reinterpret_cast<uint4*>(vo + (r - hq - hk) * a.cache.v_head_stride);
                dst[2 * p] = x0[b];
                dst[2 * p + 1] = x1[b];
            }
        }
    }
}

}  // namespace

cudaError_t launch_qk_norm_rope(const fp8bs_qk_norm_rope_args& a, cudaStream_t stream) {
    const int64_t d = a.v && a.cache.dv > a.cache.dk ? a.cache.dv : a.cache.dk;
    const int grid = static_cast<int>(a.T);
    if (d <= 64) return launch_pdl(qk_norm_rope_kernel<4>, grid, NR_THREADS, 0, stream, a);
    if (d <= 128) return launch_pdl(qk_norm_rope_kernel<8>, grid, NR_THREADS, 0, stream, a);
    return launch_pdl(qk_norm_rope_kernel<16>, grid, NR_THREADS, 0, stream, a);
}

cudaError_t read_error_norm_rope(unsigned int* out, bool clear, cudaStream_t stream) {
    return read_tu_error(out, clear, stream);
}

}  // namespace fp8bs
