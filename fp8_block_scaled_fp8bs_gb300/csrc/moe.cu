// moe.cu -- the experts of a mixture-of-experts layer for a few tokens (fp8bs_moe_experts):
// gate and up products, silu(gate) * up, its quantisation, the down product and the weighted sum over
// experts ("DeepSeek-V3 Administrator & Developer Guide", §6.4 MoE expert routing, §8.5.3
// fp8_gemm_kernel for the products).
//
// First form: one warp per row of the weights, on the CUDA cores.
#include "gemm_common.cuh"
#include "quant_math.cuh"

namespace fp8bs {

namespace {

__device__ __forceinline__ void unpack_e4m3x4(uint32_t w, float* f) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const __nv_fp8x2_storage_t p = static_cast<__nv_fp8x2_storage_t>((w >> (16 * h)) & 0xFFFFu);
        const float2 v = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(p, __NV_E4M3)));
        f[2 * h] = v.x;
        f[2 * h + 1] = v.y;
    }
}

// Dot product over nkb K blocks: lane l takes 4 codes of each block. xs: stride between blocks' scales.
__device__ __forceinline__ float dot_blocks(const uint8_t* w, const float* ws, const uint8_t* x,
                                            const float* xs, int xs_stride, int nkb, int lane) {
    float sum = 0.0f;
    for (int kb = 0; kb < nkb; ++kb) {
        float a[4], b[4];
        unpack_e4m3x4(*reinterpret_cast<const uint32_t*>(w + kb * BK + 4 * lane), a);
        unpack_e4m3x4(*reinterpret_cast<const uint32_t*>(x + kb * BK + 4 * lane), b);
        const float p = a[0] * b[0] + a[1] * b[1] + a[2] * b[2] + a[3] * b[3];
        sum = fmaf(p, ws[kb] * xs[kb * xs_stride], sum);
    }
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
    return sum;
}

// h[slot][i], slot = t * top_k + j; grid (I / 8, E)
__global__ void moe_up_kernel(const MoeArgs a, const uint8_t* x8, const float* xs, float* h) {
    grid_dependency_wait();
    const int i = blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    const int e = blockIdx.y;
    const int nkb = a.D / BK;
    const uint8_t* w13 = static_cast<const uint8_t*>(a.w13) + static_cast<int64_t>(e) * 2 * a.I * a.D;
    const float* s13 = a.s13 + static_cast<int64_t>(e) * (2 * a.I / BK) * nkb;
    for (int s = 0; s < a.T * a.top_k; ++s) {
        const int id = a.ids[s];
        if ((id < -1 || id >= a.E) && lane == 0) record_error(FP8BS_DEVERR_INDEX);
        if (id != e) continue;
        const int t = s / a.top_k;
        const float g = dot_blocks(w13 + static_cast<int64_t>(i) * a.D, s13 + (i / BK) * nkb,
                                   x8 + static_cast<int64_t>(t) * a.D, xs + t, kMoeMaxTokens, nkb, lane);
        const float u = dot_blocks(w13 + static_cast<int64_t>(a.I + i) * a.D,
                                   s13 + ((a.I + i) / BK) * nkb, x8 + static_cast<int64_t>(t) * a.D,
                                   xs + t, kMoeMaxTokens, nkb, lane);
        if (lane == 0) h[static_cast<int64_t>(s) * a.I + i] = g / (1.0f + expf(-g)) * u;
    }
}

// one warp per (slot, block of 128)
__global__ void moe_quant_kernel(const MoeArgs a, const float* h, uint8_t* h8, float* hs) {
    grid_dependency_wait();
    const int s = blockIdx.y;
    const int b = blockIdx.x;
    const int lane = threadIdx.x;
    if (a.ids[s] < 0 || a.ids[s] >= a.E) return;
    const float4 v = *reinterpret_cast<const float4*>(h + static_cast<int64_t>(s) * a.I + b * BK + 4 * lane);
    float m = fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, i));
    float sc = __fdiv_rn(fmaxf(m, 1e-4f), 448.0f);
    if (a.ue8m0) {
        uint32_t bits = __float_as_uint(sc);
        if (bits & 0x007FFFFFu) bits = (bits & 0xFF800000u) + 0x00800000u;
        sc = __uint_as_float(bits);
    }
    const uint32_t lo = pack_e4m3x2(__fdiv_rn(v.x, sc), __fdiv_rn(v.y, sc));
    const uint32_t hi = pack_e4m3x2(__fdiv_rn(v.z, sc), __fdiv_rn(v.w, sc));
    *reinterpret_cast<uint32_t*>(h8 + static_cast<int64_t>(s) * a.I + b * BK + 4 * lane) = lo | (hi << 16);
    if (lane == 0) hs[s * (a.I / BK) + b] = sc;
}

__global__ void moe_down_kernel(const MoeArgs a, const uint8_t* h8, const float* hs) {
    grid_dependency_wait();
    const int d = blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.y;
    const int nkb = a.I / BK;
    float y = 0.0f;
    for (int j = 0; j < a.top_k; ++j) {
        const int s = t * a.top_k + j;
        const int e = a.ids[s];
        if (e < 0 || e >= a.E) continue;
        const float v = dot_blocks(
            static_cast<const uint8_t*>(a.w2) + (static_cast<int64_t>(e) * a.D + d) * a.I,
            a.s2 + (static_cast<int64_t>(e) * (a.D / BK) + d / BK) * nkb,
            h8 + static_cast<int64_t>(s) * a.I, hs + s * nkb, 1, nkb, lane);
        y = fmaf(a.weights[s], v, y);
    }
    if (lane == 0) static_cast<__nv_bfloat16*>(a.y)[static_cast<int64_t>(t) * a.D + d] = __float2bfloat16_rn(y);
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
    w.x8 = take(T * D);
    w.xs = take(D / BK * kMoeMaxTokens * 4);
    w.h8 = take(slots * I);
    w.hs = take(slots * (I / BK) * 4);
    w.h32 = take(slots * I * 4);
    w.weights = take(slots * 4);
    w.ids = take(slots * 4);
    w.total = at;
    (void)E;
    return w;
}

cudaError_t launch_moe_experts(const MoeArgs& a, const MoeWorkspace& w, cudaStream_t stream) {
    uint8_t* h8 = a.ws + w.h8;
    float* hs = reinterpret_cast<float*>(a.ws + w.hs);
    float* h32 = reinterpret_cast<float*>(a.ws + w.h32);
    cudaError_t e = launch_pdl(moe_up_kernel, dim3(a.I / 8, a.E), 256, 0, stream, a, a.ws + w.x8,
                               reinterpret_cast<const float*>(a.ws + w.xs), h32);
    if (e == cudaSuccess)
        e = launch_pdl(moe_quant_kernel, dim3(a.I / BK, a.T * a.top_k), 32, 0, stream, a, h32, h8, hs);
    if (e == cudaSuccess)
        e = launch_pdl(moe_down_kernel, dim3(a.D / 8, a.T), 256, 0, stream, a, h8, hs);
    return e;
}

cudaError_t read_error_moe(unsigned int* out, bool clear, cudaStream_t stream) {
    return read_tu_error(out, clear, stream);
}

}  // namespace fp8bs
