// attention_fp8.cu -- attention of new tokens over a paged cache of e4m3 codes with one scale per page and head
// (fp8bs_paged_attention_fp8).
//
// One warp per query token and head. A lane holds DK / 32 channels of the query and DV / 32 of the output and goes
// over the keys with a running maximum and sum. Bound by the latency of each key's dot product.
#include "gemm_common.cuh"
#include "quant_math.cuh"

namespace fp8bs {

namespace {

__device__ __forceinline__ float e4m3_value(uint8_t c) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
}

template <int DK, int DV>
__global__ void __launch_bounds__(128) paged_attention_fp8_kernel(const __grid_constant__ fp8bs_paged_attention_args a,
                                                                  const float* k_scale, const float* v_scale) {
    constexpr int KP = DK / 32, VP = DV / 32;
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    if (row >= a.T * a.q_heads) return;
    const int64_t t = row / a.q_heads;
    const int h = static_cast<int>(row - t * a.q_heads);
    const int kh = h / static_cast<int>(a.q_heads / a.cache.heads);
    // the sequence of this token: the last that starts at or before it
    int64_t lo = 0, hi = a.B;
    while (hi - lo > 1) {
        const int64_t mid = (lo + hi) / 2;
        if (a.q_start[mid] <= t) lo = mid; else hi = mid;
    }
    const int64_t q0 = a.q_start[lo], n = a.q_start[lo + 1] - q0, L = a.kv_len[lo];
    if (t < q0 || t >= q0 + n) return;
    if (n > a.max_q_len || L > a.max_kv_len || L < 0 || q0 < 0 || q0 + n > a.T) {
        if (lane == 0) record_error(FP8BS_DEVERR_INDEX);
        return;
    }
    const int64_t last = L - n + (t - q0);
    const int64_t end = a.causal ? min(L, max(last + 1, int64_t{0})) : L;
    const int64_t begin = a.window > 0 ? min(L, max(last - a.window + 1, int64_t{0})) : 0;
    float q[KP], o[VP] = {}, m = -INFINITY, l = 0.0f;
    const __nv_bfloat16* qp = static_cast<const __nv_bfloat16*>(a.q) + t * a.q_token_stride + h * a.q_head_stride;
#pragma unroll
    for (int i = 0; i < KP; ++i) q[i] = __bfloat162float(qp[lane + 32 * i]);
    const int32_t* table = a.page_table + lo * a.table_stride;
    for (int64_t j = begin; j < end; ++j) {
        const int64_t page = table[j / a.cache.page_size], slot = j % a.cache.page_size;
        const bool there = page >= 0 && page < a.cache.pages;
        if (!there && lane == 0) record_error(FP8BS_DEVERR_INDEX);
        float s = 0.0f, vs = 0.0f;
        if (there) {
            const uint8_t* k = static_cast<const uint8_t*>(a.cache.k) + page * a.cache.k_page_stride +
                               slot * a.cache.k_slot_stride + kh * a.cache.k_head_stride;
#pragma unroll
            for (int i = 0; i < KP; ++i) s = fmaf(q[i], e4m3_value(k[lane + 32 * i]), s);
#pragma unroll
            for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
            s *= k_scale[page * a.cache.heads + kh] * a.scale;
            vs = v_scale[page * a.cache.heads + kh];
        }
        const float top = fmaxf(m, s);
        const float keep = m == top ? 1.0f : expf(m - top);
        const float p = s == -INFINITY ? 0.0f : expf(s - top);
        m = top;
        l = l * keep + p;
        const uint8_t* v = static_cast<const uint8_t*>(a.cache.v) + page * a.cache.v_page_stride +
                           slot * a.cache.v_slot_stride + kh * a.cache.v_head_stride;
#pragma unroll
        for (int i = 0; i < VP; ++i)
            o[i] = fmaf(there ? e4m3_value(v[lane + 32 * i]) * vs : 0.0f, p, o[i] * keep);
    }
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + row * DV;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
    for (int i = 0; i < VP; ++i) out[lane + 32 * i] = __float2bfloat16_rn(o[i] * inv);
    if (a.lse && lane == 0) a.lse[row] = l == 0.0f ? -INFINITY : m + logf(l);
}

}  // namespace

cudaError_t launch_paged_attention_fp8(const fp8bs_paged_attention_args& a, const float* k_scale, const float* v_scale,
                                       cudaStream_t stream) {
    const unsigned grid = static_cast<unsigned>((a.T * a.q_heads + 3) / 4);
    auto kernel = a.cache.dk == 64    ? paged_attention_fp8_kernel<64, 64>
                  : a.cache.dk == 128 ? paged_attention_fp8_kernel<128, 128>
                                      : paged_attention_fp8_kernel<192, 128>;
    return launch_pdl(kernel, grid, 128, 0, stream, a, k_scale, v_scale);
}

cudaError_t read_error_attention_fp8(unsigned int* out, bool clear, cudaStream_t stream) {
    return read_tu_error(out, clear, stream);
}

}  // namespace fp8bs
