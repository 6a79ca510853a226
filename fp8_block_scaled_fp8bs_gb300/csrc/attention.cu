// attention.cu -- attention of new tokens over a paged cache (fp8bs_paged_attention).
//
// First form: one warp per query token and head, one pass over the keys with the running maximum and
// sum of the softmax.
#include "gemm_common.cuh"
#include "quant_math.cuh"

namespace fp8bs {

namespace {

template <int DK, int DV>
__global__ void __launch_bounds__(256) attention_warp_kernel(const __grid_constant__ fp8bs_paged_attention_args a) {
    constexpr int NK = DK / 64, NV = DV / 64;
    grid_dependency_wait();
    const int lane = threadIdx.x & 31;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (row >= a.T * a.q_heads) return;
    const int64_t t = row / a.q_heads;
    const int head = static_cast<int>(row - t * a.q_heads);
    const int kh = head / static_cast<int>(a.q_heads / a.cache.heads);
    int b = 0;
    while (b + 1 < a.B && a.q_start[b + 1] <= t) ++b;
    const int n = a.q_start[b + 1] - a.q_start[b];
    const int64_t L = a.kv_len[b];
    const int64_t i = t - a.q_start[b];
    if ((n > a.max_q_len || L > a.max_kv_len) && lane == 0) record_error(FP8BS_DEVERR_INDEX);
    int64_t hi = a.causal ? min(L, L - n + i + 1) : L;
    int64_t lo = a.window > 0 ? max(static_cast<int64_t>(0), L - n + i - a.window + 1) : 0;
    const uint32_t* q = reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(a.q) +
                                                          t * a.q_token_stride + head * a.q_head_stride);
    float qf[2 * NK], o[2 * NV] = {};
#pragma unroll
    for (int c = 0; c < NK; ++c) {
        const uint32_t w = q[c * 32 + lane];
        qf[2 * c] = bf16_lo(w) * a.scale;
        qf[2 * c + 1] = bf16_hi(w) * a.scale;
    }
    float m = -INFINITY, l = 0.0f;
    for (int64_t j = lo; j < hi; ++j) {
        const int page = a.page_table[b * a.table_stride + j / a.cache.page_size];
        const int64_t off = j % a.cache.page_size;
        const bool ok = page >= 0 && page < a.cache.pages;
        if (!ok && lane == 0) record_error(FP8BS_DEVERR_INDEX);
        const int64_t pg = ok ? page : 0;
        const uint32_t* k = reinterpret_cast<const uint32_t*>(
            static_cast<const __nv_bfloat16*>(a.cache.k) + pg * a.cache.k_page_stride +
            off * a.cache.k_slot_stride + kh * a.cache.k_head_stride);
        const uint32_t* v = reinterpret_cast<const uint32_t*>(
            static_cast<const __nv_bfloat16*>(a.cache.v) + pg * a.cache.v_page_stride +
            off * a.cache.v_slot_stride + kh * a.cache.v_head_stride);
        float s = 0.0f;
#pragma unroll
        for (int c = 0; c < NK; ++c) {
            const uint32_t w = ok ? k[c * 32 + lane] : 0u;
            s += qf[2 * c] * bf16_lo(w) + qf[2 * c + 1] * bf16_hi(w);
        }
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        const float m2 = fmaxf(m, s);
        const float keep = expf(m - m2), p = expf(s - m2);
        l = l * keep + p;
        m = m2;
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            const uint32_t w = ok ? v[c * 32 + lane] : 0u;
            o[2 * c] = o[2 * c] * keep + p * bf16_lo(w);
            o[2 * c + 1] = o[2 * c + 1] * keep + p * bf16_hi(w);
        }
    }
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
    uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.out) + row * DV);
#pragma unroll
    for (int c = 0; c < NV; ++c) out[c * 32 + lane] = pack_bf16x2(o[2 * c] * inv, o[2 * c + 1] * inv);
    if (a.lse && lane == 0) a.lse[row] = l > 0.0f ? m + logf(l) : -INFINITY;
}

}  // namespace

AttentionPlan attention_plan(const fp8bs_paged_attention_args&, int) { return AttentionPlan{1, 1 << 30}; }

size_t attention_workspace(const fp8bs_paged_attention_args&, const AttentionPlan&) { return 0; }

cudaError_t launch_paged_attention(const fp8bs_paged_attention_args& a, const AttentionPlan&,
                                   cudaStream_t stream) {
    const dim3 grid(static_cast<unsigned>((a.T * a.q_heads + 7) / 8));
    if (a.cache.dk == 64) return launch_pdl(attention_warp_kernel<64, 64>, grid, 256, 0, stream, a);
    if (a.cache.dk == 128) return launch_pdl(attention_warp_kernel<128, 128>, grid, 256, 0, stream, a);
    return launch_pdl(attention_warp_kernel<192, 128>, grid, 256, 0, stream, a);
}

cudaError_t read_error_attention(unsigned int* out, bool clear, cudaStream_t stream) {
    return read_tu_error(out, clear, stream);
}

}  // namespace fp8bs
