// attention_fp8_tiles.cu -- attention over a paged cache of e4m3 codes for sequences of many query rows: the kernel of
// attention.cu, its keys taken as codes and its values widened on the way (attention_tiles.cuh).
//
// Measured, on inputs that change from call to call: a chunk of 4096 tokens over 8192 keys, 32 / 8 heads of 128, 318 to
// 320 us (0.66 of the products' floor in bf16; a bf16 cache 298): the tensor pipe is at 55 % and a key tile's chain
// (softmax 1750 cycles of 3700 and 180 to store P, then P V and the next S) is what lasts. Tried for it and slower: the
// next S under the softmax, P in columns of its own (409 us), the softmax in two steps, each with its own product (359;
// issued as they come 445), 64-key tiles with two S (382).
#include "attention_tiles.cuh"

namespace fp8bs {

namespace {

AttnParts parts_of(const fp8bs_paged_attention_args& a, const AttentionPlan& plan) {
    AttnParts p = {};
    p.rows = a.T * a.q_heads;
    if (plan.pieces > 1) {
        p.o = static_cast<float*>(a.workspace);
        p.ml = reinterpret_cast<float2*>(p.o + plan.pieces * p.rows * a.cache.dv);
    }
    return p;
}

template <int DK, int DV, int NQ>
cudaError_t launch_tiles(const AttentionMapsFp8& maps, const fp8bs_paged_attention_args& a, const Scales& scales,
                         const AttentionPlan& plan, int more_rows, int num_sms, cudaStream_t stream) {
    using Cfg = AttnCfg<DK, DV, NQ, true>;
    auto kernel = paged_attention_kernel<Cfg>;
    const cudaError_t e = set_smem(kernel, Cfg::SMEM);
    if (e != cudaSuccess) return e;
    const int64_t items = tile_bound(a, Cfg::ROWS) * a.cache.heads * plan.pieces;
    if (items >= INT32_MAX) return cudaErrorInvalidValue;
    const int64_t resident = static_cast<int64_t>(num_sms) * Cfg::CTAS;
    const unsigned grid = static_cast<unsigned>(items < resident ? items : resident);
    AttentionModes modes = {};
    modes.box_log2 = maps.box_log2;
    return launch_pdl(kernel, grid, Cfg::THREADS, Cfg::SMEM, stream, maps.k, maps.v, a, modes, plan.piece_len,
                      plan.pieces, parts_of(a, plan), scales, more_rows);
}

template <int DV>
cudaError_t launch_join(const fp8bs_paged_attention_args& a, const AttentionPlan& plan, cudaStream_t stream) {
    const AttnParts parts = parts_of(a, plan);
    return launch_pdl(attention_join_kernel<DV, 1, true>, static_cast<unsigned>((parts.rows + 3) / 4), 128, 0, stream,
                      parts, plan.pieces, static_cast<__nv_bfloat16*>(a.out), a.lse);
}

}  // namespace

cudaError_t launch_attention_fp8_tiles(const AttentionMapsFp8& maps, const fp8bs_paged_attention_args& a,
                                       const float* k_scale, const float* v_scale, const AttentionPlan& plan,
                                       bool two, int more_rows, int num_sms, cudaStream_t stream) {
    const Scales scales = {k_scale, v_scale};
    switch (a.cache.dk) {
        case 64:
            return two ? launch_tiles<64, 64, 2>(maps, a, scales, plan, more_rows, num_sms, stream)
                       : launch_tiles<64, 64, 1>(maps, a, scales, plan, more_rows, num_sms, stream);
        case 128:
            return two ? launch_tiles<128, 128, 2>(maps, a, scales, plan, more_rows, num_sms, stream)
                       : launch_tiles<128, 128, 1>(maps, a, scales, plan, more_rows, num_sms, stream);
        default:
            return two ? launch_tiles<192, 128, 2>(maps, a, scales, plan, more_rows, num_sms, stream)
                       : launch_tiles<192, 128, 1>(maps, a, scales, plan, more_rows, num_sms, stream);
    }
}

cudaError_t launch_attention_fp8_tiles_join(const fp8bs_paged_attention_args& a, const AttentionPlan& plan,
                                            cudaStream_t stream) {
    return a.cache.dv == 64 ? launch_join<64>(a, plan, stream) : launch_join<128>(a, plan, stream);
}

cudaError_t read_error_attention_fp8_tiles(unsigned int* out, bool clear, cudaStream_t stream) {
    return read_tu_error(out, clear, stream);
}

}  // namespace fp8bs
