// api_layer.cu -- the C ABI of the operators around the FP8 products of a decoder layer
// (include/fp8bs.h): argument and device checks. Nothing here allocates memory or synchronises.
#include <cstdint>

#include "../../include/fp8bs.h"
#include "api_util.h"
#include "kernels.h"

namespace {

bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }

constexpr int64_t kMaxDim = int64_t{1} << 31;

// A stride that keeps rows on 16-byte boundaries.
bool stride_ok(int64_t s) { return s >= 0 && s % 8 == 0; }

// Sizes and strides of a cache; pointers of k (and, with values, v).
int check_cache(const fp8bs_kv_cache& c, bool values) {
    if (c.pages < 0 || c.page_size < 1 || c.heads < 1 || c.heads >= (1 << 16) ||
        c.page_size >= kMaxDim || c.pages >= kMaxDim)
        return FP8BS_ERR_INVALID_ARG;
    if (!stride_ok(c.k_page_stride) || !stride_ok(c.k_slot_stride) || !stride_ok(c.k_head_stride))
        return FP8BS_ERR_INVALID_ARG;
    if (values &&
        (!stride_ok(c.v_page_stride) || !stride_ok(c.v_slot_stride) || !stride_ok(c.v_head_stride)))
        return FP8BS_ERR_INVALID_ARG;
    // rows must not lie on one another
    if ((c.pages > 1 && c.k_page_stride < 8) || (c.page_size > 1 && c.k_slot_stride < 8) ||
        (c.heads > 1 && c.k_head_stride < 8))
        return FP8BS_ERR_INVALID_ARG;
    if (values && ((c.pages > 1 && c.v_page_stride < 8) || (c.page_size > 1 && c.v_slot_stride < 8) ||
                   (c.heads > 1 && c.v_head_stride < 8)))
        return FP8BS_ERR_INVALID_ARG;
    if (c.pages > 0 && (!c.k || (values && !c.v))) return FP8BS_ERR_INVALID_ARG;
    if (!aligned16(c.k) || (values && !aligned16(c.v))) return FP8BS_ERR_MISALIGNED;
    return FP8BS_OK;
}

}  // namespace

extern "C" int fp8bs_qk_norm_rope(const fp8bs_qk_norm_rope_args* args, void* stream) {
    if (!args) return FP8BS_ERR_INVALID_ARG;
    fp8bs_qk_norm_rope_args a = *args;
    if (!a.v) a.cache.dv = a.cache.dk;
    const int64_t dk = a.cache.dk, dv = a.cache.dv;
    if (a.T < 0 || a.T >= kMaxDim || a.q_heads < 0 || a.q_heads >= (1 << 16))
        return FP8BS_ERR_INVALID_ARG;
    if (dk < 16 || dk > 256 || dk % 16 || dv < 16 || dv > 256 || dv % 16) return FP8BS_ERR_INVALID_ARG;
    if (a.rot_start < 0 || a.rot_start % 8 || a.rot_dim < 0 || a.rot_dim % 16 || a.rot_start > dk ||
        a.rot_dim > dk - a.rot_start)
        return FP8BS_ERR_INVALID_ARG;
    if (a.max_positions < 0 || a.max_positions >= kMaxDim) return FP8BS_ERR_INVALID_ARG;
    if (!stride_ok(a.q_token_stride) || !stride_ok(a.q_head_stride) || !stride_ok(a.k_token_stride) ||
        !stride_ok(a.k_head_stride) || (a.v && (!stride_ok(a.v_token_stride) || !stride_ok(a.v_head_stride))))
        return FP8BS_ERR_INVALID_ARG;
    const int rc = check_cache(a.cache, a.v != nullptr);
    if (rc == FP8BS_ERR_INVALID_ARG) return rc;
    if (a.T == 0) return FP8BS_OK;
    if (!a.k || !a.positions || (a.q_heads > 0 && (!a.q || !a.q_out)) ||
        (a.rot_dim > 0 && (!a.cos || !a.sin)))
        return FP8BS_ERR_INVALID_ARG;
    if (rc != FP8BS_OK) return rc;
    if (!aligned16(a.q) || !aligned16(a.k) || !aligned16(a.v) || !aligned16(a.q_out) ||
        !aligned16(a.q_weight) || !aligned16(a.k_weight) || !aligned4(a.cos) || !aligned4(a.sin) ||
        !aligned4(a.positions) || !aligned8(a.slots))
        return FP8BS_ERR_MISALIGNED;
    int sms = 0;
    const int dev = check_device(&sms);
    if (dev != FP8BS_OK) return dev;
    return status_of(fp8bs::launch_qk_norm_rope(a, static_cast<cudaStream_t>(stream)));
}

namespace {

// A cache's keys or values as fp8bs::AttentionModes says. Pages past the end read as zero.
bool make_cache_map(CUtensorMap* map, const void* base, const fp8bs_kv_cache& c, int64_t d,
                    int64_t head_stride, int64_t slot_stride, int64_t page_stride, int mode, int box_slots) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    // (the stride of an axis of length one is never used, but has to be a valid one)
    auto bytes = [&](int64_t stride, int64_t n) {
        return static_cast<cuuint64_t>(n > 1 ? stride * 2 : d * 2);
    };
    const cuuint64_t chunks = static_cast<cuuint64_t>(d / 64);
    const cuuint64_t heads = static_cast<cuuint64_t>(c.heads), pages = static_cast<cuuint64_t>(c.pages);
    const cuuint64_t slots = static_cast<cuuint64_t>(c.page_size);
    cuuint64_t dims[5], strides[4];
    cuuint32_t box[5], estr[5] = {1u, 1u, 1u, 1u, 1u};
    int rank = 5;
    if (mode == 2) {
        rank = 4;
        dims[0] = static_cast<cuuint64_t>(d), dims[1] = heads, dims[2] = slots, dims[3] = pages;
        strides[0] = bytes(head_stride, c.heads);
        strides[1] = bytes(slot_stride, c.page_size);
        strides[2] = bytes(page_stride, c.pages);
        box[0] = 64, box[1] = 1, box[2] = static_cast<cuuint32_t>(box_slots), box[3] = 1;
    } else {
        dims[0] = 64, dims[1] = 8, dims[2] = mode == 0 ? heads * chunks : chunks, dims[3] = slots / 8;
        dims[4] = mode == 0 ? pages : pages * heads;
        strides[0] = static_cast<cuuint64_t>(slot_stride) * 2;
        strides[1] = 128;
        strides[2] = static_cast<cuuint64_t>(slot_stride) * 16;
        strides[3] = mode == 0 ? bytes(page_stride, c.pages) : bytes(head_stride, c.heads);
        box[0] = 64, box[1] = 8, box[2] = static_cast<cuuint32_t>(chunks);
        box[3] = static_cast<cuuint32_t>(box_slots / 8), box[4] = 1;
    }
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, static_cast<cuuint32_t>(rank), const_cast<void*>(base),
               dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Everything but the pointers of a paged_attention call.
int check_attention_sizes(const fp8bs_paged_attention_args& a) {
    const int64_t dk = a.cache.dk, dv = a.cache.dv;
    if (!((dk == 64 && dv == 64) || (dk == 128 && dv == 128) || (dk == 192 && dv == 128)))
        return FP8BS_ERR_INVALID_ARG;
    if (a.B < 0 || a.B >= (1 << 20) || a.T < 0 || a.T >= kMaxDim || a.q_heads < 1 ||
        a.q_heads >= (1 << 16) || a.cache.heads < 1 || a.q_heads % a.cache.heads || a.window < 0 ||
        a.max_q_len < 0 || a.max_q_len > a.T || a.max_kv_len < 0 || a.max_kv_len >= kMaxDim - 1024 ||
        a.table_stride < 0 || a.T * (a.q_heads / a.cache.heads) >= kMaxDim - 1024)
        return FP8BS_ERR_INVALID_ARG;
    if (a.T > 0 && (a.B < 1 || a.max_q_len < 1)) return FP8BS_ERR_INVALID_ARG;
    if (a.cache.page_size < 1 ||
        (a.max_kv_len > 0 && a.table_stride < (a.max_kv_len - 1) / a.cache.page_size + 1))
        return FP8BS_ERR_INVALID_ARG;
    return FP8BS_OK;
}

// A window as long as the longest sequence leaves nothing out: none, so that sums with what remains stay far below
// 2^63 (callers without a window may pass the largest integer).
fp8bs_paged_attention_args without_idle_window(const fp8bs_paged_attention_args& args) {
    fp8bs_paged_attention_args a = args;
    if (a.window >= a.max_kv_len) a.window = 0;
    return a;
}

}  // namespace

extern "C" int fp8bs_paged_attention_workspace_size(const fp8bs_paged_attention_args* args,
                                                    size_t* bytes) {
    if (!args || !bytes) return FP8BS_ERR_INVALID_ARG;
    const int rc = check_attention_sizes(*args);
    if (rc != FP8BS_OK) return rc;
    int sms = 0;
    const int dev = check_device(&sms);
    if (dev != FP8BS_OK) return dev;
    const fp8bs_paged_attention_args a = without_idle_window(*args);
    *bytes = a.T == 0 ? 0 : fp8bs::attention_workspace(a, fp8bs::attention_plan(a, sms));
    return FP8BS_OK;
}

extern "C" int fp8bs_paged_attention(const fp8bs_paged_attention_args* args, void* stream) {
    if (!args) return FP8BS_ERR_INVALID_ARG;
    int rc = check_attention_sizes(*args);
    if (rc != FP8BS_OK) return rc;
    const fp8bs_paged_attention_args a = without_idle_window(*args);
    if (!stride_ok(a.q_token_stride) || !stride_ok(a.q_head_stride)) return FP8BS_ERR_INVALID_ARG;
    rc = check_cache(a.cache, true);
    if (rc == FP8BS_ERR_INVALID_ARG || a.cache.pages < 1) return FP8BS_ERR_INVALID_ARG;
    if (a.T == 0) return FP8BS_OK;
    if (!a.q || !a.q_start || !a.kv_len || !a.out || (a.max_kv_len > 0 && !a.page_table))
        return FP8BS_ERR_INVALID_ARG;
    if (rc != FP8BS_OK) return rc;
    if (!aligned16(a.q) || !aligned16(a.out) || !aligned4(a.lse) || !aligned4(a.page_table) ||
        !aligned4(a.q_start) || !aligned4(a.kv_len) || !aligned16(a.workspace))
        return FP8BS_ERR_MISALIGNED;
    int sms = 0;
    rc = check_device(&sms);
    if (rc != FP8BS_OK) return rc;
    const fp8bs::AttentionPlan plan = fp8bs::attention_plan(a, sms);
    const size_t need = fp8bs::attention_workspace(a, plan);
    if (need > 0 && (!a.workspace || a.workspace_bytes < need)) return FP8BS_ERR_INVALID_ARG;
    const fp8bs::AttentionModes modes = fp8bs::attention_modes(a.cache);
    CUtensorMap tmK, tmV;
    const fp8bs_kv_cache& c = a.cache;
    if (!make_cache_map(&tmK, c.k, c, c.dk, c.k_head_stride, c.k_slot_stride, c.k_page_stride, modes.k,
                        1 << modes.box_log2) ||
        !make_cache_map(&tmV, c.v, c, c.dv, c.v_head_stride, c.v_slot_stride, c.v_page_stride, modes.v,
                        1 << modes.box_log2))
        return FP8BS_ERR_CUDA;
    return status_of(fp8bs::launch_paged_attention(tmK, tmV, a, modes, plan, sms,
                                                   static_cast<cudaStream_t>(stream)));
}

namespace {

int check_routing(const fp8bs_moe_routing* r, int64_t D, int64_t E) {
    if (!r) return FP8BS_ERR_INVALID_ARG;
    if (D < 128 || D > 16384 || D % 128 || E < 1 || E > 512) return FP8BS_ERR_INVALID_ARG;
    if (r->top_k < 1 || r->top_k > 32 || r->groups < 1 || r->groups > 32 || E % r->groups ||
        r->topk_groups < 1 || r->topk_groups > r->groups ||
        r->top_k > r->topk_groups * (E / r->groups))
        return FP8BS_ERR_INVALID_ARG;
    if (r->score != FP8BS_SCORE_SIGMOID && r->score != FP8BS_SCORE_SOFTMAX) return FP8BS_ERR_INVALID_ARG;
    return FP8BS_OK;
}

int check_experts(const void* x, const void* w13, const float* s13, const void* w2, const float* s2,
                  void* y, int64_t T, int64_t D, int64_t I, int64_t E, int64_t top_k, int scale_fmt,
                  void* workspace, size_t workspace_bytes, fp8bs::MoeWorkspace* ws) {
    if (T < 0 || T > fp8bs::kMoeMaxTokens || D < 128 || D > 16384 || D % 128 || I < 128 || I > 16384 ||
        I % 128 || E < 1 || E > 512 || top_k < 1 || top_k > 32)
        return FP8BS_ERR_INVALID_ARG;
    if (scale_fmt != FP8BS_SCALE_FP32 && scale_fmt != FP8BS_SCALE_UE8M0) return FP8BS_ERR_INVALID_ARG;
    if (T == 0) return FP8BS_OK;
    if (!x || !w13 || !s13 || !w2 || !s2 || !y || !workspace) return FP8BS_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(w13) || !aligned16(w2) || !aligned16(y) || !aligned16(workspace) ||
        !aligned4(s13) || !aligned4(s2))
        return FP8BS_ERR_MISALIGNED;
    *ws = fp8bs::moe_workspace(T, D, I, E, top_k);
    if (workspace_bytes < ws->total) return FP8BS_ERR_INVALID_ARG;
    return FP8BS_OK;
}

int run_experts(const fp8bs::MoeWorkspace& ws, const float* weights, const int32_t* ids, const void* w13,
                const float* s13, const void* w2, const float* s2, void* y, int64_t T, int64_t D,
                int64_t I, int64_t E, int64_t top_k, int scale_fmt, void* workspace, int sms, void* stream) {
    fp8bs::MoeArgs a = {};
    a.weights = weights;
    a.ids = ids;
    a.w13 = w13;
    a.s13 = s13;
    a.w2 = w2;
    a.s2 = s2;
    a.y = y;
    a.ws = static_cast<uint8_t*>(workspace);
    a.T = static_cast<int>(T);
    a.D = static_cast<int>(D);
    a.I = static_cast<int>(I);
    a.E = static_cast<int>(E);
    a.top_k = static_cast<int>(top_k);
    a.ue8m0 = scale_fmt == FP8BS_SCALE_UE8M0;
    fp8bs::MoeMaps m;
    const int mt = fp8bs::moe_token_rows(T);
    if (!make_map(&m.w13, w13, E * 2 * I, D, 128) || !make_map(&m.w2, w2, E * D, I, 128) ||
        !make_map(&m.x8, a.ws + ws.x8, T, D, mt > 16 ? 1 : mt) || !make_map(&m.h8, a.ws + ws.h8, ws.active * T, I, mt))
        return FP8BS_ERR_CUDA;
    return status_of(fp8bs::launch_moe_experts(m, a, ws, sms, static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" int fp8bs_moe_route(const void* x, const fp8bs_moe_routing* routing, float* weights,
                               int32_t* ids, int64_t T, int64_t D, int64_t experts, void* stream) {
    const int rc = check_routing(routing, D, experts);
    if (rc != FP8BS_OK) return rc;
    if (T < 0 || T >= kMaxDim / 4) return FP8BS_ERR_INVALID_ARG;
    if (T == 0) return FP8BS_OK;
    if (!x || !weights || !ids || !routing->router_w) return FP8BS_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(routing->router_w) || !aligned4(routing->bias) ||
        !aligned4(weights) || !aligned4(ids))
        return FP8BS_ERR_MISALIGNED;
    int sms = 0;
    const int dev = check_device(&sms);
    if (dev != FP8BS_OK) return dev;
    return status_of(fp8bs::launch_moe_prepare(x, routing, weights, ids, nullptr, nullptr, T, D, experts,
                                               false, static_cast<cudaStream_t>(stream)));
}

extern "C" int fp8bs_moe_workspace_size(int64_t T, int64_t D, int64_t I, int64_t experts, int64_t top_k,
                                        size_t* bytes) {
    if (!bytes || T < 0 || T > fp8bs::kMoeMaxTokens || D < 128 || D > 16384 || D % 128 || I < 128 ||
        I > 16384 || I % 128 || experts < 1 || experts > 512 || top_k < 1 || top_k > 32)
        return FP8BS_ERR_INVALID_ARG;
    *bytes = fp8bs::moe_workspace(T, D, I, experts, top_k).total;
    return FP8BS_OK;
}

extern "C" int fp8bs_moe_experts(const void* x, const float* weights, const int32_t* ids, const void* w13,
                                 const float* s13, const void* w2, const float* s2, void* y, int64_t T,
                                 int64_t D, int64_t I, int64_t experts, int64_t top_k, int scale_fmt,
                                 void* workspace, size_t workspace_bytes, void* stream) {
    fp8bs::MoeWorkspace ws = {};
    const int rc = check_experts(x, w13, s13, w2, s2, y, T, D, I, experts, top_k, scale_fmt, workspace,
                                 workspace_bytes, &ws);
    if (rc != FP8BS_OK || T == 0) return rc;
    if (!weights || !ids) return FP8BS_ERR_INVALID_ARG;
    if (!aligned4(weights) || !aligned4(ids)) return FP8BS_ERR_MISALIGNED;
    int sms = 0;
    const int dev = check_device(&sms);
    if (dev != FP8BS_OK) return dev;
    uint8_t* base = static_cast<uint8_t*>(workspace);
    const cudaError_t e = fp8bs::launch_moe_prepare(
        x, nullptr, nullptr, nullptr, base + ws.x8, reinterpret_cast<float*>(base + ws.xs), T, D, experts,
        scale_fmt == FP8BS_SCALE_UE8M0, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return status_of(e);
    return run_experts(ws, weights, ids, w13, s13, w2, s2, y, T, D, I, experts, top_k, scale_fmt, workspace,
                       sms, stream);
}

extern "C" int fp8bs_moe_layer(const void* x, const fp8bs_moe_routing* routing, const void* w13,
                               const float* s13, const void* w2, const float* s2, void* y, int64_t T,
                               int64_t D, int64_t I, int64_t experts, int scale_fmt, void* workspace,
                               size_t workspace_bytes, void* stream) {
    int rc = check_routing(routing, D, experts);
    if (rc != FP8BS_OK) return rc;
    fp8bs::MoeWorkspace ws = {};
    rc = check_experts(x, w13, s13, w2, s2, y, T, D, I, experts, routing->top_k, scale_fmt, workspace,
                       workspace_bytes, &ws);
    if (rc != FP8BS_OK || T == 0) return rc;
    if (!routing->router_w) return FP8BS_ERR_INVALID_ARG;
    if (!aligned16(routing->router_w) || !aligned4(routing->bias)) return FP8BS_ERR_MISALIGNED;
    int sms = 0;
    const int dev = check_device(&sms);
    if (dev != FP8BS_OK) return dev;
    uint8_t* base = static_cast<uint8_t*>(workspace);
    float* weights = reinterpret_cast<float*>(base + ws.weights);
    int32_t* ids = reinterpret_cast<int32_t*>(base + ws.ids);
    const cudaError_t e = fp8bs::launch_moe_prepare(
        x, routing, weights, ids, base + ws.x8, reinterpret_cast<float*>(base + ws.xs), T, D, experts,
        scale_fmt == FP8BS_SCALE_UE8M0, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return status_of(e);
    return run_experts(ws, weights, ids, w13, s13, w2, s2, y, T, D, I, experts, routing->top_k, scale_fmt,
                       workspace, sms, stream);
}
