// attention.cu -- attention of new tokens over a paged cache (fp8bs_paged_attention).
//
// The query rows of one sequence that share a key head (token i, head g of the group: row i*G + g)
// are packed into tiles of 128, one MMA row and TMEM lane each, so that a single token of a grouped
// head still reads its keys once and a chunk fills the tensor core. Per key tile of BN keys:
//   S = Q K^T      tcgen05.mma, bf16, Q and K K-major in shared memory, S fp32 in TMEM
//   P = exp2(c S - m), m the running row maximum: one thread per row, S from TMEM, P as bf16 back
//                  into TMEM in place of S
//   O += P V       tcgen05.mma, P from TMEM, V from shared memory as the cache holds it (keys
//                  outermost: an MN-major operand), O fp32 in TMEM
// The maximum only moves when it has grown by more than 2^8 (kRescale): the tile's probabilities are then
// computed again and O is scaled in TMEM by its softmax warps; otherwise P is that much larger than 1 at most,
// which bf16 and fp32 hold without loss, and O is left alone. So no row waits for its maximum. The row sum is
// taken from P before its rounding to bf16, so lse is exact to binary32; the rounding of P (2^-9 on average per
// term) is of the size of the output's own.
// A row without keys is one whose sum is zero. A score that is not a number, or +infinite, makes the sum NaN (the
// maximum passes over NaN), and with it the row, in one piece or in many.
//
// Two forms (AttnCfg): NQ = 2 query tiles per CTA for chunks, whose softmax warps work on one tile
// while the tensor core works on the other; NQ = 1 with two S buffers for few rows.
//
// Chunks are bound by the tensor core and what feeds it: 4096 new tokens over 8192 keys, 32 query and 8 key heads
// of 128 channels, 412 GFLOP that count, take 282 us = 1.46 PFLOP/s (0.75 of a library product's rate; 298 us where the
// inputs come from HBM in every call). The tensor pipe is busy for 61 % of an SM's cycles and waits for the softmax the rest: a row of S is 128 exponentials, and
// the products with K, whose operands both come from shared memory, run at 80 instead of 64 cycles. Heads of 192 + 128
// channels take tiles of 96 keys (128 would leave room for one tile of values: 59 us instead of 56 for 2 chunks of
// 777 over 2500 keys, 16 heads).
// Decoding is bound by HBM: 64 ragged sequences of up to 8192 keys, 64 query and 8 key heads, 1.1 GB of keys and
// values, take 193 us = 5.7 TB/s (0.86 of a copy's rate); one sequence of 32785 keys takes 32 us for 134 MB, of
// which launch, first keys and join are 12.
//
// Keys and values come through TMA in boxes of as many slots as divide both the page and the tile, all
// channels of a box at once where the cache's strides allow it.
// Few rows and long keys: the key axis is cut into pieces (AttentionPlan), each CTA leaves its
// unnormalised O, maximum and sum, and a second kernel joins them in key order.
#include "attention_tiles.cuh"

namespace fp8bs {

namespace {

// Whether the two-tile form is used: where the average sequence has more rows than one tile holds. (32 sequences of
// 2048 keys, 8 heads of 128 channels, one tile and two: 128 rows 62 and 76 us, 160 rows 122 and 80, 512 rows 268 and
// 148; heads of 64 35 and 54, 82 and 61; of 192 75 and 94, 148 and 96. 4 sequences of 8192 keys, 4 heads: 128 rows 25
// and 33, 160 to 256 rows even.)
bool two_tiles(const fp8bs_paged_attention_args& a) {
    const int64_t group = a.q_heads / a.cache.heads;
    return a.T * group > 128 * a.B;
}

AttnParts attention_parts(const fp8bs_paged_attention_args& a, const AttentionPlan& plan) {
    AttnParts p = {};
    p.rows = a.T * a.q_heads;
    if (plan.pieces > 1) {
        p.o = static_cast<float*>(a.workspace);
        p.ml = reinterpret_cast<float2*>(p.o + plan.pieces * p.rows * a.cache.dv);
    }
    return p;
}

template <class Cfg>
cudaError_t launch_attention(const CUtensorMap& tmK, const CUtensorMap& tmV,
                             const fp8bs_paged_attention_args& a, const AttentionModes& modes,
                             const AttentionPlan& plan, int num_sms, cudaStream_t stream) {
    auto kernel = paged_attention_kernel<Cfg>;
    cudaError_t e = set_smem(kernel, Cfg::SMEM);
    if (e != cudaSuccess) return e;
    const AttnParts parts = attention_parts(a, plan);
    const int64_t items = tile_bound(a, Cfg::ROWS) * a.cache.heads * plan.pieces;
    if (items >= INT32_MAX) return cudaErrorInvalidValue;
    const int64_t resident = static_cast<int64_t>(num_sms) * Cfg::CTAS;
    const unsigned grid = static_cast<unsigned>(items < resident ? items : resident);
    e = launch_pdl(kernel, grid, Cfg::THREADS, Cfg::SMEM, stream, tmK, tmV, a, modes, plan.piece_len,
                   plan.pieces, parts, Scales{}, 0);
    if (e != cudaSuccess || plan.pieces == 1) return e;
    // Many pieces of few rows: four warps a row; else a warp each (more blocks than the GPU holds at once would
    // keep the next kernel from starting: 4096 rows of 8 pieces took 30 us with four warps each, none to be seen
    // with one).
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out);
    if (parts.rows <= 1024)
        return launch_pdl(attention_join_kernel<Cfg::DV, 4>, static_cast<unsigned>(parts.rows), 128, 0, stream,
                          parts, plan.pieces, out, a.lse);
    return launch_pdl(attention_join_kernel<Cfg::DV, 1>, static_cast<unsigned>((parts.rows + 3) / 4), 128, 0,
                      stream, parts, plan.pieces, out, a.lse);
}

}  // namespace

AttentionPlan attention_plan(const fp8bs_paged_attention_args& a, int num_sms) {
    return attention_plan(a, num_sms, two_tiles(a));
}

AttentionPlan attention_plan(const fp8bs_paged_attention_args& a, int num_sms, bool two) {
    const int64_t rows = two ? 256 : 128;
    const int64_t group = a.q_heads / a.cache.heads;
    // (sequences of one length, as in decoding, are counted exactly)
    const int64_t items = a.cache.heads * (a.T == a.B * a.max_q_len ? a.B * ((a.max_q_len * group + rows - 1) / rows)
                                                                    : tile_bound(a, rows));
    int64_t keys = key_span(a, rows, a.max_q_len, a.max_kv_len);
    if (keys < 1) keys = 1;
    const int64_t unit = two && a.cache.dk > 128 ? 192 : 128;       // whole key tiles
    int64_t len = keys;
    if (two) {
        // chunks that do not fill the GPU: the number of pieces with the lowest time, in keys, of the busiest
        // CTA, where a piece costs as much as 512 keys more (queries, output, its part of the join)
        int64_t best = keys;
        for (int64_t p = 2; items < num_sms && p <= 16 && keys / p >= 256; ++p) {
            const int64_t l = ((keys + p - 1) / p + unit - 1) / unit * unit;
            const int64_t time = (items * p + num_sms - 1) / num_sms * (l + 512);
            if (time < best) {
                best = time;
                len = l;
            }
        }
    } else if (items * keys < int64_t{4096} * num_sms) {
        // few rows and keys: as above, where a piece costs as much as 128 keys more, and joining p of them as much as
        // 128 + 32 p. (Cutting by one CTA's share of all keys instead, in 128 keys or more: 43.8 us instead of 30.3
        // for 14 sequences of 3183 keys, 57 instead of 43 for 5 of 9411, and around 12 instead of 9 where
        // sequences of 100 to 300 keys need no second kernel.)
        int64_t best = 0;
        for (int64_t p = 1; p <= 64 && (p == 1 || keys / p >= 64); ++p) {
            const int64_t step = p == 1 ? 64 : 128;
            const int64_t l = ((keys + p - 1) / p + step - 1) / step * step;
            const int64_t time = (items * p + num_sms - 1) / num_sms * (l + 128) + (p > 1 ? 128 + 32 * p : 0);
            if (p == 1 || time < best) {
                best = time;
                len = l;
            }
        }
    } else if (items < 8 * num_sms) {
        // many shares' worth of keys: pieces of 1024 at most, so that the longest sequence of a ragged batch does
        // not finish last on its own
        len = 1024;
    }
    // The bounds may be far above the sequences (a page table's whole width): no more pieces than kMaxPartBytes hold.
    const int64_t most = std::max<int64_t>(1, kMaxPartBytes / std::max<int64_t>(1, part_bytes(a)));
    if (len * most < keys) len = (keys + most - 1) / most;
    len = std::min<int64_t>((len + unit - 1) / unit * unit, int64_t{1} << 30);
    AttentionPlan p;
    p.piece_len = static_cast<int>(len);
    p.pieces = static_cast<int>((keys + len - 1) / len);
    return p;
}

size_t attention_workspace(const fp8bs_paged_attention_args& a, const AttentionPlan& plan) {
    if (plan.pieces == 1) return 0;
    return static_cast<size_t>(plan.pieces) * static_cast<size_t>(part_bytes(a));
}

cudaError_t launch_paged_attention(const CUtensorMap& tmK, const CUtensorMap& tmV,
                                   const fp8bs_paged_attention_args& a, const AttentionModes& modes,
                                   const AttentionPlan& plan, int num_sms, cudaStream_t stream) {
    const bool two = two_tiles(a);
    switch (a.cache.dk) {
        case 64:
            return two ? launch_attention<AttnCfg<64, 64, 2>>(tmK, tmV, a, modes, plan, num_sms, stream)
                       : launch_attention<AttnCfg<64, 64, 1>>(tmK, tmV, a, modes, plan, num_sms, stream);
        case 128:
            return two ? launch_attention<AttnCfg<128, 128, 2>>(tmK, tmV, a, modes, plan, num_sms, stream)
                       : launch_attention<AttnCfg<128, 128, 1>>(tmK, tmV, a, modes, plan, num_sms, stream);
        default:
            return two ? launch_attention<AttnCfg<192, 128, 2>>(tmK, tmV, a, modes, plan, num_sms, stream)
                       : launch_attention<AttnCfg<192, 128, 1>>(tmK, tmV, a, modes, plan, num_sms, stream);
    }
}

namespace {

// How a cache's rows of `d` channels can be fetched (AttentionModes).
int fetch_mode(const fp8bs_kv_cache& c, int64_t d, int64_t head_stride, int64_t page_stride) {
    if (c.page_size % 8 != 0) return 2;
    if (c.heads == 1 || head_stride == d) return 0;
    if (c.pages == 1 || page_stride == c.heads * head_stride)
        return c.pages * c.heads < (int64_t{1} << 31) ? 1 : 2;
    return 2;
}

}  // namespace

AttentionModes attention_modes(const fp8bs_kv_cache& c) {
    AttentionModes m;
    m.k = fetch_mode(c, c.dk, c.k_head_stride, c.k_page_stride);
    m.v = fetch_mode(c, c.dv, c.v_head_stride, c.v_page_stride);
    // slots per box: the largest power of two that divides the page and the key tiles (64 and 128, or 64 and 96)
    const int most = m.k == 2 || m.v == 2 ? 3 : c.dk > 128 ? 5 : 6;
    m.box_log2 = 0;
    while (m.box_log2 < most && c.page_size % (int64_t{2} << m.box_log2) == 0) ++m.box_log2;
    return m;
}

cudaError_t read_error_attention(unsigned int* out, bool clear, cudaStream_t stream) {
    return read_tu_error(out, clear, stream);
}

}  // namespace fp8bs
