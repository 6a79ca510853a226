// norm_rope_fp8.cu -- RMS norm of queries and keys per head, rotation by position and the write of keys and values
// into a paged cache of e4m3 codes with one power-of-two scale per page and head (fp8bs_qk_norm_rope_fp8).
//
// Bound by memory: queries 4 bytes an element, keys and values 3. Two kinds of CTAs in one launch. Queries: whole
// tokens, as in norm_rope.cu. Keys and values: the runs that begin in a window of tokens (a run: tokens of the call that
// go to one page, next to one another in rising slots), of one key head, a row to a group of LPR lanes; runs may end
// behind the window. The largest magnitudes of a run come together in shared memory, from them the page's new scale, by
// it the codes. No other CTA touches that page and head, and a maximum does not depend on the order of what it is of, so
// the same call gives the same bits. A page that grows keeps the larger of its scale and what the run asks for; where
// that is more than before, its codes are rounded again by the ratio, a power of two (exact but for codes that become
// subnormal).
//
// Measured: 8192 tokens of 32 + 8 + 8 heads of 128 channels 44 us for 185 MB and 4 of cosines and sines (0.63 of a
// copy's rate; the queries alone 25); 655 tokens of four sequences, 16 heads of 192 and 128, pages of 16 slots 10 us; 61
// sequences a token each 5 us, a launch, three loads that wait for one another and two barriers. What a CTA of keys and
// values waits for (slots, rows, positions and then cosines) bounds it, so it takes four rounds of rows with the next
// one's on its way: with a CTA per run and its rows read twice, the first case 62 us, the second 22, 200 sequences of 16
// heads 18 (now 7).
#include "norm_rows.cuh"

namespace fp8bs {

namespace {

constexpr int THREADS = 128;
constexpr int MAX_WINDOW = 64;       // tokens whose runs a CTA takes
constexpr int KEEP = 4;              // rounds of rows whose keys are kept
constexpr int FULL = 400;            // CTAs of keys and values that are enough to fill the device
constexpr int CHUNK = 512;           // tokens from which on a call is taken for one of chunks

// A run, in shared memory.
struct Run {
    int64_t page, off;       // page, slot of its first token there
    float by[2], ratio[2];   // of keys and values: 1 / the new scale; old / new scale where codes are to be rounded again
};

// A token's slot, and where it stands in its page. known: position and slot are not out of range (a negative slot is none);
// ok: a page's slot is given to it.
struct TokenSlot {
    int64_t slot, off;
    bool known, ok;
};

__device__ __forceinline__ TokenSlot token_slot(const fp8bs_qk_norm_rope_args& a, int64_t t) {
    TokenSlot s = {-1, 0, true, false};
    if (t >= 0 && t < a.T) {
        s.slot = a.slots[t];
        const int pos = a.positions[t];
        s.known = pos >= 0 && pos < a.max_positions && s.slot < a.cache.pages * a.cache.page_size;
        s.ok = s.known && s.slot >= 0;
        const int64_t size = a.cache.page_size;
        if (s.ok) s.off = (size & (size - 1)) == 0 ? s.slot & (size - 1) : s.slot % size;
    }
    return s;
}

// Whether a token continues the run of the one before it: a later slot of the same page.
__device__ __forceinline__ bool continues(const TokenSlot& before, const TokenSlot& s) {
    return before.ok && s.ok && before.slot < s.slot && before.slot >= s.slot - s.off;
}

// Codes of 8 values, by a scale's reciprocal (a power of two: the products are exact but for subnormals of binary32,
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

// MANY tokens: two warps per token of queries, whose stream is marked as not to be kept; else four.
template <int LPR, bool INTERLEAVED, bool MANY>
__global__ void __launch_bounds__(THREADS, 5) qk_norm_rope_fp8_kernel(
    const __grid_constant__ fp8bs_qk_norm_rope_args a, float* k_scale, float* v_scale, const int window,
    const unsigned windows) {
    constexpr int GROUPS = THREADS / LPR, WARPS = THREADS / 32;
    __shared__ unsigned s_starts[WARPS], s_more[WARPS], s_ok[WARPS];
    __shared__ Run s_run[MAX_WINDOW];
    __shared__ unsigned s_max[2][MAX_WINDOW];                // bits of numbers >= 0, which are in their order
    __shared__ int s_got[WARPS];
    __shared__ int s_off[THREADS];                           // slots in their pages, of the tokens that are looked at first
    __shared__ float4 s_keys[KEEP][4][THREADS];              // a thread's own
    const int tid = threadIdx.x;
    const int p = tid % LPR;
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
    auto load_weight = [&](const void* from) {
        if (!from || !rows.has) return zero16();
        const uint4* src = static_cast<const uint4*>(from);
        return Chunk16{__ldg(src + c0), __ldg(src + c1)};
    };
    // cosines and sines, 16 bytes at a time where the tables allow it (their rows are multiples of 32)
    const bool wide = ((reinterpret_cast<uintptr_t>(a.cos) | reinterpret_cast<uintptr_t>(a.sin)) & 15) == 0;
    auto load_turn = [&](int pos) {
        if (!wide) {
            rows.load_turn(a, pos, p, nr);
            return;
        }
        const int64_t at = static_cast<int64_t>(pos) * (a.rot_dim / 2);
        const float4* ct = reinterpret_cast<const float4*>(a.cos + at);
        const float4* st = reinterpret_cast<const float4*>(a.sin + at);
        const int i0 = INTERLEAVED ? p : 2 * p, i1 = INTERLEAVED ? p + nr / 2 : 2 * p + 1;
        const float4 x0 = __ldg(ct + i0), x1 = __ldg(ct + i1), y0 = __ldg(st + i0), y1 = __ldg(st + i1);
        rows.cs[0] = make_float2(x0.x, x0.y), rows.cs[1] = make_float2(x0.z, x0.w);
        rows.cs[2] = make_float2(x1.x, x1.y), rows.cs[3] = make_float2(x1.z, x1.w);
        rows.sn[0] = make_float2(y0.x, y0.y), rows.sn[1] = make_float2(y0.z, y0.w);
        rows.sn[2] = make_float2(y1.x, y1.y), rows.sn[3] = make_float2(y1.z, y1.w);
    };

    grid_dependency_wait();
    grid_launch_dependents();

    if (blockIdx.x >= windows * static_cast<unsigned>(hk)) {
        // ---- queries: two warps per token of many, whose stream is marked as not to be kept; else four
        constexpr int PER_TOKEN = MANY ? 64 : 128, BATCH = 2;
        constexpr int QGROUPS = PER_TOKEN / LPR;
        const int64_t t = static_cast<int64_t>(blockIdx.x - windows * static_cast<unsigned>(hk)) *
                              (THREADS / PER_TOKEN) + tid / PER_TOKEN;
        if (t >= a.T) return;
        const int grp = tid % PER_TOKEN / LPR;
        const int hq = static_cast<int>(a.q_heads);
        const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + t * a.q_token_stride;
        auto load_q = [&](int r) {
            if (r >= hq || !rows.has) return zero16();
            const uint4* src = reinterpret_cast<const uint4*>(q + r * a.q_head_stride);
            return MANY ? Chunk16{__ldcs(src + c0), __ldcs(src + c1)} : Chunk16{__ldg(src + c0), __ldg(src + c1)};
        };
        Chunk16 x[BATCH];
#pragma unroll
        for (int b = 0; b < BATCH; ++b) x[b] = load_q(b * QGROUPS + grp);
        const int pos = a.positions[t];
        const bool pos_ok = pos >= 0 && pos < a.max_positions;
        if ((!pos_ok || a.slots[t] >= a.cache.pages * a.cache.page_size) && tid % PER_TOKEN == 0)
            record_error(FP8BS_DEVERR_INDEX);
        rows.rotates = p < nr / 2 && pos_ok;
        if (rows.rotates) load_turn(pos);
        float2 w[8];
        unpack16(load_weight(a.q_weight), w);
        __nv_bfloat16* qo = static_cast<__nv_bfloat16*>(a.q_out) + t * hq * dk;
        for (int base = 0; base < hq; base += QGROUPS * BATCH) {
#pragma unroll
            for (int b = 0; b < BATCH; ++b) {
                if (base + b * QGROUPS >= hq) break;
                const int r = base + b * QGROUPS + grp;
                Chunk16 y = rows.row(x[b], w, a.q_weight != nullptr);
                if (!pos_ok) y = zero16();
                if (r < hq && rows.has) {
                    uint4* dst = reinterpret_cast<uint4*>(qo + static_cast<int64_t>(r) * dk);
                    if (MANY) {
                        __stcs(dst + c0, y.a);
                        __stcs(dst + c1, y.b);
                    } else {
                        dst[c0] = y.a;
                        dst[c1] = y.b;
                    }
                }
                x[b] = load_q(r + QGROUPS * BATCH);
            }
        }
        return;
    }

    // ---- the runs that begin among `window` tokens, of one key head
    const int grp = tid / LPR, warp = tid / 32, lane = tid % 32;
    const int head = static_cast<int>(blockIdx.x % static_cast<unsigned>(hk));
    const int64_t t0 = static_cast<int64_t>(blockIdx.x / static_cast<unsigned>(hk)) * window;
    // One token a thread, those of the window and of a page behind it, where its last run ends if not before.
    TokenSlot mine = {-1, 0, true, false};
    bool more = false;
    if (32 * warp < window + a.cache.page_size) {
        mine = token_slot(a, t0 + tid);
        TokenSlot before = {__shfl_up_sync(0xffffffffu, mine.slot, 1), 0, true,
                            __shfl_up_sync(0xffffffffu, mine.ok, 1) != 0};
        if (lane == 0) before = token_slot(a, t0 + tid - 1);
        more = continues(before, mine);
        s_off[tid] = static_cast<int>(mine.off);
    }
    const bool starts = tid < window && mine.ok && !more;
    // (where there are queries, theirs report it)
    if (a.q_heads == 0 && head == 0 && tid < window && !mine.known) record_error(FP8BS_DEVERR_INDEX);
    {
        const unsigned b0 = __ballot_sync(0xffffffffu, starts), b1 = __ballot_sync(0xffffffffu, more);
        const unsigned b2 = __ballot_sync(0xffffffffu, mine.ok);
        if (lane == 0) s_starts[warp] = b0, s_more[warp] = b1, s_ok[warp] = b2;
    }
    const Chunk16 weight = load_weight(a.k_weight);
    __syncthreads();
    int first = -1, runs = 0;                                // first token of a run, runs
#pragma unroll
    for (int i = MAX_WINDOW / 32 - 1; i >= 0; --i) {
        const unsigned b = i < WARPS ? s_starts[i] : 0u;
        if (b) first = 32 * i + __ffs(b) - 1;
        runs += __popc(b);
    }
    if (runs == 0) return;                                   // (uniform over the CTA)
    // tokens from e on that continue a run
    auto continuing = [&](int e) {
        const int from = e;
        while (e < THREADS) {
            const unsigned ends = ~s_more[e >> 5] >> (e & 31);
            if (ends) return e + __ffs(ends) - 1 - from;
            e = (e | 31) + 1;
        }
        return e - from;
    };
    int end = window + continuing(window);                   // behind the last row
    while (end >= THREADS) {                                 // (longer than what has been looked at)
        const bool on = continues(token_slot(a, t0 + end + tid - 1), token_slot(a, t0 + end + tid));
        const unsigned stop = ~__ballot_sync(0xffffffffu, on);
        __syncthreads();
        if (lane == 0) s_got[warp] = stop ? __ffs(stop) - 1 : 32;
        __syncthreads();
        int got = 0;
#pragma unroll
        for (int i = 0; i < WARPS; ++i)
            if (got == 32 * i) got += s_got[i];
        end += got;
        if (got < THREADS) break;
    }
    // the run of a token of the window, or of one behind it: that of the last start up to there
    auto run_of = [&](int e) {
        int run = -1;
#pragma unroll
        for (int i = 0; i < MAX_WINDOW / 32; ++i)
            if (i < WARPS && 32 * i <= e) run += __popc(s_starts[i] & (e - 32 * i >= 31 ? ~0u : (2u << (e - 32 * i)) - 1));
        return run;
    };
    float old_k = 0.0f, old_v = 0.0f;
    int run_mine = 0;
    if (starts) {
        run_mine = run_of(tid);
        Run& r = s_run[run_mine];
        r.page = mine.slot / a.cache.page_size;
        r.off = mine.off;
        s_max[0][run_mine] = s_max[1][run_mine] = 0u;
        old_k = k_scale[r.page * hk + head], old_v = v_scale[r.page * hk + head];
    }
    __syncthreads();

    const bool has_v = p < dv / 16;
    const __nv_bfloat16* from_k = static_cast<const __nv_bfloat16*>(a.k) + t0 * a.k_token_stride + head * a.k_head_stride;
    const __nv_bfloat16* from_v = static_cast<const __nv_bfloat16*>(a.v) + t0 * a.v_token_stride + head * a.v_head_stride;
    const int32_t* positions = a.positions + t0;
    // The rows, GROUPS at a time; of none of them e is -1.
    const int rounds = (end - first + GROUPS - 1) / GROUPS;
    auto row_of = [&](int i) {
        const int e = first + i * GROUPS + grp;
        return e < end && (e >= window || (s_ok[e >> 5] >> (e & 31) & 1u)) ? e : -1;
    };
    auto load_key = [&](int e) {
        if (e < 0 || !rows.has) return zero16();
        const uint4* src = reinterpret_cast<const uint4*>(from_k + e * a.k_token_stride);
        return Chunk16{__ldg(src + c0), __ldg(src + c1)};
    };
    auto load_value = [&](int e) {
        if (e < 0 || !has_v) return zero16();
        const uint4* src = reinterpret_cast<const uint4*>(from_v + e * a.v_token_stride);
        return Chunk16{__ldg(src + 2 * p), __ldg(src + 2 * p + 1)};
    };
    // Keys after norm and rotation. (Every lane calls it.)
    auto key_values = [&](int e, int pos, const Chunk16& x, float2* f) {
        rows.rotates = e >= 0 && p < nr / 2;
        if (rows.rotates) load_turn(pos);
        float2 w[8];
        unpack16(weight, w);
        rows.template values<true>(x, w, a.k_weight != nullptr, f);
    };
    // The largest magnitudes of a run, of a group's lanes: they go to those of the whole run where the group comes to
    // another one, and at the end.
    auto flush = [&](int run, float m, unsigned* to) {
#pragma unroll
        for (int i = LPR / 2; i > 0; i >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, i));
        if (run >= 0 && p == 0) atomicMax(&to[run], __float_as_uint(m));
    };
    auto largest = [](const float2* f, float m) {
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, fmaxf(fabsf(f[i].x), fabsf(f[i].y)));
        return m;
    };
    auto enter = [&](int e, int* run, float* most, const float2* f, unsigned* to) {
        const int now = e >= 0 ? run_of(e) : *run;
        if (__any_sync(0xffffffffu, now != *run)) {
            flush(*run, *most, to);
            *most = 0.0f;
            *run = now;
        }
        *most = largest(f, *most);
    };
    {
        int run = -1;
        float most = 0.0f;
#pragma unroll 1
        for (int i = 0; i < rounds; i += KEEP) {
            Chunk16 v[KEEP];
#pragma unroll
            for (int b = 0; b < KEEP; ++b) v[b] = load_value(i + b < rounds ? row_of(i + b) : -1);
#pragma unroll
            for (int b = 0; b < KEEP; ++b) {
                if (i + b >= rounds) break;
                float2 f[8];
                unpack16(v[b], f);
                enter(row_of(i + b), &run, &most, f, s_max[1]);
            }
        }
        flush(run, most, s_max[1]);
    }
    {
        // (the first rounds' keys are kept, what long runs have besides is computed again for its codes)
        int run = -1;
        float most = 0.0f;
        int e = row_of(0);
        Chunk16 x = load_key(e);
        int pos = e >= 0 ? positions[e] : 0;
#pragma unroll 1
        for (int i = 0; i < rounds; ++i) {
            const int e_next = i + 1 < rounds ? row_of(i + 1) : -1;
            const Chunk16 x_next = load_key(e_next);
            const int pos_next = e_next >= 0 ? positions[e_next] : 0;
            float2 f[8];
            key_values(e, pos, x, f);
            enter(e, &run, &most, f, s_max[0]);
            if (i < KEEP) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    s_keys[i][k][tid] = make_float4(f[2 * k].x, f[2 * k].y, f[2 * k + 1].x, f[2 * k + 1].y);
            }
            e = e_next, x = x_next, pos = pos_next;
        }
        flush(run, most, s_max[0]);
    }
    __syncthreads();
    bool grows = false;
    if (starts) {
        Run& r = s_run[run_mine];
        const float sk = grown_scale(old_k, page_scale(__uint_as_float(s_max[0][run_mine])), r.off);
        const float sv = grown_scale(old_v, page_scale(__uint_as_float(s_max[1][run_mine])), r.off);
        k_scale[r.page * hk + head] = sk;
        v_scale[r.page * hk + head] = sv;
        r.by[0] = 1.0f / sk, r.by[1] = 1.0f / sv;
        // (0: the codes that the page holds stay as they are)
        r.ratio[0] = r.off > 0 && old_k > 0.0f && old_k < sk ? old_k / sk : 0.0f;
        r.ratio[1] = r.off > 0 && old_v > 0.0f && old_v < sv ? old_v / sv : 0.0f;
        grows = r.ratio[0] != 0.0f || r.ratio[1] != 0.0f;
    }
    if (__syncthreads_or(grows)) {
        // Codes that pages hold already, by scales that have grown, before the runs' own: a warp takes a quarter of a page's
        // keys or values.
#pragma unroll 1
        for (int job = warp; job < 8 * runs; job += WARPS) {
            const Run& r = s_run[job >> 3];
            const int of = job >> 2 & 1;
            const float ratio = r.ratio[of];
            if (ratio == 0.0f) continue;
            uint8_t* codes = of == 0 ? static_cast<uint8_t*>(a.cache.k) + r.page * a.cache.k_page_stride + head * a.cache.k_head_stride
                                     : static_cast<uint8_t*>(a.cache.v) + r.page * a.cache.v_page_stride + head * a.cache.v_head_stride;
            const int64_t stride = of == 0 ? a.cache.k_slot_stride : a.cache.v_slot_stride;
            const int pieces = (of == 0 ? dk : dv) / 16;
            const int piece = lane % pieces, at_once = 32 / pieces;      // (d <= 256: 16 pieces at most)
            if (lane >= at_once * pieces) continue;
            const int64_t q0 = a.cache.page_size * (job & 3) / 4, q1 = a.cache.page_size * ((job & 3) + 1) / 4;
            for (int64_t o0 = q0 + lane / pieces; o0 < q1; o0 += 4 * at_once) {
                uint4* to[4];
                uint4 c[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int64_t o = o0 + i * at_once;
                    to[i] = o < q1 ? reinterpret_cast<uint4*>(codes + o * stride) + piece : nullptr;
                    if (o < q1) c[i] = *to[i];
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (to[i])
                        *to[i] = make_uint4(rescaled(c[i].x, ratio), rescaled(c[i].y, ratio), rescaled(c[i].z, ratio),
                                            rescaled(c[i].w, ratio));
            }
        }
        __syncthreads();
    }
#pragma unroll 1
    for (int i = 0; i < rounds; ++i) {
        const int e = row_of(i);
        const Chunk16 v = load_value(e);
        float2 f[8];
        if (i < KEEP) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float4 u = s_keys[i][k][tid];
                f[2 * k] = make_float2(u.x, u.y), f[2 * k + 1] = make_float2(u.z, u.w);
            }
        } else {
            key_values(e, e >= 0 ? positions[e] : 0, load_key(e), f);
        }
        if (e < 0) continue;
        const Run& r = s_run[run_of(e)];
        const int64_t slot = e < THREADS ? s_off[e] : a.slots[t0 + e] - r.page * a.cache.page_size;
        if (rows.has) {
            uint2* dst = reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.cache.k) + r.page * a.cache.k_page_stride +
                                                  slot * a.cache.k_slot_stride + head * a.cache.k_head_stride);
            dst[c0] = codes8(f, r.by[0]);
            dst[c1] = codes8(f + 4, r.by[0]);
        }
        if (has_v) {
            unpack16(v, f);
            const uint2 lo = codes8(f, r.by[1]), hi = codes8(f + 4, r.by[1]);
            reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.cache.v) + r.page * a.cache.v_page_stride +
                                     slot * a.cache.v_slot_stride + head * a.cache.v_head_stride)[p] =
                make_uint4(lo.x, lo.y, hi.x, hi.y);
        }
    }
}

template <int LPR, bool MANY>
cudaError_t launch_fp8(const fp8bs_qk_norm_rope_args& a, float* k_scale, float* v_scale, cudaStream_t stream) {
    // tokens per CTA of keys and values: as many as it has groups, unless the CTAs would be too few to fill the device
    int window = KEEP * THREADS / LPR;
    if (window > MAX_WINDOW) window = MAX_WINDOW;
    while (window > 1 && a.T * a.cache.heads < int64_t{FULL} * window) window /= 2;
    const unsigned windows = static_cast<unsigned>((a.T + window - 1) / window);
    const int64_t per_cta = MANY ? 2 : 1;
    const unsigned grid = windows * static_cast<unsigned>(a.cache.heads) +
                          (a.q_heads > 0 ? static_cast<unsigned>((a.T + per_cta - 1) / per_cta) : 0u);
    auto kernel = a.interleaved ? qk_norm_rope_fp8_kernel<LPR, true, MANY> : qk_norm_rope_fp8_kernel<LPR, false, MANY>;
    return launch_pdl(kernel, grid, THREADS, 0, stream, a, k_scale, v_scale, window, windows);
}

template <int LPR>
cudaError_t launch_fp8(const fp8bs_qk_norm_rope_args& a, float* k_scale, float* v_scale, cudaStream_t stream) {
    return a.T >= CHUNK ? launch_fp8<LPR, true>(a, k_scale, v_scale, stream)
                        : launch_fp8<LPR, false>(a, k_scale, v_scale, stream);
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
