// rms_norm.cu -- the residual's addition, RMS norm and the codes of the next product in one pass (fp8bs_rms_norm).
//
// One CTA per token, whose row stays in registers: PER chunks of 8 channels a thread, a block of 128 channels in 16
// neighbouring lanes. The sum of squares is one reduction over the CTA, a block's amax one over 16 lanes. Bound by
// memory: x and the residual are read once, their sum, the codes and (where asked for) the bf16 norm written once.
//
// Measured: 8192 tokens of 7168 channels, residual and codes, 65 us for 413 MB (0.95 of a copy's rate), four chunks a
// thread; five tokens 5 us on the GPU (a launch, a load and two reductions; a call of four outputs 8 to 9.5), one chunk
// a thread (fewer rows than SMs).
#include "gemm_common.cuh"
#include "quant_math.cuh"

namespace fp8bs {

namespace {

template <int PER>
__global__ void __launch_bounds__(PER == 1 ? 1024 : 512) rms_norm_kernel(const __grid_constant__ fp8bs_rms_norm_args a) {
    __shared__ float s_sum[32];
    const int chunks = static_cast<int>(a.D) / 8;
    const int64_t t = blockIdx.x;
    grid_dependency_wait();
    grid_launch_dependents();
    const uint4* x = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.x) + t * a.x_stride);
    const uint4* r = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.residual) +
                                                    (a.residual ? t * a.residual_stride : 0));
    uint4 v[PER], w[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        v[i] = c < chunks ? x[c] : make_uint4(0, 0, 0, 0);
    }
    if (a.residual) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            if (c < chunks) w[i] = r[c];
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            if (c < chunks) {
                uint32_t* p = reinterpret_cast<uint32_t*>(&v[i]);
                const uint32_t* q = reinterpret_cast<const uint32_t*>(&w[i]);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    p[k] = pack_bf16x2(bf16_lo(p[k]) + bf16_lo(q[k]), bf16_hi(p[k]) + bf16_hi(q[k]));
                reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.residual_out) + t * a.D)[c] = v[i];
            }
        }
    }
    const uint4* weight = static_cast<const uint4*>(a.weight);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c < chunks) w[i] = __ldg(weight + c);
        const uint32_t* p = reinterpret_cast<const uint32_t*>(&v[i]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            sum = fmaf(bf16_lo(p[k]), bf16_lo(p[k]), sum);
            sum = fmaf(bf16_hi(p[k]), bf16_hi(p[k]), sum);
        }
    }
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
    if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5] = sum;
    __syncthreads();
    sum = 0.0f;
    const int warps = blockDim.x >> 5;
    for (int i = 0; i < warps; ++i) sum += s_sum[i];
    const float mean = sum / static_cast<float>(a.D) + a.eps;
    float inv = rsqrtf(mean);
    {
        // a step of Newton's method, to about half the last bit (codes have borders)
        const float better = fmaf(0.5f * inv, fmaf(-mean * inv, inv, 1.0f), inv);
        if (better == better) inv = better;                      // (a mean of 0 or infinity: the root stands)
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c - static_cast<int>(threadIdx.x & 31) >= chunks) break;        // (whole warps: the reduction below)
        const bool live = c < chunks;                            // (of 16 lanes at once)
        const uint32_t* p = reinterpret_cast<const uint32_t*>(&v[i]);
        const uint32_t* q = reinterpret_cast<const uint32_t*>(&w[i]);
        float n[8], amax = 0.0f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            n[2 * k] = live ? bf16_lo(p[k]) * inv * bf16_lo(q[k]) : 0.0f;
            n[2 * k + 1] = live ? bf16_hi(p[k]) * inv * bf16_hi(q[k]) : 0.0f;
        }
        if (a.norm_out && live)
            reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.norm_out) + t * a.D)[c] =
                make_uint4(pack_bf16x2(n[0], n[1]), pack_bf16x2(n[2], n[3]), pack_bf16x2(n[4], n[5]),
                           pack_bf16x2(n[6], n[7]));
        if (a.y) {
#pragma unroll
            for (int k = 0; k < 8; ++k) amax = fmaxf(amax, fabsf(n[k]));
#pragma unroll
            for (int m = 8; m > 0; m >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
            const float s = block_scale(amax, a.scale_fmt == FP8BS_SCALE_UE8M0);
            const float rs = __frcp_rn(s);
            uint32_t out[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint32_t lo = pack_e4m3x2(div_by_scale(n[4 * k], s, rs), div_by_scale(n[4 * k + 1], s, rs));
                const uint32_t hi = pack_e4m3x2(div_by_scale(n[4 * k + 2], s, rs), div_by_scale(n[4 * k + 3], s, rs));
                out[k] = lo | hi << 16;
            }
            if (live) {
                reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.y) + t * a.D)[c] = make_uint2(out[0], out[1]);
                if ((threadIdx.x & 15) == 0) a.s[t * (a.D / BK) + c / 16] = s;
            }
        }
    }
}

template <int PER>
cudaError_t launch_rms_norm(const fp8bs_rms_norm_args& a, cudaStream_t stream) {
    const int64_t threads = (a.D / 8 + PER - 1) / PER;
    return launch_pdl(rms_norm_kernel<PER>, static_cast<unsigned>(a.T), static_cast<unsigned>((threads + 31) / 32 * 32),
                      0, stream, a);
}

}  // namespace

cudaError_t launch_rms_norm(const fp8bs_rms_norm_args& a, int num_sms, cudaStream_t stream) {
    return a.D <= 8192 && a.T <= num_sms ? launch_rms_norm<1>(a, stream) : launch_rms_norm<4>(a, stream);
}

}  // namespace fp8bs
