// moe_matvec.cu -- products of 4-bit group-scaled matrices with a few vectors
// (sm_103a): out[t, o] = sum_i W[o, i] x[t, i] (+ bias[o]) (+ out[t, o]).
#include <cuda_fp16.h>

#include "moe_launch.cuh"

namespace moe {

namespace {

template <int XT>
__device__ __forceinline__ void x8_to_float(uint4 r, float (&v)[8]) {
    if constexpr (XT == MOE_BF16) {
        bf16x8_to_float(r, v);
    } else {
        const uint32_t w4[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w4[i]));
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
}

__device__ __forceinline__ void store_out(const MatvecParams& p, int t, int o, float v) {
    const size_t at = (size_t)t * p.out_stride + o;
    if (p.bias) v += __ldg(p.bias + o);
    if (p.out_type == MOE_F32) {
        float* d = reinterpret_cast<float*>(p.out) + at;
        *d = p.accumulate ? *d + v : v;
    } else if (p.out_type == MOE_BF16) {
        __nv_bfloat16* d = reinterpret_cast<__nv_bfloat16*>(p.out) + at;
        *d = __float2bfloat16_rn(p.accumulate ? __bfloat162float(*d) + v : v);
    } else {
        __half* d = reinterpret_cast<__half*>(p.out) + at;
        *d = __float2half_rn(p.accumulate ? __half2float(*d) + v : v);
    }
}

// One warp per output row and TB rows of x: lane l takes the 8-element chunks
// l, l + 32, ... in order, then the butterfly.
template <int FMT, int XT, int TB>
__global__ void __launch_bounds__(256) matvec_kernel(const MatvecParams p) {
    const int lane = threadIdx.x & 31;
    const int64_t o = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int t0 = blockIdx.y * TB;
    pdl_wait();
    if (o < p.w.out_dim) {
        float acc[TB] = {};
        for (int c = lane; c < p.w.in_dim / 8; c += 32) {
            WChunk<FMT> ch;
            ch.load(p.w, 0, (int)o, c);
            const float cs = ch.scale(p.w, 0, (int)o, c);
            float wv[8];
            ch.decode(wv);
#pragma unroll
            for (int b = 0; b < TB; ++b) {
                const uint16_t* xr = reinterpret_cast<const uint16_t*>(p.x) + (size_t)min(t0 + b, p.n - 1) * p.x_stride;
                float xv[8];
                x8_to_float<XT>(__ldg(reinterpret_cast<const uint4*>(xr) + c), xv);
                acc[b] = fmaf(dot8(wv, xv), cs, acc[b]);
            }
        }
        const float ms = matrix_scale<FMT>(p.w, 0);
#pragma unroll
        for (int b = 0; b < TB; ++b) {
            const float v = warp_sum(acc[b]) * ms;
            if (lane == 0 && t0 + b < p.n) store_out(p, t0 + b, (int)o, v);
        }
    }
    pdl_trigger();
}

template <int FMT, int XT>
void launch_fmt(const MatvecParams& p, cudaStream_t st) {
    const int gx = (p.w.out_dim + 7) / 8;
    if (p.n == 1) launch_pdl(matvec_kernel<FMT, XT, 1>, dim3(gx, 1), 256, 0, st, p);
    else launch_pdl(matvec_kernel<FMT, XT, 4>, dim3(gx, (p.n + 3) / 4), 256, 0, st, p);
}

}  // namespace

cudaError_t launch_matvec(int fmt, int x_type, const MatvecParams& p, int num_sms, cudaStream_t st) {
    if (fmt == MOE_W_NVFP4) {
        if (x_type == MOE_BF16) launch_fmt<MOE_W_NVFP4, MOE_BF16>(p, st);
        else launch_fmt<MOE_W_NVFP4, MOE_F16>(p, st);
    } else {
        if (x_type == MOE_BF16) launch_fmt<kFmtInt4, MOE_BF16>(p, st);
        else launch_fmt<kFmtInt4, MOE_F16>(p, st);
    }
    return cudaGetLastError();
}

}  // namespace moe
