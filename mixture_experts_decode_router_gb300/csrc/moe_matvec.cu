// moe_matvec.cu -- products of 4-bit group-scaled matrices with a few vectors
// (sm_103a): out[t, o] = sum_i W[o, i] x[t, i] (+ bias[o]) (+ out[t, o]).
//
// Bound by the weight stream.  Blocks of 8 warps; a warp multiplies 16 rows
// (q4_mma.cuh) and kw warps share a tile of rows, each with every kw-th stage of
// K, their sums added in warp order through shared memory.  Blocks are
// persistent over the row tiles, the warps' copies running ahead across tiles.
#include <algorithm>
#include <mutex>

#include "moe_launch.cuh"
#include "q4_mma.cuh"

namespace moe {

namespace {

constexpr int kWarps = 8;
constexpr int kStages = 6;            // ring of each warp (5 stages in flight)
constexpr int kMaxSmem = 227 * 1024;

__device__ __forceinline__ void store_out(const MatvecParams& p, int64_t t, int o, float v) {
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

// XB: x is bf16 (else f16).  INT4 multiplies in x's type.  NVFP4 multiplies in f16:
// bf16 rows are scaled by a power of two that puts their largest value below 2^15
// (exact for elements down to 2^-32 of it) and the results scaled back.
template <int GSH, bool XB, int NT>
__global__ void __launch_bounds__(32 * kWarps) matvec_kernel(const MatvecParams p, int kw, int tp) {
    constexpr bool BF = XB && GSH != 4;
    extern __shared__ __align__(128) uint8_t dyn[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int K = p.w.in_dim, O = p.w.out_dim, row_bytes = K / 2;
    const int mw = kWarps / kw, mrow = warp / kw, kk = warp % kw;
    const int nst = (K + q4::kStageK - 1) / q4::kStageK;
    const int n_tiles = (O + 15) / 16, step = gridDim.x * mw;
    const int64_t t0 = (int64_t)blockIdx.y * tp;
    const int ntok = (int)min((int64_t)tp, (int64_t)p.n - t0);
    uint8_t* ring = dyn + (size_t)warp * kStages * q4::kStageBytes;
    float* red = reinterpret_cast<float*>(dyn + (size_t)kWarps * kStages * q4::kStageBytes);   // [warp][NT][32][4]
    float* xsc = red + kWarps * NT * 128;                                                      // [16]
    uint8_t* sx = reinterpret_cast<uint8_t*>(xsc + 16);
    const int xstride = q4::x_row_bytes(K);
    pdl_wait();

    // The copies run kStages - 1 stages ahead of the products, across tiles.
    int i_tile = blockIdx.x * mw + mrow, i_s = kk, i_slot = 0;
    auto issue = [&]() {
        if (i_s < nst && i_tile < n_tiles) {
            q4::load_stage(q4::smem_addr(ring + i_slot * q4::kStageBytes), p.w.w, i_tile * 16, O, row_bytes, i_s, lane);
            i_s += kw;
            if (i_s >= nst) { i_s = kk; i_tile += step; }
        }
        q4::cp_commit();
        i_slot = i_slot + 1 == kStages ? 0 : i_slot + 1;
    };
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) issue();

    // x in fragment order, zero past K.
    const int chunks = (xstride - 64) / 16;
    for (int b = (GSH == 4 && XB) ? warp : 0; b < ntok; b += (GSH == 4 && XB) ? kWarps : 1) {
        const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p.x) + (size_t)(t0 + b) * p.x_stride);
        uint4* dst = reinterpret_cast<uint4*>(sx + (size_t)b * xstride);
        if constexpr (GSH == 4 && XB) {
            float am = 0.f;
            for (int c = lane; c < K / 8; c += 32) {
                float v[8];
                bf16x8_to_float(src[c], v);
#pragma unroll
                for (int i = 0; i < 8; ++i) am = fmaxf(am, fabsf(v[i]));
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
            const int sh = q4::f16_shift(am);
            const float f = q4::exp2i(sh);
            if (lane == 0) xsc[b] = q4::exp2i(-sh);
            for (int c = lane; c < chunks; c += 32) {
                float v[8] = {};
                if (c < K / 8) bf16x8_to_float(src[c], v);
                uint32_t h[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const __half2 hv = __floats2half2_rn(v[2 * i] * f, v[2 * i + 1] * f);
                    h[i] = *reinterpret_cast<const uint32_t*>(&hv);
                }
                dst[c] = q4::chunk_order<GSH>(make_uint4(h[0], h[1], h[2], h[3]));
            }
        } else {
            for (int c = threadIdx.x; c < chunks; c += 32 * kWarps)
                dst[c] = q4::chunk_order<GSH>(c < K / 8 ? src[c] : make_uint4(0u, 0u, 0u, 0u));
            if (threadIdx.x == 0) xsc[b] = 1.f;
        }
    }
    __syncthreads();

    const int g = lane >> 2, t = lane & 3;
    const float ms = GSH == 4 ? __ldg(p.w.scale2) : 1.f;
    int slot = 0;
    for (int base = blockIdx.x * mw; base < n_tiles; base += step) {
        const int tile = base + mrow, row0 = tile * 16;
        const bool live = tile < n_tiles;
        float acc[NT][4];
#pragma unroll
        for (int q = 0; q < NT; ++q)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[q][i] = 0.f;
        if (live && kk < nst) {
            q4::StageScales<GSH> sc, next;
            next.load(p.w, 0, row0, O, kk, lane);
            for (int s = kk; s < nst; s += kw) {
                sc = next;
                if (s + kw < nst) next.load(p.w, 0, row0, O, s + kw, lane);
                q4::cp_wait<kStages - 2>();
                __syncwarp();
                issue();
                q4::mma_stage<GSH, BF, NT>(ring + slot * q4::kStageBytes, sx + (size_t)g * xstride + s * 512 + t * 16,
                                           xstride, ntok, sc, acc, lane);
                slot = slot + 1 == kStages ? 0 : slot + 1;
            }
        }
        if (kw > 1) {
            float4* mine = reinterpret_cast<float4*>(red) + (size_t)warp * NT * 32;
#pragma unroll
            for (int q = 0; q < NT; ++q) mine[q * 32 + lane] = make_float4(acc[q][0], acc[q][1], acc[q][2], acc[q][3]);
            __syncthreads();
            if (kk == 0) {
                for (int o = 1; o < kw; ++o)
#pragma unroll
                    for (int q = 0; q < NT; ++q) {
                        const float4 v = mine[(o * NT + q) * 32 + lane];
                        acc[q][0] += v.x; acc[q][1] += v.y; acc[q][2] += v.z; acc[q][3] += v.w;
                    }
            }
            if (base + step < n_tiles) __syncthreads();
        }
        if (live && kk == 0) {
#pragma unroll
            for (int q = 0; q < NT; ++q)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = row0 + g + 8 * (i >> 1), b = 8 * q + 2 * t + (i & 1);
                    if (row < O && b < ntok) store_out(p, t0 + b, row, acc[q][i] * (ms * xsc[b]));
                }
        }
    }
    pdl_trigger();
}

template <int GSH, bool XB, int NT>
cudaError_t launch_nt(const MatvecParams& p, int tp, int num_sms, cudaStream_t st) {
    const int K = p.w.in_dim, n_tiles = (p.w.out_dim + 15) / 16, nst = (K + q4::kStageK - 1) / q4::kStageK;
    // Warps that share a tile: as many as give every SM a block.
    int kw = 1;
    while (kw < kWarps && kw < nst && (int64_t)n_tiles * kw < (int64_t)num_sms * kWarps) kw *= 2;
    const size_t smem = (size_t)kWarps * kStages * q4::kStageBytes + (size_t)kWarps * NT * 512 + 64 +
                        (size_t)std::min<int64_t>(tp, p.n) * q4::x_row_bytes(K);
    auto kern = matvec_kernel<GSH, XB, NT>;
    static std::mutex mu;
    static bool configured[128] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) return cudaErrorInvalidDevice;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!configured[dev]) {
            const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
            if (e != cudaSuccess) return e;
            configured[dev] = true;
        }
    }
    const int per_sm = 2 * smem <= (size_t)kMaxSmem ? 2 : 1;
    const int mw = kWarps / kw;
    const int gx = std::min((n_tiles + mw - 1) / mw, num_sms * per_sm);
    launch_pdl(kern, dim3(gx, (unsigned)((p.n + tp - 1) / tp)), 32 * kWarps, smem, st, p, kw, tp);
    return cudaGetLastError();
}

template <int GSH, bool XB>
cudaError_t launch_fmt(const MatvecParams& p, int num_sms, cudaStream_t st) {
    // Tokens of a block: up to 16, as many as fit beside the rings.
    const size_t room = kMaxSmem - (size_t)kWarps * (kStages * q4::kStageBytes + 2 * 512) - 64;
    const int tp = std::min<size_t>(16, room / q4::x_row_bytes(p.w.in_dim));
    if (tp < 1) return cudaErrorInvalidValue;   // (the caller checked matvec_fits)
    const int tokens = std::min(tp, p.n);
    return tokens > 8 ? launch_nt<GSH, XB, 2>(p, tp, num_sms, st) : launch_nt<GSH, XB, 1>(p, std::min(tp, 8), num_sms, st);
}

template <int GSH>
cudaError_t launch_x(int x_type, const MatvecParams& p, int num_sms, cudaStream_t st) {
    return x_type == MOE_BF16 ? launch_fmt<GSH, true>(p, num_sms, st) : launch_fmt<GSH, false>(p, num_sms, st);
}

}  // namespace

bool matvec_fits(int K) {
    return q4::x_row_bytes(K) <= kMaxSmem - kWarps * (kStages * q4::kStageBytes + 2 * 512) - 64;
}

cudaError_t launch_matvec(int fmt, int x_type, const MatvecParams& p, int num_sms, cudaStream_t st) {
    switch (fmt) {
        case MOE_W_NVFP4: return launch_x<4>(x_type, p, num_sms, st);
        case MOE_W_INT4_G32: return launch_x<5>(x_type, p, num_sms, st);
        case MOE_W_INT4_G64: return launch_x<6>(x_type, p, num_sms, st);
        case MOE_W_INT4_G128: return launch_x<7>(x_type, p, num_sms, st);
    }
    return cudaErrorInvalidValue;
}

}  // namespace moe
