// moe_norm.cu -- residual addition and RMSNorm of rows, with an output of 16 or 32 bits, one
// of 8 bits with scales, or both (sm_103a):
//   h = x + residual, rounded to the residual's type (what residual_out holds; x without one)
//   y = h / sqrt(mean(h^2) + eps) * (weight + weight_offset)
//   out = y;  out8 = E4M3(y / s),  s = max(max |y| / 448, 2^-126) over 128 elements or the row
//
// Bound by HBM for many rows, by launch and latency for few: every element is read once,
// waits in registers (fp32) for the row's sum of squares, and is written once.  A row
// belongs to T threads of a block, each with kCh chunks of eight consecutive elements, T apart
// in chunks, all of whose loads are in flight before the first is used; rows of at most 32
// chunks a thread's kCh are one warp's, several of them to a block and no barrier.
//
// The scale of 128 elements is a maximum over 16 neighbouring lanes (a chunk is 8 elements);
// the row's, a second reduction over its threads.
#include <algorithm>

#include "moe_launch.cuh"

namespace moe {

namespace {

constexpr int kMaxThreads = 512;    // of a row
constexpr int kMaxCh = 8;           // chunks of a thread at most

// Eight consecutive elements of a row as they lie in memory.
template <int kType> struct Raw8 { uint4 v[kType == MOE_F32 ? 2 : 1]; };

__device__ __forceinline__ uint4 ld_once_v4(const void* p) {
    uint4 r;   // (not ld.global.nc: a row may be overwritten in place by the thread that read it)
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
    return r;
}

// kVec: 16-byte loads (the row is 16-byte aligned, `left` >= 8); else element by element,
// the first `left` of them, zero behind.
template <int kType, bool kVec> __device__ __forceinline__ void load8(Raw8<kType>& r, const void* row, int at, int left) {
    if constexpr (kVec) {
        const uint4* p = reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(row) + (size_t)at * (kType == MOE_F32 ? 4 : 2));
#pragma unroll
        for (int i = 0; i < (kType == MOE_F32 ? 2 : 1); ++i) r.v[i] = ld_once_v4(p + i);
    } else if constexpr (kType == MOE_F32) {
        const uint32_t* p = reinterpret_cast<const uint32_t*>(row) + at;
        uint32_t* o = reinterpret_cast<uint32_t*>(r.v);
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = i < left ? p[i] : 0u;
    } else {
        const uint16_t* p = reinterpret_cast<const uint16_t*>(row) + at;
        uint32_t* o = reinterpret_cast<uint32_t*>(r.v);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = 2 * i < left ? p[2 * i] : 0u, hi = 2 * i + 1 < left ? p[2 * i + 1] : 0u;
            o[i] = lo | (hi << 16);
        }
    }
}

template <int kType> __device__ __forceinline__ void floats8(const Raw8<kType>& r, float (&f)[8]) {
    const uint32_t* u = reinterpret_cast<const uint32_t*>(r.v);
    if constexpr (kType == MOE_F32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(u[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (kType == MOE_BF16) {
                f[2 * i] = bf16_lo(u[i]);
                f[2 * i + 1] = bf16_hi(u[i]);
            } else {
                const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
                f[2 * i] = v.x;
                f[2 * i + 1] = v.y;
            }
        }
    }
}

// Two floats as a pair of kType (16 bits each), rounded to nearest even.
template <int kType> __device__ __forceinline__ uint32_t pack2(float a, float b) {
    if constexpr (kType == MOE_BF16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&v);
    } else {
        const __half2 v = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
}

template <int kType, bool kVec> __device__ __forceinline__ void store8(void* row, int at, int left, const float (&f)[8]) {
    Raw8<kType> r;
    uint32_t* u = reinterpret_cast<uint32_t*>(r.v);
    if constexpr (kType == MOE_F32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = __float_as_uint(f[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = pack2<kType>(f[2 * i], f[2 * i + 1]);
    }
    if constexpr (kVec) {
        uint4* p = reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(row) + (size_t)at * (kType == MOE_F32 ? 4 : 2));
#pragma unroll
        for (int i = 0; i < (kType == MOE_F32 ? 2 : 1); ++i) p[i] = r.v[i];
    } else if constexpr (kType == MOE_F32) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left) reinterpret_cast<uint32_t*>(row)[at + i] = u[i];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left) reinterpret_cast<uint16_t*>(row)[at + i] = (uint16_t)(u[i >> 1] >> (16 * (i & 1)));
    }
}

template <bool kVec> __device__ __forceinline__ void store8_as(int type, void* row, int at, int left, const float (&f)[8]) {
    if (type == MOE_F32) store8<MOE_F32, kVec>(row, at, left, f);
    else if (type == MOE_BF16) store8<MOE_BF16, kVec>(row, at, left, f);
    else store8<MOE_F16, kVec>(row, at, left, f);
}

// E4M3 of a (low byte) and b, to nearest even; NaN is NaN.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}

// Sum and maximum over the T threads of a row (threadIdx.x), the same value in each.  One
// warp's by shuffles; else by warp through red[32], added in warp order.
__device__ __forceinline__ float row_sum(float v, int T, float* red) {
    v = warp_sum(v);
    if (T == 32) return v;
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = red[0];
    for (int i = 1; i < T / 32; ++i) s += red[i];
    return s;
}
__device__ __forceinline__ uint32_t row_max(uint32_t v, int T, float* red) {
    v = __reduce_max_sync(0xffffffffu, v);
    if (T == 32) return v;
    uint32_t* r = reinterpret_cast<uint32_t*>(red);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5] = v;
    __syncthreads();
    uint32_t m = r[0];
    for (int i = 1; i < T / 32; ++i) m = max(m, r[i]);
    return m;
}

// |v| as an integer of the same order, infinities and NaN above every finite value.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

constexpr uint32_t kInfBits = 0x7f800000u;

// The scale of values whose largest magnitude has the bits `most`: at least 2^-126, so that its
// reciprocal is finite; an infinity's or NaN's is itself, and the values it scales read as NaN.
__device__ __forceinline__ float scale_of(uint32_t most) {
    const float m = __uint_as_float(most);
    return most >= kInfBits ? m : fmaxf(m / 448.f, 0x1p-126f);
}

template <bool kVec> __device__ __forceinline__ void codes8(uint8_t* row, int at, int left, const float (&y)[8], float inv) {
    uint32_t u[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        u[i] = e4m3x2(y[4 * i] * inv, y[4 * i + 1] * inv) | (e4m3x2(y[4 * i + 2] * inv, y[4 * i + 3] * inv) << 16);
    if constexpr (kVec) {
        *reinterpret_cast<uint2*>(row + at) = make_uint2(u[0], u[1]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left) row[at + i] = (uint8_t)(u[i >> 2] >> (8 * (i & 3)));
    }
}

// kX: type of x.  kR: type of the residual, or -1 for none.
template <int kX, int kR, bool kVec, int kCh>
__global__ void __launch_bounds__(kMaxThreads) norm_kernel(const NormParams p) {
    __shared__ float red[32];
    const int T = blockDim.x, tid = threadIdx.x;
    const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const int H = p.H;
    constexpr int kRT = kR < 0 ? kX : kR;
    constexpr int kXs = kX == MOE_F32 ? 4 : 2, kRs = kRT == MOE_F32 ? 4 : 2;
    const bool live = row < p.n;   // (a warp's rows are the same for all its lanes; T > 32: one row a block)
    const int64_t r0 = live ? row : 0;
    const uint8_t* x = reinterpret_cast<const uint8_t*>(p.x) + r0 * p.x_stride * kXs;
    const uint8_t* res = reinterpret_cast<const uint8_t*>(p.res) + r0 * p.res_stride * kRs;
    pdl_wait();

    // Every load of the row before the first use, the weight's too (it is the same for all rows: L1).
    Raw8<kX> xr[kCh];
    Raw8<kRT> rr[kR < 0 ? 1 : kCh];
    Raw8<MOE_BF16> wr[kCh];
    const bool w16 = p.w && p.w_type != MOE_F32;
    int left[kCh];
#pragma unroll
    for (int c = 0; c < kCh; ++c) {
        const int at = (c * T + tid) * 8;
        left[c] = live ? H - at : 0;
        if (left[c] > 0) {
            load8<kX, kVec>(xr[c], x, at, left[c]);
            if constexpr (kR >= 0) load8<kRT, kVec>(rr[c], res, at, left[c]);
        }
    }
#pragma unroll
    for (int c = 0; c < kCh; ++c)
        if (w16 && left[c] > 0) {
            const int at = (c * T + tid) * 8;
            if constexpr (kVec) wr[c].v[0] = __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p.w) + at));
            else load8<MOE_BF16, false>(wr[c], p.w, at, left[c]);
        }

    float h[kCh][8];
    float ss = 0.f;
#pragma unroll
    for (int c = 0; c < kCh; ++c) {
        if (left[c] > 0) {
            floats8<kX>(xr[c], h[c]);
            if constexpr (kR >= 0) {
                float r[8];
                floats8<kRT>(rr[c], r);
#pragma unroll
                for (int i = 0; i < 8; ++i) h[c][i] += r[i];
                if constexpr (kR != MOE_F32) {   // the rows that are normalised are those that are stored
                    Raw8<kRT> st;
                    uint32_t* u = reinterpret_cast<uint32_t*>(st.v);
#pragma unroll
                    for (int i = 0; i < 4; ++i) u[i] = pack2<kRT>(h[c][2 * i], h[c][2 * i + 1]);
                    floats8<kRT>(st, h[c]);
                }
                if (p.res_out)
                    store8<kRT, kVec>(reinterpret_cast<uint8_t*>(p.res_out) + r0 * p.res_out_stride * kRs, (c * T + tid) * 8, left[c], h[c]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) ss += h[c][i] * h[c][i];
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) h[c][i] = 0.f;
        }
    }
    ss = row_sum(ss, T, red);
    const float inv_h = 1.f / (float)H;
    float pre = 1.f, rstd;
    const float mean = ss * inv_h + p.eps;
    if (mean < 3.4e38f && mean > 0x1p-100f) {
        rstd = 1.f / sqrtf(mean);
    } else {
        // Squares that left fp32's range (or a NaN): again, with the row times the power of two
        // that takes the larger of its largest magnitude and sqrt(eps) to [1, 2).
        uint32_t m = 0;
#pragma unroll
        for (int c = 0; c < kCh; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) m = max(m, abs_bits(h[c][i]));
        m = max(row_max(m, T, red), __float_as_uint(sqrtf(p.eps)));
        if (m >= kInfBits) {
            rstd = 1.f / sqrtf(mean);             // as the formula: 0 beside an infinity, NaN
        } else {
            const int e = max((int)(m >> 23) - 127, -126);
            pre = exp2i(max(-e, -126));
            float s2 = 0.f;
#pragma unroll
            for (int c = 0; c < kCh; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) s2 += (h[c][i] * pre) * (h[c][i] * pre);
            s2 = row_sum(s2, T, red);
            rstd = m == 0 ? 0.f : 1.f / sqrtf(s2 * inv_h + (p.eps * pre) * pre);   // (zeros with eps = 0: zeros)
        }
    }

    uint32_t top = 0;
#pragma unroll
    for (int c = 0; c < kCh; ++c) {
        const int at = (c * T + tid) * 8;
        uint32_t most = 0;
        if (left[c] > 0) {
            float w[8];
            if (w16) {
                if (p.w_type == MOE_BF16) floats8<MOE_BF16>(wr[c], w);
                else floats8<MOE_F16>(*reinterpret_cast<const Raw8<MOE_F16>*>(&wr[c]), w);
            } else if (p.w) {
                Raw8<MOE_F32> f;
                load8<MOE_F32, kVec>(f, p.w, at, left[c]);
                floats8<MOE_F32>(f, w);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = 1.f;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float y = (h[c][i] * pre) * rstd * (w[i] + p.w_offset);
                h[c][i] = i < left[c] ? y : 0.f;
                most = max(most, abs_bits(h[c][i]));
            }
            if (p.out)
                store8_as<kVec>(p.out_type, reinterpret_cast<uint8_t*>(p.out) + r0 * p.out_stride * (p.out_type == MOE_F32 ? 4 : 2), at, left[c], h[c]);
        }
        top = max(top, most);
        if (p.out8 && p.group) {
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
            const float s = scale_of(most);
            if (left[c] > 0) {
                if ((tid & 15) == 0) p.scale8[row * p.n_scales + at / 128] = s;
                codes8<kVec>(p.out8 + r0 * p.out8_stride, at, left[c], h[c], 1.f / s);
            }
        }
    }
    if (p.out8 && !p.group) {
        const float s = scale_of(row_max(top, T, red)), inv = 1.f / s;
        if (tid == 0 && live) p.scale8[row] = s;
#pragma unroll
        for (int c = 0; c < kCh; ++c)
            if (left[c] > 0) codes8<kVec>(p.out8 + r0 * p.out8_stride, (c * T + tid) * 8, left[c], h[c], inv);
    }
    pdl_trigger();
}

template <int kX, int kR, bool kVec, int kCh>
cudaError_t launch_ch(const NormParams& p, int T, int rows, cudaStream_t st) {
    constexpr int64_t kMaxBlocks = 0x7fffffff;
    static_assert(kMaxBlocks >= INT32_MAX, "a block for each row");
    launch_pdl(norm_kernel<kX, kR, kVec, kCh>, dim3((unsigned)((p.n + rows - 1) / rows)), dim3(T, rows), 0, st, p);
    return cudaGetLastError();
}

template <int kX, int kR, bool kVec>
cudaError_t launch_vec(const NormParams& p, int num_sms, cudaStream_t st) {
    const int chunks = (p.H + 7) / 8;
    auto threads = [&](int ch) { return ((chunks + ch - 1) / ch + 31) / 32 * 32; };
    int ch = 1;
    while (ch < kMaxCh && threads(ch) > kMaxThreads) ch *= 2;
    while (ch < 4 && (int64_t)p.n * threads(ch) > (int64_t)num_sms * 2048) ch *= 2;
    const int T = threads(ch), rows = T == 32 ? std::min(p.n, 8) : 1;
    switch (ch) {
        case 1: return launch_ch<kX, kR, kVec, 1>(p, T, rows, st);
        case 2: return launch_ch<kX, kR, kVec, 2>(p, T, rows, st);
        case 4: return launch_ch<kX, kR, kVec, 4>(p, T, rows, st);
        default: return launch_ch<kX, kR, kVec, 8>(p, T, rows, st);
    }
}

template <int kX, int kR>
cudaError_t launch_types(const NormParams& p, bool vec, int num_sms, cudaStream_t st) {
    return vec ? launch_vec<kX, kR, true>(p, num_sms, st) : launch_vec<kX, kR, false>(p, num_sms, st);
}

}  // namespace

static_assert(kMaxThreads * kMaxCh * 8 == kNormMaxHidden, "a row fits its threads");

cudaError_t launch_norm(const NormParams& p, int num_sms, cudaStream_t st) {
    // Whole 16-byte loads and stores: every row of every array starts at a multiple of 16 bytes
    // (8 for the codes) and has a multiple of eight elements.
    auto rows16 = [&](const void* a, int64_t stride, int size) {
        return !a || ((reinterpret_cast<uintptr_t>(a) % 16 == 0) && (p.n == 1 || stride * size % 16 == 0));
    };
    auto size = [](int type) { return type == MOE_F32 ? 4 : 2; };
    const bool vec = p.H % 8 == 0 && rows16(p.x, p.x_stride, size(p.x_type)) && rows16(p.res, p.res_stride, size(p.res_type)) &&
                     rows16(p.res_out, p.res_out_stride, size(p.res_type)) && rows16(p.out, p.out_stride, size(p.out_type)) &&
                     rows16(p.w, 0, 0) && reinterpret_cast<uintptr_t>(p.out8) % 8 == 0 && (p.n == 1 || p.out8_stride % 8 == 0);
    const bool f32_res = p.res && p.res_type == MOE_F32;
    switch (p.x_type) {
        case MOE_F32:
            return p.res ? launch_types<MOE_F32, MOE_F32>(p, vec, num_sms, st) : launch_types<MOE_F32, -1>(p, vec, num_sms, st);
        case MOE_BF16:
            return !p.res ? launch_types<MOE_BF16, -1>(p, vec, num_sms, st)
                 : f32_res ? launch_types<MOE_BF16, MOE_F32>(p, vec, num_sms, st)
                           : launch_types<MOE_BF16, MOE_BF16>(p, vec, num_sms, st);
        default:
            return !p.res ? launch_types<MOE_F16, -1>(p, vec, num_sms, st)
                 : f32_res ? launch_types<MOE_F16, MOE_F32>(p, vec, num_sms, st)
                           : launch_types<MOE_F16, MOE_F16>(p, vec, num_sms, st);
    }
}

}  // namespace moe
