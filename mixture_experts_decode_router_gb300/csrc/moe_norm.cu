// moe_norm.cu -- residual addition and RMSNorm of rows, with an output of 16 or 32 bits, one
// of 8 bits with scales, or both (sm_103a):
//   h = x + residual, rounded to the residual's type (what residual_out holds; x without one)
//   y = h / sqrt(mean(h^2) + eps) * (weight + weight_offset)
//   out = y;  out8 = E4M3(y / s),  s = max(max |y| / 448, 2^-126) over 128 elements or the row
//
// Every element is read once, waits in registers (fp32) for the row's sum of squares, and is
// written once.  Few rows are bound by launch and latency, many by HBM as long as the
// instructions an element stay few: products and sums in pairs (f32x2), maxima only for 8-bit
// outputs.
//
// Two kernels.  Rows of whole, aligned 16-byte chunks: a row belongs to T threads, each with
// kCh chunks of eight consecutive elements, T chunks apart, all of whose loads are in flight
// before the first is used; rows of at most 32 kCh chunks are one warp's, several of them to a
// block and no barrier.  The scale of 128 elements is a maximum over 16 neighbouring lanes.
// Any other rows: the same by single elements, neighbouring threads at neighbouring ones (eight
// a thread, one after another, took 33.8 us for 3001 x 2047 that take 22.2 so).
#include <algorithm>

#include "moe_launch.cuh"

namespace moe {

namespace {

constexpr int kThreads = 512, kWideThreads = 1024;   // of a row at most

__host__ __device__ constexpr int size_of(int type) { return type == MOE_F32 ? 4 : 2; }

// ---------------------------------------------------------------- pairs of fp32

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// Two floats of a 16-bit pair, and back (to nearest even).
template <int kType> __device__ __forceinline__ float2 unpack2(uint32_t u) {
    if constexpr (kType == MOE_BF16) return make_float2(bf16_lo(u), bf16_hi(u));
    else return __half22float2(*reinterpret_cast<const __half2*>(&u));
}
template <int kType> __device__ __forceinline__ uint32_t pack2(float2 v) {
    if constexpr (kType == MOE_BF16) {
        const __nv_bfloat162 q = __floats2bfloat162_rn(v.x, v.y);
        return *reinterpret_cast<const uint32_t*>(&q);
    } else {
        const __half2 q = __floats2half2_rn(v.x, v.y);
        return *reinterpret_cast<const uint32_t*>(&q);
    }
}

// ---------------------------------------------------------------- chunks of eight elements

template <int kType> struct Raw8 { uint4 v[kType == MOE_F32 ? 2 : 1]; };

__device__ __forceinline__ uint4 ld_once_v4(const void* p) {
    uint4 r;   // (not ld.global.nc: a row may be overwritten in place by the thread that read it)
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
    return r;
}
template <int kType> __device__ __forceinline__ void load8(Raw8<kType>& r, const uint8_t* row, int at) {
#pragma unroll
    for (int i = 0; i < size_of(kType) / 2; ++i) r.v[i] = ld_once_v4(row + (size_t)at * size_of(kType) + 16 * i);
}
template <int kType> __device__ __forceinline__ void floats8(const Raw8<kType>& r, float2 (&f)[4]) {
    const uint32_t* u = reinterpret_cast<const uint32_t*>(r.v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (kType == MOE_F32) f[i] = make_float2(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1]));
        else f[i] = unpack2<kType>(u[i]);
    }
}
template <int kType> __device__ __forceinline__ void store8(uint8_t* row, int at, const float2 (&f)[4]) {
    uint8_t* d = row + (size_t)at * size_of(kType);
    if constexpr (kType == MOE_F32) {
        *reinterpret_cast<float4*>(d) = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
        *reinterpret_cast<float4*>(d + 16) = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
    } else {
        *reinterpret_cast<uint4*>(d) = make_uint4(pack2<kType>(f[0]), pack2<kType>(f[1]), pack2<kType>(f[2]), pack2<kType>(f[3]));
    }
}

// ---------------------------------------------------------------- rows

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
// The larger of two magnitudes, a NaN before both (one instruction, where abs_bits takes two).
__device__ __forceinline__ float max_abs(float m, float v) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(m), "f"(fabsf(v)));
    return r;
}

// The scale of values whose largest magnitude has the bits `most`: at least 2^-126, so that its
// reciprocal is finite; an infinity's or NaN's is itself, and the values it scales read as NaN.
__device__ __forceinline__ float scale_of(uint32_t most) {
    const float m = __uint_as_float(most);
    return most >= kInfBits ? m : fmaxf(m * (1.f / 448.f), 0x1p-126f);
}
// 1 / s of a scale (2^-126 to 2^120, or as above), within a step of fp32.
__device__ __forceinline__ float reciprocal(float s) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
    return r;
}
// E4M3 of a pair (x in the low byte), to nearest even; NaN is NaN.
__device__ __forceinline__ uint32_t e4m3x2(float2 v) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(v.y), "f"(v.x));
    return r;
}

// 1 / sqrt(mean(h^2) + eps) from this thread's sum of squares.  If squares left fp32's range (or
// met a NaN), from the row times the power of two that takes the larger of its largest magnitude and
// sqrt(eps) to [1, 2), by which h is then multiplied.
template <int N> __device__ __forceinline__ float row_rstd(float ss, float2 (&h)[N], const NormParams& p, int T, float* red) {
    const float inv_h = 1.f / (float)p.H;
    const float mean = row_sum(ss, T, red) * inv_h + p.eps;
    if (mean < 3.4e38f && mean > 0x1p-100f) return 1.f / sqrtf(mean);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) m = max(m, max(abs_bits(h[i].x), abs_bits(h[i].y)));
    m = max(row_max(m, T, red), __float_as_uint(sqrtf(p.eps)));
    if (m >= kInfBits) return 1.f / sqrtf(mean);   // as the formula: 0 beside an infinity, NaN
    if (m == 0) return 0.f;                        // zeros with eps = 0
    const float pre = exp2i(max(-max((int)(m >> 23) - 127, -126), -126));
    float s2 = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        h[i] = __fmul2_rn(h[i], both(pre));
        s2 += h[i].x * h[i].x + h[i].y * h[i].y;
    }
    return 1.f / sqrtf(row_sum(s2, T, red) * inv_h + (p.eps * pre) * pre);
}

// One row from what get(c, xr, rr) gives of chunk c of x and the residual, and weight16(c) of a 16-bit
// weight.  in[c]: the thread has a chunk c.  live: the row is one (else it only takes part in the
// reductions).
template <int kX, int kR, int kCh, typename Get, typename Weight16>
__device__ __forceinline__ void norm_row(const NormParams& p, int64_t row, bool live, int T, const bool (&in)[kCh], float* red, Get get,
                                         Weight16 weight16) {
    constexpr int kRT = kR < 0 ? kX : kR;
    const int tid = threadIdx.x;
    const int64_t r0 = live ? row : 0;
    uint8_t* res_out = reinterpret_cast<uint8_t*>(p.res_out) + r0 * p.res_out_stride * size_of(kRT);
    const bool w16 = p.w && p.w_type != MOE_F32;
    float2 h[kCh * 4], ss = make_float2(0.f, 0.f);
#pragma unroll
    for (int c = 0; c < kCh; ++c) {
        float2(&hc)[4] = *reinterpret_cast<float2(*)[4]>(&h[4 * c]);
        if (in[c]) {
            Raw8<kX> xr;
            Raw8<kRT> rr;
            get(c, xr, rr);
            floats8<kX>(xr, hc);
            if constexpr (kR >= 0) {
                float2 r[4];
                floats8<kRT>(rr, r);
#pragma unroll
                for (int i = 0; i < 4; ++i) hc[i] = __fadd2_rn(hc[i], r[i]);
                if constexpr (kR != MOE_F32) {   // the rows that are normalised are those that are stored
                    const uint4 st = make_uint4(pack2<kRT>(hc[0]), pack2<kRT>(hc[1]), pack2<kRT>(hc[2]), pack2<kRT>(hc[3]));
                    if (p.res_out) *reinterpret_cast<uint4*>(res_out + (size_t)(c * T + tid) * 16) = st;
                    floats8<kRT>(Raw8<kRT>{{st}}, hc);
                } else if (p.res_out) {
                    store8<MOE_F32>(res_out, (c * T + tid) * 8, hc);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) ss = __ffma2_rn(hc[i], hc[i], ss);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) hc[i] = make_float2(0.f, 0.f);
        }
    }
    const float2 rstd = both(row_rstd(ss.x + ss.y, h, p, T, red));

    uint32_t top = 0;
#pragma unroll
    for (int c = 0; c < kCh; ++c) {
        float2(&y)[4] = *reinterpret_cast<float2(*)[4]>(&h[4 * c]);
        const int at = (c * T + tid) * 8;
        if (in[c]) {
            float2 w[4];
            if (w16) {
                const uint4 wr = weight16(c);
                if (p.w_type == MOE_BF16) floats8<MOE_BF16>(Raw8<MOE_BF16>{{wr}}, w);
                else floats8<MOE_F16>(Raw8<MOE_F16>{{wr}}, w);
            } else if (p.w) {
                const float4* f = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p.w) + at);
                const float4 a = __ldg(f), b = __ldg(f + 1);
                w[0] = make_float2(a.x, a.y); w[1] = make_float2(a.z, a.w);
                w[2] = make_float2(b.x, b.y); w[3] = make_float2(b.z, b.w);
            } else {
                w[0] = w[1] = w[2] = w[3] = both(1.f);
            }
            if (p.w_offset != 0.f) {
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = __fadd2_rn(w[i], both(p.w_offset));
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = __fmul2_rn(__fmul2_rn(y[i], rstd), w[i]);
            if (p.out) {
                uint8_t* out = reinterpret_cast<uint8_t*>(p.out) + r0 * p.out_stride * size_of(p.out_type);
                if (p.out_type == MOE_BF16) store8<MOE_BF16>(out, at, y);
                else if (p.out_type == MOE_F16) store8<MOE_F16>(out, at, y);
                else store8<MOE_F32>(out, at, y);
            }
        }
        if (p.out8) {
            float m = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) m = max_abs(max_abs(m, y[i].x), y[i].y);
            uint32_t most = in[c] ? __float_as_uint(m) : 0u;
            if (p.group) {
#pragma unroll
                for (int o = 1; o < 16; o <<= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
                const float s = scale_of(most);
                if (in[c]) {
                    if ((tid & 15) == 0) p.scale8[row * p.n_scales + at / 128] = s;
                    const float2 inv = both(reciprocal(s));
                    *reinterpret_cast<uint2*>(p.out8 + r0 * p.out8_stride + at) =
                        make_uint2(e4m3x2(__fmul2_rn(y[0], inv)) | e4m3x2(__fmul2_rn(y[1], inv)) << 16, e4m3x2(__fmul2_rn(y[2], inv)) | e4m3x2(__fmul2_rn(y[3], inv)) << 16);
                }
            } else {
                top = max(top, most);
            }
        }
    }
    if (p.out8 && !p.group) {
        const float s = scale_of(row_max(top, T, red));
        const float2 inv = both(reciprocal(s));
        if (tid == 0 && live) p.scale8[row] = s;
#pragma unroll
        for (int c = 0; c < kCh; ++c) {
            const float2* y = &h[4 * c];
            if (in[c])
                *reinterpret_cast<uint2*>(p.out8 + r0 * p.out8_stride + (c * T + tid) * 8) =
                    make_uint2(e4m3x2(__fmul2_rn(y[0], inv)) | e4m3x2(__fmul2_rn(y[1], inv)) << 16, e4m3x2(__fmul2_rn(y[2], inv)) | e4m3x2(__fmul2_rn(y[3], inv)) << 16);
        }
    }
}

// kX: type of x.  kR: type of the residual, or -1 for none.  Rows of whole aligned chunks.  kWide:
// rows so long that their threads have no registers for loads in flight.
template <int kX, int kR, int kCh, bool kWide>
__global__ void __launch_bounds__(kWide ? kWideThreads : kThreads, kWide || kR == MOE_F32 ? 1 : 2) norm_kernel(const NormParams p) {
    __shared__ float red[32];
    constexpr int kRT = kR < 0 ? kX : kR;
    const int T = blockDim.x, tid = threadIdx.x;
    const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const bool live = row < p.n;   // (whole warps: T > 32 means one row a block)
    const int64_t r0 = live ? row : 0;
    const uint8_t* x = reinterpret_cast<const uint8_t*>(p.x) + r0 * p.x_stride * size_of(kX);
    const uint8_t* res = reinterpret_cast<const uint8_t*>(p.res) + r0 * p.res_stride * size_of(kRT);
    bool in[kCh];
#pragma unroll
    for (int c = 0; c < kCh; ++c) in[c] = live && (c * T + tid) * 8 < p.H;
    pdl_wait();
    pdl_trigger();   // (the next kernel's launch overlaps this one; it waits for its end)

    // Every load of the row before the first use; of a thread's only chunk the weight's too.
    Raw8<kX> xr[kCh];
    Raw8<kRT> rr[kR < 0 ? 1 : kCh];
    uint4 wr = make_uint4(0u, 0u, 0u, 0u);
    auto load_w16 = [&](int c) { return __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p.w) + (c * T + tid) * 8)); };
    if constexpr (!kWide) {
#pragma unroll
        for (int c = 0; c < kCh; ++c)
            if (in[c]) {
                load8<kX>(xr[c], x, (c * T + tid) * 8);
                if constexpr (kR >= 0) load8<kRT>(rr[c], res, (c * T + tid) * 8);
            }
        if (kCh == 1 && in[0] && p.w && p.w_type != MOE_F32) wr = load_w16(0);
    }
    norm_row<kX, kR, kCh>(
        p, row, live, T, in, red,
        [&](int c, Raw8<kX>& a, Raw8<kRT>& b) {
            if constexpr (kWide) {
                load8<kX>(a, x, (c * T + tid) * 8);
                if constexpr (kR >= 0) load8<kRT>(b, res, (c * T + tid) * 8);
            } else {
                a = xr[c];
                if constexpr (kR >= 0) b = rr[c];
            }
        },
        [&](int c) { return kCh == 1 ? wr : load_w16(c); });
}

// ---------------------------------------------------------------- rows of any alignment

template <int kType> __device__ __forceinline__ float load1(const void* row, int at) {
    if constexpr (kType == MOE_F32) return reinterpret_cast<const float*>(row)[at];
    const uint16_t u = reinterpret_cast<const uint16_t*>(row)[at];
    return unpack2<kType>(u).x;
}
// Elements i T + tid of the weight (1 without one), plus its offset.
template <int kType, int kE> __device__ __forceinline__ void load_weight(const NormParams& p, int T, float (&w)[kE]) {
#pragma unroll
    for (int i = 0; i < kE; ++i) {
        const int at = i * T + (int)threadIdx.x;
        if constexpr (kType == MOE_F32) {
            w[i] = at < p.H ? __ldg(reinterpret_cast<const float*>(p.w) + at) : 0.f;
        } else {
            const uint16_t u = at < p.H ? __ldg(reinterpret_cast<const uint16_t*>(p.w) + at) : (uint16_t)0;
            w[i] = unpack2<kType>(u).x;
        }
    }
}
template <int kE> __device__ __forceinline__ void load_weight_as(const NormParams& p, int T, float (&w)[kE]) {
    if (!p.w) {
#pragma unroll
        for (int i = 0; i < kE; ++i) w[i] = 1.f;
    } else if (p.w_type == MOE_F32) load_weight<MOE_F32>(p, T, w);
    else if (p.w_type == MOE_BF16) load_weight<MOE_BF16>(p, T, w);
    else load_weight<MOE_F16>(p, T, w);
#pragma unroll
    for (int i = 0; i < kE; ++i) w[i] += p.w_offset;
}
template <int kType> __device__ __forceinline__ void store1(void* row, int at, float v) {
    if constexpr (kType == MOE_F32) reinterpret_cast<float*>(row)[at] = v;
    else reinterpret_cast<uint16_t*>(row)[at] = (uint16_t)pack2<kType>(make_float2(v, 0.f));
}
__device__ __forceinline__ void store1_as(int type, void* row, int at, float v) {
    if (type == MOE_F32) store1<MOE_F32>(row, at, v);
    else if (type == MOE_BF16) store1<MOE_BF16>(row, at, v);
    else store1<MOE_F16>(row, at, v);
}

// A row a block, element i T + tid the thread's i-th of kE (T a multiple of 128: the scale of 128
// elements is a maximum over four warps).
template <int kX, int kR, int kE, int kMost>
__global__ void __launch_bounds__(kMost) norm_any_kernel(const NormParams p) {
    __shared__ float red[32];
    __shared__ __align__(16) uint32_t tops[kE * (kMost / 32)];
    constexpr int kRT = kR < 0 ? kX : kR;
    const int T = blockDim.x, tid = threadIdx.x, H = p.H;
    const int64_t row = blockIdx.x;
    const uint8_t* x = reinterpret_cast<const uint8_t*>(p.x) + row * p.x_stride * size_of(kX);
    const uint8_t* res = reinterpret_cast<const uint8_t*>(p.res) + row * p.res_stride * size_of(kRT);
    uint8_t* res_out = reinterpret_cast<uint8_t*>(p.res_out) + row * p.res_out_stride * size_of(kRT);
    pdl_wait();
    pdl_trigger();   // (the next kernel's launch overlaps this one; it waits for its end)
    float2 h[kE / 2];
    float rv[kR < 0 ? 1 : kE];
    auto each = [&](int i) -> float& { return i & 1 ? h[i / 2].y : h[i / 2].x; };
#pragma unroll
    for (int i = 0; i < kE; ++i) {
        const int at = i * T + tid;
        each(i) = at < H ? load1<kX>(x, at) : 0.f;
        if constexpr (kR >= 0) rv[i] = at < H ? load1<kRT>(res, at) : 0.f;
    }
    // The weight before the first store, behind which its loads would wait one by one.
    float w[kE];
    constexpr bool kEarly = kE < 32;
    if (kEarly) load_weight_as(p, T, w);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < kE; ++i) {
        float& v = each(i);
        if constexpr (kR >= 0) {
            v += rv[i];
            if constexpr (kR != MOE_F32) v = unpack2<kRT>(pack2<kRT>(make_float2(v, 0.f))).x;
            if (p.res_out && i * T + tid < H) store1<kRT>(res_out, i * T + tid, v);
        }
        ss = fmaf(v, v, ss);
    }
    const float rstd = row_rstd(ss, h, p, T, red);
    if (!kEarly) load_weight_as(p, T, w);
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kE; ++i) {
        const int at = i * T + tid;
        float& y = each(i);
        if (at < H) {
            y = (y * rstd) * w[i];
            if (p.out) store1_as(p.out_type, reinterpret_cast<uint8_t*>(p.out) + row * p.out_stride * size_of(p.out_type), at, y);
        }
        if (p.out8) {
            const uint32_t m = at < H ? abs_bits(y) : 0u;
            if (p.group) {
                const uint32_t most = __reduce_max_sync(0xffffffffu, m);
                if ((tid & 31) == 0) tops[i * (T / 32) + tid / 32] = most;
            } else {
                top = max(top, m);
            }
        }
    }
    if (p.out8) {
        float s = 0.f;
        if (p.group) {
            __syncthreads();
        } else {
            s = scale_of(row_max(top, T, red));
            if (tid == 0) p.scale8[row] = s;
        }
#pragma unroll
        for (int i = 0; i < kE; ++i) {
            const int at = i * T + tid;
            if (at >= H) break;
            if (p.group) {
                const uint4 m = *reinterpret_cast<const uint4*>(&tops[i * (T / 32) + tid / 128 * 4]);
                s = scale_of(max(max(m.x, m.y), max(m.z, m.w)));
                if (tid % 128 == 0) p.scale8[row * p.n_scales + at / 128] = s;
            }
            p.out8[row * p.out8_stride + at] = (uint8_t)e4m3x2(make_float2(each(i) * reciprocal(s), 0.f));
        }
    }
}

// ---------------------------------------------------------------- launches

template <int kX, int kR>
cudaError_t launch_types(const NormParams& p, bool chunks, int num_sms, cudaStream_t st) {
    if (!chunks) {
        auto go = [&](auto kern, int e) {
            launch_pdl(kern, dim3((unsigned)p.n), dim3(((p.H + e - 1) / e + 127) / 128 * 128), 0, st, p);
            return cudaGetLastError();
        };
        // Elements of a thread: four while the rows' threads all run at once, else eight, as many
        // as long rows ask for (2047 elements: 152 rows 3.4 us with 4, 4.1 with 8; 4000 rows 38.7 and 35.2).
        const int few = (p.H + 3) / 4;
        if (few <= kThreads && (int64_t)p.n * few <= (int64_t)num_sms * 2048) return go(norm_any_kernel<kX, kR, 4, kThreads>, 4);
        if (p.H <= 8 * kThreads) return go(norm_any_kernel<kX, kR, 8, kThreads>, 8);
        if (p.H <= 16 * kThreads) return go(norm_any_kernel<kX, kR, 16, kThreads>, 16);
        return go(norm_any_kernel<kX, kR, 32, kWideThreads>, 32);
    }
    const int n8 = p.H / 8;
    auto threads = [&](int ch) { return ((n8 + ch - 1) / ch + 31) / 32 * 32; };
    auto go = [&](auto kern, int ch) {
        const int T = threads(ch), rows = T == 32 ? std::min(p.n, 8) : 1;
        launch_pdl(kern, dim3((unsigned)((p.n + rows - 1) / rows)), dim3(T, rows), 0, st, p);
        return cudaGetLastError();
    };
    // Chunks of a thread: one while the rows' threads all run at once, else as many as its registers
    // hold (two of two fp32 rows).
    constexpr int kMost = kX == MOE_F32 && kR == MOE_F32 ? 2 : 4;
    int ch = 1;
    while (threads(ch) > kThreads) ch *= 2;
    while (ch < kMost && (int64_t)p.n * threads(ch) > (int64_t)num_sms * 2048) ch *= 2;
    if (ch > kMost) return go(norm_kernel<kX, kR, 4, true>, 4);
    if (ch == 1) return go(norm_kernel<kX, kR, 1, false>, 1);
    if (ch == 2) return go(norm_kernel<kX, kR, 2, false>, 2);
    if constexpr (kMost == 4) return go(norm_kernel<kX, kR, 4, false>, 4);
    return cudaErrorInvalidValue;
}

}  // namespace

static_assert(kWideThreads * 32 == kNormMaxHidden, "a row fits its threads");

cudaError_t launch_norm(const NormParams& p, int num_sms, cudaStream_t st) {
    // Whole 16-byte loads and stores: every row of every array starts at a multiple of 16 bytes
    // (8 for the codes) and has a multiple of eight elements.
    auto rows16 = [&](const void* a, int64_t stride, int size) {
        return !a || ((reinterpret_cast<uintptr_t>(a) % 16 == 0) && (p.n == 1 || stride * size % 16 == 0));
    };
    const bool chunks = p.H % 8 == 0 && rows16(p.x, p.x_stride, size_of(p.x_type)) && rows16(p.res, p.res_stride, size_of(p.res_type)) &&
                        rows16(p.res_out, p.res_out_stride, size_of(p.res_type)) && rows16(p.out, p.out_stride, size_of(p.out_type)) &&
                        rows16(p.w, 0, 0) &&
                        (!p.out8 || (reinterpret_cast<uintptr_t>(p.out8) % 8 == 0 && (p.n == 1 || p.out8_stride % 8 == 0)));
    const bool f32_res = p.res && p.res_type == MOE_F32;
    switch (p.x_type) {
        case MOE_F32:
            return p.res ? launch_types<MOE_F32, MOE_F32>(p, chunks, num_sms, st) : launch_types<MOE_F32, -1>(p, chunks, num_sms, st);
        case MOE_BF16:
            return !p.res ? launch_types<MOE_BF16, -1>(p, chunks, num_sms, st)
                 : f32_res ? launch_types<MOE_BF16, MOE_F32>(p, chunks, num_sms, st)
                           : launch_types<MOE_BF16, MOE_BF16>(p, chunks, num_sms, st);
        default:
            return !p.res ? launch_types<MOE_F16, -1>(p, chunks, num_sms, st)
                 : f32_res ? launch_types<MOE_F16, MOE_F32>(p, chunks, num_sms, st)
                           : launch_types<MOE_F16, MOE_F16>(p, chunks, num_sms, st);
    }
}

}  // namespace moe
