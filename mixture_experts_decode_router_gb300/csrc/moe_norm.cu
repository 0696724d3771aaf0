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
// A row belongs to T threads, each with kCh chunks of eight consecutive elements, T chunks apart, all of
// whose loads are in flight before the first is used; rows of at most 32 kCh chunks are one warp's,
// several of them to a block and no barrier.  The scale of 128 elements is a maximum over 16
// neighbouring lanes.
//
// Rows that are not of whole chunks at addresses of whole chunks (kAny): a chunk is cut from the two
// aligned 16 bytes (fp32: three) that it lies in, each of which holds a byte of the row; outputs go
// through a warp's staging, from which lanes take the aligned 16 bytes (of codes 8) of the span of its
// 32 chunks, and what is left before and behind them by elements.  A warp writes its own elements only,
// so rows may still be overwritten in place.  (By single elements, neighbouring threads at
// neighbouring ones: 22 us for 3001 x 2047 that take 17.5 so, 250 for 5000 x 7168 that take 76.)
#include <algorithm>
#include <type_traits>

#include "moe_launch.cuh"

namespace moe {

namespace {

constexpr int kThreads = 512, kWideThreads = 1024;   // of a row at most
constexpr int kNoCodes = 0, kRow = 1, kGroups = 2;   // out8's scales: none, of the row, of 128 elements

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

// ---------------------------------------------------------------- the same at any address

// The 16 bytes from byte `at` (even) of two neighbouring ones, and the 8 bytes from any byte of 16.
__device__ __forceinline__ uint4 cut16(const uint4& a, const uint4& b, int at) {
    const uint32_t r[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t s[7], t[5];
#pragma unroll
    for (int i = 0; i < 7; ++i) s[i] = at & 4 ? r[i + 1] : r[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) t[i] = at & 8 ? s[i + 2] : s[i];
    const int bits = 8 * (at & 3);
    return make_uint4(__funnelshift_r(t[0], t[1], bits), __funnelshift_r(t[1], t[2], bits), __funnelshift_r(t[2], t[3], bits),
                      __funnelshift_r(t[3], t[4], bits));
}
__device__ __forceinline__ uint2 cut8(const uint2& a, const uint2& b, int at) {
    const uint32_t r0 = at & 4 ? a.y : a.x, r1 = at & 4 ? b.x : a.y, r2 = at & 4 ? b.y : b.x;
    const int bits = 8 * (at & 3);
    return make_uint2(__funnelshift_r(r0, r1, bits), __funnelshift_r(r1, r2, bits));
}
// The aligned 16 bytes that eight elements of a row lie in; zeros for those that hold nothing of the row.
template <int kType> struct Around8 { uint4 v[kType == MOE_F32 ? 3 : 2]; };
__device__ __forceinline__ uint4 ld_v4(const void* p) {
    uint4 r;
    asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
    return r;
}
template <int kType> __device__ __forceinline__ void load_around(Around8<kType>& r, const uint8_t* row, int at, int H) {
    const uint8_t *a = row + (size_t)at * size_of(kType), *end = row + (size_t)H * size_of(kType);
    const int off = (int)(reinterpret_cast<uintptr_t>(a) & 15);
    a -= off;
    constexpr int kN = size_of(kType) / 2;      // 16 bytes of eight elements
#pragma unroll
    for (int i = 0; i <= kN; ++i) r.v[i] = i == 0 || ((i < kN || off) && a + 16 * i < end) ? ld_v4(a + 16 * i) : make_uint4(0u, 0u, 0u, 0u);
}
template <int kType> __device__ __forceinline__ Raw8<kType> cut_around(const Around8<kType>& r, const uint8_t* row) {
    const int off = (int)(reinterpret_cast<uintptr_t>(row) & 15);
    Raw8<kType> q;
#pragma unroll
    for (int i = 0; i < size_of(kType) / 2; ++i) q.v[i] = cut16(r.v[i], r.v[i + 1], off);
    return q;
}
// What a warp's lanes have of `n` elements from `to` on, eight a lane, through its staging of 1 KB.
// Of 16 bits ...
__device__ __forceinline__ void put16(uint8_t* to, int n, const uint4& v, uint8_t* stage) {
    const int lane = threadIdx.x & 31, off = (int)(reinterpret_cast<uintptr_t>(to) & 15);
    if (off == 0 && n == 256) {
        reinterpret_cast<uint4*>(to)[lane] = v;
        return;
    }
    uint4* s = reinterpret_cast<uint4*>(stage);
    s[lane] = v;
    __syncwarp();
    const int head = (16 - off & 15) / 2, whole = max(0, n - head) / 8;
    if (lane < whole) *reinterpret_cast<uint4*>(to + 2 * head + 16 * lane) = cut16(s[lane], s[min(lane + 1, 31)], 2 * head);
    if (lane < n - 8 * whole) {
        const int e = lane < head ? lane : 8 * whole + lane;
        reinterpret_cast<uint16_t*>(to)[e] = reinterpret_cast<const uint16_t*>(stage)[e];
    }
    __syncwarp();
}
// ... of 8 ...
__device__ __forceinline__ void put8(uint8_t* to, int n, const uint2& v, uint8_t* stage) {
    const int lane = threadIdx.x & 31, off = (int)(reinterpret_cast<uintptr_t>(to) & 7);
    if (off == 0 && n == 256) {
        reinterpret_cast<uint2*>(to)[lane] = v;
        return;
    }
    uint2* s = reinterpret_cast<uint2*>(stage);
    s[lane] = v;
    __syncwarp();
    const int head = 8 - off & 7, whole = max(0, n - head) / 8;
    if (lane < whole) *reinterpret_cast<uint2*>(to + head + 8 * lane) = cut8(s[lane], s[min(lane + 1, 31)], head);
    if (lane < n - 8 * whole) {
        const int e = lane < head ? lane : 8 * whole + lane;
        to[e] = stage[e];
    }
    __syncwarp();
}
// ... and of 32.
__device__ __forceinline__ void put32(uint8_t* to, int n, const float2 (&f)[4], uint8_t* stage) {
    const int lane = threadIdx.x & 31;
    float4* s = reinterpret_cast<float4*>(stage) + 2 * lane;
    s[0] = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
    s[1] = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (32 * i + lane < n) reinterpret_cast<float*>(to)[32 * i + lane] = reinterpret_cast<const float*>(stage)[32 * i + lane];
    __syncwarp();
}
template <int kType> __device__ __forceinline__ uint4 pack8(const float2 (&f)[4]) {
    return make_uint4(pack2<kType>(f[0]), pack2<kType>(f[1]), pack2<kType>(f[2]), pack2<kType>(f[3]));
}
// Eight elements of which `n` are the row's: zeros for the others.
__device__ __forceinline__ void first_of8(float2 (&f)[4], int n) {
    if (n >= 8) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (2 * i >= n) f[i].x = 0.f;
        if (2 * i + 1 >= n) f[i].y = 0.f;
    }
}

// ---------------------------------------------------------------- rows

// Sum and maximum over the T threads of a row (threadIdx.x), the same value in each.  One
// warp's by shuffles; more than one warp's through red, 32 words that nothing else uses.
__device__ __forceinline__ float row_sum(float v, int T, float* red) {
    v = warp_sum(v);
    if (T == 32) return v;
    const int lane = threadIdx.x & 31;
    if (lane == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    return warp_sum(lane < T / 32 ? red[lane] : 0.f);
}
__device__ __forceinline__ uint32_t row_max(uint32_t v, int T, float* red) {
    v = __reduce_max_sync(0xffffffffu, v);
    if (T == 32) return v;
    uint32_t* r = reinterpret_cast<uint32_t*>(red);
    const int lane = threadIdx.x & 31;
    if (lane == 0) r[threadIdx.x >> 5] = v;
    __syncthreads();
    return __reduce_max_sync(0xffffffffu, lane < T / 32 ? r[lane] : 0u);
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

// A group's scale, and what takes values to their codes' quotients by it.  y is t times the root's part m in [1, 2), so
// y / (max |y| / 448) is t times 448 / max |t|, which m does not enter: from t, whose products of 16-bit numbers are
// exact, a quotient at a border of E4M3 falls as exact arithmetic has it.  (A row of 16-bit elements has many there: from y
// and the scale, each rounded, some 5400 of 8192 x 7168 codes were the neighbouring ones, and none so.)  The scale is the
// quotient of y's largest (a product with 1 / 448 is another number for half of all magnitudes, and is corrected by what it
// leaves: Markstein, 1990); the factor is a sum of two fp32, off by some 2^-46 of it, so that a product with it is
// rounded once.  (Selects for the rare scales: with branches 8192 x 7168 took 1.5 us more.)
struct Factor {
    float scale;
    float2 hi, lo;
    __device__ __forceinline__ Factor(float top, float m) {      // top: max |t|
        const float v = top * m, q = v * (1.f / 448.f), s = fmaf(fmaf(q, -448.f, v), 1.f / 448.f, q);
        const bool finite = v < INFINITY;        // (of y: top may still be)
        scale = finite ? fmaxf(s, 0x1p-126f) : v;
        top = finite ? top : v;
        float up = 1.f, r;
        if (scale < 0x1p-100f) up = 0x1p64f;     // (what r is taken of stays above fp32's smallest)
        top *= up;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(top * (1.f / 448.f)));
        float rest = fmaf(-top, r, 448.f) * (1.f / 448.f) * r;
        if (!finite) rest = 0.f;                 // (a number by an infinity is 0)
        r *= up;
        rest *= up;
        if (scale == 0x1p-126f) r = m * 0x1p126f, rest = 0.f;      // the smallest scale there is: y 2^126
        hi = both(r);
        lo = both(rest);
    }
    __device__ __forceinline__ float2 times(float2 t) const { return __ffma2_rn(t, hi, __fmul2_rn(t, lo)); }
};
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
    m = max(row_max(m, T, red + 32), __float_as_uint(sqrtf(p.eps)));
    if (m >= kInfBits) return 1.f / sqrtf(mean);   // as the formula: 0 beside an infinity, NaN
    if (m == 0) return 0.f;                        // zeros with eps = 0
    const float pre = exp2i(max(-max((int)(m >> 23) - 127, -126), -126));
    float s2 = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        h[i] = __fmul2_rn(h[i], both(pre));
        s2 += h[i].x * h[i].x + h[i].y * h[i].y;
    }
    return 1.f / sqrtf(row_sum(s2, T, red + 64) * inv_h + (p.eps * pre) * pre);
}

// One row from what get(c, xr, rr) gives of chunk c of x and the residual, and weight16(c) of a 16-bit
// weight.  in[c]: the thread has a chunk c.  live: the row is one (else it only takes part in the
// reductions).  stage: kAny's, of the warp.
template <int kX, int kR, int kCh, bool kAny, int kCodes, typename Get, typename Weight16, typename Weight32>
__device__ __forceinline__ void norm_row(const NormParams& p, int64_t row, bool live, int T, const bool (&in)[kCh], float* red, uint8_t* stage,
                                         Get get, Weight16 weight16, Weight32 weight32) {
    constexpr int kRT = kR < 0 ? kX : kR;
    const int tid = threadIdx.x;
    const int64_t r0 = live ? row : 0;
    uint8_t* res_out = reinterpret_cast<uint8_t*>(p.res_out) + r0 * p.res_out_stride * size_of(kRT);

    const bool w16 = p.w && p.w_type != MOE_F32;
    // kAny: where the warp's chunks c begin, and how many elements they have.
    auto span = [&](int c) { return (c * T + (tid & ~31)) * 8; };
    auto within = [&](int c) { return live ? min(256, p.H - span(c)) : 0; };
    auto codes = [&](const float2* t, const Factor& f) {
        return make_uint2(e4m3x2(f.times(t[0])) | e4m3x2(f.times(t[1])) << 16, e4m3x2(f.times(t[2])) | e4m3x2(f.times(t[3])) << 16);
    };
    float2 h[kCh * 4], ss = make_float2(0.f, 0.f);
#pragma unroll
    for (int c = 0; c < kCh; ++c) {
        float2(&hc)[4] = *reinterpret_cast<float2(*)[4]>(&h[4 * c]);
        uint4 st = make_uint4(0u, 0u, 0u, 0u);
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
                    st = pack8<kRT>(hc);
                    if (!kAny && p.res_out) *reinterpret_cast<uint4*>(res_out + (size_t)(c * T + tid) * 16) = st;
                    floats8<kRT>(Raw8<kRT>{{st}}, hc);
                } else if (!kAny && p.res_out) {
                    store8<MOE_F32>(res_out, (c * T + tid) * 8, hc);
                }
            }
            if constexpr (kAny) first_of8(hc, p.H - (c * T + tid) * 8);
#pragma unroll
            for (int i = 0; i < 4; ++i) ss = __ffma2_rn(hc[i], hc[i], ss);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) hc[i] = make_float2(0.f, 0.f);
        }
        if constexpr (kAny && kR >= 0) {
            if (p.res_out && within(c) > 0) {
                uint8_t* to = res_out + (size_t)span(c) * size_of(kRT);
                if constexpr (kR == MOE_F32) put32(to, within(c), hc, stage);
                else put16(to, within(c), st, stage);
            }
        }
    }
    // With codes, the root's power of two (exact), and the rest of it, m, only on the way to out and the scales (Factor).
    const float root = row_rstd(ss.x + ss.y, h, p, T, red);
    const uint32_t root_bits = __float_as_uint(root);
    const bool apart = kCodes != kNoCodes && root_bits < kInfBits;
    const float2 rstd = both(apart ? __uint_as_float(root_bits & kInfBits) : root);
    const float m = apart ? __uint_as_float((root_bits & ~kInfBits) | 0x3f800000u) : 1.f;

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
                floats8<MOE_F32>(weight32(c), w);
            } else {
                w[0] = w[1] = w[2] = w[3] = both(1.f);
            }
            if (p.w_offset != 0.f) {
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = __fadd2_rn(w[i], both(p.w_offset));
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = __fmul2_rn(__fmul2_rn(y[i], rstd), w[i]);
            if constexpr (kAny) first_of8(y, p.H - at);
        }
        if (kCodes == kNoCodes || p.out) {
            float2 z[4] = {y[0], y[1], y[2], y[3]};
            if constexpr (kCodes != kNoCodes) {
#pragma unroll
                for (int i = 0; i < 4; ++i) z[i] = __fmul2_rn(z[i], both(m));
            }
            if constexpr (kAny) {
                if (within(c) > 0) {
                    uint8_t* to = reinterpret_cast<uint8_t*>(p.out) + (r0 * p.out_stride + span(c)) * size_of(p.out_type);
                    if (p.out_type == MOE_F32) put32(to, within(c), z, stage);
                    else put16(to, within(c), p.out_type == MOE_BF16 ? pack8<MOE_BF16>(z) : pack8<MOE_F16>(z), stage);
                }
            } else if (in[c]) {
                uint8_t* out = reinterpret_cast<uint8_t*>(p.out) + r0 * p.out_stride * size_of(p.out_type);
                if (p.out_type == MOE_BF16) store8<MOE_BF16>(out, at, z);
                else if (p.out_type == MOE_F16) store8<MOE_F16>(out, at, z);
                else store8<MOE_F32>(out, at, z);
            }
        }
        if constexpr (kCodes != kNoCodes) {
            float top8 = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) top8 = max_abs(max_abs(top8, y[i].x), y[i].y);
            uint32_t most = in[c] ? __float_as_uint(top8) : 0u;
            if constexpr (kCodes == kGroups) {
#pragma unroll
                for (int o = 1; o < 16; o <<= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
                const Factor f(__uint_as_float(most), m);
                if (in[c] && (tid & 15) == 0) p.scale8[row * p.n_scales + at / 128] = f.scale;
                const uint2 q = codes(y, f);
                if constexpr (kAny) {
                    if (within(c) > 0) put8(p.out8 + r0 * p.out8_stride + span(c), within(c), q, stage);
                } else if (in[c]) {
                    *reinterpret_cast<uint2*>(p.out8 + r0 * p.out8_stride + at) = q;
                }
            } else {
                top = max(top, most);
            }
        }
    }
    if constexpr (kCodes == kRow) {
        const Factor f(__uint_as_float(row_max(top, T, red + 96)), m);
        if (tid == 0 && live) p.scale8[row] = f.scale;
#pragma unroll
        for (int c = 0; c < kCh; ++c) {
            const uint2 q = codes(&h[4 * c], f);
            if constexpr (kAny) {
                if (within(c) > 0) put8(p.out8 + r0 * p.out8_stride + span(c), within(c), q, stage);
            } else if (in[c]) {
                *reinterpret_cast<uint2*>(p.out8 + r0 * p.out8_stride + (c * T + tid) * 8) = q;
            }
        }
    }
}

// kX: type of x.  kR: type of the residual, or -1 for none.  kWide: rows so long that their threads have
// no registers for loads in flight.  kCodes: out8's scales.  (Kernels of their own: with all three in one, 2048 x 7168
// without codes took 16.1 us that take 14.6 so, 8192 x 7168 in groups 71.6 that take 68.1.)
template <int kX, int kR, int kCh, bool kWide, bool kAny, int kCodes>
__global__ void __launch_bounds__(kWide ? kWideThreads : kThreads, kWide || kR == MOE_F32 ? 1 : 2) norm_kernel(const NormParams p) {
    __shared__ float red[4 * 32];
    __shared__ __align__(16) uint8_t staging[kAny ? (kWide ? kWideThreads : kThreads) * 32 : 16];
    constexpr int kRT = kR < 0 ? kX : kR;
    const int T = blockDim.x, tid = threadIdx.x;
    uint8_t* stage = staging + (kAny ? (threadIdx.y * T + tid) / 32 * 1024 : 0);
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
    using RawX = std::conditional_t<kAny, Around8<kX>, Raw8<kX>>;
    using RawR = std::conditional_t<kAny, Around8<kRT>, Raw8<kRT>>;
    auto load = [&](int c, RawX& a, RawR& b) {
        const int at = (c * T + tid) * 8;
        if constexpr (kAny) {
            load_around<kX>(a, x, at, p.H);
            if constexpr (kR >= 0) load_around<kRT>(b, res, at, p.H);
        } else {
            load8<kX>(a, x, at);
            if constexpr (kR >= 0) load8<kRT>(b, res, at);
        }
    };
    RawX xr[kCh];
    RawR rr[kR < 0 ? 1 : kCh];
    const uint8_t* w = reinterpret_cast<const uint8_t*>(p.w);
    auto load_w16 = [&](int c) {
        if constexpr (kAny) {
            Around8<MOE_BF16> r;
            load_around<MOE_BF16>(r, w, (c * T + tid) * 8, p.H);
            return cut_around<MOE_BF16>(r, w).v[0];
        } else {
            return __ldg(reinterpret_cast<const uint4*>(w) + (c * T + tid));
        }
    };
    auto load_w32 = [&](int c) {
        Raw8<MOE_F32> r;
        if constexpr (kAny) {
            Around8<MOE_F32> a;
            load_around<MOE_F32>(a, w, (c * T + tid) * 8, p.H);
            r = cut_around<MOE_F32>(a, w);
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) r.v[i] = __ldg(reinterpret_cast<const uint4*>(w) + 2 * (c * T + tid) + i);
        }
        return r;
    };
    uint4 wr = make_uint4(0u, 0u, 0u, 0u);
    if constexpr (!kWide) {
#pragma unroll
        for (int c = 0; c < kCh; ++c)
            if (in[c]) load(c, xr[c], rr[kR < 0 ? 0 : c]);
        if (kCh == 1 && in[0] && p.w && p.w_type != MOE_F32) wr = load_w16(0);
    }
    norm_row<kX, kR, kCh, kAny, kCodes>(
        p, row, live, T, in, red, stage,
        [&](int c, Raw8<kX>& a, Raw8<kRT>& b) {
            if constexpr (kWide) load(c, xr[0], rr[0]);
            const int i = kWide ? 0 : c;
            if constexpr (kAny) {
                a = cut_around<kX>(xr[i], x);
                if constexpr (kR >= 0) b = cut_around<kRT>(rr[i], res);
            } else {
                a = xr[i];
                if constexpr (kR >= 0) b = rr[i];
            }
        },
        [&](int c) { return kCh == 1 ? wr : load_w16(c); }, load_w32);
}

// ---------------------------------------------------------------- launches

template <int kX, int kR, int kCodes>
cudaError_t launch_types(const NormParams& p, bool chunks, int num_sms, cudaStream_t st) {
    const int n8 = (p.H + 7) / 8;
    auto threads = [&](int ch) { return ((n8 + ch - 1) / ch + 31) / 32 * 32; };
    auto go = [&](auto kern, int ch) {
        const int T = threads(ch), rows = T == 32 ? std::min(p.n, 8) : 1;
        launch_pdl(kern, dim3((unsigned)(((int64_t)p.n + rows - 1) / rows)), dim3(T, rows), 0, st, p);
        return cudaGetLastError();
    };
    // Chunks of a thread: one while the rows' threads all run at once, else as many as its registers
    // hold (two of two fp32 rows, and where each comes with its neighbours, but without a residual four: 8000 rows
    // of 1001 11.6 us against 13.9 with two).
    constexpr int kMost = kX == MOE_F32 && kR == MOE_F32 ? 2 : 4;
    constexpr int kMostAny = kR < 0 && kX != MOE_F32 ? 4 : 2;
    const int most = chunks ? kMost : kMostAny;
    int ch = 1;
    while (threads(ch) > kThreads) ch *= 2;
    while (ch < most && (int64_t)p.n * threads(ch) > (int64_t)num_sms * 2048) ch *= 2;
    if (!chunks) {
        if (ch > most) return go(norm_kernel<kX, kR, 4, true, true, kCodes>, 4);
        if constexpr (kMostAny == 4) if (ch == 4) return go(norm_kernel<kX, kR, 4, false, true, kCodes>, 4);
        return ch == 1 ? go(norm_kernel<kX, kR, 1, false, true, kCodes>, 1) : go(norm_kernel<kX, kR, 2, false, true, kCodes>, 2);
    }
    if (ch > most) return go(norm_kernel<kX, kR, 4, true, false, kCodes>, 4);
    if (ch == 1) return go(norm_kernel<kX, kR, 1, false, false, kCodes>, 1);
    if (ch == 2) return go(norm_kernel<kX, kR, 2, false, false, kCodes>, 2);
    if constexpr (kMost == 4) return go(norm_kernel<kX, kR, 4, false, false, kCodes>, 4);
    return cudaErrorInvalidValue;
}

template <int kCodes>
cudaError_t launch_codes(const NormParams& p, bool chunks, int num_sms, cudaStream_t st) {
    const bool f32_res = p.res && p.res_type == MOE_F32;
    switch (p.x_type) {
        case MOE_F32:
            return p.res ? launch_types<MOE_F32, MOE_F32, kCodes>(p, chunks, num_sms, st) : launch_types<MOE_F32, -1, kCodes>(p, chunks, num_sms, st);
        case MOE_BF16:
            return !p.res ? launch_types<MOE_BF16, -1, kCodes>(p, chunks, num_sms, st)
                 : f32_res ? launch_types<MOE_BF16, MOE_F32, kCodes>(p, chunks, num_sms, st)
                           : launch_types<MOE_BF16, MOE_BF16, kCodes>(p, chunks, num_sms, st);
        default:
            return !p.res ? launch_types<MOE_F16, -1, kCodes>(p, chunks, num_sms, st)
                 : f32_res ? launch_types<MOE_F16, MOE_F32, kCodes>(p, chunks, num_sms, st)
                           : launch_types<MOE_F16, MOE_F16, kCodes>(p, chunks, num_sms, st);
    }
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
    return !p.out8 ? launch_codes<kNoCodes>(p, chunks, num_sms, st)
         : p.group ? launch_codes<kGroups>(p, chunks, num_sms, st) : launch_codes<kRow>(p, chunks, num_sms, st);
}

}  // namespace moe
