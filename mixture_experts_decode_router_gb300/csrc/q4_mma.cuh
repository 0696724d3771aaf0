// q4_mma.cuh -- products of 4-bit weight tiles with up to 16 vectors on one warp
// (sm_103a), shared by the matrix-vector kernel and the INT4 expert kernels.
//
// A decode product reads each weight once and multiplies it with a handful of
// tokens: at 6.8 TB/s of 4-bit codes a GB300 has ~2.7 lane instructions for each
// weight, so what bounds it after HBM is the instructions between the load and
// the multiply.  The codes therefore go from shared memory straight into the
// registers of a warp-level m16n8k16 MMA (16 weight rows, 8 tokens), which does
// the multiplying and the summing over lanes; a tcgen05 tile of 128 rows would
// first have to be written, dequantised, to tensor memory.
//
//  * A warp owns 16 weight rows and walks its K range in stages of 256 codes
//    (128 bytes a row, 2 KB), which it copies itself, some stages ahead, with
//    16-byte cp.async (zero-filled past the matrix).  Warps share nothing but x.
//  * 16-byte chunk c of row r sits at chunk c ^ (r & 7), so the fragment reads
//    below touch every bank once.
//  * The order of K inside an MMA is free as long as both operands agree: lane
//    (g, t) takes the word of codes 32 j + 8 t .. + 7 of rows g and g + 8, so one
//    word of each row feeds two MMAs and all 32 codes of a step lie in one group.
//    Its nibbles i and i + 4 form one 16-bit pair (INT4), so x is stored with
//    the elements of every 8 in the order 0 4 1 5 2 6 3 7.
//  * INT4 value = (q - z) s: q goes under the exponent of 128 (bf16) or of 1024 and
//    64 (f16), the well-known way from small integers to floats without a conversion;
//    less that exponent's value + z is the exact difference; the MMA sums
//    a group in fp32, and s multiplies that sum in fp32.  No weight is rounded, and
//    x enters as it is.  (Measured and not kept: masked codes as f16 subnormals with
//    -z taken away by a second MMA, or by the groups' sums of x, after scaling x
//    into range: as many instructions, and the scaling of x on top.  The same with a
//    scale and a sum of x for each group: 354 instead of 417 instructions a stage, 15%
//    fewer, in the same time.  Codes as e4m3 numbers in m16n8k32 MMAs: those run as two
//    f16 MMAs and conversions of both operands, 800 instructions a stage.)
//  * What bounds it: about 420 warp instructions a stage (16 x 256 codes) with groups of
//    32, at 0.6 an SM's scheduler and cycle; the ALU pipe is 36-45% busy, the tensor pipe
//    15%, DRAM 40%.
//  * NVFP4: e2m1 times e4m3 is exact in f16; scale2 multiplies the result.  bf16
//    rows of x are scaled by a power of two that puts their largest value below
//    2^15 (exact for elements down to 2^-32 of it; below, they round at 2^-40 of
//    it) and the results scaled back.
#pragma once

#include <cuda_fp16.h>

#include "moe_internal.cuh"

namespace moe {
namespace q4 {

constexpr int kStageK = 256;          // codes of a row in a stage
constexpr int kStageBytes = 16 * 128;

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// The same, with zeros when !valid (src is not read then).
__device__ __forceinline__ void cp16_or_zero(uint32_t dst, const void* src, bool valid) {
    const int n = valid ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// A lane's part of the copies of 16 weight rows: rows lane / 8 + 4 i, chunk lane % 8
// of one stage after another.
struct RowCopy {
    const uint8_t* src;    // row lane / 8, chunk lane % 8 of the next stage
    int rows;              // rows of the tile inside the matrix
    uint32_t d0;           // lane's place in a stage; row r + 4's chunk is the other of bit 2
    __device__ __forceinline__ void start(const uint8_t* w, int64_t row, int rows_left, int row_bytes, int s, int lane) {
        const int r0 = lane >> 3;
        src = w + (row + r0) * row_bytes + s * 128 + (lane & 7) * 16;
        rows = rows_left;
        d0 = r0 * 128 + (((lane & 7) ^ r0) << 4);
    }
    // The next stage, number s, into dst; `step` stages on after it.  full_stages:
    // stages that lie inside the row.
    __device__ __forceinline__ void issue(uint32_t dst, int s, int step, int row_bytes, int full_stages,
                                          const uint8_t* any, int lane) {
        const uint32_t d = dst + d0, e = dst + (d0 ^ 64u);
        const size_t r4 = (size_t)(4 * row_bytes);
        if (rows >= 16 && s < full_stages) {
            cp16(d, src);
            cp16(e + 512, src + r4);
            cp16(d + 1024, src + 2 * r4);
            cp16(e + 1536, src + 3 * r4);
        } else {
            const bool in = s * 128 + (lane & 7) * 16 < row_bytes;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const bool ok = in && (lane >> 3) + 4 * i < rows;
                cp16_or_zero(((i & 1) ? e : d) + 512 * i, ok ? src + i * r4 : any, ok);
            }
        }
        src += step * 128;
    }
};

// d += A B, or (FIRST) d = A B; 16-bit operands bf16 (BF) or f16, fp32 sums.
template <bool BF, bool FIRST>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    if constexpr (FIRST) {
        if constexpr (BF)
            asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                         : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                         : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
        else
            asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                         : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                         : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
    } else {
        if constexpr (BF)
            asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                         : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                         : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
        else
            asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                         : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                         : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    }
}

__device__ __forceinline__ uint32_t lop_and_or(uint32_t a, uint32_t mask, uint32_t orv) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(a), "r"(mask), "r"(orv));   // (a & mask) | orv
    return d;
}

// The eight codes of w less the zero point, as pairs (i, i + 4), exact.  zz: two
// copies of 128 + z (bf16) or 1024 + z (f16); z64 (f16): of 64 + z.  In f16 a
// nibble in bits 4-7 under the exponent of 64 is 64 + q, which saves two shifts.
template <bool BF>
__device__ __forceinline__ void int4_pairs(uint32_t w, uint32_t zz, uint32_t z64, uint32_t (&p)[4]) {
    if constexpr (BF) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t v = lop_and_or(w >> (4 * i), 0x000f000fu, 0x43004300u);
            asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(p[i]) : "r"(v), "r"(zz));
        }
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t v = w >> (8 * h);
            asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(p[2 * h]) : "r"(lop_and_or(v, 0x000f000fu, 0x64006400u)), "r"(zz));
            asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(p[2 * h + 1]) : "r"(lop_and_or(v, 0x00f000f0u, 0x54005400u)), "r"(z64));
        }
    }
}
// Two copies of 128 (bf16) or 1024 (f16), to whose last places z is added.
template <bool BF> constexpr uint32_t kZeroBase = BF ? 0x43004300u : 0x64006400u;
// Two copies of 64 + z from those of 1024 + z.
__device__ __forceinline__ constexpr uint32_t zero64(uint32_t zz) { return zz * 16u + (0x54005400u - 0x64006400u * 16u); }

// NVFP4: the eight codes of w (pairs of neighbours) times the block scale, exact in f16.
__device__ __forceinline__ void nvfp4_pairs(uint32_t w, uint32_t s2, uint32_t (&p)[4]) {
    asm("{ .reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3; }"
        : "=r"(p[0]), "=r"(p[1]), "=r"(p[2]), "=r"(p[3])
        : "r"(w));
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(p[i]) : "r"(s2));
}

// Scales of one stage (and INT4 zero points) as this lane holds them, loaded a
// stage ahead and left as loaded until the stage is multiplied.  GSH: log2 of the
// INT4 group, or 4 for NVFP4; Z: zero points.
//  INT4: lane (g, t) holds groups t, t + 4, .. of the stage for rows g, g + 8; a
//    group's values are shuffled from lane t.
//  NVFP4: all sixteen block scales of the two rows, four words each.
template <int GSH, bool Z> struct StageScales {
    static constexpr int kGroups = kStageK >> GSH;            // groups of a stage
    static constexpr int kHold = GSH == 4 ? 4 : (kGroups + 3) / 4;
    uint32_t v[2][kHold], z[2][Z ? kHold : 1];
};

// A lane's part of the loads of a tile's scales, one stage after another.
template <int GSH, bool Z> struct ScaleLoad {
    using S = StageScales<GSH, Z>;
    const uint8_t* sp;     // first value of the lane (INT4: group t of row g; NVFP4: block 0 of row g)
    const uint8_t* zp;
    bool has_zero;         // (Z kernels take matrices without zero points too)
    int rows;              // rows of the tile inside the matrix
    // row: the tile's first row in the stack.
    __device__ __forceinline__ void start(const QMatDev& m, int64_t row, int rows_left, int s, int lane) {
        const int g = lane >> 2, t = GSH == 4 ? 0 : lane & 3;
        const size_t at = (size_t)(row + g) * (m.in_dim >> GSH) + s * S::kGroups + t;
        sp = reinterpret_cast<const uint8_t*>(m.scale) + (GSH == 4 ? at : 2 * at);
        if constexpr (Z) {
            has_zero = m.zero != nullptr;
            zp = m.zero + (has_zero ? at : 0);
        }
        rows = rows_left;
    }
    // The next stage, number s; `step` stages on after it.
    __device__ __forceinline__ void load(S& o, int s, int step, int in_dim, int lane) {
        const int g = lane >> 2, t = lane & 3, per_row = in_dim >> GSH;
        const int left = per_row - s * S::kGroups;               // groups of the row from this stage on
        if constexpr (GSH == 4) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint8_t* q8 = sp + (size_t)(8 * h) * per_row;
                const bool in = g + 8 * h < rows;
                if ((in_dim & 255) == 0) {   // rows of whole stages: 4-byte aligned words
#pragma unroll
                    for (int q = 0; q < 4; ++q) o.v[h][q] = in ? __ldg(reinterpret_cast<const uint32_t*>(q8) + q) : 0u;
                } else {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint32_t u = 0;
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (in && 4 * q + i < left) u |= (uint32_t)__ldg(q8 + 4 * q + i) << (8 * i);
                        o.v[h][q] = u;
                    }
                }
            }
            sp += step * S::kGroups;
        } else {
            const unsigned short* s16 = reinterpret_cast<const unsigned short*>(sp);
            if (rows >= 16 && left >= S::kGroups) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int q = 0; q < S::kHold; ++q)
                        if (S::kGroups >= 4 || t < S::kGroups) {
                            o.v[h][q] = __ldg(s16 + (size_t)(8 * h) * per_row + 4 * q);
                            if constexpr (Z) o.z[h][q] = has_zero ? __ldg(zp + (size_t)(8 * h) * per_row + 4 * q) : 8;
                        }
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int q = 0; q < S::kHold; ++q) {
                        const bool ok = g + 8 * h < rows && t + 4 * q < S::kGroups && t + 4 * q < left;
                        o.v[h][q] = ok ? (uint32_t)__ldg(s16 + (size_t)(8 * h) * per_row + 4 * q) : 0u;
                        if constexpr (Z) o.z[h][q] = ok && has_zero ? (uint32_t)__ldg(zp + (size_t)(8 * h) * per_row + 4 * q) : 8u;
                    }
            }
            sp += step * (2 * S::kGroups);
            if constexpr (Z) if (has_zero) zp += step * S::kGroups;
        }
    }
};

// What a warp's lanes read of the vectors, as offsets from the block's shared
// memory: chunk t of tokens g (and g + 8).  Past the last token a lane reads the
// last one's row again: its column of the result is not used.
template <int NT> struct XView {
    uint32_t at[NT];
    __device__ __forceinline__ void start(uint32_t x0, int xstride, int ntok, int lane) {
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int q = 0; q < NT; ++q) at[q] = x0 + min(8 * q + g, ntok - 1) * xstride + t * 16;
    }
};

// One stage of one matrix: acc[NT] += (16 rows x 256 codes at offset st) x (256
// elements of each of 8 NT tokens, stage s of the view).
template <int GSH, bool Z, bool BF, int NT>
__device__ __forceinline__ void mma_stage(const uint8_t* sm, uint32_t st, const XView<NT>& x, int s,
                                          const StageScales<GSH, Z>& sc, float (&acc)[NT][4], int lane) {
    const int g = lane >> 2, t = lane & 3;
    const uint32_t w_at = st + g * 128 + (g << 4) + 4 * t;
    uint32_t xa[NT];
#pragma unroll
    for (int q = 0; q < NT; ++q) xa[q] = x.at[q] + (uint32_t)s * (2 * kStageK);
    float d[NT][4];
    uint32_t zz[2] = {kZeroBase<BF> + 0x00080008u, kZeroBase<BF> + 0x00080008u}, z64[2] = {zero64(zz[0]), zero64(zz[1])};
    // Rows g and g + 8 of each held group in one word.
    constexpr int kHold = StageScales<GSH, Z>::kHold;
    uint32_t ps[kHold], pz[kHold];
    if constexpr (GSH != 4) {
#pragma unroll
        for (int q = 0; q < kHold; ++q) {
            ps[q] = __byte_perm(sc.v[0][q], sc.v[1][q], 0x5410);
            if constexpr (Z) pz[q] = __byte_perm(sc.z[0][q], sc.z[1][q], 0x5410) + kZeroBase<BF>;
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t w0 = *reinterpret_cast<const uint32_t*>(sm + (w_at ^ (uint32_t)(j << 4)));
        const uint32_t w1 = *reinterpret_cast<const uint32_t*>(sm + (w_at ^ (uint32_t)(j << 4)) + 1024);
        uint4 b[NT];
#pragma unroll
        for (int q = 0; q < NT; ++q) b[q] = *reinterpret_cast<const uint4*>(sm + xa[q] + j * 64);
        uint32_t p0[4], p1[4];
        if constexpr (GSH == 4) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                // Block 2 j + t / 2: byte 2 (j & 1) + t / 2 of word j / 2, twice.
                const uint32_t by = __byte_perm(sc.v[h][j >> 1], 0u, (2 * (j & 1) + (t >> 1)) * 0x11);
                uint32_t s2;
                asm("{ .reg .b16 c; cvt.u16.u32 c, %1; cvt.rn.f16x2.e4m3x2 %0, c; }" : "=r"(s2) : "r"(by));
                if (h == 0) nvfp4_pairs(w0, s2, p0);
                else nvfp4_pairs(w1, s2, p1);
            }
#pragma unroll
            for (int q = 0; q < NT; ++q) {
                mma16816<BF, false>(acc[q], p0[0], p1[0], p0[1], p1[1], b[q].x, b[q].y);
                mma16816<BF, false>(acc[q], p0[2], p1[2], p0[3], p1[3], b[q].z, b[q].w);
            }
        } else {
            constexpr int kPer = (1 << GSH) / 32;   // steps of a group
            const int grp = j / kPer, from = (lane & 28) | (grp & 3);
            if constexpr (Z) {
                if (j % kPer == 0) {
                    const uint32_t u = __shfl_sync(0xffffffffu, pz[grp / 4], from);
                    zz[0] = __byte_perm(u, 0u, 0x1010);
                    zz[1] = __byte_perm(u, 0u, 0x3232);
                    if constexpr (!BF) {
                        z64[0] = zero64(zz[0]);
                        z64[1] = zero64(zz[1]);
                    }
                }
            }
            int4_pairs<BF>(w0, zz[0], z64[0], p0);
            int4_pairs<BF>(w1, zz[1], z64[1], p1);
#pragma unroll
            for (int q = 0; q < NT; ++q) {
                if (j % kPer == 0) mma16816<BF, true>(d[q], p0[0], p1[0], p0[1], p1[1], b[q].x, b[q].y);
                else mma16816<BF, false>(d[q], p0[0], p1[0], p0[1], p1[1], b[q].x, b[q].y);
                mma16816<BF, false>(d[q], p0[2], p1[2], p0[3], p1[3], b[q].z, b[q].w);
            }
            if (j % kPer == kPer - 1) {
                const uint32_t u = __shfl_sync(0xffffffffu, ps[grp / 4], from);
                const float fs[2] = {__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u)};
#pragma unroll
                for (int q = 0; q < NT; ++q)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[q][i] = fmaf(fs[i >> 1], d[q][i], acc[q][i]);
            }
        }
    }
}

// Bytes between token rows in shared memory: whole stages of 16-bit elements, and
// 64 bytes so that neighbouring rows' chunks fall into different banks.
__host__ __device__ inline int x_row_bytes(int K) { return (K + kStageK - 1) / kStageK * (2 * kStageK) + 64; }
// The eight 16-bit elements of a chunk in the order the fragments take them.
template <int GSH>
__device__ __forceinline__ uint4 chunk_order(uint4 u) {
    if constexpr (GSH == 4) return u;
    return make_uint4(__byte_perm(u.x, u.z, 0x5410), __byte_perm(u.x, u.z, 0x7632), __byte_perm(u.y, u.w, 0x5410),
                      __byte_perm(u.y, u.w, 0x7632));
}

// One bf16 row as f16, scaled by a power of two, by one warp: dst [chunks] (zero
// past K); returns the factor that scales a result back.  kU: loads of a lane in
// flight; a row of at most 32 kU chunks is read once.
template <int kU>
__device__ __forceinline__ float scaled_row(const uint4* src, int K8, int chunks, uint4* dst, int lane) {
    uint4 u[kU];
    auto load = [&](int c0) {
#pragma unroll
        for (int i = 0; i < kU; ++i) {
            const int c = c0 + 32 * i + lane;
            u[i] = c < K8 ? src[c] : make_uint4(0u, 0u, 0u, 0u);
        }
    };
    auto largest = [&](bool finite) {
        float am = 0.f;
        for (int c0 = 0; c0 < K8; c0 += 32 * kU) {
            load(c0);
#pragma unroll
            for (int i = 0; i < kU; ++i) {
                float v[8];
                bf16x8_to_float(u[i], v);
#pragma unroll
                for (int e = 0; e < 8; ++e) {   // (NaN keeps its column NaN by itself)
                    const float a = fabsf(v[e]);
                    am = fmaxf(am, finite && a == INFINITY ? 0.f : a);
                }
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
        return am;
    };
    float am = largest(false);
    if (am == INFINITY) am = largest(true);   // an infinity stays one at any scale; the rest has to stay finite
    const int sh = f16_shift(am);
    const float f = exp2i(sh);
    for (int c0 = 0; c0 < chunks; c0 += 32 * kU) {
        if (K8 > 32 * kU) load(c0);
#pragma unroll
        for (int i = 0; i < kU; ++i) {
            const int c = c0 + 32 * i + lane;
            float v[8];
            bf16x8_to_float(u[i], v);
            uint32_t h[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const __half2 hv = __floats2half2_rn(v[2 * e] * f, v[2 * e + 1] * f);
                h[e] = *reinterpret_cast<const uint32_t*>(&hv);
            }
            if (c < chunks) dst[c] = make_uint4(h[0], h[1], h[2], h[3]);
        }
    }
    return exp2i(-sh);
}

}  // namespace q4
}  // namespace moe
