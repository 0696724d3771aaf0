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
//    (128 bytes a row, 2 KB), which it copies itself, several stages ahead, with
//    16-byte cp.async (zero-filled past the matrix).  Warps share nothing but x.
//  * 16-byte chunk c of row r sits at chunk c ^ (r & 7), so the fragment reads
//    below touch every bank once.
//  * The order of K inside an MMA is free as long as both operands agree: lane
//    (g, t) takes the word of codes 32 j + 8 t .. + 7 of rows g and g + 8, so one
//    word of each row feeds two MMAs and all 32 codes of a step lie in one group.
//    Its nibbles i and i + 4 form one 16-bit pair (INT4), so x is stored with
//    the elements of every 8 in the order 0 4 1 5 2 6 3 7.
//  * INT4 value = (q - z) s: q goes under the exponent of 128 (bf16) or 1024
//    (f16), less 128 + z (1024 + z) is the exact difference; the MMA sums a
//    group in fp32, and s multiplies that sum in fp32.  Nothing is rounded.
//  * NVFP4 value = e2m1 e4m3 scale2: the product of the two small floats is exact
//    in f16; scale2 multiplies the result.
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
// 16 bytes global -> shared; zeros when !valid (src is not read then).
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool valid) {
    const int n = valid ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Weight rows row0 .. row0 + 15 of the matrix whose code rows (`row_bytes` each)
// start at w: the 128 bytes of stage s, into dst (swizzled).
__device__ __forceinline__ void load_stage(uint32_t dst, const uint8_t* w, int row0, int rows, int row_bytes, int s,
                                           int lane) {
    const int c = lane & 7, byte = s * 128 + c * 16;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * i + (lane >> 3);
        const bool ok = row0 + r < rows && byte < row_bytes;
        cp16(dst + r * 128 + ((c ^ (r & 7)) << 4), ok ? w + (size_t)(row0 + r) * row_bytes + byte : w, ok);
    }
}

template <bool BF>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    if constexpr (BF)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t lop_and_or(uint32_t a, uint32_t mask, uint32_t orv) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(a), "r"(mask), "r"(orv));   // (a & mask) | orv
    return d;
}

// The eight codes of w less the zero point, as pairs (i, i + 4), exact.  zz: two
// copies of 128 + z (bf16) or 1024 + z (f16).
template <bool BF>
__device__ __forceinline__ void int4_pairs(uint32_t w, uint32_t zz, uint32_t (&p)[4]) {
    if constexpr (BF) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t v = lop_and_or(w >> (4 * i), 0x000f000fu, 0x43004300u);
            asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(p[i]) : "r"(v), "r"(zz));
        }
    } else {
        // A nibble in bits 4-7 is 16 q under the exponent of 1024: (1024 + 16 q) / 16
        // - (64 + z) = q - z, exact, and saves the shift.
        const uint32_t w8 = w >> 8;
        uint32_t zh;   // 64 + z = (1024 + z) - 960
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(zh) : "r"(zz), "r"(0x63806380u));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t v = h ? w8 : w;
            const uint32_t lo = lop_and_or(v, 0x000f000fu, 0x64006400u);
            const uint32_t hi = lop_and_or(v, 0x00f000f0u, 0x64006400u);
            asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(p[2 * h]) : "r"(lo), "r"(zz));
            asm("{ .reg .b32 n; neg.f16x2 n, %2; fma.rn.f16x2 %0, %1, %3, n; }"
                : "=r"(p[2 * h + 1]) : "r"(hi), "r"(zh), "r"(0x2c002c00u));
        }
    }
}

// Two copies of 128 + z (bf16) or 1024 + z (f16).
template <bool BF>
__device__ __forceinline__ uint32_t zero_pair(uint32_t z) {
    if constexpr (BF) {
        const __nv_bfloat162 v = __float2bfloat162_rn((float)(128u + z));
        return *reinterpret_cast<const uint32_t*>(&v);
    } else {
        const __half2 v = __float2half2_rn((float)(1024u + z));
        return *reinterpret_cast<const uint32_t*>(&v);
    }
}

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
// stage ahead.  GSH: log2 of the INT4 group, or 4 for NVFP4.
//  INT4: lane (g, t) holds groups t, t + 4, .. of the stage for rows g, g + 8, as
//    (bf16 scale << 16) | zero point; a group's value is shuffled from lane t.
//  NVFP4: the blocks of the lane's own words, 2 j + t / 2: e4m3 bytes, eight a row.
template <int GSH> struct StageScales {
    static constexpr int kGroups = kStageK >> GSH;            // groups of a stage
    static constexpr int kHold = GSH == 4 ? 2 : (kGroups + 3) / 4;
    uint32_t v[2][kHold];

    __device__ __forceinline__ void load(const QMatDev& m, size_t row_base, int row0, int rows, int s, int lane) {
        const int g = lane >> 2, t = lane & 3, per_row = m.in_dim >> GSH;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int row = row0 + g + 8 * h;
            const size_t at = (row_base + row) * per_row + (size_t)s * kGroups;
            if constexpr (GSH == 4) {
                const uint8_t* sp = reinterpret_cast<const uint8_t*>(m.scale) + at;
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    uint32_t u = 0;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {   // words j = 4 q + i of the stage
                        const int b = 2 * (4 * q + i) + (t >> 1);
                        if (row < rows && s * kGroups + b < per_row) u |= (uint32_t)__ldg(sp + b) << (8 * i);
                    }
                    v[h][q] = u;
                }
            } else {
#pragma unroll
                for (int q = 0; q < kHold; ++q) {
                    const int b = t + 4 * q;
                    uint32_t u = 8u;
                    if (b < kGroups && row < rows && s * kGroups + b < per_row) {
                        u = (uint32_t)__ldg(reinterpret_cast<const unsigned short*>(m.scale) + at + b) << 16;
                        u |= m.zero ? (uint32_t)__ldg(m.zero + at + b) : 8u;
                    }
                    v[h][q] = u;
                }
            }
        }
    }
};

// One stage of one matrix: acc[NT] += (16 rows x 256 codes at st) x (256 elements
// of each of 8 NT tokens).  xs: the chunk of this stage and lane, token row g (row
// stride xstride bytes); ntok: tokens whose rows exist (the others are zero).
template <int GSH, bool BF, int NT>
__device__ __forceinline__ void mma_stage(const uint8_t* st, const uint8_t* xs, int xstride, int ntok,
                                          const StageScales<GSH>& sc, float (&acc)[NT][4], int lane) {
    const int g = lane >> 2, t = lane & 3;
    const uint8_t* wp = st + g * 128 + 4 * t;
    float d[NT][4];
    uint32_t zz[2] = {0u, 0u};
    float fs[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t w0 = *reinterpret_cast<const uint32_t*>(wp + ((j ^ g) << 4));
        const uint32_t w1 = *reinterpret_cast<const uint32_t*>(wp + 1024 + ((j ^ g) << 4));
        uint4 b[NT];
#pragma unroll
        for (int q = 0; q < NT; ++q) {
            b[q] = make_uint4(0u, 0u, 0u, 0u);
            if (8 * q + g < ntok) b[q] = *reinterpret_cast<const uint4*>(xs + (size_t)(8 * q) * xstride + j * 64);
        }
        uint32_t p0[4], p1[4];
        if constexpr (GSH == 4) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t by = (sc.v[h][j >> 2] >> (8 * (j & 3))) & 0xffu;
                uint32_t s2;
                asm("{ .reg .b16 c; cvt.u16.u32 c, %1; cvt.rn.f16x2.e4m3x2 %0, c; }" : "=r"(s2) : "r"(by * 0x101u));
                if (h == 0) nvfp4_pairs(w0, s2, p0);
                else nvfp4_pairs(w1, s2, p1);
            }
#pragma unroll
            for (int q = 0; q < NT; ++q) {
                mma16816<BF>(acc[q], p0[0], p1[0], p0[1], p1[1], b[q].x, b[q].y);
                mma16816<BF>(acc[q], p0[2], p1[2], p0[3], p1[3], b[q].z, b[q].w);
            }
        } else {
            constexpr int kPer = (1 << GSH) / 32;   // steps of a group
            if (j % kPer == 0) {
                const int grp = j / kPer;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t u = __shfl_sync(0xffffffffu, sc.v[h][grp / 4], (lane & 28) | (grp & 3));
                    fs[h] = __uint_as_float(u & 0xffff0000u);
                    zz[h] = zero_pair<BF>(u & 0xffu);
                }
#pragma unroll
                for (int q = 0; q < NT; ++q)
#pragma unroll
                    for (int i = 0; i < 4; ++i) d[q][i] = 0.f;
            }
            int4_pairs<BF>(w0, zz[0], p0);
            int4_pairs<BF>(w1, zz[1], p1);
#pragma unroll
            for (int q = 0; q < NT; ++q) {
                mma16816<BF>(d[q], p0[0], p1[0], p0[1], p1[1], b[q].x, b[q].y);
                mma16816<BF>(d[q], p0[2], p1[2], p0[3], p1[3], b[q].z, b[q].w);
            }
            if (j % kPer == kPer - 1)
#pragma unroll
                for (int q = 0; q < NT; ++q)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[q][i] = fmaf(fs[i >> 1], d[q][i], acc[q][i]);
        }
    }
}

// The eight 16-bit elements of a chunk in the order the fragments take them.
template <int GSH>
__device__ __forceinline__ uint4 chunk_order(uint4 u) {
    if constexpr (GSH == 4) return u;
    return make_uint4(__byte_perm(u.x, u.z, 0x5410), __byte_perm(u.x, u.z, 0x7632), __byte_perm(u.y, u.w, 0x5410),
                      __byte_perm(u.y, u.w, 0x7632));
}

// Bytes between token rows in shared memory: whole stages of 16-bit elements, and
// 64 bytes so that neighbouring rows' chunks fall into different banks.
__host__ __device__ inline int x_row_bytes(int K) { return (K + kStageK - 1) / kStageK * (2 * kStageK) + 64; }

// 2^e as a float, e in [-126, 127].
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// The power of two that takes values of magnitude at most amax into f16 with the
// largest below 2^15 (1 for zero, infinite or NaN amax), as an exponent.
__device__ __forceinline__ int f16_shift(float amax) {
    const int e = (int)(__float_as_uint(amax) >> 23) & 0xff;
    if (amax == 0.f || e == 255) return 0;
    return min(126, 14 - (e - 127));
}

}  // namespace q4
}  // namespace moe
