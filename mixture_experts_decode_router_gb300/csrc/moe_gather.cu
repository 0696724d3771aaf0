// moe_gather.cu -- the grouped path's small memory-bound kernels around the
// tensor-core GEMMs (sm_103a): gathering the token rows into expert order
// before them, and combining the weighted expert rows after them.
#include <algorithm>

#include "moe_launch.cuh"

namespace moe {

namespace {

// xs[p, :] = x[perm[p] / k, :] for the grouped routes, and xh = x (the shared
// expert's operand); 16-bit values as the tiles take them (F16: f16 for the FP8
// and NVFP4 tiles, else bf16).  The tensor-core kernels' TMA copies therefore
// read only workspace buffers: x itself is read here with plain loads, so it
// may also live in pinned host memory.
template <bool F16>
__device__ __forceinline__ uint4 to_tile16(uint4 v) {
    if constexpr (F16) {
        uint32_t w4[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float lo = __uint_as_float(w4[q] << 16), hi = __uint_as_float(w4[q] & 0xffff0000u);
            w4[q] = pack_f16_sat(lo, hi);
        }
        return make_uint4(w4[0], w4[1], w4[2], w4[3]);
    }
    return v;
}

// One warp per destination row (the row's source index read once), its lanes
// taking 16-byte chunks lane, lane + 32, ...: kU chunks per lane loaded before
// any is stored, so a row costs one round of load latency, not one per chunk.
// With a pre-expert RMSNorm weight nw, the rows copied are the normalised ones,
// with the norm kernel's arithmetic (rms_inv_warp, then rms_apply8): a first
// pass over the row sums its squares in the same chunk order (lane l's chunks
// l, l + 32, ... in order, then the butterfly), so the values are that
// kernel's, bit for bit.  (NORM: whether nw is given -- its own instance, so
// that the plain copy keeps its small register count.)
template <bool F16, bool NORM>
__global__ void __launch_bounds__(256) gather_kernel(const uint16_t* __restrict__ x, int n, int H, int k,
                                                     const int32_t* __restrict__ perm,
                                                     const int32_t* __restrict__ offsets, int E,
                                                     uint16_t* __restrict__ xs, uint16_t* __restrict__ xh,
                                                     const uint16_t* __restrict__ nw, float eps, int early) {
    constexpr int kU = 8;
    pdl_wait();
    if (early) pdl_trigger();
    const int n_routes = offsets[E];
    const int rows = n_routes + n;
    const int C8 = H >> 3;
    const int lane = threadIdx.x & 31;
    const int nwarps = gridDim.x * (blockDim.x >> 5);
    for (int r = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); r < rows; r += nwarps) {
        const bool routed = r < n_routes;
        const int t = routed ? perm[r] / k : r - n_routes;
        const uint4* src = reinterpret_cast<const uint4*>(x + (size_t)t * H);
        uint4* dst = reinterpret_cast<uint4*>(routed ? xs + (size_t)r * H : xh + (size_t)(r - n_routes) * H);
        if (NORM && C8 <= 32 * kU) {
            // The whole row in one round: the lane's chunks and their norm
            // weights loaded together, then the sum of squares, then the stores.
            uint4 v[kU], wv[kU];
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const int c = lane + 32 * u;
                if (c < C8) {
                    v[u] = __ldg(src + c);
                    wv[u] = __ldg(reinterpret_cast<const uint4*>(nw) + c);
                }
            }
            float ss = 0.f;
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                if (lane + 32 * u < C8) {
                    float f[8];
                    bf16x8_to_float(v[u], f);
#pragma unroll
                    for (int i = 0; i < 8; ++i) ss = fmaf(f[i], f[i], ss);
                }
            }
            ss = warp_sum(ss);
            const float inv = rsqrtf(ss / (float)H + eps);
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const int c = lane + 32 * u;
                if (c < C8) dst[c] = to_tile16<F16>(rms_apply8(v[u], wv[u], inv));
            }
            continue;
        }
        float inv = 0.f;
        if (NORM) {   // a longer row: its sum of squares first, then the copy below
            float ss = 0.f;
            for (int c0 = lane; c0 < C8; c0 += 32 * kU) {
                uint4 v[kU];
#pragma unroll
                for (int u = 0; u < kU; ++u) {
                    const int c = c0 + 32 * u;
                    if (c < C8) v[u] = __ldg(src + c);
                }
#pragma unroll
                for (int u = 0; u < kU; ++u) {
                    if (c0 + 32 * u < C8) {
                        float f[8];
                        bf16x8_to_float(v[u], f);
#pragma unroll
                        for (int i = 0; i < 8; ++i) ss = fmaf(f[i], f[i], ss);
                    }
                }
            }
            ss = warp_sum(ss);
            inv = rsqrtf(ss / (float)H + eps);
        }
        for (int c0 = lane; c0 < C8; c0 += 32 * kU) {
            uint4 v[kU];
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const int c = c0 + 32 * u;
                if (c < C8) {
                    v[u] = __ldg(src + c);
                    if (NORM) v[u] = rms_apply8(v[u], __ldg(reinterpret_cast<const uint4*>(nw) + c), inv);
                }
            }
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const int c = c0 + 32 * u;
                if (c < C8) dst[c] = to_tile16<F16>(v[u]);
            }
        }
    }
    pdl_trigger();
}

// The same rows for the INT4 tiles: f16 under a power of two each, which puts the row's largest
// finite value below 2^15 and whose exponent goes to exps.  Exact for values down to 2^-29 of it
// (a BF16 value has 8 significand bits), at any magnitude; an infinity stays one.
//
// Beside them, the weight rows' exponents: f16 holds (code - zero point) times a scale, so each
// row's scales are multiplied by the power of two that puts the largest below 2^9 (127 of which
// f16 holds), which the epilogue undoes.  (Scales below 2^-22 of their row's largest lose bits,
// as they would in any one row of f16 operands.)  A warp takes 32 rows of one matrix, of the
// experts that have tokens, as many lanes a row as it has loads of 16 bytes (8 scales; 4 bytes
// where rows are no multiple of 16), four loads of a lane in flight.  768 tokens of hidden 2048,
// 256 experts, groups of 32: the kernel 31 us, the call 411 (4-byte loads: 58 and 436).
__device__ __forceinline__ void weight_row_exps(const WeightRows& wr, const int32_t* __restrict__ active, int n_active) {
    const int lane = threadIdx.x & 31, wpb = blockDim.x >> 5;
    const int per = (2 * wr.I + wr.H) / 32, routed = n_active * per, units = routed + (wr.S > 0 ? (2 * wr.S + wr.H) / 32 : 0);
    for (int unit = blockIdx.x * wpb + (threadIdx.x >> 5); unit < units; unit += gridDim.x * wpb) {
        const bool sh = unit >= routed;
        const int a = sh ? 0 : unit / per, r = (sh ? unit - routed : unit - a * per) * 32, W = sh ? wr.S : wr.I;
        const int m = r < W ? 0 : (r < 2 * W ? 1 : 2);
        // The first row in its matrix's stack.
        const int64_t row0 = (r - m * W) + (sh ? 0 : (int64_t)(__ldg(active + a) - wr.e_begin) * (m < 2 ? W : wr.H));
        const int ng = (m < 2 ? wr.H : W) >> wr.gshift;
        const uint16_t* s = (m == 0 ? (sh ? wr.sh_scale[0] : wr.scale[0]) : m == 1 ? (sh ? wr.sh_scale[1] : wr.scale[1])
                                                                           : (sh ? wr.sh_scale[2] : wr.scale[2])) + row0 * ng;
        int8_t* out = wr.exps + (sh ? wr.shared(m) : wr.routed(m)) + row0;
        const bool vec = ng % 8 == 0 && reinterpret_cast<uintptr_t>(s) % 16 == 0;
        const int words = vec ? ng / 8 : (ng + 1) / 2;   // loads of a row
        const int lg = words >= 32 ? 5 : 32 - __clz(words - 1), lanes = 1 << lg, l = lane & (lanes - 1);   // (words >= 1)
        for (int q0 = 0; q0 < lanes; q0 += 4) {
            uint32_t am[4] = {0u, 0u, 0u, 0u};   // magnitude bits; those of an infinity or NaN count as 0
            for (int w = l; w < words; w += lanes) {
                uint4 b[4];
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const uint16_t* p = s + (size_t)(((q0 + v) << (5 - lg)) + (lane >> lg)) * ng + (vec ? 8 : 2) * w;
                    b[v] = make_uint4(0u, 0u, 0u, 0u);
                    if (q0 + v >= lanes) continue;
                    if (vec) b[v] = __ldg(reinterpret_cast<const uint4*>(p));
                    else if (ng % 2 == 0) b[v].x = __ldg(reinterpret_cast<const uint32_t*>(p));   // (4-byte aligned arrays)
                    else b[v].x = __ldg(p) | (2 * w + 1 < ng ? (uint32_t)__ldg(p + 1) << 16 : 0u);
                }
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const uint32_t b4[4] = {b[v].x, b[v].y, b[v].z, b[v].w};
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint32_t lo = b4[q] & 0x7fffu, hi = (b4[q] >> 16) & 0x7fffu;
                        am[v] = max(am[v], max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
                    }
                }
            }
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                for (int o = 1; o < lanes; o <<= 1) am[v] = max(am[v], __shfl_xor_sync(0xffffffffu, am[v], o));
                if (l == 0 && q0 + v < lanes)
                    out[((q0 + v) << (5 - lg)) + (lane >> lg)] = am[v] == 0u ? 0 : (int8_t)min(126, 8 - ((int)(am[v] >> 7) - 127));
            }
        }
    }
}

template <bool NORM>
__global__ void __launch_bounds__(256) gather_scaled_kernel(const uint16_t* __restrict__ x, int n, int H, int k,
                                                            const int32_t* __restrict__ perm,
                                                            const int32_t* __restrict__ offsets, int E,
                                                            uint16_t* __restrict__ xs, uint16_t* __restrict__ xh,
                                                            const uint16_t* __restrict__ nw, float eps,
                                                            int32_t* __restrict__ exps, const WeightRows wr,
                                                            const int32_t* __restrict__ active,
                                                            const Ctrl* __restrict__ ctrl, int early) {
    constexpr int kU = NORM ? 4 : 8;
    pdl_wait();
    if (early) pdl_trigger();
    const int n_routes = offsets[E], rows = n_routes + n, C8 = H >> 3;
    const int lane = threadIdx.x & 31, nwarps = gridDim.x * (blockDim.x >> 5);
    for (int r = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); r < rows; r += nwarps) {
        const bool routed = r < n_routes;
        const int t = routed ? perm[r] / k : r - n_routes;
        const uint4* src = reinterpret_cast<const uint4*>(x + (size_t)t * H);
        uint4* dst = reinterpret_cast<uint4*>(routed ? xs + (size_t)r * H : xh + (size_t)(r - n_routes) * H);
        const float inv = NORM ? rms_inv_warp(reinterpret_cast<const uint16_t*>(src), H, eps, lane) : 0.f;
        uint4 v[kU];
        auto load = [&](int c0) {
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const int c = c0 + 32 * u;
                v[u] = c < C8 ? __ldg(src + c) : make_uint4(0u, 0u, 0u, 0u);
            }
            if constexpr (NORM) {
#pragma unroll
                for (int u = 0; u < kU; ++u) {
                    const int c = c0 + 32 * u;
                    if (c < C8) v[u] = rms_apply8(v[u], __ldg(reinterpret_cast<const uint4*>(nw) + c), inv);
                }
            }
        };
        // The largest finite magnitude, of BF16 bits: those of an infinity or NaN count as 0.
        uint32_t am = 0u;
        for (int c0 = lane; c0 < C8 + lane; c0 += 32 * kU) {
            load(c0);
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const uint32_t w4[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint32_t lo = w4[q] & 0x7fffu, hi = (w4[q] >> 16) & 0x7fffu;
                    am = max(am, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
                }
            }
        }
        am = __reduce_max_sync(0xffffffffu, am);
        const int sh = f16_shift(__uint_as_float(am << 16));
        const float f = exp2i(sh);
        for (int c0 = lane; c0 < C8; c0 += 32 * kU) {
            if (C8 > 32 * kU) load(c0);
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                if (c0 + 32 * u >= C8) continue;
                float e[8];
                bf16x8_to_float(v[u], e);
                uint32_t o[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const __half2 h = __floats2half2_rn(e[2 * q] * f, e[2 * q + 1] * f);
                    o[q] = *reinterpret_cast<const uint32_t*>(&h);
                }
                dst[c0 + 32 * u] = make_uint4(o[0], o[1], o[2], o[3]);
            }
        }
        if (lane == 0) exps[routed ? r : n * k + (r - n_routes)] = sh;
    }
    weight_row_exps(wr, active, ctrl->n_active);
    pdl_trigger();
}

// out[t, h] = bf16( sum_j y[inv[t*k + j], h] (slot order) + y_sh[t, h] ), for
// calls whose down kernel does not run the combine itself.
__global__ void __launch_bounds__(256) combine_kernel(const float* __restrict__ y, const float* __restrict__ ysh,
                                                      const int32_t* __restrict__ inv, int n, int H, int k,
                                                      int has_shared, int accumulate, uint16_t* __restrict__ out,
                                                      int early) {
    pdl_wait();
    if (early) pdl_trigger();
    combine_range<false>(y, ysh, inv, n, H, k, has_shared, accumulate, out,
                         blockIdx.x * (int64_t)blockDim.x + threadIdx.x, (int64_t)gridDim.x * blockDim.x);
    pdl_trigger();
}

// SiLU(g) u of the INT4 experts as the f16 rows of the down product: each row times the power
// of two that puts its largest finite value below 2^15, its exponent to exps.  One rounding to
// 11 significand bits, down to 2^-29 of that value, at any magnitude; an infinity stays one.
// One warp a row; a row of up to 32 kU chunks of 8 is read once.
__global__ void __launch_bounds__(256) act_rows_kernel(const float* __restrict__ act, const float* __restrict__ act_sh,
                                                       int n, int I, int S, const int32_t* __restrict__ offsets, int E,
                                                       uint16_t* __restrict__ as, uint16_t* __restrict__ ash,
                                                       int32_t* __restrict__ exps, int n_routes_max, int early) {
    constexpr int kU = 4;
    pdl_wait();
    if (early) pdl_trigger();
    const int n_routes = offsets[E], rows = n_routes + (S > 0 ? n : 0);
    const int lane = threadIdx.x & 31, nwarps = gridDim.x * (blockDim.x >> 5);
    for (int r = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); r < rows; r += nwarps) {
        const bool routed = r < n_routes;
        const int rr = routed ? r : r - n_routes, width = routed ? I : S, C8 = width >> 3;
        const float4* src = reinterpret_cast<const float4*>((routed ? act : act_sh) + (size_t)rr * width);
        uint4* dst = reinterpret_cast<uint4*>((routed ? as : ash) + (size_t)rr * width);
        float4 v[kU][2];
        auto load = [&](int c0) {
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const int c = c0 + 32 * u;
                v[u][0] = c < C8 ? src[2 * c] : make_float4(0.f, 0.f, 0.f, 0.f);
                v[u][1] = c < C8 ? src[2 * c + 1] : make_float4(0.f, 0.f, 0.f, 0.f);
            }
        };
        float am = 0.f;
        for (int c0 = lane; c0 < C8 + lane; c0 += 32 * kU) {
            load(c0);
#pragma unroll
            for (int u = 0; u < kU; ++u)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    am = fmaxf(am, fmaxf(fmaxf(finite_abs(v[u][h].x), finite_abs(v[u][h].y)),
                                         fmaxf(finite_abs(v[u][h].z), finite_abs(v[u][h].w))));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
        const int sh = f16_shift(am);
        const float f = exp2i(sh);
        for (int c0 = lane; c0 < C8; c0 += 32 * kU) {
            if (C8 > 32 * kU) load(c0);
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                auto pair = [&](float x, float y) {
                    const __half2 h = __floats2half2_rn(x * f, y * f);
                    return *reinterpret_cast<const uint32_t*>(&h);
                };
                if (c0 + 32 * u < C8)
                    dst[c0 + 32 * u] = make_uint4(pair(v[u][0].x, v[u][0].y), pair(v[u][0].z, v[u][0].w),
                                                  pair(v[u][1].x, v[u][1].y), pair(v[u][1].z, v[u][1].w));
            }
        }
        if (lane == 0) exps[routed ? rr : n_routes_max + rr] = sh;
    }
    pdl_trigger();
}

// dst = src, n16 16-byte words (x staged from pinned host memory).
__global__ void __launch_bounds__(256) copy16_kernel(const uint4* __restrict__ src, uint4* __restrict__ dst,
                                                     size_t n16) {
    pdl_wait();
    for (size_t i = blockIdx.x * (size_t)blockDim.x + threadIdx.x; i < n16; i += (size_t)gridDim.x * blockDim.x)
        dst[i] = src[i];
    pdl_trigger();
}

}  // namespace

cudaError_t launch_copy16(const void* src, void* dst, size_t bytes, int num_sms, cudaStream_t st) {
    const size_t n16 = bytes / 16;
    const int grid = (int)std::min<size_t>((size_t)num_sms, (n16 + 255) / 256);
    launch_pdl(copy16_kernel, grid > 0 ? grid : 1, 256, 0, st, static_cast<const uint4*>(src),
               static_cast<uint4*>(dst), n16);
    return cudaGetLastError();
}

cudaError_t launch_gather(int fmt, const uint16_t* x, int n, int H, int k, const int32_t* perm,
                          const int32_t* offsets, int E, uint16_t* xs, uint16_t* xh, const uint16_t* norm_w,
                          float eps, int32_t* exps, const WeightRows& wr, const int32_t* active, const Ctrl* ctrl, bool early, int num_sms, cudaStream_t st) {
    const int grid = 2 * num_sms;
    if (exps) {
        launch_pdl(norm_w ? gather_scaled_kernel<true> : gather_scaled_kernel<false>, 4 * num_sms, 256, 0, st, x, n, H, k, perm,
                   offsets, E, xs, xh, norm_w, eps, exps, wr, active, ctrl, early ? 1 : 0);
        return cudaGetLastError();
    }
    auto kern = fmt != MOE_W_BF16 ? (norm_w ? gather_kernel<true, true> : gather_kernel<true, false>)
                                  : (norm_w ? gather_kernel<false, true> : gather_kernel<false, false>);
    launch_pdl(kern, grid, 256, 0, st, x, n, H, k, perm, offsets, E, xs, xh, norm_w, eps, early ? 1 : 0);
    return cudaGetLastError();
}

cudaError_t launch_act_rows(const float* act, const float* act_sh, int n, int I, int S, const int32_t* offsets, int E,
                            uint16_t* as, uint16_t* ash, int32_t* exps, int n_routes_max, bool early, int num_sms,
                            cudaStream_t st) {
    launch_pdl(act_rows_kernel, 2 * num_sms, 256, 0, st, act, act_sh, n, I, S, offsets, E, as, ash, exps, n_routes_max,
               early ? 1 : 0);
    return cudaGetLastError();
}

cudaError_t launch_combine(const float* y, const float* ysh, const int32_t* inv, int n, int H, int k,
                           int has_shared, int accumulate, uint16_t* out, bool early, int num_sms, cudaStream_t st) {
    launch_pdl(combine_kernel, 2 * num_sms, 256, 0, st, y, ysh, inv, n, H, k, has_shared, accumulate, out,
               early ? 1 : 0);
    return cudaGetLastError();
}

}  // namespace moe
