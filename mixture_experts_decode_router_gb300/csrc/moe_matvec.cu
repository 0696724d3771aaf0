// moe_matvec.cu -- products of 4-bit group-scaled matrices with a few vectors
// (sm_103a): out[t, o] = sum_i W[o, i] x[t, i] (+ bias[o]) (+ out[t, o]).
//
// Bound by the instructions on the weight stream (q4_mma.cuh).  On GB300: 100003 x 2048,
// groups of 32, six tokens 31.0 us (3.8 TB/s); 7168 x 7168 with zero points, one token
// 8.9 us (3.2 TB/s); 2048 x 2048 3.0 us, launch and latency; 7168 x 2048 NVFP4, 16
// tokens 8.0 us, the staging of x in every block.  Without the products the
// first takes 21 us.  (Stretches of stages that split the tiles of a part evenly over a
// block's warps, which balances the rounds, took 35 us where this took 33.4: the copies
// of a block's warps then lie apart in K.)
//
// Blocks of 8 or 16 warps; a warp multiplies 16 rows
// (q4_mma.cuh) and kw warps share a tile of rows, each with every kw-th stage of
// K, their sums added in warp order through shared memory.  Blocks are
// persistent over the row tiles, the warps' copies running ahead across tiles.
#include <algorithm>
#include <mutex>

#include "moe_launch.cuh"
#include "q4_mma.cuh"

namespace moe {

namespace {

constexpr int kMaxKw = 8;             // warps that share a tile at most
constexpr int kStages = 3;            // ring of each warp (2 stages in flight)
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

// Shared memory of a block: the warps' rings, the results' factors, the
// rows of x, and (kw > 1) the warps' sums.
struct Smem {
    uint32_t factor, x, red, total;
};
__host__ __device__ inline Smem smem_plan(int warps, int K, int nt, int ntok, int kw) {
    Smem m;
    m.factor = warps * kStages * q4::kStageBytes;   // of each token's result
    m.x = m.factor + 64;
    m.red = m.x + (uint32_t)ntok * q4::x_row_bytes(K);
    m.total = m.red + (kw > 1 ? warps * nt * 512 : 0);
    return m;
}

// XB: x is bf16 (else f16).
template <int GSH, bool Z, bool XB, int NT, int kWarps>
__global__ void __launch_bounds__(32 * kWarps, kWarps > 8 ? 1 : NT == 1 ? 3 : 2) matvec_kernel(const MatvecParams p, int kw, int tp) {
    extern __shared__ __align__(128) uint8_t dyn[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int K = p.w.in_dim, O = p.w.out_dim, row_bytes = K / 2;
    const int mw = kWarps / kw, mrow = warp / kw, kk = warp % kw;
    const int nst = (K + q4::kStageK - 1) / q4::kStageK;
    const int n_tiles = (O + 15) / 16, step = gridDim.x * mw;
    const int64_t t0 = (int64_t)blockIdx.y * tp;
    const int ntok = (int)min((int64_t)tp, (int64_t)p.n - t0);
    const Smem sm = smem_plan(kWarps, K, NT, ntok, kw);
    const uint32_t ring = warp * kStages * q4::kStageBytes;
    pdl_wait();

    // The copies run kStages - 1 stages ahead of the products, across tiles, and
    // the scales' loads one.
    const uint32_t dyn_a = q4::smem_addr(dyn);
    const int full = row_bytes / 128;
    int i_tile = kk < nst ? blockIdx.x * mw + mrow : n_tiles, i_s = kk, i_slot = 0;
    q4::RowCopy cp;
    cp.start(p.w.w, (int64_t)i_tile * 16, O - i_tile * 16, row_bytes, kk, lane);
    auto issue = [&]() {
        if (i_tile < n_tiles) {
            cp.issue(dyn_a + ring + i_slot * q4::kStageBytes, i_s, kw, row_bytes, full, p.w.w, lane);
            i_s += kw;
            if (i_s >= nst) {
                i_s = kk;
                i_tile += step;
                cp.start(p.w.w, (int64_t)i_tile * 16, O - i_tile * 16, row_bytes, kk, lane);
            }
        }
        q4::cp_commit();
        i_slot = i_slot + 1 == kStages ? 0 : i_slot + 1;
    };
    int n_tile = i_tile, n_s = kk;
    q4::StageScales<GSH, Z> sc, next;
    q4::ScaleLoad<GSH, Z> sl;
    sl.start(p.w, (int64_t)n_tile * 16, O - n_tile * 16, kk, lane);
    auto load_scales = [&]() {
        if (n_tile < n_tiles) {
            sl.load(next, n_s, kw, K, lane);
            n_s += kw;
            if (n_s >= nst) {
                n_s = kk;
                n_tile += step;
                sl.start(p.w, (int64_t)n_tile * 16, O - n_tile * 16, kk, lane);
            }
        }
    };
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) issue();
    load_scales();

    // x in fragment order, zero behind each row.
    const int xstride = q4::x_row_bytes(K), K8 = K / 8, chunks = nst * (q4::kStageK / 8);
    float* factor = reinterpret_cast<float*>(dyn + sm.factor);
    auto row = [&](int b) {
        return reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p.x) + (size_t)(t0 + b) * p.x_stride);
    };
    if constexpr (GSH == 4 && XB) {
        for (int b = warp; b < ntok; b += kWarps) {
            const float f = q4::scaled_row<NT == 1 && kWarps == 8 ? 4 : 8>(row(b), K8, chunks, reinterpret_cast<uint4*>(dyn + sm.x + b * xstride), lane);
            if (lane == 0) factor[b] = f * __ldg(p.w.scale2);
        }
    } else {
        // kU loads of a thread are made before any is stored.  Long rows, and a single one,
        // are taken by all threads one by one; shorter ones a stage a warp (2048 elements,
        // 16 tokens: 11.3 us by rows, 8.6 us so; 7168, 9 tokens: 16.0 us against 17.7).
        constexpr int kU = 4;
        const bool by_rows = ntok == 1 || chunks >= 3 * 32 * kWarps;
        for (int b = 0; by_rows && b < ntok; ++b) {
            const uint4* src = row(b);
            uint4* dst = reinterpret_cast<uint4*>(dyn + sm.x + b * xstride);
            for (int c0 = threadIdx.x; c0 < chunks; c0 += kU * 32 * kWarps) {
                uint4 v[kU];
#pragma unroll
                for (int u = 0; u < kU; ++u) {
                    const int c = c0 + u * 32 * kWarps;
                    v[u] = c < K8 ? src[c] : make_uint4(0u, 0u, 0u, 0u);
                }
#pragma unroll
                for (int u = 0; u < kU; ++u) {
                    const int c = c0 + u * 32 * kWarps;
                    if (c < chunks) dst[c] = q4::chunk_order<GSH>(v[u]);
                }
            }
        }
        const int units = by_rows ? 0 : ntok * nst;
        for (int u0 = warp; u0 < units; u0 += kU * kWarps) {
            uint4 v[kU];
#pragma unroll
            for (int i = 0; i < kU; ++i) {
                const int u = u0 + i * kWarps, b = u / nst, c = (u - b * nst) * 32 + lane;
                v[i] = u < units && c < K8 ? row(b)[c] : make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
            for (int i = 0; i < kU; ++i) {
                const int u = u0 + i * kWarps, b = u / nst, c = (u - b * nst) * 32 + lane;
                if (u < units) reinterpret_cast<uint4*>(dyn + sm.x + b * xstride)[c] = q4::chunk_order<GSH>(v[i]);
            }
        }
        if (threadIdx.x < 16) factor[threadIdx.x] = GSH == 4 ? __ldg(p.w.scale2) : 1.f;
    }
    __syncthreads();
    q4::XView<NT> x;
    x.start(sm.x, xstride, ntok, lane);

    const int g = lane >> 2, t = lane & 3;
    int slot = 0;
    for (int base = blockIdx.x * mw; base < n_tiles; base += step) {
        const int tile = base + mrow, row0 = tile * 16;
        const bool live = tile < n_tiles;
        float acc[NT][4];
#pragma unroll
        for (int q = 0; q < NT; ++q)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[q][i] = 0.f;
        if (live) {
            for (int s = kk; s < nst; s += kw) {
                sc = next;
                load_scales();
                q4::cp_wait<kStages - 2>();
                __syncwarp();
                issue();
                q4::mma_stage<GSH, Z, XB && GSH != 4, NT>(dyn, ring + slot * q4::kStageBytes, x, s, sc, acc, lane);
                slot = slot + 1 == kStages ? 0 : slot + 1;
            }
        }
        if (kw > 1) {
            float4* mine = reinterpret_cast<float4*>(dyn + sm.red) + (size_t)warp * NT * 32;
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
                    if (row < O && b < ntok) store_out(p, t0 + b, row, acc[q][i] * factor[b]);
                }
        }
    }
    pdl_trigger();
}

template <int GSH, bool Z, bool XB, int NT, int kWarps>
cudaError_t launch_warps(const MatvecParams& p, int tp, int kw, int num_sms, cudaStream_t st) {
    const int n_tiles = (p.w.out_dim + 15) / 16;
    const size_t smem = smem_plan(kWarps, p.w.in_dim, NT, std::min(tp, p.n), kw).total;
    auto kern = matvec_kernel<GSH, Z, XB, NT, kWarps>;
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
    const int per_sm = kWarps > 8 ? 1 : std::max(1, std::min(3, (int)((size_t)kMaxSmem / (smem + 1024))));
    const int mw = kWarps / kw;
    const int gx = std::min((n_tiles + mw - 1) / mw, num_sms * per_sm);
    // (A grid has at most 65535 rows of blocks.)
    constexpr int64_t kMaxY = 65535;
    MatvecParams q = p;
    for (int64_t n0 = 0; n0 < p.n; n0 += kMaxY * tp) {
        q.n = (int)std::min<int64_t>(p.n - n0, kMaxY * tp);
        q.x = static_cast<const uint16_t*>(p.x) + n0 * p.x_stride;
        q.out = static_cast<uint8_t*>(p.out) + n0 * p.out_stride * (p.out_type == MOE_F32 ? 4 : 2);
        launch_pdl(kern, dim3(gx, (unsigned)((q.n + tp - 1) / tp)), 32 * kWarps, smem, st, q, kw, tp);
    }
    return cudaGetLastError();
}

template <int GSH, bool Z, bool XB, int NT>
cudaError_t launch_nt(const MatvecParams& p, int tp, int num_sms, cudaStream_t st) {
    const int K = p.w.in_dim, n_tiles = (p.w.out_dim + 15) / 16, nst = (K + q4::kStageK - 1) / q4::kStageK;
    // Warps that share a tile: as many as give every SM about its 24 warps (a
    // 7168 x 7168 product with one token: 10.6 us with 8, 9.1 us so).
    int kw = 1;
    while (kw < kMaxKw && kw < nst && (int64_t)n_tiles * kw < (int64_t)num_sms * 20) kw *= 2;
    // Rows of x so long that an SM has room for one block of 8 warps: 16 warps, if their
    // rings fit (7168 x 2048 NVFP4, 16 tokens: 9.1 us with 8, 8.2 us with 16).
    const int tokens = std::min(tp, p.n);
    if (2 * (smem_plan(8, K, NT, tokens, kw).total + 1024) > (uint32_t)kMaxSmem &&
        smem_plan(16, K, NT, tokens, kw).total <= (uint32_t)kMaxSmem)
        return launch_warps<GSH, Z, XB, NT, 16>(p, tp, kw, num_sms, st);
    return launch_warps<GSH, Z, XB, NT, 8>(p, tp, kw, num_sms, st);
}

template <int GSH, bool Z, bool XB>
cudaError_t launch_fmt(const MatvecParams& p, int num_sms, cudaStream_t st) {
    // Tokens of a block: up to 16, as many as fit beside the rings.
    const int64_t room = kMaxSmem - (int64_t)smem_plan(8, p.w.in_dim, 2, 0, kMaxKw).total;
    int tp = (int)std::min<int64_t>(16, room / q4::x_row_bytes(p.w.in_dim));
    if (tp < 1) return cudaErrorInvalidValue;   // (matvec_fits says no)
    if (p.n > tp && tp < 16) tp = std::min(tp, 8);   // (two groups of eight rather than one of nine to fifteen and a rest)
    const int tokens = std::min(tp, p.n);
    return tokens > 8 ? launch_nt<GSH, Z, XB, 2>(p, tp, num_sms, st) : launch_nt<GSH, Z, XB, 1>(p, std::min(tp, 8), num_sms, st);
}

template <int GSH>
cudaError_t launch_x(int x_type, const MatvecParams& p, int num_sms, cudaStream_t st) {
    if constexpr (GSH != 4) {
        if (p.w.zero)
            return x_type == MOE_BF16 ? launch_fmt<GSH, true, true>(p, num_sms, st) : launch_fmt<GSH, true, false>(p, num_sms, st);
    }
    return x_type == MOE_BF16 ? launch_fmt<GSH, false, true>(p, num_sms, st) : launch_fmt<GSH, false, false>(p, num_sms, st);
}

}  // namespace

// The longest row of x that the interface admits; one fits beside the rings.
constexpr int kMaxIn = 57344;
static_assert(8 * (kStages * q4::kStageBytes + 1024) + 64 + kMaxIn * 2 + 64 + 512 <= kMaxSmem,
              "a row of x fits");
bool matvec_fits(int K) { return K <= kMaxIn; }

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
