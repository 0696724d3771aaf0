// moe_experts_q4.cu -- the INT4 experts of a decode batch (sm_103a).
//
// A decode batch gives an expert a handful of tokens, so its products are bound by
// the stream of its 4-bit matrices; a warp multiplies 16 weight rows with up to 16
// tokens straight from the codes (q4_mma.cuh), without the dequantised tile in
// tensor memory that a 128-row tcgen05 tile needs.
//
//   gate_up   item = (tokens of one expert, 8 tiles of 16 rows of I): a block's
//             8 warps take a tile each, gate and up, the tokens' rows staged in
//             shared memory in chunks of K; a = SiLU(g) u -> act (fp32)
//   down      item = (the same tokens, 8 tiles of 16 rows of H):
//             y[p, h] = weight (route p) Wd a (fp32); the combine kernel adds a
//             token's rows in slot order
//   One token, or a few: gate_up_n1 and down_n1 take a token's routes as they are (no
//   grouping), split K over a block's warps, and down_n1 adds the slots and writes the
//   output.
//
// act enters the down product as f16, each token's chunk of 768 (one token: 256) scaled by a power of
// two that puts its largest finite value below 2^15: one rounding to 11 significand bits
// down to 2^-29 of that value, at any magnitude.  Chunks and order of every sum
// depend on the layer's sizes alone within each of the two forms: a token's bits do not
// depend on the other tokens of its batch, and do differ between the batches that take
// their routes one by one (one token, or a few) and the larger ones.
//
// On GB300 (hidden 2048, intermediate 512, 8 of 256 experts and a shared one): one token
// 9.7 us (1.5 TB/s), 16 tokens with groups of 64 and zero points 64 us (2.8 TB/s), 256
// rows with groups of 32 205 us (2.2 TB/s); hidden 7168, intermediate 2048, 8 of 64
// experts, 64 tokens 473 us (3.1 TB/s).  The copies and the staging alone take 41, 125
// and 306 us of the last three; the rest is what the warps' instructions do not overlap.
// (Measured and not kept: the rows of x prepared once by a kernel of their own and read
// through L1 by warps that share nothing, 70, 273 and 547 us; two row tiles a warp for
// each staging, 67, 226 and 511 us; four blocks an SM with rings of two stages, 85, 229
// and 586 us.)
#include <algorithm>
#include <mutex>

#include "moe_launch.cuh"
#include "q4_mma.cuh"

namespace moe {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kStages = 3;                 // ring of each warp
constexpr int kRing = kWarps * kStages * q4::kStageBytes;
constexpr int kStages2 = 2;                // of one token's gate and up together
constexpr int kRing2 = kWarps * kStages2 * 2 * q4::kStageBytes;
constexpr int kActStages = 3;              // stages of a chunk of act
constexpr int kXBytes = 16 * (kActStages * 512 + 64);   // rows of x or act in shared memory (25.6 KB: three blocks an SM)
constexpr int kMaxSmem = 227 * 1024;

// 256 kN fp32 values of one act row (zero past `left`) as f16 chunks for the fragments,
// by one warp; returns the factor that scales results back.
template <int kN>
__device__ __forceinline__ float stage_act(const float* src, int left, uint8_t* dst, int lane) {
    float v[kN][8];   // chunks of 8
#pragma unroll
    for (int i = 0; i < kN; ++i) {
        const int c = lane + 32 * i;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
        if (c * 8 < left) {
            a = __ldcg(reinterpret_cast<const float4*>(src) + 2 * c);
            b = __ldcg(reinterpret_cast<const float4*>(src) + 2 * c + 1);
        }
        v[i][0] = a.x; v[i][1] = a.y; v[i][2] = a.z; v[i][3] = a.w;
        v[i][4] = b.x; v[i][5] = b.y; v[i][6] = b.z; v[i][7] = b.w;
    }
    auto largest = [&](bool finite) {
        float am = 0.f;
#pragma unroll
        for (int i = 0; i < kN; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float a = fabsf(v[i][e]);
                am = fmaxf(am, finite && a == INFINITY ? 0.f : a);
            }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
        return am;
    };
    float am = largest(false);
    if (am == INFINITY) am = largest(true);   // an infinity stays one at any scale; the rest has to stay finite
    const int sh = f16_shift(am);
    const float f = exp2i(sh);
#pragma unroll
    for (int i = 0; i < kN; ++i) {
        auto pair = [&](int x, int y) {
            const __half2 h = __floats2half2_rn(v[i][x] * f, v[i][y] * f);
            return *reinterpret_cast<const uint32_t*>(&h);
        };
        reinterpret_cast<uint4*>(dst)[lane + 32 * i] = make_uint4(pair(0, 4), pair(1, 5), pair(2, 6), pair(3, 7));
    }
    return exp2i(-sh);
}

__device__ __forceinline__ float shared_gate(const float* sg_logit, int t) {
    return sg_logit ? 1.0f / (1.0f + expf(-__ldg(sg_logit + t))) : 1.0f;
}

// One item's products by one block: see the file's head.  NT: 8-token tiles.
struct Item {
    bool sh;
    int le, pos0, ntok, tile0;   // expert in its stack, first sorted row, tokens, first 16-row tile
};

template <int GSH, bool Z, bool GU, int TILE, int NT>
__device__ __forceinline__ void run_item(const Q4Params& p, const Item& it, uint8_t* dyn, bool& waited) {
    constexpr int kMats = GU ? 2 : 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int out = GU ? (it.sh ? p.S : p.I) : p.H, K = GU ? p.H : (it.sh ? p.S : p.I);
    const int nst = (K + q4::kStageK - 1) / q4::kStageK, row_bytes = K / 2, full = row_bytes / 128;
    const int row0 = (it.tile0 + warp) * 16, rows = out - row0;
    const int64_t srow = (int64_t)it.le * out + row0;        // the tile's first row in the stack
    const bool live = rows > 0;
    const uint32_t ring = warp * kStages * q4::kStageBytes, ring_a = q4::smem_addr(dyn) + ring;
    float* factor = reinterpret_cast<float*>(dyn + kRing);   // [16] of the chunk (down)
    float* weight = factor + 16;                             // [16] of the token (down)
    const uint32_t x0 = kRing + 128;
    const QMatDev& m0 = GU ? (it.sh ? p.sh_gate : p.gate) : (it.sh ? p.sh_down : p.down);
    const QMatDev& m1 = it.sh ? p.sh_up : p.up;
    // Stages of a chunk; a token's row of a chunk in shared memory.
    const int cs = GU ? min(nst, (kXBytes / it.ntok - 64) / 512) : min(nst, kActStages);
    const int xstride = (GU ? cs : kActStages) * 512 + 64;

    // Stages in the order chunk, matrix, stage; the copies run kStages - 1 ahead and
    // the scales' loads one.
    struct Walk {
        int s, m, c0;
        __device__ __forceinline__ bool next(int cs, int nst) {   // whether the matrix or the chunk changes
            if (++s < min(c0 + cs, nst)) return false;
            if (++m == kMats) { m = 0; c0 += cs; }
            s = c0;
            return true;
        }
    };
    Walk wi{0, 0, 0}, wn{0, 0, 0};
    int i_slot = 0;
    q4::RowCopy cp;
    q4::ScaleLoad<GSH, Z> sl;
    q4::StageScales<GSH, Z> sc, nx;
    auto issue = [&]() {
        if (live && wi.s < nst) {
            cp.issue(ring_a + i_slot * q4::kStageBytes, wi.s, 1, row_bytes, full, m0.w, lane);
            if (wi.next(cs, nst)) cp.start(wi.m ? m1.w : m0.w, srow, rows, row_bytes, wi.s, lane);
        }
        q4::cp_commit();
        i_slot = i_slot + 1 == kStages ? 0 : i_slot + 1;
    };
    auto load_scales = [&]() {
        if (live && wn.s < nst) {
            sl.load(nx, wn.s, 1, K, lane);
            if (wn.next(cs, nst)) sl.start(wn.m ? m1 : m0, srow, rows, wn.s, lane);
        }
    };
    cp.start(m0.w, srow, rows, row_bytes, 0, lane);
    sl.start(m0, srow, rows, 0, lane);
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) issue();
    load_scales();
    [[maybe_unused]] int token = 0;   // lane b's token
    if (GU && TILE > 8 && lane < it.ntok) token = it.sh ? it.pos0 + lane : __ldg(p.perm + it.pos0 + lane) / p.k;
    if (!GU && !waited) {
        pdl_wait();
        pdl_trigger();
        waited = true;
    }
    if (!GU && threadIdx.x < it.ntok) {
        const int b = it.pos0 + threadIdx.x;
        weight[threadIdx.x] = it.sh ? shared_gate(p.sg_logit, b) : __ldg(p.route_w + __ldg(p.perm + b));
    }

    q4::XView<NT> x;
    x.start(x0, xstride, it.ntok, lane);
    float acc[kMats][NT][4], total[NT][4];
#pragma unroll
    for (int q = 0; q < NT; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            total[q][i] = 0.f;
#pragma unroll
            for (int m = 0; m < kMats; ++m) acc[m][q][i] = 0.f;
        }
    int slot = 0;
    const int g = lane >> 2, t = lane & 3;
    for (int c0 = 0; c0 < nst; c0 += cs) {
        if (c0 > 0) __syncthreads();   // every warp is done with the chunk before
        if constexpr (GU) {
            // Elements [c0, c0 + cs) stages of each token's row, zero past K.  Segments of
            // up to 16 tokens: a warp a stage of a row, kU of them loaded before any is
            // stored (256 rows of 8 of 256 experts: 214 us by single chunks, 208 us so);
            // shorter ones by single chunks (16 tokens: 64 us, 66 us the other way).
            const int k8 = K / 8, chunks = cs * 32;
            if constexpr (TILE > 8) {
                constexpr int kU = 4;
                const int units = it.ntok * cs;
                for (int u0 = warp; u0 < units; u0 += kU * kWarps) {
                    uint4 v[kU];
#pragma unroll
                    for (int i = 0; i < kU; ++i) {
                        const int u = u0 + i * kWarps, b = u / cs, cc = (c0 + u - b * cs) * 32 + lane;
                        const int tok = __shfl_sync(0xffffffffu, token, min(b, it.ntok - 1));
                        v[i] = u < units && cc < k8 ? __ldg(reinterpret_cast<const uint4*>(p.x + (size_t)tok * K) + cc)
                                                    : make_uint4(0u, 0u, 0u, 0u);
                    }
#pragma unroll
                    for (int i = 0; i < kU; ++i) {
                        const int u = u0 + i * kWarps, b = u / cs, c = (u - b * cs) * 32 + lane;
                        if (u < units) *reinterpret_cast<uint4*>(dyn + x0 + b * xstride + c * 16) = q4::chunk_order<GSH>(v[i]);
                    }
                }
            } else {
                for (int i = threadIdx.x; i < it.ntok * chunks; i += kThreads) {
                    const int b = i / chunks, c = i - b * chunks, cc = c0 * 32 + c;
                    uint4 v = make_uint4(0u, 0u, 0u, 0u);
                    if (cc < k8) {
                        const int tok = it.sh ? it.pos0 + b : __ldg(p.perm + it.pos0 + b) / p.k;
                        v = __ldg(reinterpret_cast<const uint4*>(p.x + (size_t)tok * K) + cc);
                    }
                    *reinterpret_cast<uint4*>(dyn + x0 + b * xstride + c * 16) = q4::chunk_order<GSH>(v);
                }
            }
        } else {
            const float* a = it.sh ? p.act_sh : p.act;
            for (int b = warp; b < it.ntok; b += kWarps) {
                const float f = stage_act<kActStages>(a + (size_t)(it.pos0 + b) * K + c0 * q4::kStageK, K - c0 * q4::kStageK,
                                          dyn + x0 + b * xstride, lane);
                if (lane == 0) factor[b] = f;
            }
        }
        __syncthreads();
        if (live) {
#pragma unroll
            for (int m = 0; m < kMats; ++m)
                for (int s = c0; s < min(c0 + cs, nst); ++s) {
                    sc = nx;
                    load_scales();
                    q4::cp_wait<kStages - 2>();
                    __syncwarp();
                    issue();
                    q4::mma_stage<GSH, Z, GU, NT>(dyn, ring + slot * q4::kStageBytes, x, s - c0, sc, acc[m], lane);
                    slot = slot + 1 == kStages ? 0 : slot + 1;
                }
            if constexpr (!GU) {
#pragma unroll
                for (int q = 0; q < NT; ++q)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int b = 8 * q + 2 * t + (i & 1);
                        total[q][i] = fmaf(acc[0][q][i], factor[min(b, it.ntok - 1)], total[q][i]);
                        acc[0][q][i] = 0.f;
                    }
            }
        }
    }
    if (live) {
        float* dst = GU ? (it.sh ? p.act_sh : p.act) : (it.sh ? p.y_sh : p.y);
#pragma unroll
        for (int q = 0; q < NT; ++q)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = g + 8 * (i >> 1), b = 8 * q + 2 * t + (i & 1);
                if (r < rows && b < it.ntok) {
                    const float v = GU ? silu(acc[0][q][i]) * acc[kMats - 1][q][i] : total[q][i] * weight[b];
                    dst[(size_t)(it.pos0 + b) * out + row0 + r] = v;
                }
            }
    }
}

// TILE: tokens of a segment, 8 or 16.
template <int GSH, bool Z, bool GU, int TILE>
__global__ void __launch_bounds__(kThreads, TILE == 8 ? 3 : 2) experts_q4_kernel(const Q4Params p) {
    extern __shared__ __align__(128) uint8_t dyn[];
    // The down kernel's first item starts its weights before it waits for gate_up, whose
    // own wait, before it let this kernel start, covered the grouping.
    bool waited = GU;
    if (GU) {
        pdl_wait();
        pdl_trigger();
    }
    const int n_rsegs = __ldcg(&p.ctrl->n_rsegs);
    const int n_ssegs = p.S > 0 ? (p.n + TILE - 1) / TILE : 0;
    const int gr = ((GU ? p.I : p.H) + 16 * kWarps - 1) / (16 * kWarps), gs = ((GU ? p.S : p.H) + 16 * kWarps - 1) / (16 * kWarps);
    const int items = n_ssegs * gs + n_rsegs * gr;
    for (int i = blockIdx.x; i < items; i += gridDim.x) {
        Item it;
        it.sh = i < n_ssegs * gs;
        if (it.sh) {
            const int s = i / gs;
            it.le = 0;
            it.pos0 = s * TILE;
            it.ntok = min(TILE, p.n - it.pos0);
            it.tile0 = (i - s * gs) * kWarps;
        } else {
            const int j = i - n_ssegs * gs, s = j / gr;
            it.le = __ldcg(p.segs + 3 * s) - p.e_begin;
            it.pos0 = __ldcg(p.segs + 3 * s + 1);
            it.ntok = __ldcg(p.segs + 3 * s + 2);
            it.tile0 = (j - s * gr) * kWarps;
        }
        if (i != (int)blockIdx.x) __syncthreads();   // the item before is done with shared memory
        if (TILE == 8 || it.ntok <= 8) run_item<GSH, Z, GU, TILE, 1>(p, it, dyn, waited);
        else if constexpr (TILE > 8) run_item<GSH, Z, GU, TILE, 2>(p, it, dyn, waited);
    }
    if (!waited) pdl_wait();   // (a block without items)
}

// ---------------------------------------------------------------- one token a block

// One block per (slot, 16 rows of I) and (shared expert, 16 rows of S): its warps take
// every eighth stage of gate and up together, their sums added in warp order.  (One
// matrix after the other, and act staged in chunks of 768: the two kernels took 12.8 us
// at hidden 2048, intermediate 512, eight experts and a shared one, and take 9.7 us.)
template <int GSH, bool Z>
__global__ void __launch_bounds__(kThreads, 3) gate_up_n1_kernel(const Q4Params p) {
    extern __shared__ __align__(128) uint8_t dyn[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tr = (p.I + 15) / 16, tile = blockIdx.x, tok = blockIdx.y;
    const bool sh = tile >= p.k * tr;
    const int slot = sh ? p.k : tile / tr, row0 = (sh ? tile - p.k * tr : tile % tr) * 16;
    const int out = sh ? p.S : p.I, K = p.H, row_bytes = K / 2, full = row_bytes / 128;
    const int nst = (K + q4::kStageK - 1) / q4::kStageK;
    pdl_wait();
    pdl_trigger();
    const int e = sh ? 0 : __ldg(p.idx + tok * p.k + slot);
    if (!sh && (e < p.e_begin || e >= p.e_end)) return;   // not held here: down skips it too
    const int64_t srow = (int64_t)(sh ? 0 : e - p.e_begin) * out + row0;
    const QMatDev& m0 = sh ? p.sh_gate : p.gate;
    const QMatDev& m1 = sh ? p.sh_up : p.up;
    constexpr uint32_t kSlot = 2 * q4::kStageBytes;            // of gate and of up
    const uint32_t ring = warp * kStages2 * kSlot, ring_a = q4::smem_addr(dyn) + ring;
    float* red = reinterpret_cast<float*>(dyn + kRing2);       // [2][kWarps][16]
    const uint32_t x0 = kRing2 + 2 * kWarps * 16 * 4;
    int i_s = warp, n_s = warp, i_slot = 0, slot_s = 0;
    q4::RowCopy cp[2];
    q4::ScaleLoad<GSH, Z> sl[2];
    q4::StageScales<GSH, Z> sc[2], nx[2];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        cp[m].start(m ? m1.w : m0.w, srow, out - row0, row_bytes, i_s, lane);
        sl[m].start(m ? m1 : m0, srow, out - row0, n_s, lane);
    }
    auto issue = [&]() {
        if (i_s < nst) {
#pragma unroll
            for (int m = 0; m < 2; ++m)
                cp[m].issue(ring_a + i_slot * kSlot + m * q4::kStageBytes, i_s, kWarps, row_bytes, full, m0.w, lane);
            i_s += kWarps;
        }
        q4::cp_commit();
        i_slot = i_slot + 1 == kStages2 ? 0 : i_slot + 1;
    };
    auto load_scales = [&]() {
        if (n_s < nst) {
#pragma unroll
            for (int m = 0; m < 2; ++m) sl[m].load(nx[m], n_s, kWarps, K, lane);
            n_s += kWarps;
        }
    };
#pragma unroll
    for (int s = 0; s < kStages2 - 1; ++s) issue();
    load_scales();
    for (int c = threadIdx.x; c < nst * 32; c += kThreads)
        *reinterpret_cast<uint4*>(dyn + x0 + c * 16) =
            q4::chunk_order<GSH>(c < K / 8 ? __ldg(reinterpret_cast<const uint4*>(p.x + (size_t)tok * K) + c) : make_uint4(0u, 0u, 0u, 0u));
    __syncthreads();
    q4::XView<1> x;
    x.start(x0, 0, 1, lane);
    float acc[2][1][4] = {};
    for (int s = warp; s < nst; s += kWarps) {
#pragma unroll
        for (int m = 0; m < 2; ++m) sc[m] = nx[m];
        load_scales();
        q4::cp_wait<kStages2 - 2>();
        __syncwarp();
        issue();
#pragma unroll
        for (int m = 0; m < 2; ++m)
            q4::mma_stage<GSH, Z, true, 1>(dyn, ring + slot_s * kSlot + m * q4::kStageBytes, x, s, sc[m], acc[m], lane);
        slot_s = slot_s + 1 == kStages2 ? 0 : slot_s + 1;
    }
    if ((lane & 3) == 0) {   // column 0: rows g and g + 8
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            red[(m * kWarps + warp) * 16 + (lane >> 2)] = acc[m][0][0];
            red[(m * kWarps + warp) * 16 + (lane >> 2) + 8] = acc[m][0][2];
        }
    }
    __syncthreads();
    if (threadIdx.x < 16 && row0 + (int)threadIdx.x < out) {
        float gu[2];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            gu[m] = red[m * kWarps * 16 + threadIdx.x];
            for (int w = 1; w < kWarps; ++w) gu[m] += red[(m * kWarps + w) * 16 + threadIdx.x];
        }
        (sh ? p.act_sh + (size_t)tok * p.S : p.act + (size_t)(tok * p.k + slot) * p.I)[row0 + threadIdx.x] = silu(gu[0]) * gu[1];
    }
}

// One block per 16 rows of H: its warps take every eighth of all slots' stages (the
// shared expert's last), each stage's sum weighted, added in warp order, and written.
template <int GSH, bool Z>
__global__ void __launch_bounds__(kThreads, 3) down_n1_kernel(const Q4Params p) {
    extern __shared__ __align__(128) uint8_t dyn[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row0 = blockIdx.x * 16, rows = p.H - row0, tok = blockIdx.y;
    const int32_t* idx = p.idx + tok * p.k;
    const int nr = (p.I + q4::kStageK - 1) / q4::kStageK, ns = (p.S + q4::kStageK - 1) / q4::kStageK;
    const int units = p.k * nr + ns;
    const uint32_t ring = warp * kStages * q4::kStageBytes, ring_a = q4::smem_addr(dyn) + ring;
    float* red = reinterpret_cast<float*>(dyn + kRing);             // [kWarps][16]
    float* cf = red + kWarps * 16;                                  // weight and factor of each unit
    const uint32_t x0 = kRing + kWarps * 64 + ((units * 4 + 15) & ~15);
    // (What comes before the wait does not depend on gate_up, whose own wait, before it
    // let this kernel start, covered the routing.)
    // Unit u: stage u % nr of slot u / nr, then the shared expert's stages.
    struct Unit {
        int slot, s, e, K;
        bool held;
    };
    auto unit = [&](int u) {
        Unit a;
        const bool sh = u >= p.k * nr;
        a.slot = sh ? p.k : u / nr;
        a.s = sh ? u - p.k * nr : u - a.slot * nr;
        a.K = sh ? p.S : p.I;
        const int e = sh ? 0 : __ldcg(idx + a.slot);
        a.held = sh || (e >= p.e_begin && e < p.e_end);
        a.e = sh ? 0 : e - p.e_begin;
        return a;
    };
    int ui = warp, un = warp, i_slot = 0, slot_s = 0;
    q4::RowCopy cp;
    q4::ScaleLoad<GSH, Z> sl;
    q4::StageScales<GSH, Z> sc, nx;
    auto issue = [&]() {
        if (ui < units) {
            const Unit a = unit(ui);
            const QMatDev& m = a.slot == p.k ? p.sh_down : p.down;
            if (a.held) {
                cp.start(m.w, (int64_t)a.e * p.H + row0, rows, a.K / 2, a.s, lane);
                cp.issue(ring_a + i_slot * q4::kStageBytes, a.s, 1, a.K / 2, a.K / 256, m.w, lane);
            }
            ui += kWarps;
        }
        q4::cp_commit();
        i_slot = i_slot + 1 == kStages ? 0 : i_slot + 1;
    };
    auto load_scales = [&]() {
        if (un < units) {
            const Unit a = unit(un);
            if (a.held) {
                sl.start(a.slot == p.k ? p.sh_down : p.down, (int64_t)a.e * p.H + row0, rows, a.s, lane);
                sl.load(nx, a.s, 1, a.K, lane);
            }
            un += kWarps;
        }
    };
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) issue();
    load_scales();
    pdl_wait();
    pdl_trigger();
    // Every slot's act, a warp a stage.
    for (int u = warp; u < units; u += kWarps) {
        const Unit a = unit(u);
        if (!a.held) continue;
        const float* src = (a.slot == p.k ? p.act_sh + (size_t)tok * p.S : p.act + (size_t)(tok * p.k + a.slot) * p.I) + a.s * q4::kStageK;
        const float f = stage_act<1>(src, a.K - a.s * q4::kStageK, dyn + x0 + u * 512, lane);
        if (lane == 0) cf[u] = f * (a.slot == p.k ? shared_gate(p.sg_logit, tok) : __ldg(p.route_w + tok * p.k + a.slot));
    }
    __syncthreads();
    float total[4] = {0.f, 0.f, 0.f, 0.f};
    for (int u = warp; u < units; u += kWarps) {
        const Unit a = unit(u);
        sc = nx;
        load_scales();
        q4::cp_wait<kStages - 2>();
        __syncwarp();
        issue();
        if (a.held) {
            q4::XView<1> x;
            x.start(x0 + u * 512, 0, 1, lane);
            float acc[1][4] = {};
            q4::mma_stage<GSH, Z, false, 1>(dyn, ring + slot_s * q4::kStageBytes, x, 0, sc, acc, lane);
            const float w = cf[u];
#pragma unroll
            for (int i = 0; i < 4; ++i) total[i] = fmaf(acc[0][i], w, total[i]);
        }
        slot_s = slot_s + 1 == kStages ? 0 : slot_s + 1;
    }
    if ((lane & 3) == 0) {
        red[warp * 16 + (lane >> 2)] = total[0];
        red[warp * 16 + (lane >> 2) + 8] = total[2];
    }
    __syncthreads();
    if (threadIdx.x < 16 && (int)threadIdx.x < rows) {
        float v = red[threadIdx.x];
        for (int w = 1; w < kWarps; ++w) v += red[w * 16 + threadIdx.x];
        uint16_t* o = p.out + (size_t)tok * p.H + row0 + threadIdx.x;
        if (p.accumulate) v += __uint_as_float((uint32_t)*o << 16);
        const __nv_bfloat16 b = __float2bfloat16_rn(v);
        *o = *reinterpret_cast<const uint16_t*>(&b);
    }
}

size_t gate_up_n1_smem(int H) { return kRing2 + 2 * kWarps * 64 + (size_t)q4::x_row_bytes(H); }
size_t down_n1_smem(int k, int I, int S) {
    const size_t units = (size_t)k * ((I + q4::kStageK - 1) / q4::kStageK) + (S + q4::kStageK - 1) / q4::kStageK;
    return kRing + kWarps * 64 + ((units * 4 + 15) & ~size_t(15)) + units * 512;
}

template <typename Kern>
cudaError_t launch_smem(Kern kern, int slot, size_t smem, dim3 grid, cudaStream_t st, const Q4Params& p) {
    static std::mutex mu;
    static size_t configured[128][64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) return cudaErrorInvalidDevice;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (configured[dev][slot] < smem) {
            const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
            if (e != cudaSuccess) return e;
            configured[dev][slot] = smem;
        }
    }
    launch_pdl(kern, grid, kThreads, smem, st, p);
    return cudaGetLastError();
}

// Blocks of the general kernels: every SM's share of the items there can be.
template <int GSH, bool Z, int SLOT>
cudaError_t launch_fmt(const Q4Params& p, bool gate_up, int tile, int num_sms, cudaStream_t st) {
    const size_t smem = kRing + 128 + kXBytes;
    const int per_sm = tile == 8 ? 3 : 2;
    const dim3 grid(num_sms * per_sm);
    if (p.per_token) {
        if (gate_up)
            return launch_smem(gate_up_n1_kernel<GSH, Z>, SLOT * 6, gate_up_n1_smem(p.H),
                               dim3(p.k * ((p.I + 15) / 16) + (p.S + 15) / 16, p.n), st, p);
        return launch_smem(down_n1_kernel<GSH, Z>, SLOT * 6 + 1, down_n1_smem(p.k, p.I, p.S), dim3((p.H + 15) / 16, p.n), st, p);
    }
    if (tile == 8)
        return gate_up ? launch_smem(experts_q4_kernel<GSH, Z, true, 8>, SLOT * 6 + 2, smem, grid, st, p)
                       : launch_smem(experts_q4_kernel<GSH, Z, false, 8>, SLOT * 6 + 3, smem, grid, st, p);
    return gate_up ? launch_smem(experts_q4_kernel<GSH, Z, true, 16>, SLOT * 6 + 4, smem, grid, st, p)
                   : launch_smem(experts_q4_kernel<GSH, Z, false, 16>, SLOT * 6 + 5, smem, grid, st, p);
}

}  // namespace

bool q4_n1_fits(int H, int k, int I, int S) {
    return gate_up_n1_smem(H) <= (size_t)kMaxSmem && down_n1_smem(k, I, S) <= (size_t)kMaxSmem;
}

cudaError_t launch_experts_q4(int fmt, const Q4Params& p, bool gate_up, int tile, int num_sms, cudaStream_t st) {
    const bool z = p.zero;
    switch (fmt) {
        case MOE_W_INT4_G32: return z ? launch_fmt<5, true, 0>(p, gate_up, tile, num_sms, st) : launch_fmt<5, false, 1>(p, gate_up, tile, num_sms, st);
        case MOE_W_INT4_G64: return z ? launch_fmt<6, true, 2>(p, gate_up, tile, num_sms, st) : launch_fmt<6, false, 3>(p, gate_up, tile, num_sms, st);
        case MOE_W_INT4_G128: return z ? launch_fmt<7, true, 4>(p, gate_up, tile, num_sms, st) : launch_fmt<7, false, 5>(p, gate_up, tile, num_sms, st);
    }
    return cudaErrorInvalidValue;
}

}  // namespace moe
