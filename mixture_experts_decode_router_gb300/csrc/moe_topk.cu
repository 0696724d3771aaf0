// moe_topk.cu -- top-k routing of rows of logits (sm_103a): softmax or sigmoid
// scores, a balance bias, group-limited selection, any number of rows.
//
// Which expert a row chooses hangs on the order of near scores, and a whole number
// has no tolerance, so the order is that of the scores in 64 bits.  FP64 is scarce
// on a GB300 (a warp's instruction takes 16 cycles), so a row is first decided in
// 32 bits with a certificate: every comparison the choice hangs on -- neighbours
// among the chosen, the last chosen against the best left, the last kept group
// against the best left -- has to be clear by more than the 32-bit errors allow.  A
// row that is not clear is decided again, with the scores of its contenders in 64
// bits (~0.5% of rows of spread logits over 256 experts).
//
// One warp per row; lane l holds the V experts l V .. l V + V - 1 in registers.  The
// chosen come out of k + 1 rounds of one redux each: a lane's scores are order-
// preserving integers with the expert's index in the low bits (so equal scores go to
// the lower index), sorted in lists of 8, and the lane whose head wins shifts its
// list.  Bound by instruction issue: ~400 of a warp for 256 experts, 8 chosen.
#include <cuda_fp16.h>

#include <algorithm>
#include <mutex>

#include "moe_launch.cuh"

namespace moe {

namespace {

constexpr int kRowWarps = 4;   // rows per block

struct TopkParams {
    const void* logits;
    int64_t row_stride;
    int ns;
    int64_t pstride;
    float* lsum;
    int n, E, k;
    Routing r;
    const float* bias;
    int norm;
    float scale;
    int32_t* idx;
    float* w;
};

template <int TYPE>
__device__ __forceinline__ float load_logit(const TopkParams& p, int64_t t, int e) {
    const size_t at = (size_t)(t * p.row_stride) + e;
    if constexpr (TYPE == MOE_BF16)
        return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(p.logits)[at] << 16);
    if constexpr (TYPE == MOE_F16) return __half2float(reinterpret_cast<const __half*>(p.logits)[at]);
    const float* l = reinterpret_cast<const float*>(p.logits) + at;
    float v = l[0];
    for (int u = 1; u < p.ns; ++u) v += l[(size_t)u * p.pstride];
    return v;
}

// The k selected experts of a row from its logits sl [E]: lane j < k returns the
// expert of slot j.  sc: E doubles of scratch.  Group g's score by lane g.
__device__ __noinline__ int select_exact(const TopkParams& p, const float* sl, double* sc, int lane) {
    const bool biased = mode_has_bias(p.r.mode), sig = mode_sigmoid(p.r.mode);
    double m = 0., z = 1.;
    if (!sig && (biased || p.r.top2)) {
        m = -INFINITY;
        for (int e = lane; e < p.E; e += 32) m = fmax(m, (double)sl[e]);
        for (int o = 16; o > 0; o >>= 1) m = fmax(m, __shfl_xor_sync(0xffffffffu, m, o));
        z = 0.;
        for (int e = lane; e < p.E; e += 32) z += exp((double)sl[e] - m);
        for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    }
    auto prob = [&](float l) { return sig ? 1. / (1. + exp(-(double)l)) : exp((double)l - m) / z; };
    auto clean = [](double s) { return s != s ? -(double)INFINITY : s; };   // NaN ranks last
    for (int e = lane; e < p.E; e += 32) sc[e] = clean(biased ? prob(sl[e]) + p.bias[e] : (double)sl[e]);
    __syncwarp();
    uint32_t alive = 0xffffffffu;
    const int size = p.E / p.r.groups;
    if (p.r.groups > 1) {
        double a = -INFINITY, b = -INFINITY;
        if (lane < p.r.groups) {
            for (int i = 0; i < size; ++i) {
                const int e = lane * size + i;
                const double s = p.r.top2 && !biased ? clean(prob(sl[e])) : sc[e];
                if (s > a) { b = a; a = s; }
                else if (s > b) b = s;
            }
            if (p.r.top2 && size > 1) a += b;
        }
        int ahead = 0;
        for (int g = 0; g < p.r.groups; ++g) {
            const double o = __shfl_sync(0xffffffffu, a, g);
            ahead += (o > a || (o == a && g < lane)) ? 1 : 0;
        }
        alive = __ballot_sync(0xffffffffu, lane < p.r.groups && ahead < p.r.kept);
    }
    // Round j takes the best (score, lower index) behind round j - 1's.
    double last = INFINITY;
    int last_e = -1, mine = 0;
    for (int j = 0; j < p.k; ++j) {
        double best = -INFINITY;
        int best_e = 1 << 30;
        for (int e = lane; e < p.E; e += 32) {
            const double s = sc[e];
            if (!((alive >> (e / size)) & 1u) && p.r.groups > 1) continue;
            if (!(s < last || (s == last && e > last_e))) continue;
            if (s > best || (s == best && e < best_e)) { best = s; best_e = e; }
        }
        for (int o = 16; o > 0; o >>= 1) {
            const double s = __shfl_xor_sync(0xffffffffu, best, o);
            const int e = __shfl_xor_sync(0xffffffffu, best_e, o);
            if (s > best || (s == best && e < best_e)) { best = s; best_e = e; }
        }
        last = best;
        last_e = best_e;
        if (lane == j) mine = best_e;
    }
    return mine;
}

// The weights of the selected logits (lane j < k holds slot j's logit l):
// p, renormalised over the k when norm, times scale.  Renormalised weights are
// ratios, formed from exp(l - M) with M the largest selected logit (sigmoid: at
// most 0), so that they neither overflow nor vanish together.  Softmax without
// renormalising takes the row's largest logit m and sum z of exp(l - m).
__device__ __forceinline__ float row_weight(const TopkParams& p, float l, float m, float z, int lane) {
    const bool in = lane < p.k, sig = mode_sigmoid(p.r.mode);
    float v;
    if (p.norm) {
        float M = in ? l : -INFINITY;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        if (sig) {
            M = fminf(M, 0.f);
            v = l > 0.f ? 1.f / (1.f + expf(-l)) : expf(l - M) / (1.f + expf(l));
        } else {
            v = expf(l - M);
        }
        if (M == -INFINITY && !(l != l)) v = 0.f;
        if (!in) v = 0.f;
        const float tot = warp_sum(v);
        v = tot == 0.f ? 0.f : v / tot;
    } else if (sig) {
        v = 1.f / (1.f + expf(-l));
    } else {
        v = m == -INFINITY && !(l != l) ? 0.f : expf(l - m) / z;
    }
    return v * p.scale;
}

// fp32 as an unsigned integer of the same order (-0 as +0).
__device__ __forceinline__ uint32_t ordered(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t k) {
    return __uint_as_float(k ^ ((k & 0x80000000u) ? 0x80000000u : 0xffffffffu));
}

// V values of a row from expert e0 on; -inf past E.
template <int TYPE, int V>
__device__ __forceinline__ void load_values(const TopkParams& p, int64_t t, int e0, bool vec, float (&l)[V]) {
    constexpr int kPer = TYPE == MOE_F32 ? 4 : 8;   // elements of 16 bytes
    if (V >= kPer && vec) {
        const size_t at = (size_t)(t * p.row_stride) + e0;
#pragma unroll
        for (int c = 0; c < V / kPer; ++c) {
            if (e0 + c * kPer >= p.E) {   // (E is whole vectors)
#pragma unroll
                for (int i = 0; i < kPer; ++i) l[c * kPer + i] = -INFINITY;
                continue;
            }
            if constexpr (TYPE == MOE_F32) {
                const float4 v = __ldg(reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p.logits) + at) + c);
                l[4 * c] = v.x; l[4 * c + 1] = v.y; l[4 * c + 2] = v.z; l[4 * c + 3] = v.w;
            } else {
                const uint4 v = __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p.logits) + at) + c);
                const uint32_t w4[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if constexpr (TYPE == MOE_BF16) {
                        l[8 * c + 2 * i] = bf16_lo(w4[i]);
                        l[8 * c + 2 * i + 1] = bf16_hi(w4[i]);
                    } else {
                        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w4[i]));
                        l[8 * c + 2 * i] = f.x;
                        l[8 * c + 2 * i + 1] = f.y;
                    }
                }
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) l[i] = e0 + i < p.E ? load_logit<TYPE>(p, t, e0 + i) : -INFINITY;
}

template <int N> __device__ __forceinline__ void sort_desc(uint32_t (&v)[N]) {   // odd-even merge network, N a power of two
#pragma unroll
    for (int q = 1; q < N; q <<= 1)
#pragma unroll
        for (int r = q; r > 0; r >>= 1)
#pragma unroll
            for (int j = r % q; j + r < N; j += 2 * r)
#pragma unroll
                for (int i = 0; i < r; ++i)
                    if (i + j + r < N && (i + j) / (2 * q) == (i + j + r) / (2 * q)) {
                        const uint32_t a = max(v[i + j], v[i + j + r]), b = min(v[i + j], v[i + j + r]);
                        v[i + j] = a;
                        v[i + j + r] = b;
                    }
}

// TYPE: of the logits.  V: experts of a lane (32 V >= E).
template <int TYPE, int V>
__global__ void __launch_bounds__(32 * kRowWarps, V <= 8 ? 6 : 1) topk_rows_kernel(const TopkParams p, int vec) {
    constexpr int W = V < 8 ? V : 8, L = V / W;      // lists of W
    extern __shared__ __align__(16) uint8_t dyn[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int E = p.E, k = p.k, e0 = lane * V;
    // Per warp: logits and selection scores [32 V], 64-bit scratch [E] (256 bytes at least).
    float* sl = reinterpret_cast<float*>(dyn) + (size_t)warp * (64 * V);
    float* ss = sl + 32 * V;
    double* sc = reinterpret_cast<double*>(dyn + (size_t)kRowWarps * 256 * V) + (size_t)warp * max(E, 32);
    const bool biased = mode_has_bias(p.r.mode), sig = mode_sigmoid(p.r.mode);
    const int size = E / p.r.groups;                 // experts of a group
    const bool need_p = biased || (p.r.groups > 1 && p.r.top2);
    const bool need_z = !sig && (need_p || !p.norm);
    const uint32_t ibits = E <= 256 ? 8 : (E <= 512 ? 9 : 10), imask = (1u << ibits) - 1u;
    const float bucket = exp2f((float)ibits - 22.f);
    pdl_wait();

    for (int64_t t = (int64_t)blockIdx.x * kRowWarps + warp; t < p.n; t += (int64_t)gridDim.x * kRowWarps) {
        float l[V];
        load_values<TYPE, V>(p, t, e0, vec != 0, l);
        if (p.lsum)
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (e0 + i < E) p.lsum[(size_t)t * E + e0 + i] = l[i];
        __syncwarp();   // the row before is done with shared memory
#pragma unroll
        for (int i = 0; i < V; ++i) sl[e0 + i] = l[i];

        // Softmax over the row: the largest logit and the sum of exp(l - m).
        float m = -INFINITY, z = 1.f;
        if (need_z) {
#pragma unroll
            for (int i = 0; i < V; ++i) m = fmaxf(m, l[i]);
            m = unordered(__reduce_max_sync(0xffffffffu, ordered(m)));
            z = 0.f;
#pragma unroll
            for (int i = 0; i < V; ++i) z += expf(l[i] - m);
            z = warp_sum(z);
        }
        // Selection scores.  Errors in 32 bits: of a sigmoid 2^-21 (ex2 and rcp within
        // 2^-22, its argument's rounding times s (1 - s)); of a softmax 2^-18 of itself
        // (the argument's rounding, the sum); of the sum with the bias half an ulp.
        float s[V];
        float perr = 0.f;                                // error of a p
        if (need_p) {
            const float rz = 1.f / z;
#pragma unroll
            for (int i = 0; i < V; ++i)
                s[i] = sig ? __fdividef(1.f, 1.f + __expf(-l[i])) : expf(l[i] - m) * rz;
            if (biased)
#pragma unroll
                for (int i = 0; i < V; ++i) s[i] += e0 + i < E ? __ldg(p.bias + e0 + i) : 0.f;
            perr = sig ? 0x1p-21f : 0x1p-18f * rz;
        }
        bool clear = true, gclear = true;
        uint32_t alive = 0xffffffffu;                    // bit i: expert e0 + i may be chosen
        if (p.r.groups > 1) {
            // Group scores: the sum of the two best p (+ bias), or the best selection score.
            const bool by_p = p.r.top2 || biased;
            const bool lanes = size % V == 0 && ((size / V) & (size / V - 1)) == 0;   // groups are 2^j whole lanes
            float a = -INFINITY, b = -INFINITY;
            int grp;
            if (lanes) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float v = by_p ? s[i] : l[i];
                    b = fmaxf(b, fminf(a, v));
                    a = fmaxf(a, v);
                }
                for (int o = 1; o < size / V; o <<= 1) {
                    const float a2 = __shfl_xor_sync(0xffffffffu, a, o), b2 = __shfl_xor_sync(0xffffffffu, b, o);
                    b = fmaxf(fminf(a, a2), fmaxf(b, b2));
                    a = fmaxf(a, a2);
                }
                grp = lane / (size / V);
            } else {
                if (by_p) {
#pragma unroll
                    for (int i = 0; i < V; ++i) ss[e0 + i] = s[i];
                }
                __syncwarp();
                grp = lane;
                if (lane < p.r.groups) {
                    const float* src = (by_p ? ss : sl) + lane * size;
                    for (int i = 0; i < size; ++i) {
                        b = fmaxf(b, fminf(a, src[i]));
                        a = fmaxf(a, src[i]);
                    }
                }
                __syncwarp();
            }
            const float gs = p.r.top2 ? (size > 1 ? a + b : a) : a;
            const int per = lanes ? size / V : 1;        // lanes of a group
            int ahead = 0;
            for (int g = 0; g < p.r.groups; ++g) {
                const float o = __shfl_sync(0xffffffffu, gs, g * per);
                ahead += (o > gs || (o == gs && g < grp)) ? 1 : 0;
            }
            const bool in = grp < p.r.groups, keep = in && ahead < p.r.kept;
            const float worst = unordered(__reduce_min_sync(0xffffffffu, keep ? ordered(gs) : 0xffffffffu));
            const float best = unordered(__reduce_max_sync(0xffffffffu, in && !keep ? ordered(gs) : ordered(-INFINITY)));
            if (by_p && p.r.kept < p.r.groups)
                clear = worst - best > 4.f * perr + 0x1p-21f * fmaxf(fabsf(worst), fabsf(best));
            // (The best logits decide exactly, but a NaN is for the 64-bit path.)
            else if (!(worst >= best)) clear = false;
            gclear = __all_sync(0xffffffffu, clear);
            const uint32_t kept = lanes ? 0u : __ballot_sync(0xffffffffu, keep);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const bool on = lanes ? keep : ((kept >> ((e0 + i) / size)) & 1u) != 0u;
                if (!on) alive &= ~(1u << i);
            }
        }
        if (!biased)
#pragma unroll
            for (int i = 0; i < V; ++i) s[i] = l[i];
        const float serr = biased ? perr : 0.f;

        uint32_t key[L][W];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float v = s[i] == s[i] ? s[i] : -INFINITY;   // NaN ranks last
            if (biased) ss[e0 + i] = s[i];
            const bool on = e0 + i < E && ((alive >> i) & 1u);
            key[i / W][i % W] = on ? (ordered(v) & ~imask) | (imask - (uint32_t)(e0 + i)) : 0u;
        }
#pragma unroll
        for (int q = 0; q < L; ++q) sort_desc(key[q]);
        uint32_t mine = 0u;
        for (int j = 0; j <= k; ++j) {                    // one more than k: the best left
            uint32_t h = key[0][0];
#pragma unroll
            for (int q = 1; q < L; ++q) h = max(h, key[q][0]);
            const uint32_t w = __reduce_max_sync(0xffffffffu, h);
            if (lane == j) mine = w;                      // (k = 32: the last is dropped and not needed, see below)
#pragma unroll
            for (int q = 0; q < L; ++q)
                if (key[q][0] == w) {
#pragma unroll
                    for (int i = 0; i + 1 < W; ++i) key[q][i] = key[q][i + 1];
                    key[q][W - 1] = 0u;
                }
        }
        __syncwarp();
        int e = (int)(imask - (mine & imask));
        const float* rank = biased ? ss : sl;
        float sj = mine != 0u ? rank[e] : -INFINITY;
        {
            const float nx = __shfl_down_sync(0xffffffffu, sj, 1);
            const int ne = __shfl_down_sync(0xffffffffu, e, 1);
            const bool last_in = __shfl_down_sync(0xffffffffu, mine != 0u ? 1 : 0, 1) == 0;
            if (lane < k) {
                // What the index bits hide of a score (two scores that close are within a binade).
                const float trunc = fmaxf(fabsf(sj), fabsf(nx)) * bucket + 1e-38f;
                const float tol = 2.f * serr + (biased ? 0x1p-22f * fabsf(sj) : 0.f);
                bool ok;
                if (lane == 31) ok = false;               // (32 chosen: the best left was not kept)
                else if (lane == k - 1 && last_in) ok = true;   // nothing is left
                else if (serr > 0.f || (TYPE == MOE_F32 && lane == k - 1)) ok = sj - nx > tol + (lane == k - 1 ? trunc : 0.f);
                else ok = sj > nx || (sj == nx && e < ne);
                clear = clear && ok;
            }
        }
        if (!__all_sync(0xffffffffu, clear)) {
            // Not clear.  With the kept groups clear, the choice is among the experts
            // whose score reaches the k-th one's, less what the index bits and the
            // errors hide: one lane each, if they are at most 32.
            const float at_k = __shfl_sync(0xffffffffu, sj, k - 1);
            const float thr = at_k - (fabsf(at_k) * (2.f * bucket) + 2.f * serr + 0x1p-21f * fabsf(at_k) + 1e-38f);
            uint32_t cand = 0u;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (e0 + i < E && s[i] >= thr) cand |= 1u << i;
            cand &= alive;
            int before = __popc(cand);
            const int own = before;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, before, o);
                if (lane >= o) before += y;
            }
            const int total = __shfl_sync(0xffffffffu, before, 31);
            // (-inf or NaN at the k-th, a softmax with a bias, unclear groups: every score in 64 bits.)
            if (gclear && at_k > -3.0e38f && total <= 32 && !(biased && !sig)) {
                int* list = reinterpret_cast<int*>(sc);
                int at = before - own;
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if ((cand >> i) & 1u) list[at++] = e0 + i;
                __syncwarp();
                const int ce = lane < total ? list[lane] : 0;
                double v = (double)sl[ce];
                if (biased) v = 1. / (1. + exp(-v)) + (double)__ldg(p.bias + ce);
                // As integers of the same order.
                long long q = __double_as_longlong(v + 0.0);
                q ^= (long long)((unsigned long long)(q >> 63) >> 1);
                int ahead = 0;
                for (int i = 0; i < total; ++i) {
                    const long long o = __shfl_sync(0xffffffffu, q, i);
                    ahead += (o > q || (o == q && i < lane)) ? 1 : 0;   // (the list is in index order)
                }
                __syncwarp();
                if (lane < total && ahead < k) list[32 + ahead] = ce;
                __syncwarp();
                e = lane < k ? list[32 + lane] : 0;
                __syncwarp();
            } else {
                e = select_exact(p, sl, sc, lane);
            }
        }
        const float v = row_weight(p, lane < k ? sl[e] : 0.f, m, z, lane);
        if (lane < k) {
            p.idx[(size_t)t * k + lane] = e;
            p.w[(size_t)t * k + lane] = v;
        }
    }
    pdl_trigger();
}

template <int TYPE, int V>
cudaError_t launch_rows(const TopkParams& p, int num_sms, cudaStream_t st) {
    constexpr int kPer = TYPE == MOE_F32 ? 4 : 8;
    const size_t esize = TYPE == MOE_F32 ? 4 : 2;
    const int vec = p.ns == 1 && reinterpret_cast<uintptr_t>(p.logits) % 16 == 0 && p.row_stride * esize % 16 == 0 && p.E % kPer == 0;
    const int64_t blocks = ((int64_t)p.n + kRowWarps - 1) / kRowWarps;
    const size_t smem = (size_t)kRowWarps * (256 * V + std::max(8 * p.E, 256));   // <= 64 KB
    static std::mutex mu;
    static bool configured[128] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) return cudaErrorInvalidDevice;
    auto kern = topk_rows_kernel<TYPE, V>;
    if (V == 32) {
        std::lock_guard<std::mutex> lock(mu);
        if (!configured[dev]) {
            const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 64 * 1024);
            if (e != cudaSuccess) return e;
            configured[dev] = true;
        }
    }
    const int grid = (int)std::min<int64_t>(blocks, (int64_t)num_sms * 8);
    launch_pdl(kern, grid, 32 * kRowWarps, smem, st, p, vec);
    return cudaGetLastError();
}

template <int TYPE>
cudaError_t launch_type(const TopkParams& p, int num_sms, cudaStream_t st) {
    if (p.E <= 32) return launch_rows<TYPE, 1>(p, num_sms, st);
    if (p.E <= 64) return launch_rows<TYPE, 2>(p, num_sms, st);
    if (p.E <= 128) return launch_rows<TYPE, 4>(p, num_sms, st);
    if (p.E <= 256) return launch_rows<TYPE, 8>(p, num_sms, st);
    if (p.E <= 512) return launch_rows<TYPE, 16>(p, num_sms, st);
    return launch_rows<TYPE, 32>(p, num_sms, st);
}

}  // namespace

cudaError_t launch_topk_rows(const void* logits, int dtype, int64_t row_stride, int ns, int64_t pstride, float* lsum,
                             int n, int E, int k, int32_t routing, const float* bias, int norm, float scale,
                             int32_t* idx, float* w, int num_sms, cudaStream_t st) {
    TopkParams p{logits, row_stride, ns, pstride, lsum, n, E, k, routing_of(routing), bias, norm, scale, idx, w};
    if (dtype == MOE_F32) return launch_type<MOE_F32>(p, num_sms, st);
    if (dtype == MOE_BF16) return launch_type<MOE_BF16>(p, num_sms, st);
    return launch_type<MOE_F16>(p, num_sms, st);
}

}  // namespace moe
