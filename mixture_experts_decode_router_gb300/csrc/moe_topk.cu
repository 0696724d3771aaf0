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
// list.  Bound by instruction issue: about 850 of a warp for a row of 256 sigmoid scores
// with a bias, 8 groups and 8 chosen, at 0.59 a scheduler and cycle: 32768 such rows take
// 37 us on GB300, 0.91 TB/s of fp32 logits; one row 3.2 us, most of it launch and
// latency.  (Every score in 64 bits: 1116 us and 28 us.)
#include <cuda_fp16.h>

#include <algorithm>
#include <climits>
#include <mutex>

#include "moe_launch.cuh"

namespace moe {

namespace {

constexpr int kRowWarps = 4;   // rows per block
constexpr int kMinBlocks = 6;  // blocks of an SM (256 experts and fewer)

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

// A double as a signed integer of the same order (-0 as +0); NaN as the lowest.
__device__ __forceinline__ long long ordered64(double v) {
    const long long q = __double_as_longlong(v + 0.0);
    return v != v ? LLONG_MIN : q ^ (long long)((unsigned long long)(q >> 63) >> 1);
}

// The k selected experts of a row from its logits sl [E], every score in 64 bits:
// lane j < k returns the expert of slot j.  sc: E 64-bit words of scratch.
__device__ __noinline__ int select_exact(const TopkParams& p, const float* sl, double* sc, int lane) {
    const bool biased = mode_has_bias(p.r.mode), sig = mode_sigmoid(p.r.mode);
    long long* key = reinterpret_cast<long long*>(sc);   // the scores, as integers of their order
    double m = 0., z = 1.;
    if (!sig && (biased || (p.r.groups > 1 && p.r.top2))) {
        float mf = -INFINITY;
        for (int e = lane; e < p.E; e += 32) mf = fmaxf(mf, sl[e]);
        for (int o = 16; o > 0; o >>= 1) mf = fmaxf(mf, __shfl_xor_sync(0xffffffffu, mf, o));
        m = mf;
        z = 0.;
        for (int e = lane; e < p.E; e += 32) z += exp((double)sl[e] - m);
        for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    }
    auto prob = [&](float l) { return sig ? 1. / (1. + exp(-(double)l)) : exp((double)l - m) / z; };
    const int size = p.E / p.r.groups;
    const bool by_p = biased || (p.r.groups > 1 && p.r.top2);
    uint32_t alive = 0xffffffffu;
    if (p.r.groups > 1) {
        // Group scores by p (+ bias), or by the logits.
        for (int e = lane; e < p.E; e += 32) {
            const double v = by_p ? prob(sl[e]) + (biased ? (double)__ldg(p.bias + e) : 0.) : (double)sl[e];
            sc[e] = v != v ? -(double)INFINITY : v;
        }
        __syncwarp();
        double a = -INFINITY, b = -INFINITY;
        if (lane < p.r.groups) {
            for (int i = 0; i < size; ++i) {
                const double s = sc[lane * size + i];
                if (s > a) { b = a; a = s; }
                else if (s > b) b = s;
            }
            if (p.r.top2 && size > 1) a += b;
        }
        __syncwarp();
        const long long mine = ordered64(a);
        int ahead = 0;
        for (int g = 0; g < p.r.groups; ++g) {
            const long long o = __shfl_sync(0xffffffffu, mine, g);
            ahead += (o > mine || (o == mine && g < lane)) ? 1 : 0;
        }
        alive = __ballot_sync(0xffffffffu, lane < p.r.groups && ahead < p.r.kept);
    }
    for (int e = lane; e < p.E; e += 32) {
        if (p.r.groups > 1 && biased) key[e] = ordered64(sc[e]);
        else key[e] = ordered64(biased ? prob(sl[e]) + (double)__ldg(p.bias + e) : (double)sl[e]);
        if (key[e] == LLONG_MIN) key[e] = ordered64(-(double)INFINITY);   // NaN ranks with -inf
    }
    __syncwarp();
    // Round j takes the best (score, lower index) behind round j - 1's.
    long long last = LLONG_MAX;
    int last_e = -1, mine_e = 0;
    for (int j = 0; j < p.k; ++j) {
        long long best = LLONG_MIN;
        int best_e = 1 << 30;
        for (int e = lane; e < p.E; e += 32) {
            const long long s = key[e];
            if (p.r.groups > 1 && !((alive >> (e / size)) & 1u)) continue;
            if (!(s < last || (s == last && e > last_e))) continue;
            if (s > best) { best = s; best_e = e; }
        }
        for (int o = 16; o > 0; o >>= 1) {
            const long long s = __shfl_xor_sync(0xffffffffu, best, o);
            const int e = __shfl_xor_sync(0xffffffffu, best_e, o);
            if (s > best || (s == best && e < best_e)) { best = s; best_e = e; }
        }
        last = best;
        last_e = best_e;
        if (lane == j) mine_e = best_e;
    }
    return mine_e;
}

// The weights of the selected logits (lane j < k holds slot j's logit l):
// p, renormalised over the k when norm, times scale.  Renormalised weights are
// ratios, formed from exp(l - M) with M the largest selected logit (sigmoid: at
// most 0), so that they neither overflow nor vanish together.  Softmax without
// renormalising takes the row's largest logit m and sum z of exp(l - m).  (expf and whole
// quotients: __expf is off by an ulp for each unit of its argument, 60 ulps of a sigmoid's
// weight at a logit of -60; it saves nothing that 32768 rows show.)
__device__ __forceinline__ float row_weight(const TopkParams& p, float l, float m, float z, int lane) {
    const bool in = lane < p.k, sig = mode_sigmoid(p.r.mode);
    float v = sig ? 1.f / (1.f + expf(-l)) : expf(l - m) / z;
    if (!p.norm) return (m == -INFINITY && !sig && !(l != l) ? 0.f : v) * p.scale;
    // Softmax ratios, and sigmoids that are all small, from the largest selected logit.
    if (!sig || !__any_sync(0xffffffffu, in && l > -60.f)) {
        float M = in ? l : -INFINITY;
        for (int o = 1; o < p.k; o <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        M = __shfl_sync(0xffffffffu, M, 0);
        v = expf(l - M);   // (a small sigmoid is exp(l) to within its rounding)
        if (M == -INFINITY && !(l != l)) v = 0.f;
    }
    if (!in) v = 0.f;
    float tot = v;
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) tot += __shfl_xor_sync(0xffffffffu, tot, o);
    if (p.k > 8) {
        tot += __shfl_xor_sync(0xffffffffu, tot, 8);
        tot += __shfl_xor_sync(0xffffffffu, tot, 16);
    }
    return tot == 0.f ? 0.f : v / tot * p.scale;
}

// V floats of a lane to and from shared memory (16-byte aligned when V is a multiple of 4).
template <int V> __device__ __forceinline__ void put(float* d, const float (&v)[V]) {
    if constexpr (V % 4 == 0) {
#pragma unroll
        for (int i = 0; i < V; i += 4) *reinterpret_cast<float4*>(d + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) d[i] = v[i];
    }
}
template <int V> __device__ __forceinline__ void get(const float* d, float (&v)[V]) {
    if constexpr (V % 4 == 0) {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const float4 f = *reinterpret_cast<const float4*>(d + i);
            v[i] = f.x; v[i + 1] = f.y; v[i + 2] = f.z; v[i + 3] = f.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = d[i];
    }
}

// fp32 as an unsigned integer of the same order.
__device__ __forceinline__ uint32_t ordered(float v) {
    const uint32_t b = __float_as_uint(v);
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

// The experts e0 + i (i < V) of all lanes that `in` picks, in index order, to list (the
// first 32); returns how many there are.
template <int V, typename In>
__device__ __forceinline__ int compact(In in, int e0, int lane, int* list) {
    uint32_t cand = 0u;
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (in(i)) cand |= 1u << i;
    int before = __popc(cand);
    const int own = before;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += y;
    }
    const int total = __shfl_sync(0xffffffffu, before, 31);
    int at = before - own;
#pragma unroll
    for (int i = 0; i < V; ++i)
        if ((cand >> i) & 1u) {
            if (at < 32) list[at] = e0 + i;
            ++at;
        }
    __syncwarp();
    return total;
}

// TYPE: of the logits.  V: experts of a lane (32 V >= E).
template <int TYPE, int V>
__global__ void __launch_bounds__(32 * kRowWarps, V <= 8 ? kMinBlocks : 1) topk_rows_kernel(const TopkParams p, int vec) {
    constexpr int W = V < 8 ? V : 8, L = V / W;      // lists of W
    extern __shared__ __align__(16) uint8_t dyn[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int E = p.E, k = p.k, e0 = lane * V;
    // The bias [32 V]; per warp: logits and selection scores [32 V], 64-bit scratch [E]
    // (256 bytes at least).
    float* sb = reinterpret_cast<float*>(dyn);
    float* sl = sb + 32 * V + (size_t)warp * (64 * V);
    float* ss = sl + 32 * V;
    double* sc = reinterpret_cast<double*>(dyn + (size_t)(1 + 2 * kRowWarps) * 128 * V) + (size_t)warp * max(E, 32);
    // Bit i: expert e0 + i exists.
    const uint32_t valid = E - e0 >= V ? 0xffffffffu : (E > e0 ? (1u << (E - e0)) - 1u : 0u);
    const bool biased = mode_has_bias(p.r.mode), sig = mode_sigmoid(p.r.mode);
    const int size = E / p.r.groups;                 // experts of a group
    const bool need_p = biased || (p.r.groups > 1 && p.r.top2);
    const bool need_z = !sig && (need_p || !p.norm);
    const uint32_t ibits = E <= 256 ? 8 : (E <= 512 ? 9 : 10), imask = (1u << ibits) - 1u;
    const float bucket = exp2f((float)ibits - 22.f);
    // Groups of 2^j whole lanes: every lane of a group holds its scores; other sizes: lane
    // g those of group g.
    const bool lanes = size % V == 0 && ((size / V) & (size / V - 1)) == 0;
    const int per = lanes ? size / V : 1, grp = lane / per, e_grp = e0 / size;
    const bool in = grp < p.r.groups;
    pdl_wait();
    if (biased) {
        for (int i = threadIdx.x; i < 32 * V; i += 32 * kRowWarps) sb[i] = i < E ? __ldg(p.bias + i) : 0.f;
        __syncthreads();
    }

    for (int64_t t = (int64_t)blockIdx.x * kRowWarps + warp; t < p.n; t += (int64_t)gridDim.x * kRowWarps) {
        float l[V];
        load_values<TYPE, V>(p, t, e0, vec != 0, l);
        if (p.lsum)
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (e0 + i < E) p.lsum[(size_t)t * E + e0 + i] = l[i];
        __syncwarp();   // the row before is done with shared memory
        put<V>(sl + e0, l);

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
#pragma unroll
        for (int i = 0; i < V; ++i) s[i] = l[i];
        if (need_p) {
            const float rz = 1.f / z;
#pragma unroll
            for (int i = 0; i < V; ++i)
                s[i] = sig ? __fdividef(1.f, 1.f + __expf(-l[i])) : expf(l[i] - m) * rz;
            if (biased) {
                float b[V];
                get<V>(sb + e0, b);
#pragma unroll
                for (int i = 0; i < V; ++i) s[i] += b[i];
            }
            perr = sig ? 0x1p-21f : 0x1p-18f * rz;
        }
        bool clear = true, gclear = true;
        uint32_t alive = valid;                          // bit i: expert e0 + i may be chosen
        if (p.r.groups > 1) {
            // Group scores: the sum of the two best p (+ bias), or the best selection score.
            const bool by_p = need_p;
            float a = -INFINITY, b = -INFINITY;
            if (lanes) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    b = fmaxf(b, fminf(a, s[i]));
                    a = fmaxf(a, s[i]);
                }
                for (int o = 1; o < per; o <<= 1) {
                    const float a2 = __shfl_xor_sync(0xffffffffu, a, o), b2 = __shfl_xor_sync(0xffffffffu, b, o);
                    b = fmaxf(fminf(a, a2), fmaxf(b, b2));
                    a = fmaxf(a, a2);
                }
            } else {
                put<V>(ss + e0, s);
                __syncwarp();
                if (lane < p.r.groups) {
                    const float* src = ss + lane * size;
                    for (int i = 0; i < size; ++i) {
                        b = fmaxf(b, fminf(a, src[i]));
                        a = fmaxf(a, src[i]);
                    }
                }
                __syncwarp();
            }
            const bool two = p.r.top2 && size > 1;
            const float gs = (two ? a + b : a) + 0.f;
            // Ranks by integers of the scores' order with the group in the low bits.
            const uint32_t gk = in ? (ordered(gs) & ~31u) | (31u - grp) : 0u;
            int ahead = 0;
            for (int g = 0; g < p.r.groups; ++g) ahead += __shfl_sync(0xffffffffu, gk, g * per) > gk ? 1 : 0;
            bool keep = in && ahead < p.r.kept;
            if (p.r.kept < p.r.groups) {
                // Whether every kept group is clear of every other: the lowest that the scores of
                // the kept can be against the highest of the rest.  A score is off by `tol` of
                // itself, and, of p (+ bias), by the errors of its p and the roundings of its
                // terms.  These go with the terms: a sum of two large biases of opposite sign has
                // them whole.  (tol 0 of logits: the scores are exact.  An infinite score is exact,
                // its terms' roundings do not reach it; a NaN is clear of none.)
                const float terms = two ? fabsf(a) + fabsf(b) : fabsf(a);
                const float fix = by_p ? (two ? 2.f : 1.f) * perr + 0x1p-22f * terms : 1e-38f;
                auto apart = [&](float tol) {
                    const bool exact = tol == 0.f && !by_p;
                    const float err = exact || fabsf(gs) == INFINITY ? 0.f : fix + tol * fabsf(gs);
                    const float lo = gs == gs ? gs - err : -INFINITY, hi = gs == gs ? gs + err : INFINITY;
                    const float worst = unordered(__reduce_min_sync(0xffffffffu, keep ? ordered(lo) : 0xffffffffu));
                    const float best = unordered(__reduce_max_sync(0xffffffffu, in && !keep ? ordered(hi) : 0u));
                    return exact ? worst >= best : worst > best;
                };
                // (The index hides 32 ulps of a score in fp32, nothing of 16-bit logits.)
                clear = apart(TYPE == MOE_F32 || by_p ? 0x1p-17f : 0.f);
                if (!clear) {                             // the whole scores
                    ahead = 0;
                    for (int g = 0; g < p.r.groups; ++g) {
                        const float o = __shfl_sync(0xffffffffu, gs, g * per);
                        ahead += (o > gs || (o == gs && g < grp)) ? 1 : 0;
                    }
                    keep = in && ahead < p.r.kept;
                    clear = apart(0.f);
                    if (by_p && !__all_sync(0xffffffffu, clear) && (sig || !biased)) {
                        // The experts that can be a group's two best (or best) in 64 bits, one lane
                        // each; without a bias the softmax's common factor is left out.
                        // (An infinite score is exact: less an error that goes with it, it would be NaN.)
                        const float from = p.r.top2 ? b : a;
                        const float low = fabsf(from) == INFINITY ? from : from - 4.f * perr - 0x1p-21f * fabsf(from);
                        int* list = reinterpret_cast<int*>(sc);
                        const int total = compact<V>([&](int i) {
                            const int ge = lanes ? grp * per : min((e0 + i) / size, 31);   // the lane that holds the group's scores
                            const float lo = __shfl_sync(0xffffffffu, low, ge);
                            return ((valid >> i) & 1u) && s[i] >= lo;
                        }, e0, lane, list);
                        if (total <= 32) {
                            const int ce = lane < total ? list[lane] : 0;
                            double v = sig ? 1. / (1. + exp(-(double)sl[ce])) : exp((double)sl[ce] - (double)m);
                            if (biased) v += (double)sb[ce];
                            const int cg = lane < total ? ce / size : 64;
                            double va = -INFINITY, vb = -INFINITY;
                            for (int i = 0; i < total; ++i) {
                                const double o = __shfl_sync(0xffffffffu, v, i);
                                if (__shfl_sync(0xffffffffu, cg, i) != grp) continue;
                                if (ordered64(o) > ordered64(va)) { vb = va; va = o; }
                                else if (ordered64(o) > ordered64(vb)) vb = o;
                            }
                            const long long q = ordered64(p.r.top2 && size > 1 ? va + vb : va);
                            ahead = 0;
                            for (int g = 0; g < p.r.groups; ++g) {
                                const long long o = __shfl_sync(0xffffffffu, q, g * per);
                                ahead += (o > q || (o == q && g < grp)) ? 1 : 0;
                            }
                            keep = in && ahead < p.r.kept;
                            clear = true;
                        }
                        __syncwarp();
                    }
                }
            }
            gclear = __all_sync(0xffffffffu, clear);
            const uint32_t kept = lanes ? 0u : __ballot_sync(0xffffffffu, keep);
            if (lanes) {
                if (!keep) alive = 0u;
            } else {
                int gi = e_grp, r = e0 - gi * size;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    if (!((kept >> (gi & 31)) & 1u)) alive &= ~(1u << i);
                    if (++r == size) { r = 0; ++gi; }
                }
            }
        }
        if (!biased)
#pragma unroll
            for (int i = 0; i < V; ++i) s[i] = l[i];
        const float serr = biased ? perr : 0.f;

        if (biased) put<V>(ss + e0, s);
        uint32_t key[L][W];
        bool nan = false;
        const uint32_t c0 = imask - (uint32_t)e0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            nan = nan || s[i] != s[i];
            const uint32_t o = ordered(biased ? s[i] : s[i] + 0.0f);   // (-0 ties with +0)
            key[i / W][i % W] = (alive & (1u << i)) ? (o & ~imask) | (c0 - i) : 0u;
        }
        // A NaN ranks last: by the 64-bit path.  (Past E the logits are -inf.)
        if (nan && valid) clear = false;
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
            for (int q = 0; q < L; ++q) {
                const bool won = key[q][0] == w;
#pragma unroll
                for (int i = 0; i + 1 < W; ++i) key[q][i] = won ? key[q][i + 1] : key[q][i];
                key[q][W - 1] = won ? 0u : key[q][W - 1];
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
            int* list = reinterpret_cast<int*>(sc);
            const int total = compact<V>([&](int i) { return ((alive >> i) & 1u) && s[i] >= thr; }, e0, lane, list);
            // (Infinite scores, NaN, a softmax with a bias, unclear groups: every score in 64 bits.)
            if (gclear && !__any_sync(0xffffffffu, nan) && fabsf(at_k) < 3.0e38f && total >= k && total <= 32 && !(biased && !sig)) {
                const int ce = lane < total ? list[lane] : 0;
                // By their whole 32-bit scores, if these are clear; else in 64 bits.
                const float v32 = lane < total ? (biased ? ss : sl)[ce] : -INFINITY;
                int ahead = 0;
                bool close = false;
                const float near = 2.f * serr + 0x1p-22f * fabsf(v32);
                for (int i = 0; i < total; ++i) {
                    const float o = __shfl_sync(0xffffffffu, v32, i);
                    ahead += (o > v32 || (o == v32 && i < lane)) ? 1 : 0;   // (the list is in index order)
                    close = close || (i != lane && fabsf(o - v32) <= near);
                }
                if (biased && __any_sync(0xffffffffu, lane < total && close)) {
                    const long long q = ordered64(1. / (1. + exp(-(double)sl[ce])) + (double)sb[ce]);
                    ahead = 0;
                    for (int i = 0; i < total; ++i) {
                        const long long o = __shfl_sync(0xffffffffu, q, i);
                        ahead += (o > q || (o == q && i < lane)) ? 1 : 0;
                    }
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
    const size_t smem = (size_t)128 * V + (size_t)kRowWarps * (256 * V + std::max(8 * p.E, 256));   // <= 68 KB
    static std::mutex mu;
    static bool configured[128] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) return cudaErrorInvalidDevice;
    auto kern = topk_rows_kernel<TYPE, V>;
    if (V == 32) {
        std::lock_guard<std::mutex> lock(mu);
        if (!configured[dev]) {
            const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 68 * 1024);
            if (e != cudaSuccess) return e;
            configured[dev] = true;
        }
    }
    const int grid = (int)std::min<int64_t>(blocks, (int64_t)num_sms * (V <= 8 ? kMinBlocks : 2));   // one wave
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
