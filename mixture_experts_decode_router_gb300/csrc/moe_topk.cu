// moe_topk.cu -- top-k routing of rows of logits (sm_103a): softmax or sigmoid
// scores, a balance bias, group-limited selection, any number of rows.
//
// One warp per row.  Scores are held in 64 bits: which expert a row chooses
// hangs on the order of near values, and a whole number has no tolerance.
#include <cuda_fp16.h>

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
__device__ __forceinline__ int select_exact(const TopkParams& p, const float* sl, double* sc, int lane) {
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

template <int TYPE>
__global__ void __launch_bounds__(32 * kRowWarps) topk_rows_kernel(const TopkParams p) {
    extern __shared__ __align__(16) uint8_t dyn[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    double* sc = reinterpret_cast<double*>(dyn) + (size_t)warp * p.E;
    float* sl = reinterpret_cast<float*>(reinterpret_cast<double*>(dyn) + (size_t)kRowWarps * p.E) + (size_t)warp * p.E;
    const int64_t t = (int64_t)blockIdx.x * kRowWarps + warp;
    pdl_wait();
    if (t < p.n) {
        float m = -INFINITY;
        for (int e = lane; e < p.E; e += 32) {
            const float l = load_logit<TYPE>(p, t, e);
            sl[e] = l;
            if (p.lsum) p.lsum[(size_t)t * p.E + e] = l;
            m = fmaxf(m, l);
        }
        __syncwarp();
        float z = 0.f;
        if (!p.norm && !mode_sigmoid(p.r.mode)) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            for (int e = lane; e < p.E; e += 32) z += expf(sl[e] - m);
            z = warp_sum(z);
        }
        const int e = select_exact(p, sl, sc, lane);
        const float v = row_weight(p, lane < p.k ? sl[e] : 0.f, m, z, lane);
        if (lane < p.k) {
            p.idx[(size_t)t * p.k + lane] = e;
            p.w[(size_t)t * p.k + lane] = v;
        }
    }
    pdl_trigger();
}

}  // namespace

cudaError_t launch_topk_rows(const void* logits, int dtype, int64_t row_stride, int ns, int64_t pstride, float* lsum,
                             int n, int E, int k, int32_t routing, const float* bias, int norm, float scale,
                             int32_t* idx, float* w, int num_sms, cudaStream_t st) {
    TopkParams p{logits, row_stride, ns, pstride, lsum, n, E, k, routing_of(routing), bias, norm, scale, idx, w};
    const int grid = (int)(((int64_t)n + kRowWarps - 1) / kRowWarps);
    const size_t smem = (size_t)kRowWarps * E * 12;   // <= 48 KB for E <= 1024
    if (dtype == MOE_F32) launch_pdl(topk_rows_kernel<MOE_F32>, grid, 32 * kRowWarps, smem, st, p);
    else if (dtype == MOE_BF16) launch_pdl(topk_rows_kernel<MOE_BF16>, grid, 32 * kRowWarps, smem, st, p);
    else launch_pdl(topk_rows_kernel<MOE_F16>, grid, 32 * kRowWarps, smem, st, p);
    return cudaGetLastError();
}

}  // namespace moe
