// moe_launch.cuh -- kernel parameter blocks and launch entry points used by
// the C ABI layer (moe_capi.cu).  Internal to libmoe_gb300.
#pragma once

#include <cuda.h>

#include <algorithm>

#include "moe_internal.cuh"

namespace moe {

struct GateUpParams {
    const uint16_t* x;
    int n, H, I, S, k;
    QMatDev gate, up, sh_gate, sh_up;
    const int32_t* counts;
    const int32_t* offsets;
    const int32_t* perm;
    const int32_t* active;
    const Ctrl* ctrl;
    float* act;      // [n*k, I], row = route id t*k + j
    float* act_sh;   // [n, S]
};

struct DownParams {
    int n, H, I, S, k, E;
    int e_begin, e_end;      // routes to experts outside [e_begin, e_end) contribute nothing
    int accumulate;          // out = BF16(out + result)
    QMatDev down, sh_down;
    const int32_t* idx;
    const float* w;
    const float* act;
    const float* act_sh;
    const float* sg_logit;   // NULL = shared gate 1
    uint16_t* out;
};

// INT4 streaming path (moe_experts_q4.cu).
struct Q4Params {
    const uint16_t* x;       // [n, H] the experts' input
    int n, H, I, S, k;
    QMatDev gate, up, down, sh_gate, sh_up, sh_down;
    bool zero;               // any matrix has zero points
    int e_begin, e_end;      // experts held here
    const int32_t* segs;     // [n_rsegs][3] (n > 1)
    const int32_t* perm;     // sorted position -> route id (n > 1)
    const Ctrl* ctrl;
    bool per_token;          // each token's routes as they are (a few tokens)
    const int32_t* idx;      // [n, k] (per token)
    const float* route_w;    // [n*k]
    const float* sg_logit;   // shared gate logits or NULL
    float* act;              // [n*k, I] by sorted position (per token: by route)
    float* act_sh;           // [n, S]
    float* y;                // [n*k, H] weighted rows (n > 1)
    float* y_sh;             // [n, H]
    uint16_t* out;           // [n, H] (per token)
    int accumulate;
};
bool q4_n1_fits(int H, int k, int I, int S);   // whether the per-token kernels' shared memory suffices
cudaError_t launch_experts_q4(int fmt, const Q4Params& p, bool gate_up, int tile, int num_sms, cudaStream_t st);

// Grouped tensor-core path (moe_grouped_tc.cu).
struct TcMaps {
    CUtensorMap w[2];    // routed weights: (gate, up) or (down)
    CUtensorMap ws[2];   // shared-expert weights
    CUtensorMap b;       // routed activations (expert-sorted rows)
    CUtensorMap bs;      // shared-expert activations (token rows)
};

struct TcParams {
    int out_dim, in_dim;     // routed matrix [out, in] per expert
    int sh_out, sh_in;       // shared matrix (sh_out == 0: no shared expert)
    int n, k;
    int e_base;              // global index of the weight stacks' first expert
    const int32_t* segs;     // [n_rsegs][3] = (expert, first sorted row, tokens)
    const Ctrl* ctrl;
    const void* scale[2];    // routed scales (FP8 fp32 blocks / NVFP4 E4M3 bytes)
    const void* sh_scale[2];
    const float* scale2[2];  // NVFP4 per-expert fp32
    const float* sh_scale2[2];
    const uint8_t* zero[2];     // INT4 zero points, or NULL
    const uint8_t* sh_zero[2];
    int gshift;                 // INT4: log2 of the group size
    const int32_t* row_exp;     // INT4: the power of two by which each row of x (down: of act) was multiplied
    const int32_t* row_exp_sh;
    const int8_t* wexp[2];      // INT4: the power of two by which each weight row's scales are multiplied
    const int8_t* sh_wexp[2];
    void* act_out;           // gate_up: sorted SiLU(g)*u rows [n*k, I] (bf16 / f16; INT4: fp32)
    void* act_sh_out;        // gate_up: shared [n, S]
    float* y;                // down: weighted rows [n*k, H]
    float* y_sh;             // down: gated shared rows [n, H]
    const float* route_w;    // [n*k] routing weights (by route id)
    const int32_t* perm;     // sorted position -> route id
    const float* sg_logit;   // shared gate logits or NULL
    int32_t* err;            // Ctrl::err
    const void* zero4;       // 4 zero bytes (stand-in scale source past the last row)
    // Down kernel only: after every tile, a grid barrier and the combine
    // (out = BF16(sum_j y[inv[t*k + j]] in slot order + y_sh[t] (+ out))).
    int combine;             // 0: the combine runs as a kernel of its own
    const int32_t* inv;      // route id -> sorted position (-1: dropped)
    uint16_t* out;           // [n, H] BF16 (device or mapped pinned host memory)
    int has_shared, accumulate;
    uint32_t* tc_count;      // Ctrl::tc_count
    uint32_t* tc_gen;        // Ctrl::tc_gen
};

bool build_tc_maps(int fmt, bool gate_up, const moe_weights_t* w, int E, int H, int I, int S, int n,
                   int n_routes_max, const void* act_routed, const void* act_shared, TcMaps* maps);
cudaError_t launch_grouped_tc(int fmt, bool gate_up, const TcMaps& maps, const TcParams& p, int num_sms,
                              cudaStream_t st);
cudaError_t launch_copy16(const void* src, void* dst, size_t bytes, int num_sms, cudaStream_t st);
// norm_w (may be null): the pre-expert RMSNorm weight; the rows gathered are
// then the normalised ones (the norm kernel's values).  exps (INT4): each row enters as f16
// times the power of two whose exponent goes there (n k rows of xs, then those of xh), and wr's
// exponents of the weight rows of the active experts and the shared one are formed.
cudaError_t launch_gather(int fmt, const uint16_t* x, int n, int H, int k, const int32_t* perm,
                          const int32_t* offsets, int E, uint16_t* xs, uint16_t* xh, const uint16_t* norm_w,
                          float eps, int32_t* exps, const WeightRows& wr, const int32_t* active, const Ctrl* ctrl, bool early, int num_sms, cudaStream_t st);
// INT4: the rows of SiLU(g) u (fp32) as f16 times a power of two each, whose exponents go to
// exps (n_routes_max rows of as, then those of ash).
cudaError_t launch_act_rows(const float* act, const float* act_sh, int n, int I, int S, const int32_t* offsets, int E,
                            uint16_t* as, uint16_t* ash, int32_t* exps, int n_routes_max, bool early, int num_sms,
                            cudaStream_t st);
cudaError_t launch_combine(const float* y, const float* ysh, const int32_t* inv, int n, int H, int k,
                           int has_shared, int accumulate, uint16_t* out, bool early, int num_sms, cudaStream_t st);

// Fused single-token kernel (moe_fused_n1.cu).
struct FusedParams {
    const uint16_t* x;
    int H, E, k, I, S, routing, norm;
    float scale;
    int e_begin, e_end;       // local experts (expert parallelism)
    int accumulate;           // out = BF16(out + result)
    const uint16_t* norm_w;   // pre-expert RMSNorm weight or NULL
    float eps;
    const uint16_t* router;
    const uint16_t* gw;       // shared-gate weight or NULL
    const float* bias;
    QMatDev gate, up, down, sh_gate, sh_up, sh_down;
    float* logits;            // [E]
    float* sg_logit;          // [1]
    float* act;               // [k * I]
    float* act_sh;            // [S]
    int32_t* idx_out;         // [k]
    float* w_out;             // [k]
    uint16_t* out;            // [H]
    Ctrl* ctrl;
    int rpc;                  // output columns per CTA
    uint32_t row_bytes, drow_bytes, dsh_row_bytes;
    uint32_t off_x, off_xe, off_lg, off_sc, off_sel, off_cand, off_down, off_act, off_part, off_shgu, off_bar,
        smem_bytes;
    int n_cand;
};

bool fused_plan(const moe_config_t* c, int num_sms, FusedParams* p);
cudaError_t launch_fused_n1(int fmt, const FusedParams& p, int num_sms, cudaStream_t st);

cudaError_t launch_router(const uint16_t* x, int n, int H, const uint16_t* wr, int E,
                          const uint16_t* gw, float* logits, float* sg_logit, int num_sms,
                          cudaStream_t st);
// Tensor-core router (moe_router_tc.cu): partial logits [splits][n][E] of the
// BF16 router (rows E) for device-resident x, each multiplied by *scale when
// scale is not null; the caller checked router_tc_fits.
cudaError_t launch_router_tc(const uint16_t* x, int n, int H, const uint16_t* wr, int E, float* part,
                             int32_t* err, const float* scale, bool early, cudaStream_t st);
// The NVFP4 router [E, H] as BF16 (exact: E2M1 code times E4M3 block scale),
// for the tensor-core router, which multiplies its partials by scale2.
cudaError_t launch_router_nvfp4_expand(const QMatDev& wq, int E, int H, uint16_t* out, bool early, int num_sms,
                                       cudaStream_t st);
// 2-D TMA map over a row-major [rows, cols] matrix of `esize`-byte elements, rows `stride` elements
// apart (0: cols) (moe_grouped_tc.cu).
bool make_map(CUtensorMap* m, const void* base, CUtensorMapDataType dt, int esize, uint64_t cols,
              uint64_t rows, uint32_t box_cols, uint32_t box_rows, CUtensorMapSwizzle swizzle, uint64_t stride = 0);
bool make_map_pairs(CUtensorMap* m, const void* base, CUtensorMapDataType dt, uint64_t cols, uint64_t rows, int apart);
cudaError_t launch_router_nvfp4(const uint16_t* x, int n, int H, const QMatDev& wq, int E, float* logits,
                                cudaStream_t st);
// logits: ns partial rows per token ([ns][n][E], ns = 1 for a plain logit
// matrix), summed in order; lsum (may be null) receives the sums.
cudaError_t launch_topk(const float* logits, int ns, float* lsum, int n, int E, int k, int routing, const float* bias,
                        int norm, float scale, int32_t* idx, float* w, cudaStream_t st);
// Top-k routing of rows of logits (moe_topk.cu).  ns > 1 (fp32 only): a row's
// logits are the sums, in order, of ns partial rows pstride elements apart;
// lsum (may be null) receives them, rows E apart.
cudaError_t launch_topk_rows(const void* logits, int dtype, int64_t row_stride, int ns, int64_t pstride, float* lsum,
                             int n, int E, int k, int32_t routing, const float* bias, int norm, float scale,
                             int32_t* idx, float* w, int num_sms, cudaStream_t st);
// out[t, :] = W x[t, :] for a 4-bit W (moe_matvec.cu).
struct MatvecParams {
    QMatDev w;
    const float* bias;
    const void* x;
    int64_t x_stride;
    int n;
    void* out;
    int64_t out_stride;
    int out_type, accumulate;
};
bool matvec_fits(int K);   // whether a row of x fits beside the kernel's rings
cudaError_t launch_matvec(int fmt, int x_type, const MatvecParams& p, int num_sms, cudaStream_t st);

// Residual addition and RMSNorm of rows (moe_norm.cu).  Strides in elements.
constexpr int kNormMaxHidden = 32768;
struct NormParams {
    const void *x, *res, *w;   // res, w may be null
    int x_type, res_type, w_type, out_type;
    int64_t x_stride, res_stride, res_out_stride, out_stride, out8_stride;
    void *res_out, *out;       // may be null
    uint8_t* out8;             // may be null
    float* scale8;             // [n, n_scales]
    int n, H, n_scales;
    int group;                 // a scale for each 128 elements (else for the row)
    float eps, w_offset;
};
cudaError_t launch_norm(const NormParams& p, int num_sms, cudaStream_t st);

// Low-rank adapters of rows (moe_lora.cu; many rows: moe_lora_tc.cu).  Strides in elements.
struct LoraParams {
    const uint16_t *a, *b;     // [L, r, K], [L, O, r]
    const float* scale;        // [L] or null
    const uint16_t* x;
    const int32_t* idx;        // [n]
    const void* base;          // or null
    void* out;
    int64_t x_stride, base_stride, out_stride;
    int n, K, O, r, L, out_type;
    bool x_host, out_host;     // x; base or out: it is pinned host memory
    int32_t* err;              // where a bounded wait that gives up leaves its code; no output while one is there.  Null: in the workspace
    // Set by launch_lora.
    int vec;                   // elements of base's and out's rows that can be read at once: 8, 4 or 1
    bool copy;                 // rows without an adapter are to be written
    int groups;                // few rows: clusters that are launched, or 0 for one a row
    // The rows sorted by adapter, or null: runs (adapter, or -1 for none; first position; rows), the
    // runs of adapters before those of none.  ctrl->n_active runs of adapters, n_rsegs in all.
    const int32_t *segs, *perm;
    Ctrl* ctrl;
};
size_t lora_workspace(int64_t n, int L, int K, int O, int r);
cudaError_t launch_lora(const LoraParams& p, int x_type, void* ws, cudaStream_t st);
// Runs of at most 128 rows through the tensor cores' kernels, v's partial sums [splits][n][r] in part.
constexpr int kLoraTile = 128;
// Blocks that a call aims at: two on each of GB300's 152 SMs.  (A constant, since the size of a workspace follows from it: on a
// GPU of fewer SMs blocks wait for their turn.)
constexpr int kLoraBlocks = 304;
constexpr int kLoraMaxSplits = 8;
constexpr int kLoraErrFirst = 31, kLoraErrLast = 37;   // codes of the bounded waits (anything else is memory not cleared yet)
inline int64_t lora_part_rows(int64_t n) {   // of splits * n, and of every smaller n's
    return std::min<int64_t>(kLoraMaxSplits * n, (int64_t)kLoraBlocks * kLoraTile + 2 * n);
}
// Whether the tensor maps of a call can be made; `maps` receives them (x by
// single rows, A, B, x by 32 rows, B by pairs of rows).
bool lora_maps(const LoraParams& p, int x_type, CUtensorMap (&maps)[5]);
cudaError_t launch_lora_tc(const LoraParams& p, int x_type, const CUtensorMap (&maps)[5], float* part, int max_segs, cudaStream_t st);

// tile: routes of a segment at most.
cudaError_t launch_group(const int32_t* idx, int nk, int E, int tile, int e_begin, int e_end, int32_t* counts,
                         int32_t* offsets, int32_t* perm, int32_t* inv, int32_t* active, int32_t* segs,
                         Ctrl* ctrl, cudaStream_t st);
cudaError_t launch_topk_group(const float* logits, int ns, int n, int E, int k, int routing, const float* bias,
                              int norm, float scale, int32_t* idx, float* w, int tile, int e_begin, int e_end, int32_t* counts,
                              int32_t* offsets, int32_t* perm, int32_t* inv, int32_t* active, int32_t* segs,
                              Ctrl* ctrl, const uint16_t* x, const uint16_t* gw, float* sg_logit, int H, bool early,
                              int num_sms, cudaStream_t st);
// Whether launch_topk_group can form the shared gate's logit (gw != null) for
// E experts and hidden size H.
bool topk_group_gate_fits(int E, int H);
cudaError_t launch_rmsnorm(const uint16_t* x, int n, int H, const uint16_t* w, float eps, uint16_t* xe,
                           cudaStream_t st);
cudaError_t launch_gate_up_tm(int fmt, const GateUpParams& gu, int num_sms, cudaStream_t st);
cudaError_t launch_down_blend_tm(int fmt, const DownParams& dn, int num_sms, cudaStream_t st);

}  // namespace moe
