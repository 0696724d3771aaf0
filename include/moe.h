/*
 * moe.h -- C ABI of the GB300 (sm_103a) Mixture-of-Experts decode-layer forward.
 *
 * One library, libmoe_gb300.so, computes the MoE layer of a decoder for a
 * decode-sized batch of N tokens (N = 1..256 and beyond), on one GPU:
 *
 *   router   logits[t,e] = sum_h x[t,h] * Wr[e,h]                 (fp32)
 *   top-k    softmax: rank logits, p = softmax over all E logits;
 *            sigmoid+bias: rank sigmoid(l)+bias, p = sigmoid(l);
 *            (also softmax+bias, sigmoid alone, and group-limited selection)
 *            w = p / sum_topk p if norm_topk_prob; w *= routed_scaling_factor
 *   experts  per (token t, slot j), e = idx[t,j]:
 *            d = Wd[e] (SiLU(Wg[e] x_t) * (Wu[e] x_t)),  SiLU(g) = g/(1+exp(-g))
 *   shared   ds = the same SwiGLU with the shared expert's three matrices
 *   blend    out[t] = sum_j w[t,j] d[t,j] + g_s ds,
 *            g_s = sigmoid(x_t . shared_gate_w), or 1 without a gate weight
 *
 * The operation is the one the pages "metrale_model_layers/layers/moe/forward.rs"
 * (MoeLayer::forward: gate, topk, exp_gate_up, exp_silu_down and wsum_blend
 * steps), "spark_model/layers/moe/forward_token_major.rs"
 * (forward_token_major_decode: gate GEMM, batched top-k, gate+up, silu+down,
 * weighted sum and blend for N tokens) and
 * "metrale_model_layers/layers/moe/forward_fp8_grouped_router.rs"
 * (grouped_route: router logits and top-k written as [m*top_k] indices and
 * fp32 weights) describe.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - Every pointer marked "device" is a CUDA device (or managed) address on the
 *    current device; the caller owns every buffer (weights, input, outputs,
 *    workspace).  The library never allocates, frees or synchronises: each call
 *    only enqueues kernels on `stream` and returns.
 *  - The layer input x (moe_route, moe_experts, moe_forward) and output out
 *    (moe_experts, moe_forward) may instead be pinned (page-locked) host
 *    memory mapped into the device's address space (cudaHostAlloc, or any
 *    pinned allocation under unified addressing).  The kernels then reach x
 *    and out over the host link (NVLink-C2C on Grace systems) and no copy is
 *    needed before or after the call: one token's kernel reads x directly;
 *    for more tokens the call first copies x into the workspace with a kernel
 *    of its own, so that its other kernels read it from device memory.  Host
 *    memory that is not pinned is refused (MOE_ERR_HOST_MEMORY).  idx, w,
 *    logits, the weights and the workspace stay in device memory.
 *  - Device pointers must be 16-byte aligned (MOE_ERR_ALIGNMENT otherwise),
 *    except the scale and scale2 arrays of moe_qmat_t, which need 4 bytes (so
 *    that one rank's slice of a stacked scale array can be passed as it is).
 *  - All arguments are validated on the host before anything is enqueued; an
 *    error status means nothing was launched.  There is no fallback path: a
 *    configuration the kernels do not cover is refused by name
 *    (MOE_ERR_UNSUPPORTED), never computed some other way.
 *  - Asynchronous device faults are not reported by the call that enqueued
 *    the work; they surface from the next CUDA call as usual.
 *  - n == 0 is a valid no-op (MOE_OK, nothing launched).
 *  - The workspace is scratch the layer reuses across its steps.  Its first 256
 *    bytes are a control block that must be zero before the first call (for
 *    example cudaMemsetAsync(ws, 0, 256, stream) after allocating it); every
 *    call leaves it valid for the next one.  The rest is not meaningful between
 *    calls.  Two
 *    calls that run at the same time on the GPU must not share a workspace.
 *  - Device-side failures that the kernels detect themselves (a bounded wait
 *    that gave up after 2 s, or a control block that was not zeroed) end the
 *    kernel early and set an error word in the workspace: read it with
 *    moe_workspace_check().  The output of such a call is not valid.
 *
 * Tensor layouts (row-major, C order)
 * -----------------------------------
 *  x            BF16  [N, H]
 *  router_w     BF16  [E, H]  (each expert's router row contiguous)
 *  routed gate, up:   [E, I, H];  routed down: [E, H, I]
 *  shared gate, up:   [1, S, H];  shared down: [1, H, S]
 *  For a stacked [E, out, in] matrix the formats are
 *   MOE_W_BF16      w: BF16 [E, out, in]; scale, scale2 unused (NULL)
 *   MOE_W_FP8_B128  w: FP8 E4M3 bytes [E, out, in];
 *                   scale: fp32 [E, ceil(out/128), ceil(in/128)];
 *                   value = e4m3(w) * scale[o/128][i/128]
 *   MOE_W_NVFP4     w: bytes [E, out, in/2], two E2M1 codes per byte, the
 *                   element with even `in` index in the low nibble;
 *                   scale: FP8 E4M3 bytes [E, out, in/16] (one per 16 elements);
 *                   scale2: fp32 [E];
 *                   value = e2m1(code) * e4m3(scale[o][i/16]) * scale2[e]
 *   MOE_W_INT4_G32, MOE_W_INT4_G64, MOE_W_INT4_G128 (groups of G = 32, 64, 128)
 *                   w: bytes [E, out, in/2], two codes 0..15 per byte, the
 *                   element with even `in` index in the low nibble;
 *                   scale: BF16 [E, out, in/G] (one per G elements along in);
 *                   zero: bytes [E, out, in/G], 0..15, or NULL (every zero
 *                   point is 8); value = (code - zero[o][i/G]) * scale[o][i/G];
 *                   every reduction length (H, I and S) is a multiple of G.
 *                   INT4 experts have fp32's range at any number of tokens:
 *                   SiLU(g) u (and, on the expert-grouped path, x and the
 *                   scales) enter the products as f16 under a power of two for
 *                   each row, or for each 256 or 768 elements of a row.  Values
 *                   below 2^-29 (scales: 2^-22) of the largest that shares their
 *                   power of two lose bits there.
 *  idx          int32 [N, k], slots in descending selection score
 *  w            fp32  [N, k]
 *  logits       fp32  [N, E]
 *  out          BF16  [N, H] (round to nearest even from fp32)
 */
#ifndef MOE_GB300_MOE_H
#define MOE_GB300_MOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_ABI_VERSION 2

/* A CUDA stream handle (the same object as cudaStream_t; NULL = legacy default stream). */
typedef struct CUstream_st* moe_stream_t;

typedef enum {
    MOE_OK = 0,
    MOE_ERR_NULL = 1,            /* a required pointer is NULL                              */
    MOE_ERR_INVALID_CONFIG = 2,  /* a size, enum or flag is out of range or inconsistent    */
    MOE_ERR_UNSUPPORTED = 3,     /* valid, but outside what the kernels cover (named refusal)*/
    MOE_ERR_WORKSPACE = 4,       /* workspace missing or smaller than moe_workspace_bytes()  */
    MOE_ERR_CUDA = 5,            /* a CUDA call failed while enqueueing (cudaGetLastError)   */
    MOE_ERR_ALIGNMENT = 6,       /* a device pointer is not aligned (16 bytes; 4 for scales) */
    MOE_ERR_ALIAS = 7,           /* `out` overlaps `x`                                       */
    MOE_ERR_HOST_MEMORY = 8      /* `x` or `out` is host memory that is not pinned (page-locked) */
} moe_status_t;

/* Scores p of the experts (softmax over all E, or sigmoid, of the logits) and
 * the selection score s that ranks them: the logit itself, or p + the correction
 * bias in the *_BIAS modes (the bias only selects, it enters no weight). */
typedef enum {
    MOE_ROUTE_SOFTMAX = 0,
    MOE_ROUTE_SIGMOID_BIAS = 1,
    MOE_ROUTE_SOFTMAX_BIAS = 2,
    MOE_ROUTE_SIGMOID = 3
} moe_routing_t;
/* Group-limited routing: the experts form `groups` groups of E / groups
 * consecutive ones (at most 32 groups, of equal size), the `kept` groups with
 * the best group scores stay (ties: the lower group), and the top-k is taken
 * among their experts, of which there must be at least k.  A group's score is
 * its best selection score, or the sum of its two best p (+ bias) (of the one,
 * in a group of one). */
typedef enum { MOE_GROUP_MAX = 0, MOE_GROUP_TOP2 = 1 } moe_group_score_t;
/* The routing word of moe_config_t and moe_topk_config_t: a moe_routing_t
 * alone, or one with groups. */
#define MOE_ROUTING(mode, groups, kept, score) \
    ((int32_t)((mode) | ((groups) << 8) | ((kept) << 16) | ((score) << 24)))
typedef enum { MOE_F32 = 0, MOE_BF16 = 1, MOE_F16 = 2 } moe_dtype_t;
typedef enum {
    MOE_W_BF16 = 0,
    MOE_W_FP8_B128 = 1,
    MOE_W_NVFP4 = 2,
    MOE_W_INT4_G32 = 3,
    MOE_W_INT4_G64 = 4,
    MOE_W_INT4_G128 = 5
} moe_wfmt_t;
/* Expert-stage algorithm.  AUTO: one token runs the single-token kernel,
 * 2-3 tokens the token-major kernels, 4 or more the expert-grouped
 * tensor-core GEMM; INT4 experts run streaming kernels of their own while an
 * expert has at most 20 tokens on average (n k <= 20 E), the expert-grouped
 * GEMM above.  The two explicit values force one (tests); TOKEN_MAJOR
 * with one token still runs the single-token kernel (same arithmetic). */
typedef enum { MOE_PATH_AUTO = 0, MOE_PATH_TOKEN_MAJOR = 1, MOE_PATH_GROUPED = 2 } moe_path_t;

/* Pre-expert RMSNorm (the pre_expert_norm step of MoeLayer::forward, page
 * "metrale_model_layers/layers/moe/forward.rs"): with a norm weight, the routed
 * and shared experts take xe = BF16(x / sqrt(mean(x^2) + eps) * w); the router
 * and the shared-expert gate keep x.
 *
 * Expert parallelism (the EP branch of MoeLayer::forward and
 * forward_token_major_decode): a call with [expert_begin, expert_end) holds
 * only those experts -- the routed weight stacks have expert_end - expert_begin
 * entries, indexed from expert_begin -- and routes to other experts contribute
 * nothing; routing is still computed over all E.  With exclude_shared = 1 the
 * output is one rank's partial: the caller sums the partials over ranks (an
 * all-reduce) and adds the shared expert once, with a call that holds no
 * experts (expert_begin = expert_end = E) and accumulate = 1: it adds the
 * (gated) shared expert into the summed output, as the pages' residual_add /
 * moe_batched_blend after the all-reduce do.  A call that holds no experts and
 * is given neither idx nor w skips routing (it computes only the shared-gate
 * logit); on one token it still routes.
 *
 * accumulate = 1: every output element is BF16(out + result), with out read
 * on entry (rounded once, in fp32); out must then hold n x H valid values.
 *
 * NVFP4 router (the gate_nvfp4 / w4a16_gemm branch of the router step on the
 * same page): router_fmt = MOE_W_NVFP4 takes the router from router_q, an
 * NVFP4 matrix [E, H] in the expert layout below with one expert (w: bytes
 * [E, H/2]; scale: E4M3 [E, H/16]; scale2: one fp32), multiplying the BF16
 * activations; router_w is then unused (may be NULL).  One token then runs the
 * token-major kernels (the single-token kernel reads a BF16 router).  On the
 * expert-grouped path the router is expanded to BF16 in the workspace (each
 * code times its block scale, exact) for the tensor-core router, which applies
 * scale2 to its partial logits; the workspace then holds E x H BF16 more.
 *
 * Layer configuration (the config fields hidden_size, num_experts,
 * num_experts_per_tok, moe_intermediate_size, shared_expert_intermediate_size,
 * norm_topk_prob and routed_scaling_factor of the pages' layer).
 * Limits: 1 <= num_experts <= 1024; 1 <= top_k <= min(num_experts, 32);
 * hidden, inter > 0 and multiples of 32; shared_inter >= 0 and a multiple of 32
 * (0 = no shared expert); routed_scaling_factor finite. */
typedef struct {
    int32_t hidden;                 /* H */
    int32_t num_experts;            /* E */
    int32_t top_k;                  /* k */
    int32_t inter;                  /* I  (routed expert intermediate size) */
    int32_t shared_inter;           /* S  (shared expert intermediate size; 0 = none) */
    int32_t routing;                /* moe_routing_t or MOE_ROUTING(...) */
    int32_t norm_topk_prob;         /* 0 or 1 */
    float   routed_scaling_factor;
    int32_t expert_fmt;             /* moe_wfmt_t: routed and shared experts alike */
    int32_t path;                   /* moe_path_t */
    /* ABI version 2 (a zero-filled tail keeps the version-1 behaviour): */
    float   rms_norm_eps;           /* epsilon of the pre-expert RMSNorm (when a norm weight is given) */
    int32_t expert_begin;           /* expert parallelism: this call holds experts   */
    int32_t expert_end;             /*   [expert_begin, expert_end); 0 and 0 = all E  */
    int32_t exclude_shared;         /* 1: leave the shared expert out of the output  */
    int32_t accumulate;             /* 1: out = BF16(out + layer output)             */
    int32_t router_fmt;             /* MOE_W_BF16 (router_w) or MOE_W_NVFP4 (router_q) */
} moe_config_t;

/* (An unnamed union is C11; GNU compilers take it in any mode.) */
#ifdef __GNUC__
#define MOE_EXTENSION __extension__
#else
#define MOE_EXTENSION
#endif
/* One stacked expert matrix (device pointers; see the layouts above). */
typedef struct {
    const void*  w;
    const void*  scale;    /* FP8: fp32 block scales; NVFP4: E4M3 bytes; INT4: BF16; BF16: NULL */
#if defined(__cplusplus) || defined(__GNUC__) || (defined(__STDC_VERSION__) && __STDC_VERSION__ >= 201112L)
    MOE_EXTENSION union {
        const float*   scale2;   /* NVFP4: fp32 [E]; BF16, FP8: NULL */
        const uint8_t* zero;     /* INT4: zero points [E, out, in/G], or NULL (8) */
    };
#else   /* C without unnamed unions: INT4 zero points are cast into scale2 */
    const float* scale2;
#endif
} moe_qmat_t;

/* All weights of one layer (device pointers).  The shared-expert matrices are
 * ignored (may be NULL) when shared_inter == 0. */
typedef struct {
    const void*  router_w;          /* BF16 [E, H] */
    const float* correction_bias;   /* fp32 [E]; required by the *_BIAS modes, else must be NULL */
    moe_qmat_t   gate, up, down;    /* routed experts */
    moe_qmat_t   sh_gate, sh_up, sh_down;   /* shared expert (E = 1) */
    const void*  shared_gate_w;     /* BF16 [H] or NULL (then the shared gate is 1) */
    /* ABI version 2: */
    const void*  pre_expert_norm_w; /* BF16 [H] or NULL: RMSNorm of the experts' input */
    moe_qmat_t   router_q;          /* NVFP4 router [E, H] when router_fmt = MOE_W_NVFP4 */
} moe_weights_t;

/* Bytes of workspace a call with up to `max_tokens` tokens needs (a multiple
 * of 256).  Returns 0 if `cfg` is NULL or invalid, or max_tokens < 0. */
size_t moe_workspace_bytes(const moe_config_t* cfg, int32_t max_tokens);

/* Router and top-k for n tokens (the pages' gate and topk steps, grouped_route).
 * The router runs where moe_forward's would for the same cfg and n: a BF16
 * router on the grouped path (cfg->path, or n > 3 under MOE_PATH_AUTO) on the
 * tensor cores (fp32 accumulation per K range, the ranges summed in a fixed
 * order), otherwise on the CUDA cores; so moe_route + moe_experts is
 * moe_forward bit for bit.
 * The routing words MOE_ROUTE_SOFTMAX and MOE_ROUTE_SIGMOID_BIAS alone rank
 * scores computed in fp32 (sigmoid(l) + bias of two experts can tie or change
 * places there within their fp32 errors); every other word ranks them in 64
 * bits, as moe_topk does with any word.
 *   x       device BF16 [n, H]
 *   idx     device int32 [n, k]   (out) selected experts, descending score
 *   w       device fp32  [n, k]   (out) routing weights
 *   logits  device fp32  [n, E]   (out, optional: NULL = not returned)
 *   ws      device workspace of at least moe_workspace_bytes(cfg, n) bytes
 * Errors: MOE_ERR_NULL, MOE_ERR_INVALID_CONFIG, MOE_ERR_UNSUPPORTED,
 * MOE_ERR_WORKSPACE, MOE_ERR_ALIGNMENT, MOE_ERR_HOST_MEMORY, MOE_ERR_CUDA. */
moe_status_t moe_route(const moe_config_t* cfg, const moe_weights_t* wts,
                       const void* x, int32_t n,
                       int32_t* idx, float* w, float* logits,
                       void* ws, size_t ws_bytes, moe_stream_t stream);

/* Routed experts, shared expert and blend for n tokens given their routing
 * (the pages' exp_gate_up, exp_silu_down and wsum_blend steps).
 *   x     device BF16 [n, H] (the layer input: with a pre-expert norm weight
 *         the experts take its RMSNorm, and the shared gate takes x itself)
 *   idx   device int32 [n, k]; an entry outside [expert_begin, expert_end)
 *         (all of [0, E) by default) is dropped (that slot contributes
 *         nothing), so a bad index never reads outside the weights
 *   w     device fp32  [n, k]
 *   out   device BF16 [n, H] (out); must not overlap x
 * Errors: as moe_route, plus MOE_ERR_ALIAS. */
moe_status_t moe_experts(const moe_config_t* cfg, const moe_weights_t* wts,
                         const void* x, int32_t n,
                         const int32_t* idx, const float* w,
                         void* out, void* ws, size_t ws_bytes, moe_stream_t stream);

/* The whole layer: moe_route then moe_experts on one stream.
 *   idx, w  optional device outputs ([n, k] int32 / fp32); NULL = kept in the
 *           workspace only. */
moe_status_t moe_forward(const moe_config_t* cfg, const moe_weights_t* wts,
                         const void* x, int32_t n, void* out,
                         int32_t* idx, float* w,
                         void* ws, size_t ws_bytes, moe_stream_t stream);

/* moe_forward with stage markers, for profiling (the per-stage timing the
 * pages' `prof!` macro in MoeLayer::forward takes with a stream sync, done here
 * with device events and no sync).
 *   events    array of n_events cudaEvent_t handles (cast to void*) created by
 *             the caller on the current device; marker i is recorded with
 *             cudaEventRecord(events[i], stream) for i < n_events
 *   n_marks   (out, optional) markers the call reached
 * Markers: 0 before the first kernel, then one after each stage, in launch
 * order.  One token on the single-token kernel: 2 markers (before, after).
 * Token-major kernels: 5 (router, top-k + grouping, gate+up, down+blend).
 * INT4 streaming kernels: 6 (router, top-k + grouping, gate+up, down, combine);
 * where the tokens take their routes one by one (one token, or up to four whose
 * experts take at most 64 MB together) 5 (router, top-k, gate+up, down+blend).
 * Grouped tensor-core path: 7 (router, top-k + grouping, gather, gate+up, down,
 * combine).  The pre-expert RMSNorm, when present, runs at the start of the
 * stage after top-k + grouping.
 * Errors: as moe_forward, plus MOE_ERR_NULL for events == NULL with n_events > 0. */
moe_status_t moe_forward_timed(const moe_config_t* cfg, const moe_weights_t* wts,
                               const void* x, int32_t n, void* out,
                               int32_t* idx, float* w,
                               void* ws, size_t ws_bytes, moe_stream_t stream,
                               void* const* events, int32_t n_events, int32_t* n_marks);

/* Bytes of the static device workspace of moe_forward_static_ws. */
#define MOE_STATIC_WORKSPACE_BYTES ((size_t)16 << 20)

/* moe_forward for callers that cannot allocate device memory (no counterpart
 * in the pages: an addition of this library).  A plugin whose host owns every
 * allocation, or code that is recording a CUDA graph (where cudaMalloc is not
 * allowed), may have input and output buffers but no way to get a workspace.
 * This call takes none: its scratch is one file-scope device array of
 * MOE_STATIC_WORKSPACE_BYTES that every GPU which loads the library keeps until
 * the process exits.  It allocates nothing and calls no allocating routine.
 *   Arguments, outputs and errors: as moe_forward, without ws / ws_bytes.
 *   A call that would need more than MOE_STATIC_WORKSPACE_BYTES of workspace
 *   (moe_workspace_bytes(cfg, n)) returns MOE_ERR_WORKSPACE and launches nothing.
 *   The first call on each device looks up the array's device address and
 *   clears its control block on `stream`, then synchronises `stream`; make
 *   that first call before any stream capture (a first call on a stream that
 *   is being captured returns MOE_ERR_UNSUPPORTED and launches nothing).
 *   Every call shares the one array: calls whose work overlaps on the GPU
 *   (other streams, other host threads) race on it and must be serialised by
 *   the caller.
 *   Device-side failures (a bounded wait that gave up; a control block left
 *   dirty by such a call, which makes every later one-token call refuse and
 *   leave `out` unwritten) are recorded in the array's control block and are
 *   not returned by this call: read and clear them with
 *   moe_static_workspace_check(). */
moe_status_t moe_forward_static_ws(const moe_config_t* cfg, const moe_weights_t* wts,
                                   const void* x, int32_t n, void* out,
                                   int32_t* idx, float* w, moe_stream_t stream);

/* moe_workspace_check for the static workspace of moe_forward_static_ws on the
 * current device (no counterpart in the pages: an addition of this library).
 * Reads, then clears, the array's device error word and resets its
 * single-token barrier word, so the next static call runs; synchronises
 * `stream`.
 *   device_error (out)  as moe_workspace_check: 0, 11-17, 1-8 or 20.
 *   workspace    (out, optional) the array's device address on this device
 *                (NULL = not returned); the library owns it.
 * The first use on a device runs the set-up of moe_forward_static_ws.
 * Errors: MOE_ERR_NULL (device_error NULL), MOE_ERR_UNSUPPORTED (`stream` is
 * being captured into a graph), MOE_ERR_CUDA. */
moe_status_t moe_static_workspace_check(int32_t* device_error, void** workspace, moe_stream_t stream);

/* Reads, then clears, the device error word of a workspace, and resets the
 * single-token kernel's and the grouped down kernel's barrier words (which a
 * call that ended early leaves non-zero) and the routed-token count, so the
 * workspace serves the next call.  Synchronises `stream` (the only entry
 * point that does).
 *   device_error (out)  0: no failure since the last check; 11-17: a bounded
 *                       wait of the single-token kernel gave up; 1-5: a bounded
 *                       wait of the grouped tensor-core kernels gave up (8: the
 *                       down kernel's grid barrier before its combine); 6-7:
 *                       one of the tensor-core router's; 31-37: one of
 *                       moe_lora's, in its workspace, or moe_lora_checked's,
 *                       in its errors; 20: the workspace
 *                       control block was not zeroed before use.  An FP8
 *                       call on the grouped path made while an error is
 *                       pending does not write out (its down kernel, which
 *                       also combines, skips the combine); check (and so
 *                       clear) after a failure.
 * Errors: MOE_ERR_NULL, MOE_ERR_ALIGNMENT, MOE_ERR_WORKSPACE (ws_bytes < 256),
 * MOE_ERR_CUDA. */
moe_status_t moe_workspace_check(void* ws, size_t ws_bytes, int32_t* device_error,
                                 moe_stream_t stream);

/* Routing of one call, from logits the caller holds (moe_topk). */
typedef struct {
    int32_t num_experts;            /* E, 1..1024 */
    int32_t top_k;                  /* k, 1..min(E, 32) */
    int32_t routing;                /* moe_routing_t or MOE_ROUTING(...) */
    int32_t norm_topk_prob;         /* 0 or 1 */
    float   routed_scaling_factor;  /* finite */
    int32_t logits_type;            /* moe_dtype_t */
} moe_topk_config_t;

/* Top-k routing of n rows of logits: the pages' topk step on its own, for a
 * router product the caller made, and for any number of rows.  moe_route and
 * moe_forward route through the same kernel when their routing word is not one
 * of MOE_ROUTE_SOFTMAX and MOE_ROUTE_SIGMOID_BIAS alone.
 *   logits      device [n, E] of logits_type, rows row_stride elements apart
 *               (row_stride >= E; any element alignment)
 *   bias        device fp32 [E] (*_BIAS modes; 4-byte aligned), else NULL
 *   idx, w      device int32 / fp32 [n, k] (out), slots in descending
 *               selection score, equal scores by ascending expert index
 * Selection is that of the scores in 64 bits, for any finite or infinite bias.
 * A NaN score ranks as -inf does (a softmax of -inf alone is NaN: such a row
 * takes experts by index); a group score of inf - inf ranks last.
 * w = p, divided by the sum of the k selected p if norm_topk_prob, times
 * routed_scaling_factor; a row whose selected logits are all -inf gets w = 0.
 * logits may also be pinned host memory.  No workspace; n == 0 is a no-op.
 * Errors: MOE_ERR_NULL, MOE_ERR_INVALID_CONFIG, MOE_ERR_UNSUPPORTED (more than
 * 32 groups), MOE_ERR_ALIGNMENT (a pointer is not aligned to its element),
 * MOE_ERR_HOST_MEMORY, MOE_ERR_CUDA. */
moe_status_t moe_topk(const moe_topk_config_t* cfg, const void* logits, int64_t row_stride, const float* bias,
                      int32_t n, int32_t* idx, float* w, moe_stream_t stream);

/* One 4-bit weight matrix [out_features, in_features] (moe_matvec). */
typedef struct {
    int32_t out_features;           /* 1..2^28 */
    int32_t in_features;            /* > 0, a multiple of 32 and of the group size, <= 57344 */
    int32_t w_fmt;                  /* MOE_W_INT4_G32 / G64 / G128 or MOE_W_NVFP4 */
    int32_t x_type;                 /* MOE_BF16 or MOE_F16 */
    int32_t out_type;               /* moe_dtype_t */
    int32_t accumulate;             /* 1: out = rounded(out + result) */
} moe_matvec_config_t;

/* out[t, o] = sum_i W[o, i] x[t, i] (+ bias[o]) (+ out[t, o]) for the n rows of
 * x: the matrix-vector product of the layer's 4-bit formats for a decode batch,
 * as the experts use it, for the dense projections around the layer.  fp32
 * accumulation, one rounding to out_type.  A row's result does not depend on
 * the other rows.  The weights cross HBM once for each 16 rows of x while
 * in_features <= 5376, for each 8 up to 10752, and for as many as 175040 bytes
 * hold at 2 in_features + 64 each beyond (5 at 16384, 1 at 57344).
 *   w           the matrix, in the layouts above with E = 1 (its w 16-byte
 *               aligned, scale and scale2 4)
 *   bias        device fp32 [out_features] (4-byte aligned), or NULL
 *   x           device [n, in_features], rows x_stride elements apart; 16-byte
 *               aligned, x_stride >= in_features and a multiple of 8
 *   out         device [n, out_features], rows out_stride >= out_features
 *               elements apart, aligned to its element; must not overlap x
 * x and out may also be pinned host memory.  No workspace; n == 0 is a no-op.
 * Errors: MOE_ERR_NULL, MOE_ERR_INVALID_CONFIG, MOE_ERR_UNSUPPORTED (a weight
 * format of 8 or 16 bits, more than 57344 in_features or 2^28 out_features), MOE_ERR_ALIGNMENT, MOE_ERR_ALIAS,
 * MOE_ERR_HOST_MEMORY, MOE_ERR_CUDA. */
moe_status_t moe_matvec(const moe_matvec_config_t* cfg, const moe_qmat_t* w, const float* bias, const void* x,
                        int64_t x_stride, int32_t n, void* out, int64_t out_stride, moe_stream_t stream);

/* Residual addition and RMSNorm of rows (moe_norm). */
typedef struct {
    int32_t hidden;                 /* H, 1..32768 */
    int32_t x_type;                 /* moe_dtype_t */
    int32_t residual_type;          /* of residual and residual_out: x_type or MOE_F32 */
    int32_t weight_type;            /* moe_dtype_t */
    int32_t out_type;               /* moe_dtype_t */
    int32_t scale_group;            /* elements of a row that share a scale of out8: 128, or 0 for the whole row */
    float   eps;                    /* >= 0 */
    float   weight_offset;          /* added to the weight: 0, or 1 where weights are stored about 0 */
} moe_norm_config_t;

/* The norm between two layers, for any number of rows: a layer's output x is
 * added to the residual stream, and the sum, normalised, is the next input --
 * in 16 or 32 bits, in 8 bits with scales (the FP8 experts' E4M3 and their
 * blocks of 128 along a reduction), or both.  (The layer's own pre-expert norm
 * has neither a residual nor an 8-bit output.)
 *   h = x + residual in fp32, rounded to the residual's type; x without one
 *   y = h / sqrt(mean(h^2) + eps) * (weight + weight_offset)      (fp32)
 *   residual_out = h;  out = y, rounded to out_type;
 *   scale8[g] = max(max |y| / 448, 2^-126) over the group g;  out8 = E4M3(y / scale8[g])
 *   (scale8 from y as an fp32 out holds it; codes, to nearest even, from
 *   h (weight + weight_offset) and its largest, which the root does not enter: of
 *   16-bit h and weights, weight_offset 0, as exact arithmetic has them)
 *   x, residual     device [n, H]; residual may be NULL
 *   weight          device [H], or NULL (1)
 *   residual_out    device [n, H] (out), or NULL; may be residual itself
 *   out             device [n, H] (out), or NULL; may be x itself (of one type)
 *   out8, scale8    device E4M3 bytes [n, H] and fp32 [n, ceil(H / 128)] or [n] (out),
 *                   or NULL; one of out and out8 is given
 * Rows are *_stride >= H elements apart; every pointer is aligned to its
 * element.  Where all of them (and the strides) are multiples of 16 bytes (8 for
 * out8) and H of 8, rows are read and written 16 bytes at a time.  Other rows
 * are read by the aligned 16 bytes around their elements: bytes beside a row
 * may be read with it (within the 16 that hold its first or last element),
 * and are never written.
 * Outputs overlap nothing else, from their first row to their last.
 * h^2 may leave fp32's range: such a row is normalised all the same.  A row of
 * zeros with eps = 0 gives zeros.  An infinity in h makes NaN of itself and
 * zeros of the rest, a NaN the whole row; the scale of a group with an infinity
 * or a NaN in y is that, and the values it stands for are NaN.
 * All of these but weight may also be pinned host memory.  No workspace;
 * n == 0 is a no-op.
 * Errors: MOE_ERR_NULL, MOE_ERR_INVALID_CONFIG, MOE_ERR_UNSUPPORTED (more than
 * 32768 elements), MOE_ERR_ALIGNMENT, MOE_ERR_ALIAS, MOE_ERR_HOST_MEMORY,
 * MOE_ERR_CUDA. */
moe_status_t moe_norm(const moe_norm_config_t* cfg, const void* x, int64_t x_stride, const void* residual,
                      int64_t residual_stride, const void* weight, int32_t n, void* residual_out,
                      int64_t residual_out_stride, void* out, int64_t out_stride, void* out8, int64_t out8_stride,
                      float* scale8, moe_stream_t stream);

/* Low-rank adapters of one projection (moe_lora). */
typedef struct {
    int32_t in_features;            /* a multiple of 8, at most 2^20 */
    int32_t out_features;           /* 1..2^28 */
    int32_t rank;                   /* a multiple of 8, at most 128 (an adapter of less is filled with zeros) */
    int32_t num_adapters;           /* 1..1024 */
    int32_t x_type;                 /* of x and of both matrices: MOE_BF16 or MOE_F16 */
    int32_t out_type;               /* of base and out: moe_dtype_t */
} moe_lora_config_t;

/* Bytes of workspace a call with up to `max_rows` rows needs (a multiple of
 * 256).  Returns 0 if `cfg` is NULL or invalid, or max_rows < 0. */
size_t moe_lora_workspace_bytes(const moe_lora_config_t* cfg, int32_t max_rows);

/* out[t] = base[t] + scale[e] B_e (A_e x[t]),  e = idx[t]: the adapters of many
 * requests at once beside a projection that they share (moe_matvec's, or any
 * other), whose result is `base`.  A row whose e is outside [0, num_adapters)
 * has no adapter: out[t] = base[t].
 *   a           device [num_adapters, rank, in_features] (16-byte aligned)
 *   b           device [num_adapters, out_features, rank] (16-byte aligned)
 *   scale       device fp32 [num_adapters], or NULL (1)
 *   x           device [n, in_features], rows x_stride elements apart; 16-byte
 *               aligned, x_stride >= in_features and a multiple of 8
 *   idx         device int32 [n], in any order
 *   base        device [n, out_features], rows base_stride elements apart, or
 *               NULL (zeros); may be out itself
 *   out         device [n, out_features] (out), rows out_stride elements apart;
 *               overlaps nothing else but base where it is that, from the first
 *               row to the last
 *   ws          device workspace (16-byte aligned) of at least
 *               moe_lora_workspace_bytes(cfg, n) bytes, of which no other
 *               argument has any; it need not be cleared,
 *               and keeps nothing between calls but the error word of the last,
 *               for moe_workspace_check (256 bytes: it is not used, and may be
 *               any address).  Where a wait of the product with A gave up, out
 *               is not written; of the one with B, some of it is
 * base and out are aligned to their element.  fp32 sums; A_e x[t] enters the
 * second product in 16 bits of precision for outputs of 16 bits, in 24 for
 * fp32 outputs; one rounding to out_type, after the addition of base.  (As a
 * sum of 16-bit parts, of which some are 0 or of the other sign: an infinity
 * in b may come out as NaN where the formula has an infinity.)
 * x, base and out may also be pinned host memory; n == 0 is a no-op.
 * Errors: MOE_ERR_NULL, MOE_ERR_INVALID_CONFIG, MOE_ERR_UNSUPPORTED (a rank
 * over 128, more than 1024 adapters, 2^20 in_features or 2^28 out_features),
 * MOE_ERR_WORKSPACE, MOE_ERR_ALIGNMENT, MOE_ERR_ALIAS, MOE_ERR_HOST_MEMORY,
 * MOE_ERR_CUDA. */
moe_status_t moe_lora(const moe_lora_config_t* cfg, const void* a, const void* b, const float* scale, const void* x,
                      int64_t x_stride, const int32_t* idx, int32_t n, const void* base, int64_t base_stride, void* out,
                      int64_t out_stride, void* ws, size_t ws_bytes, moe_stream_t stream);

/* moe_lora for a workspace that does not outlive the call: the code of a bounded
 * wait that gives up goes to `errors` (device, 256 bytes, 16-byte aligned, zeros
 * before the first call; of any number of calls, on any streams), where it stays
 * until moe_workspace_check(errors, 256, ...) reads and clears it.  Calls whose
 * workspace is above 256 bytes do not write out while it is there (the others
 * have no such waits); what is no such code there is not looked at. */
moe_status_t moe_lora_checked(const moe_lora_config_t* cfg, const void* a, const void* b, const float* scale, const void* x,
                              int64_t x_stride, const int32_t* idx, int32_t n, const void* base, int64_t base_stride, void* out,
                              int64_t out_stride, void* ws, size_t ws_bytes, void* errors, moe_stream_t stream);

/* Static description of a status code (never NULL). */
const char* moe_status_string(moe_status_t status);

/* MOE_ABI_VERSION of the built library. */
int32_t moe_abi_version(void);

#ifdef __cplusplus
}
#endif
#endif /* MOE_GB300_MOE_H */
