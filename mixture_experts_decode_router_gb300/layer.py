"""A thin holder that turns torch weight tensors into the C structs of
``include/moe.h`` and calls the library.  Marshalling only: no arithmetic of
the layer happens here.
"""

from __future__ import annotations

from ctypes import addressof
from dataclasses import fields, is_dataclass
from typing import Optional

import torch

from . import binding as B
from .synth import (FMT_BF16, FMT_FP8_B128, FMT_INT4_G128, FMT_INT4_G32, FMT_INT4_G64, FMT_NVFP4, INT4_GROUP,
                    ROUTE_SIGMOID, ROUTE_SIGMOID_BIAS, ROUTE_SOFTMAX, ROUTE_SOFTMAX_BIAS, LayerConfig,
                    LayerWeights, QMatT)

_FMT = {FMT_BF16: B.MOE_W_BF16, FMT_FP8_B128: B.MOE_W_FP8_B128, FMT_NVFP4: B.MOE_W_NVFP4,
        FMT_INT4_G32: B.MOE_W_INT4_G32, FMT_INT4_G64: B.MOE_W_INT4_G64, FMT_INT4_G128: B.MOE_W_INT4_G128}
_PATH = {"auto": B.MOE_PATH_AUTO, "token_major": B.MOE_PATH_TOKEN_MAJOR,
         "grouped": B.MOE_PATH_GROUPED}


_MODE = {ROUTE_SOFTMAX: B.MOE_ROUTE_SOFTMAX, ROUTE_SIGMOID_BIAS: B.MOE_ROUTE_SIGMOID_BIAS,
         ROUTE_SOFTMAX_BIAS: B.MOE_ROUTE_SOFTMAX_BIAS, ROUTE_SIGMOID: B.MOE_ROUTE_SIGMOID}
_SCORE = {"max": B.MOE_GROUP_MAX, "top2": B.MOE_GROUP_TOP2}
_TYPE = {torch.float32: B.MOE_F32, torch.bfloat16: B.MOE_BF16, torch.float16: B.MOE_F16}


def routing_word(routing: str, num_groups: int = 1, topk_groups: int = 1, group_score: str = "top2") -> int:
    """The C routing word of a routing name and its groups (1 = no groups)."""
    mode = _MODE[routing]
    if num_groups == 1:
        return mode
    if not (0 < num_groups < 256 and 0 < topk_groups < 256):
        raise ValueError("num_groups and topk_groups are 1..255")
    return B.MOE_ROUTING(mode, num_groups, topk_groups, _SCORE[group_score])


def make_config(cfg: LayerConfig, path: str = "auto", experts=None,
                exclude_shared: bool = False, accumulate: bool = False) -> B.moe_config_t:
    """``experts`` = (begin, end): the routed experts this call holds (expert
    parallelism; None = all).  ``exclude_shared``: leave the shared expert out.
    ``accumulate``: add the layer's output into ``out``."""
    c = B.moe_config_t()
    c.hidden, c.num_experts, c.top_k = cfg.hidden, cfg.num_experts, cfg.top_k
    c.inter, c.shared_inter = cfg.inter, cfg.shared_inter
    c.routing = routing_word(cfg.routing, cfg.num_groups, cfg.topk_groups, cfg.group_score)
    c.norm_topk_prob = 1 if cfg.norm_topk_prob else 0
    c.routed_scaling_factor = cfg.routed_scaling_factor
    c.expert_fmt = _FMT[cfg.expert_fmt]
    c.path = _PATH[path]
    c.rms_norm_eps = cfg.rms_norm_eps
    if experts is not None:
        c.expert_begin, c.expert_end = int(experts[0]), int(experts[1])
    c.exclude_shared = 1 if exclude_shared else 0
    c.accumulate = 1 if accumulate else 0
    c.router_fmt = _FMT[cfg.router_fmt]
    return c


_BYTES = {torch.uint8, torch.int8}
_E4M3 = _BYTES | {torch.float8_e4m3fn}
_E2M1 = _BYTES | {t for t in (getattr(torch, "float4_e2m1fn_x2", None),) if t is not None}


def _check_4bit(q: QMatT, n: int, out: int, inp: int) -> None:
    """The arrays of n 4-bit matrices [out, inp] are those of their format: the kernels see only
    addresses, and read them by these sizes and types."""
    def is_a(t, cols, types):
        return (t is not None and t.dtype in types and t.dim() > 0 and t.shape[-1] == cols
                and t.numel() == n * out * cols and t.is_contiguous())
    if q.fmt == FMT_NVFP4:
        if not (is_a(q.w, inp // 2, _E2M1) and is_a(q.scale, inp // 16, _E4M3)):
            raise ValueError("NVFP4 is E2M1 pairs [out, in/2] and E4M3 scales [out, in/16], in bytes")
        if q.zero is not None or q.scale2 is None or q.scale2.dtype != torch.float32 or q.scale2.numel() != n \
                or not q.scale2.is_contiguous():
            raise ValueError("NVFP4 has one float32 scale2 a matrix and no zero points")
    else:
        G = INT4_GROUP[q.fmt]
        if inp % G or not (is_a(q.w, inp // 2, _BYTES) and is_a(q.scale, inp // G, {torch.bfloat16})):
            raise ValueError(f"{q.fmt} is pairs of codes [out, in/2], in bytes, and bfloat16 scales [out, in/{G}]")
        if q.scale2 is not None or not (q.zero is None or is_a(q.zero, inp // G, _BYTES)):
            raise ValueError(f"{q.fmt} has zero points [out, in/{G}], in bytes, or none, and no scale2")


def _qmat(q: Optional[QMatT]) -> B.moe_qmat_t:
    m = B.moe_qmat_t()
    if q is None:
        return m
    m.w = q.w.data_ptr()
    m.scale = q.scale.data_ptr() if q.scale is not None else None
    if q.scale2 is not None:
        m.scale2 = q.scale2.data_ptr()
    elif q.zero is not None:
        m.zero = q.zero.data_ptr()
    return m


def make_weights(lw: LayerWeights) -> B.moe_weights_t:
    w = B.moe_weights_t()
    w.router_w = lw.router_w.data_ptr()
    w.correction_bias = lw.correction_bias.data_ptr() if lw.correction_bias is not None else None
    w.gate, w.up, w.down = _qmat(lw.gate), _qmat(lw.up), _qmat(lw.down)
    w.sh_gate, w.sh_up, w.sh_down = _qmat(lw.sh_gate), _qmat(lw.sh_up), _qmat(lw.sh_down)
    w.shared_gate_w = lw.shared_gate_w.data_ptr() if lw.shared_gate_w is not None else None
    w.pre_expert_norm_w = (lw.pre_expert_norm_w.data_ptr() if lw.pre_expert_norm_w is not None
                           else None)
    w.router_q = _qmat(lw.router_q)
    return w


def _tensors(o) -> list:
    """The tensors of a weights dataclass, those of its matrices included."""
    if isinstance(o, torch.Tensor):
        return [o]
    return [t for f in fields(o) for t in _tensors(getattr(o, f.name))] if is_dataclass(o) else []


def _made(stream, *shape, **kw) -> torch.Tensor:
    """An output of a call on `stream`: that stream's memory, in use on the current one."""
    current = None if stream is None else torch.cuda.current_stream(kw["device"])
    if current is None or B._stream(stream) == current.cuda_stream:
        return torch.empty(*shape, **kw)
    raw, dev = B._stream(stream), kw["device"]   # (ExternalStream(0) would be a new stream)
    with torch.cuda.stream(torch.cuda.ExternalStream(raw, dev) if raw else torch.cuda.default_stream(dev)):
        t = torch.empty(*shape, **kw)
    t.record_stream(current)
    return t


class MoeLayer:
    """One MoE layer on the current CUDA device.

    ``forward(x)`` runs router, top-k, experts and blend through ``moe_forward``
    on the current torch stream and returns ``(out, idx, w)``.

    Expert parallelism: with ``experts=(begin, end)`` the weight stacks of
    ``weights`` hold only those experts (``synth.expert_slice``) and the output
    is this rank's partial; ``exclude_shared`` leaves the shared expert out;
    ``accumulate`` adds the result into ``out`` (which must then be given).
    """

    def __init__(self, weights: LayerWeights, max_tokens: int, path: str = "auto",
                 experts=None, exclude_shared: bool = False, accumulate: bool = False):
        self.weights = weights
        self.cfg = weights.cfg
        self.accumulate = accumulate
        self.c_cfg = make_config(self.cfg, path, experts, exclude_shared, accumulate)
        self.c_w = make_weights(weights)
        self._held = _tensors(weights)   # the memory that c_w points to
        self.ws_bytes = B.moe_workspace_bytes(self.c_cfg, max_tokens)
        if self.ws_bytes == 0:
            raise B.MoeError("invalid layer configuration")
        if self.cfg.expert_fmt in INT4_GROUP:
            self._check_int4()
        dev = self._device = weights.router_w.device
        # The control block (first 256 bytes) must start at zero; calls keep it zero.
        self.ws = torch.zeros(self.ws_bytes, dtype=torch.uint8, device=dev)
        self.max_tokens = max_tokens
        calls = B.tensor_calls()
        self._experts, self._forward = calls.experts, calls.forward

    def _check_int4(self) -> None:
        """The arrays of the matrices that this layer's calls read."""
        c, lw = self.c_cfg, self.weights
        held = c.num_experts if c.expert_begin == c.expert_end == 0 else c.expert_end - c.expert_begin
        stacks = [("gate", held, c.inter, c.hidden), ("up", held, c.inter, c.hidden), ("down", held, c.hidden, c.inter)]
        shared = 0 if c.exclude_shared else c.shared_inter
        stacks += [("sh_gate", 1, shared, c.hidden), ("sh_up", 1, shared, c.hidden), ("sh_down", 1, c.hidden, shared)]
        for name, n, out, inp in stacks:
            q = getattr(lw, name)
            if n * out * inp == 0:
                continue
            if q is None or q.fmt != self.cfg.expert_fmt:
                raise ValueError(f"{name} is an {self.cfg.expert_fmt} matrix")
            _check_4bit(q, n, out, inp)
            if any(t is not None and t.device != lw.router_w.device for t in (q.w, q.scale, q.zero)):
                raise ValueError("weights on one device")

    def forward(self, x: torch.Tensor, out=None, idx=None, w=None, stream=None,
                routing: bool = True):
        """``routing=False``: do not return the routing (idx and w are None), so
        a call that holds no routed expert can skip it."""
        return self._forward(addressof(self.c_cfg), addressof(self.c_w), self.ws, self.ws_bytes, x, out, idx, w, routing,
                             stream if stream is None else B._stream(stream))

    def device_error(self, stream=None) -> int:
        """Reads and clears the workspace's device error word (syncs the stream)."""
        s, v = B.moe_workspace_check(self.ws, self.ws_bytes, stream)
        B.check(s)
        return v

    def route(self, x: torch.Tensor, logits: bool = True, stream=None):
        dev, H = self._device, self.cfg.hidden
        if x.dtype != torch.bfloat16 or x.dim() < 1 or x.numel() != x.shape[0] * H or not x.is_contiguous():
            raise ValueError("x is contiguous bfloat16 [n, hidden]")
        if dev.type != "cuda" or dev.index != torch.cuda.current_device() or not (x.device == dev or x.is_pinned()):
            raise ValueError("x is on the current device, which is the layer's, or in pinned host memory")
        n, k, E = x.shape[0], self.cfg.top_k, self.cfg.num_experts
        idx = _made(stream, n, k, dtype=torch.int32, device=dev)
        w = _made(stream, n, k, dtype=torch.float32, device=dev)
        lg = _made(stream, n, E, dtype=torch.float32, device=dev) if logits else None
        B.check(B.moe_route(self.c_cfg, self.c_w, x, n, idx, w, lg, self.ws, self.ws_bytes, stream))
        return idx, w, lg

    def experts(self, x: torch.Tensor, idx: torch.Tensor, w: torch.Tensor, stream=None):
        return self._experts(addressof(self.c_cfg), addressof(self.c_w), self.ws, self.ws_bytes, x, idx, w,
                             stream if stream is None else B._stream(stream))


class MoeTopk:
    """Top-k routing of logits the caller holds (``moe_topk``): ``forward(logits)``
    returns ``(idx, w)`` of ``[n, num_experts]`` fp32, bf16 or fp16 logits, whose
    rows may be strided.

    ``routing`` is "softmax" or "sigmoid"; ``bias`` (fp32 ``[num_experts]``) is added
    to the scores for the selection only.  ``num_groups`` > 1 limits the selection
    to the ``topk_groups`` groups of best ``group_score`` ("max", or "top2": the sum
    of the group's two best scores).
    """

    def __init__(self, num_experts: int, top_k: int, routing: str = "softmax",
                 bias: Optional[torch.Tensor] = None, num_groups: int = 1, topk_groups: int = 1,
                 group_score: str = "top2", norm_topk_prob: bool = True, routed_scaling_factor: float = 1.0):
        if bias is not None and (bias.dtype != torch.float32 or bias.shape != (num_experts,)
                                 or not bias.is_contiguous()):
            raise ValueError("bias is contiguous float32 [num_experts]")
        name = {"softmax": (ROUTE_SOFTMAX, ROUTE_SOFTMAX_BIAS),
                "sigmoid": (ROUTE_SIGMOID, ROUTE_SIGMOID_BIAS)}[routing][bias is not None]
        c = B.moe_topk_config_t()
        c.num_experts, c.top_k = num_experts, top_k
        c.routing = routing_word(name, num_groups, topk_groups, group_score)
        c.norm_topk_prob = 1 if norm_topk_prob else 0
        c.routed_scaling_factor = routed_scaling_factor
        self.num_experts, self.top_k, self.bias, self.c_cfg = num_experts, top_k, bias, c
        self._topk = B.tensor_calls().topk

    def forward(self, logits: torch.Tensor, idx=None, w=None, stream=None):
        return self._topk(addressof(self.c_cfg), self.bias, logits, idx, w, stream if stream is None else B._stream(stream))


class MoeMatvec:
    """Products of one 4-bit matrix with a few vectors (``moe_matvec``): ``forward(x)``
    returns ``[n, out]`` of ``out_dtype`` for bf16 or fp16 ``x`` ``[n, in]``, whose rows
    may be strided.  ``weights``: a ``QMatT`` ``[out, in/2]`` (INT4 groups or NVFP4);
    ``bias``: fp32 ``[out]``; ``accumulate`` adds the result into ``out`` (which must
    then be given).
    """

    def __init__(self, weights: QMatT, bias: Optional[torch.Tensor] = None, out_dtype=torch.bfloat16,
                 accumulate: bool = False):
        q = weights
        out_f, in_f = q.w.shape[-2], 2 * q.w.shape[-1]
        if q.w.numel() != out_f * in_f // 2 or not all(
                t is None or t.is_contiguous() for t in (q.w, q.scale, q.scale2, q.zero, bias)):
            raise ValueError("one contiguous matrix [out, in/2] and its scales")
        if q.fmt == FMT_NVFP4 or q.fmt in INT4_GROUP:
            _check_4bit(q, 1, out_f, in_f)
        if bias is not None and (bias.dtype != torch.float32 or bias.shape != (out_f,)):
            raise ValueError("bias is float32 [out]")
        c = B.moe_matvec_config_t()
        c.out_features, c.in_features, c.w_fmt = out_f, in_f, _FMT[q.fmt]
        c.out_type, c.accumulate = _TYPE[out_dtype], 1 if accumulate else 0
        self.c_cfg, self.c_w = c, _qmat(q)
        self._held = q, bias, (q.w, q.scale, q.scale2, q.zero)   # the memory that c_w and the bias point to
        self.out_dtype = out_dtype
        self.in_features, self.out_features, self.accumulate = in_f, out_f, accumulate
        dev = q.w.get_device()
        if any(t is not None and t.get_device() != dev for t in (q.scale, q.scale2, q.zero, bias)):
            raise ValueError("weights and bias on one device")
        self._matvec = B.tensor_calls().matvec
        self._bias, self._device = 0 if bias is None else bias.data_ptr(), dev

    @property
    def weights(self) -> QMatT:
        return self._held[0]

    @property
    def bias(self) -> Optional[torch.Tensor]:
        return self._held[1]

    def forward(self, x: torch.Tensor, out=None, stream=None):
        return self._matvec(addressof(self.c_cfg), addressof(self.c_w), self._bias, self._device, x, out, stream if stream is None else B._stream(stream))
