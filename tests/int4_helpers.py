"""Host copies of layers with INT4 group-scaled experts for the oracle."""

from __future__ import annotations

from oracle import moe_oracle as O
from tests.moe_helpers import LazyExperts, bf16_bits


def host_int4(q) -> O.QMat:
    return O.QMat(q.fmt, LazyExperts(q.w), LazyExperts(q.scale, as_uint16=True),
                  zero=LazyExperts(q.zero) if q.zero is not None else None)


def int4_oracle_layer(lw) -> O.OracleLayer:
    c = lw.cfg
    return O.OracleLayer(
        hidden=c.hidden, num_experts=c.num_experts, top_k=c.top_k, inter=c.inter, shared_inter=c.shared_inter,
        routing=c.routing, norm_topk_prob=c.norm_topk_prob, routed_scaling_factor=c.routed_scaling_factor,
        router_w=bf16_bits(lw.router_w), gate=host_int4(lw.gate), up=host_int4(lw.up), down=host_int4(lw.down),
        sh_gate=host_int4(lw.sh_gate) if lw.sh_gate is not None else None,
        sh_up=host_int4(lw.sh_up) if lw.sh_up is not None else None,
        sh_down=host_int4(lw.sh_down) if lw.sh_down is not None else None,
        correction_bias=lw.correction_bias.cpu().numpy() if lw.correction_bias is not None else None,
        shared_gate_w=bf16_bits(lw.shared_gate_w) if lw.shared_gate_w is not None else None,
        pre_expert_norm_w=bf16_bits(lw.pre_expert_norm_w) if lw.pre_expert_norm_w is not None else None,
        rms_norm_eps=c.rms_norm_eps)
