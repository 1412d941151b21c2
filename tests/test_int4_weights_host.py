"""The layer's calls refuse routed experts that are stored in another form than the config names, before
anything is launched.  No GPU is needed: what gets past the checks is refused for lying on the host."""
from __future__ import annotations

import pytest
import torch

import mixture_experts_layer_37_b200 as M

T, D, FFN, E, K = 4, 192, 320, 4, 1


@pytest.fixture(scope="module", autouse=True)
def built():
    from mixture_experts_layer_37_b200 import build
    build.build()


def names(act):
    return (("w_gate", D, FFN), ("w_up", D, FFN), ("w_down", FFN, D)) if act == "swiglu" else \
        (("w1", D, FFN), ("w2", FFN, D))


def int4_weights(act, group, experts=E):
    w = {}
    for n, k, c in names(act):
        w[n] = torch.zeros(experts, c, -(-k // 128) * 64, dtype=torch.uint8)
        w[n + "_scale"] = torch.zeros(experts, -(-k // group), c)
    if act != "swiglu":
        w["b1"], w["b2"] = torch.zeros(experts, FFN).bfloat16(), torch.zeros(experts, D).bfloat16()
    return w


def config(act="swiglu", weights="int4_g32"):
    return M.MoEConfig(T=T, d=D, ffn=FFN, E=E, k=K, act=act, capacity_factor=0.0, weights=weights)


def calls(cfg, w):
    """Every call that takes the routed experts' weights."""
    ws = type("W", (), {"ptr": 1 << 20, "nbytes": 0})()
    x = torch.zeros(T, D).bfloat16()
    one = torch.zeros(1, dtype=torch.int32)
    yield "MoELayer", lambda: M.MoELayer(cfg, w)
    yield "moe_expert_ffn", lambda: M.moe_expert_ffn(cfg, w, x, one, x, ws, stream=0)
    yield "moe_forward", lambda: M.moe_forward(cfg, w, x, {}, ws, stream=0)
    yield "moe_forward_profiled", lambda: M.moe_forward_profiled(cfg, w, x, {}, ws, [], stream=0)
    yield "moe_forward_hostio", lambda: M.moe_forward_hostio(cfg, w, x, x, {}, x, x, ws, stream=0)
    yield "moe_dp_finish", lambda: M.moe_dp_finish(cfg, T, one, one, 1, 0, w, x, {}, ws, stream=0)
    yield "moe_pipeline_create", lambda: M.Pipeline(cfg, w)
    yield "moe_ep_expert_ffn", lambda: M.moe_ep_expert_ffn(cfg, T, 1, w, x, x, one, x, ws, stream=0)


def refused(cfg, w, match):
    for name, f in calls(cfg, w):
        with pytest.raises(M.MoEError, match=f"{name}: .*{match}"):
            f()


@pytest.mark.parametrize("act", ["swiglu", "gelu_bias"])
@pytest.mark.parametrize("have,want", [(128, 32), (64, 32), (128, 64), (32, 128)])
def test_scales_of_another_group_length(act, have, want):
    refused(config(act, f"int4_g{want}"), int4_weights(act, have), "_scale of int4_g")


@pytest.mark.parametrize("act", ["swiglu", "gelu_bias"])
def test_each_tensor_is_looked_at(act):
    cfg = config(act)
    good = int4_weights(act, 32)
    refused(cfg, good, "tensors on a CUDA device")           # all that is wrong with these
    for n in [n for n in good if n not in ("b1", "b2")]:
        t = good[n]
        for bad in (t[:, :-8].contiguous(), t[:-1], t.to(torch.int8), t.transpose(1, 2).contiguous().transpose(1, 2),
                    torch.empty(t.shape, dtype=t.dtype, device="meta")):
            match = "a contiguous tensor" if bad.device.type == "cpu" or n != names(act)[0][0] else "contiguous|CUDA"
            refused(cfg, {**good, n: bad}, match)


def test_codes_under_another_format():
    w4 = int4_weights("swiglu", 64)
    w8 = {n: torch.zeros(E, k, c, dtype=torch.int8) for n, k, c in names("swiglu")}
    w16 = {n: torch.zeros(E, k, c).bfloat16() for n, k, c in names("swiglu")}
    refused(config(weights="native"), w4, "holds codes")
    refused(config(weights="int8"), w4, "holds codes")
    refused(config(weights="native"), w8, "holds codes")
    refused(config(weights="int4_g64"), w8, "a contiguous tensor")
    refused(config(weights="int4_g64"), w16, "a contiguous tensor")


def test_expert_parallel_ranks_hold_their_part():
    cfg = config()
    ws = type("W", (), {"ptr": 1 << 20, "nbytes": 0})()
    x, o = torch.zeros(T, D).bfloat16(), torch.zeros(3, dtype=torch.int32)
    whole = int4_weights("swiglu", 32)
    for w, match in ((whole, "a contiguous tensor"), (M.local_expert_weights(whole, 2, 1), "tensors on a CUDA device")):
        with pytest.raises(M.MoEError, match=match):
            M.moe_ep_expert_ffn(cfg, T, 2, w, x, x, o, x, ws, stream=0)
