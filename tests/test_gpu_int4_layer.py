"""The whole layer on 4-bit experts beside shared experts, padding and drops, against the float64 oracle on the
weights that the codes stand for (exact in bf16 here: scales are powers of two)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import mixture_experts_layer_37_b200 as M
import workloads as W
from gpu_common import host_f64, mask_dev, out_close, to_dev, weights_dev
from oracle import moe_oracle as O

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act,group,T,kw", [
    ("swiglu", 64, 300, dict(n_shared=2, pad_fraction=0.2, capacity_factor=0.8)),
    ("gelu_bias", 32, 300, dict(n_shared=1, capacity_factor=1.0)),
    ("swiglu", 128, 1, dict(capacity_factor=0.0, n_shared=1)),
    ("gelu_bias", 128, 700, dict(pad_fraction=0.5, capacity_factor=0.6)),
])
def test_layer_with_all_that_surrounds_the_experts(act, group, T, kw):
    wl = W.Workload("int4_all", T=T, d=192, ffn=320, E=6, k=2, act=act, dtype="bf16", seed=91, weights=f"int4_g{group}",
                    **kw)
    inp = W.make_inputs(wl)
    wd = weights_dev(wl, inp)
    for n in ("w_gate", "w_up", "w_down") if act == "swiglu" else ("w1", "w2"):
        w = wd[n].float()
        K = w.shape[1]
        G = -(-K // group)
        pad = torch.nn.functional.pad(w, (0, 0, 0, G * group - K)).view(w.shape[0], G, group, -1)
        scale = torch.exp2(torch.ceil(torch.log2(pad.abs().amax(2) / 7)))
        rows = torch.repeat_interleave(scale, group, dim=1)[:, :K]
        q = torch.round(w / rows).clamp(-8, 7)
        wd[n], wd[n + "_scale"] = M.moe_pack_int4(q.to(torch.int8)), scale.contiguous()
        stands = (q * rows).bfloat16()
        assert torch.equal(stands.float(), q * rows)
        inp[n] = stands.view(torch.int16).cpu().numpy().view(np.uint16)
    cfg, x, mask = M.MoEConfig.of(wl), to_dev(inp["x"]), mask_dev(inp)
    layer = M.MoELayer(cfg, wd)
    first = layer.forward(x, token_mask=mask)["out"].clone()
    layer.check()
    layer.capture(x, token_mask=mask)
    layer.outputs["out"].zero_()
    out = layer.replay()
    torch.cuda.synchronize()
    assert torch.equal(out["out"], first)
    r = O.route(wl, inp)
    same = (out["topk_idx"].cpu().numpy() == r["idx"]).all(axis=1) & \
        ((out["slot"].cpu().numpy() >= 0) == (r["slot"] >= 0)).all(axis=1)
    toks = np.arange(T)[same]
    assert len(toks) >= 0.9 * T
    ref = O.forward(wl, inp, routing=r, tokens=toks)
    ok, err, scale = out_close(host_f64(first)[toks], ref["out"], wl.dtype)
    assert ok, f"max err {err} vs scale {scale}"
