"""Data-parallel shards on 4-bit experts, emulated on one GPU: bit for bit one forward over the whole batch."""
import pytest
import torch

import mixture_experts_layer_37_b200 as M
import workloads as W
from gpu_common import to_dev, weights_dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act,group,bounds", [("swiglu", 32, [0, 70, 71, 190]), ("gelu_bias", 128, [0, 100, 190]),
                                              ("swiglu", 64, [0, 190])])
def test_shards_equal_the_whole_batch(act, group, bounds):
    wl = W.Workload("dp_int4", T=190, d=192, ffn=320, E=4, k=2, act=act, dtype="bf16", capacity_factor=0.8, seed=71,
                    weights=f"int4_g{group}")
    inp = W.make_inputs(wl)
    cfg = M.MoEConfig.of(wl)
    wd = M.quantize_expert_weights(cfg, weights_dev(wl, inp))
    x = to_dev(inp["x"])
    whole = M.MoELayer(cfg, wd).forward(x)
    assert (whole["slot"] < 0).any(), "the case must exercise drops"
    world, shards = len(bounds) - 1, []
    for t0, t1 in zip(bounds, bounds[1:]):
        c = M.MoEConfig.of(wl.with_(T=t1 - t0))
        s = dict(c=c, x=x[t0:t1], o=M.allocate_outputs(c), ws=M.Workspace(c, nbytes=M.moe_dp_workspace_size(c, wl.T)),
                 lc=torch.zeros(wl.E, dtype=torch.int32, device="cuda"),
                 lp=torch.zeros(wl.E, dtype=torch.float64, device="cuda"),
                 lr=torch.zeros(1, dtype=torch.int32, device="cuda"))
        s["o"]["src_assign"] = torch.empty(max(M.moe_dp_max_rows(c, wl.T), 1), dtype=torch.int32, device="cuda")
        M.moe_dp_route(c, wl.T, wd, s["x"], s["o"], s["lc"], s["lp"], s["ws"], local_real=s["lr"])
        shards.append(s)
    counts, psum, real = (torch.stack([s[n] for s in shards]) for n in ("lc", "lp", "lr"))
    for r, s in enumerate(shards):
        M.moe_dp_finish(s["c"], wl.T, counts, psum, world, r, wd, s["x"], s["o"], s["ws"], all_real=real)
        assert M.moe_check_device_status(s["ws"])[0] == M.MOE_OK
    assert torch.equal(torch.cat([s["o"]["out"] for s in shards]), whole["out"])
