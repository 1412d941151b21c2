"""Products and expert FFNs with 4-bit weights: storage form and quantiser
exactly, products against float64 on the dequantised weights.

Tolerances (u = 2^-24, A = the sum over the absolute values of its terms):
code times activation is exact and a group's 32..128 products are summed by the
tensor cores (at most 2 u of A per step of 16), the groups and the parts of K
by fp32 FMA: (K / 8 + 64) u A covers both; an output rounded to bf16 adds half a
step, 2^-8 of its value.  The FFN rounds its inner activation to bf16 once:
2^-8 of its terms more.
"""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import mixture_experts_layer_37_b200 as M

pytestmark = pytest.mark.gpu
U, HALF = 2.0 ** -24, 2.0 ** -8


def rand(shape, std, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g, dtype=torch.float64) * std).to(dtype)


def pack_plain(q):
    """Storage form of codes q int8 [E, K, N] (numpy), from its description, code by code."""
    E, K, N = q.shape
    blocks = -(-K // 128)
    out = np.full((E, N, blocks * 128), 8, dtype=np.uint8)   # by nibble
    for k in range(K):
        b, r = divmod(k, 128)
        i, r = divmod(r, 32)
        t, j = divmod(r, 8)
        nib = j // 2 if j % 2 == 0 else 4 + j // 2
        out[:, :, b * 128 + (4 * t + i) * 8 + nib] = q[:, k, :] + 8
    return out[:, :, 0::2] | (out[:, :, 1::2] << 4)


def offsets_of(counts):
    return [0] + np.cumsum(counts).tolist()


@pytest.mark.parametrize("E,K,N", [(1, 8, 8), (2, 200, 40), (3, 128, 136), (1, 1032, 64)])
def test_pack_is_the_stated_layout(E, K, N):
    q = torch.randint(-8, 8, (E, K, N), dtype=torch.int8, generator=torch.Generator().manual_seed(K))
    got = M.moe_pack_int4(q.cuda()).cpu().numpy()
    want = pack_plain(q.numpy())
    assert np.array_equal(got, want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_quantise_codes_and_scales_exact(dtype, group):
    E, K, N = 2, 328, 72
    w = rand((E, K, N), 0.02, dtype, 5)
    w[0, :, 1] = 0.0
    w[1, 64:128, 2] = 3.0
    codes, scale = M.moe_quantize_int4(w.cuda(), group)
    G = -(-K // group)
    wf = w.float().numpy()
    want_s = np.zeros((E, G, N), dtype=np.float32)
    want_q = np.zeros((E, K, N), dtype=np.int8)
    for g in range(G):
        part = wf[:, g * group:(g + 1) * group]
        s = (np.abs(part).max(axis=1) / np.float32(7.0)).astype(np.float32)
        want_s[:, g] = s
        with np.errstate(divide="ignore", invalid="ignore"):
            q = np.rint((part / s[:, None]).astype(np.float32))
        want_q[:, g * group:(g + 1) * group] = np.where(s[:, None] > 0, np.clip(q, -7, 7), 0)
    assert np.array_equal(scale.cpu().numpy().view(np.uint32), want_s.view(np.uint32))
    assert np.array_equal(codes.cpu().numpy(), pack_plain(want_q))


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_quantise_shows_values_without_a_code(bad, group):
    """A group that holds an infinity or NaN gets the scale NaN and codes 0; the other groups keep theirs, and the
    product is NaN in that expert's column alone."""
    E, K, N, k, n = 2, 328, 72, 130, 5
    w = rand((E, K, N), 0.02, torch.bfloat16, 6)
    codes, scale = (t.cpu() for t in M.moe_quantize_int4(w.cuda(), group))
    w[1, k, n] = bad
    c2, s2 = M.moe_quantize_int4(w.cuda(), group)
    want = scale.clone()
    want[1, k // group, n] = float("nan")
    assert torch.equal(torch.isnan(s2.cpu()), torch.isnan(want))
    assert torch.equal(s2.cpu().nan_to_num(7.0), want.nan_to_num(7.0))
    others = torch.ones(E, N, dtype=torch.bool)
    others[1, n] = False
    assert torch.equal(c2.cpu()[others], codes[others])
    g = M.GroupedConfig(rows=6, E=E, K=K, N=N)
    ws = M.Workspace(None, nbytes=M.moe_grouped_workspace_size(g))
    y = torch.empty(6, N, device="cuda", dtype=torch.bfloat16)
    M.moe_grouped_gemm_int4(g, rand((6, K), 1.0, torch.bfloat16, 7).cuda(), c2, s2,
                            torch.tensor([0, 2, 6], dtype=torch.int32, device="cuda"), y, ws, group)
    expect = torch.zeros(6, N, dtype=torch.bool)
    expect[2:, n] = True
    assert torch.equal(torch.isnan(y.cpu()), expect)


# counts per expert, rows behind the last one, K, N
SHAPES = [
    ([1], 0, 8, 8),
    ([1, 0, 1], 0, 2048, 64),
    ([2] * 64, 0, 256, 128),
    ([3, 0, 9, 1, 17], 2, 200, 328),
    ([0, 0], 3, 128, 64),
    ([40, 0, 33, 7, 64], 1, 360, 136),
    ([8, 100], 0, 1032, 520),
    ([1, 2], 0, 9000, 40),
    ([70], 0, 2600, 72),
    ([300, 0, 5], 1, 640, 264),
]


def case(shape, group, seed=0):
    counts, behind, K, N = shape
    E, off = len(counts), offsets_of(counts)
    rows = off[-1] + behind
    x = rand((rows, K), 1.0, torch.bfloat16, seed + 1)
    x[off[-1]:] = math.nan
    G = -(-K // group)
    gen = torch.Generator().manual_seed(seed + 2)
    q = torch.randint(-8, 8, (E, K, N), dtype=torch.int8, generator=gen)
    s = (torch.rand((E, G, N), generator=gen) * 0.01 + 0.002)
    b = rand((E, N), 0.5, torch.bfloat16, seed + 3)
    g = M.GroupedConfig(rows=rows, E=E, K=K, N=N)
    return g, off, x, q, s, b, M.Workspace(None, nbytes=M.moe_grouped_workspace_size(g))


def weight(q, s, group, e):
    return q[e].double() * torch.repeat_interleave(s[e].double(), group, dim=0)[:q.shape[1]]


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"E{len(s[0])}_R{sum(s[0])}_K{s[2]}_N{s[3]}")
def test_product(shape, group, with_bias):
    g, off, x, q, s, b, ws = case(shape, group)
    y = torch.full((g.rows, g.N), 5.0, dtype=torch.bfloat16, device="cuda")
    o = torch.tensor(off, dtype=torch.int32).cuda()
    M.moe_grouped_gemm_int4(g, x.cuda(), M.moe_pack_int4(q.cuda()), s.cuda(), o, y, ws, group,
                            bias=b.cuda() if with_bias else None)
    assert M.moe_check_device_status(ws)[0] == M.MOE_OK
    for e in range(g.E):
        xe, we = x[off[e]:off[e + 1]].double(), weight(q, s, group, e)
        be = b[e].double() if with_bias else torch.zeros(g.N, dtype=torch.float64)
        ref, mag = xe @ we + be, xe.abs() @ we.abs() + be.abs()
        err = (y[off[e]:off[e + 1]].double().cpu() - ref).abs()
        tol = (g.K / 8 + 64) * U * mag + HALF * ref.abs() + 1e-37
        assert (err <= tol).all(), float((err / tol).max())
    assert (y[off[-1]:] == 5.0).all()


def test_values_stay_in_their_row_and_expert():
    """NaN in a row, in an expert's scales and behind K reach nothing else."""
    g, off, x, q, s, b, ws = case(([3, 5, 20], 0, 136, 72), 64)
    x[off[1]] = math.nan
    s[0] = math.inf
    codes = M.moe_pack_int4(q.cuda())
    codes[:, :, 64 + 16 * 1:] = 255   # block 1 holds k = 128..135 in its first words; the rest stands for no k
    keep = M.moe_pack_int4(q.cuda())
    for k in range(128, 136):
        word = 0
        codes[:, :, 64 + word * 4:64 + word * 4 + 4] = keep[:, :, 64 + word * 4:64 + word * 4 + 4]
    y = torch.empty((g.rows, g.N), dtype=torch.bfloat16, device="cuda")
    M.moe_grouped_gemm_int4(g, x.cuda(), codes, s.cuda(), torch.tensor(off, dtype=torch.int32).cuda(), y, ws, 64)
    for e in (1, 2):
        for r in range(off[e], off[e + 1]):
            if r == off[1]:
                assert torch.isnan(y[r]).all()
                continue
            we = weight(q, s, 64, e)
            ref, mag = x[r].double() @ we, x[r].double().abs() @ we.abs()
            assert ((y[r].double().cpu() - ref).abs() <= (g.K / 8 + 64) * U * mag + HALF * ref.abs() + 1e-37).all()


def test_bad_offsets_are_refused_on_the_device():
    g, off, x, q, s, b, ws = case(([30, 30, 30], 0, 64, 72), 32)
    y = torch.full((g.rows, g.N), 5.0, dtype=torch.bfloat16, device="cuda")
    M.moe_grouped_gemm_int4(g, x.cuda(), M.moe_pack_int4(q.cuda()), s.cuda(),
                            torch.tensor([0, 30, 20, 91], dtype=torch.int32).cuda(), y, ws, 32)
    assert M.moe_check_device_status(ws) == (M.MOE_ERR_RANGE, 0x501)
    assert (y[30:] == 5.0).all() and not (y[:30] == 5.0).all()


@pytest.mark.parametrize("act", ["swiglu", "gelu_bias"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("counts,d,ffn", [([2, 0, 1, 5], 128, 192), ([1] * 16, 320, 64), ([30, 50], 192, 320)])
def test_expert_ffn(act, group, counts, d, ffn):
    E, off = len(counts), offsets_of(counts)
    T = off[-1]
    cfg = M.MoEConfig(T=T, d=d, ffn=ffn, E=E, k=1, act=act, capacity_factor=0.0, weights=f"int4_g{group}")
    names = (("w_gate", d, ffn), ("w_up", d, ffn), ("w_down", ffn, d)) if act == "swiglu" else \
        (("w1", d, ffn), ("w2", ffn, d))
    w = {n: rand((E, K, N), 0.1, torch.bfloat16, i) for i, (n, K, N) in enumerate(names)}
    if act == "gelu_bias":
        w["b1"], w["b2"] = rand((E, ffn), 0.1, torch.bfloat16, 8), rand((E, d), 0.1, torch.bfloat16, 9)
    wd = M.quantize_expert_weights(cfg, {n: v.cuda() for n, v in w.items()})
    x = rand((T, d), 1.0, torch.bfloat16, 7)
    ws = M.Workspace(cfg)
    y = torch.empty((T, d), dtype=torch.bfloat16, device="cuda")
    M.moe_expert_ffn(cfg, wd, x.cuda(), torch.tensor(off, dtype=torch.int32).cuda(), y, ws)
    assert M.moe_check_device_status(ws)[0] == M.MOE_OK

    def deq(n, e):   # w / scale rounded, times scale: what moe_quantize_int4 states (checked above)
        s = wd[n + "_scale"][e].cpu()
        sk = torch.repeat_interleave(s, group, dim=0)[:w[n].shape[1]]
        return torch.where(sk > 0, torch.clamp(torch.round(w[n][e].float() / sk), -7, 7), 0.0).double() * sk.double()

    for e in range(E):
        xe = x[off[e]:off[e + 1]].double()
        if act == "swiglu":
            wg, wu, wo = deq("w_gate", e), deq("w_up", e), deq("w_down", e)
            g, u = xe @ wg, xe @ wu
            ga, ua = xe.abs() @ wg.abs(), xe.abs() @ wu.abs()
            s = torch.sigmoid(g)
            h = g * s * u
            amp = 1.1 * ga * u.abs() + (g * s).abs() * ua + h.abs()
            bias = torch.zeros(d, dtype=torch.float64)
        else:
            w1, wo, bias = deq("w1", e), deq("w2", e), w["b2"][e].double()
            p = xe @ w1 + w["b1"][e].double()
            h = p * 0.5 * (1 + torch.erf(p / math.sqrt(2)))
            amp = 1.13 * (xe.abs() @ w1.abs() + w["b1"][e].double().abs()) + h.abs()
        ref = h @ wo + bias
        c = 2 * (max(d, ffn) / 8 + 64) * U
        tol = c * (amp @ wo.abs() + bias.abs()) + 1.01 * HALF * (h.abs() @ wo.abs()) + 1.01 * HALF * ref.abs()
        err = (y[off[e]:off[e + 1]].double().cpu() - ref).abs()
        assert (err <= tol).all(), float((err / tol).max())


def test_layer_forward_captured_on_another_stream_and_again():
    """The whole layer on 4-bit experts: the same bits eagerly, on a side stream and replayed, and equal to
    its own stages called one by one."""
    T, d, ffn, E, k = 24, 128, 192, 8, 2
    cfg = M.MoEConfig(T=T, d=d, ffn=ffn, E=E, k=k, capacity_factor=0.0, weights="int4_g64")
    w = {"w_router": rand((d, E), 0.3, torch.bfloat16, 1), "w_gate": rand((E, d, ffn), 0.1, torch.bfloat16, 2),
         "w_up": rand((E, d, ffn), 0.1, torch.bfloat16, 3), "w_down": rand((E, ffn, d), 0.1, torch.bfloat16, 4)}
    wd = M.quantize_expert_weights(cfg, {n: v.cuda() for n, v in w.items()})
    wd["w_router"] = w["w_router"].cuda()
    x = rand((T, d), 1.0, torch.bfloat16, 5).cuda()
    layer = M.MoELayer(cfg, wd)
    first = layer.forward(x)["out"].clone()
    layer.check()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.outputs["out"].zero_()
        again = layer.forward(x)["out"].clone()
    torch.cuda.synchronize()
    assert torch.equal(first, again)
    layer.capture(x)
    layer.outputs["out"].zero_()
    out = layer.replay()
    torch.cuda.synchronize()
    assert torch.equal(out["out"], first)
    rows = M.moe_max_rows(cfg)
    x_perm, y_perm = (torch.zeros((rows, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    x_perm.copy_(x[out["src_assign"].long() // k])
    M.moe_expert_ffn(cfg, wd, x_perm, out["offsets"], y_perm, layer.ws)
    o2 = torch.zeros_like(x)
    M.moe_combine(cfg, y_perm, out["slot"], out["topk_w"], o2)
    assert torch.equal(o2, first)


def test_expert_parallel_ranks_equal_the_whole_batch():
    """Two emulated expert-parallel ranks on 4-bit experts: bit for bit one forward over the batch (tiles of 16
    tokens or 64 sum each output in the same order)."""
    import workloads as W
    from test_gpu_ep import run_emulated
    from gpu_common import to_dev, weights_dev
    wl = W.Workload("ep_int4", T=190, d=128, ffn=192, E=4, k=2, act="swiglu", dtype="bf16", capacity_factor=1.0, seed=61,
                    weights="int4_g32")
    inp = W.make_inputs(wl)
    cfg = M.MoEConfig.of(wl)
    wd = M.quantize_expert_weights(cfg, weights_dev(wl, inp))
    x = to_dev(inp["x"])
    whole = M.MoELayer(cfg, wd).forward(x)["out"]
    ranks = run_emulated(wl, [0, 77, 190], wd, x)
    for s in ranks:
        assert M.moe_check_device_status(s["ws"])[0] == M.MOE_OK
    assert torch.equal(torch.cat([s["out"]["out"] for s in ranks]), whole)


def test_pipeline_on_4_bit_experts():
    T, d, ffn, E, k = 16, 64, 128, 4, 2
    cfg = M.MoEConfig(T=T, d=d, ffn=ffn, E=E, k=k, capacity_factor=0.0, weights="int4_g128")
    w = {"w_router": rand((d, E), 0.3, torch.bfloat16, 1), "w_gate": rand((E, d, ffn), 0.1, torch.bfloat16, 2),
         "w_up": rand((E, d, ffn), 0.1, torch.bfloat16, 3), "w_down": rand((E, ffn, d), 0.1, torch.bfloat16, 4)}
    wd = M.quantize_expert_weights(cfg, {n: v.cuda() for n, v in w.items()})
    layer = M.MoELayer(cfg, wd)
    with M.Pipeline(cfg, wd) as pipe:
        xs = [rand((T, d), 1.0, torch.bfloat16, 10 + i).pin_memory() for i in range(3)]
        outs = [torch.empty((T, d), dtype=torch.bfloat16).pin_memory() for _ in xs]
        aux = [torch.empty(1).pin_memory() for _ in xs]
        for x, o, a in zip(xs, outs, aux):
            pipe.submit(x, o, a)
        pipe.wait()
        pipe.check()
    for x, o in zip(xs, outs):
        assert torch.equal(layer.forward(x.cuda())["out"].cpu(), o)


@pytest.mark.parametrize("rows", [1, 15, 16, 17, 33, 64, 65, 129, 400])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_tile_borders(rows, group):
    """One expert's rows around the tiles' borders, K and N around the blocks'; the same bits from one call of all
    rows and from calls of each part of them."""
    for K, N in ((120, 120), (128, 128), (136, 136), (256, 264), (392, 24)):
        g, off, x, q, s, b, ws = case(([rows, 2], 0, K, N), group, seed=rows + K)
        codes, sd, o = M.moe_pack_int4(q.cuda()), s.cuda(), torch.tensor(off, dtype=torch.int32).cuda()
        y = torch.zeros((g.rows, N), dtype=torch.bfloat16, device="cuda")
        xd = x.cuda()
        M.moe_grouped_gemm_int4(g, xd, codes, sd, o, y, ws, group)
        assert M.moe_check_device_status(ws)[0] == M.MOE_OK
        for e in range(2):
            xe, we = x[off[e]:off[e + 1]].double(), weight(q, s, group, e)
            ref, mag = xe @ we, xe.abs() @ we.abs()
            err = (y[off[e]:off[e + 1]].double().cpu() - ref).abs()
            tol = (K / 8 + 64) * U * mag + HALF * ref.abs() + 1e-37
            assert (err <= tol).all(), (K, N, float((err / tol).max()))
        one = M.GroupedConfig(rows=1, E=2, K=K, N=N)
        y1 = torch.zeros((1, N), dtype=torch.bfloat16, device="cuda")
        M.moe_grouped_gemm_int4(one, xd[rows - 1:rows].contiguous(), codes, sd, torch.tensor([0, 1, 1], dtype=torch.int32).cuda(),
                                y1, ws, group)
        assert torch.equal(y1[0], y[rows - 1])


def test_many_units_and_empty_experts():
    """Long streams over many tiles per CTA, with experts that hold no row between others: the rings' parities."""
    for group in (32, 64, 128):
        for counts, K, N in (([0, 3] * 32, 2176, 1160), ([70, 0, 130], 2304, 2048)):
            g, off, x, q, s, b, ws = case((counts, 0, K, N), group, seed=3)
            y = torch.zeros((g.rows, N), dtype=torch.bfloat16, device="cuda")
            xd, qd, sd = x.cuda(), q.cuda(), s.cuda()
            for _ in range(3):
                M.moe_grouped_gemm_int4(g, xd, M.moe_pack_int4(qd), sd, torch.tensor(off, dtype=torch.int32).cuda(), y, ws,
                                        group)
            assert M.moe_check_device_status(ws)[0] == M.MOE_OK
            for e in range(g.E):
                if off[e] == off[e + 1]:
                    continue
                we = (qd[e].double() * torch.repeat_interleave(sd[e].double(), group, dim=0)[:K])
                xe = xd[off[e]:off[e + 1]].double()
                ref, mag = xe @ we, xe.abs() @ we.abs()
                err = (y[off[e]:off[e + 1]].double() - ref).abs()
                assert (err <= (K / 8 + 64) * U * mag + HALF * ref.abs() + 1e-37).all()


WIDE_ROWS = [31, 32, 33, 47, 48, 49, 63, 64, 65, 95, 97, 129]


@pytest.mark.parametrize("rows", WIDE_ROWS)
@pytest.mark.parametrize("group", [32, 64, 128])
def test_wide_tile_borders(rows, group):
    """Columns enough for the tiles of 32 and 64 tokens: rows around the borders of the tiles and of the tokens that
    four of their warps take, a ragged last tile of columns, NaN rows behind."""
    test_product(([rows, 2], 1, 200, 6152), group, True)


@pytest.mark.parametrize("act", ["swiglu", "gelu_bias"])
@pytest.mark.parametrize("rows", [31, 33, 48, 49, 64, 65])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_expert_ffn_wide_tile_borders(act, rows, group):
    test_expert_ffn(act, group, [rows, 2], 64, 6144)
