"""Grouped products, their gradients and the FFN's backward pass where the arithmetic or the offsets are extreme,
against float64.  Tolerances as in test_gpu_grouped: (n + 8) u A for fp32 chains, (n / 4 + 64) u A for the tensor
cores' sums (u = 2^-24, A = the sum over the absolute values of the terms), half a step of the output's type."""
from __future__ import annotations

import math

import pytest
import torch

import mixture_experts_layer_37_b200 as M
from test_gpu_grouped import DT, HALF, U, check, rand
from test_gpu_int4 import pack_plain, weight

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ offsets that give two experts the same rows
OVERLAPS = [
    [0, 900, 0, 900],                                  # the third expert has the first one's rows again
    [0, 400, 200, 600, 600, 900],                      # and a part of them
    [300, 310, 0, 305, 305, 900],                      # and all of them, from further ahead
    [0, 500] + [500] * 36 + [100, 300, 900],           # an expert of the other half of the warp's lanes
]


def accepted(off, rows):
    """[(first row, rows)] by the stated rule, one expert after the other."""
    out, end = [], 0
    for a, b in zip(off, off[1:]):
        good = 0 <= a <= b <= rows
        out.append((a, b - a) if good and (a >= end or a == b) else (0, 0))
        end = max(end, b if good else 0)
    return out


@pytest.mark.parametrize("off", OVERLAPS, ids=lambda o: f"E{len(o) - 1}_{o[0]}_{o[2]}")
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_claimed_twice_belong_to_the_first(dtype, off):
    E, rows, K, N, dt = len(off) - 1, 900, 72, 136, DT[dtype]
    g = M.GroupedConfig(rows=rows, E=E, K=K, N=N, dtype=dtype)
    ws = M.Workspace(None, nbytes=M.moe_grouped_workspace_size(g))
    x, dy, w = rand((rows, K), 1.0, dt, 1), rand((rows, N), 0.1, dt, 2), rand((E, K, N), 0.05, dt, 3)
    xd, dyd, wd, o = x.cuda(), dy.cuda(), w.cuda(), torch.tensor(off, dtype=torch.int32).cuda()
    y = torch.full((rows, N), 5.0, dtype=dt, device="cuda")
    dx = torch.full((rows, K), 5.0, dtype=dt, device="cuda")
    dw, db = torch.full((E, K, N), 5.0, device="cuda"), torch.full((E, N), 5.0, device="cuda")
    for f in (lambda: M.moe_grouped_gemm(g, xd, wd, o, y, ws), lambda: M.moe_grouped_gemm_grad_x(g, dyd, wd, o, dx, ws),
              lambda: M.moe_grouped_gemm_grad_w(g, xd, dyd, o, dw, ws, db=db)):
        f()
        assert M.moe_check_device_status(ws) == (M.MOE_ERR_RANGE, 0x501)
    written = torch.zeros(rows, dtype=torch.bool)
    for e, (a, n) in enumerate(accepted(off, rows)):
        assert not written[a:a + n].any()
        written[a:a + n] = True
        xe, de, we = x[a:a + n].double(), dy[a:a + n].double(), w[e].double()
        check(y[a:a + n], xe @ we, xe.abs() @ we.abs(), K, dt)
        check(dx[a:a + n], de @ we.t(), de.abs() @ we.abs().t(), N, dt)
        check(dw[e], xe.t() @ de, xe.abs().t() @ de.abs(), n, dt)
        check(db[e], de.sum(0), de.abs().sum(0), n, torch.float32)
    assert (y.cpu()[~written] == 5.0).all() and (dx.cpu()[~written] == 5.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_claimed_twice_with_rows_in_parts(dtype):
    """The same where each expert's rows are summed in parts."""
    rows, K, N, dt = 9000, 40, 64, DT[dtype]
    off = [0, 9000, 2000, 9000]
    g = M.GroupedConfig(rows=rows, E=3, K=K, N=N, dtype=dtype)
    n = M.moe_grouped_workspace_size(g)
    assert n > 64 * 1024
    ws = M.Workspace(None, nbytes=n)
    x, dy = rand((rows, K), 1.0, dt, 1), rand((rows, N), 0.1, dt, 2)
    dw, db = torch.empty((3, K, N), device="cuda"), torch.empty((3, N), device="cuda")
    M.moe_grouped_gemm_grad_w(g, x.cuda(), dy.cuda(), torch.tensor(off, dtype=torch.int32).cuda(), dw, ws, db=db)
    assert M.moe_check_device_status(ws) == (M.MOE_ERR_RANGE, 0x501)
    x, dy = x.double(), dy.double()
    check(dw[0], x.t() @ dy, x.abs().t() @ dy.abs(), rows, dt)
    check(db[0], dy.sum(0), dy.abs().sum(0), rows, torch.float32)
    assert (dw[1:] == 0).all() and (db[1:] == 0).all()


@pytest.mark.parametrize("off", OVERLAPS, ids=lambda o: f"E{len(o) - 1}_{o[0]}_{o[2]}")
def test_int4_rows_claimed_twice_belong_to_the_first(off):
    E, rows, K, N, group = len(off) - 1, 900, 136, 72, 64
    g = M.GroupedConfig(rows=rows, E=E, K=K, N=N)
    ws = M.Workspace(None, nbytes=M.moe_grouped_workspace_size(g))
    gen = torch.Generator().manual_seed(4)
    q = torch.randint(-8, 8, (E, K, N), dtype=torch.int8, generator=gen)
    s = torch.rand((E, -(-K // group), N), generator=gen) * 0.01 + 0.002
    x = rand((rows, K), 1.0, torch.bfloat16, 5)
    y = torch.full((rows, N), 5.0, dtype=torch.bfloat16, device="cuda")
    codes = torch.from_numpy(pack_plain(q.numpy())).cuda()
    M.moe_grouped_gemm_int4(g, x.cuda(), codes, s.cuda(), torch.tensor(off, dtype=torch.int32).cuda(), y, ws, group)
    assert M.moe_check_device_status(ws) == (M.MOE_ERR_RANGE, 0x501)
    written = torch.zeros(rows, dtype=torch.bool)
    for e, (a, n) in enumerate(accepted(off, rows)):
        written[a:a + n] = True
        we, xe = weight(q, s, group, e), x[a:a + n].double()
        ref, mag = xe @ we, xe.abs() @ we.abs()
        tol = (K / 8 + 64) * U * mag + HALF[torch.bfloat16] * ref.abs() + 1e-37
        assert ((y[a:a + n].double().cpu() - ref).abs() <= tol).all()
    assert (y.cpu()[~written] == 5.0).all()


# ------------------------------------------------------------------ what is there is added once
@pytest.mark.parametrize("counts,K,N", [
    ([16384], 2048, 2048),                  # 32 runs of rows for each accumulator, whole tiles
    ([5000, 0, 1, 3111], 1304, 1320),       # ragged tiles of rows and of columns, an expert without rows
    ([700, 1500], 2048, 1064),
    ([512, 513, 40], 1672, 1688),
], ids=lambda v: str(v) if isinstance(v, list) else None)
def test_accumulating_adds_the_finished_sum_once(counts, K, N):
    """fp32 gradients of bf16 rows, not in parts: with `accumulate` exactly what is there plus the sum that the call
    without it gives, in one rounding, however much larger what is there may be."""
    off = [0]
    for n in counts:
        off.append(off[-1] + n)
    g = M.GroupedConfig(rows=off[-1] + 3, E=len(counts), K=K, N=N)
    nb = M.moe_grouped_workspace_size(g)
    ws = M.Workspace(None, nbytes=nb)
    gen = torch.Generator(device="cuda").manual_seed(K)
    x = torch.randn((g.rows, K), generator=gen, device="cuda").bfloat16()
    dy = torch.randn((g.rows, N), generator=gen, device="cuda").bfloat16()
    o = torch.tensor(off, dtype=torch.int32).cuda()
    total = torch.empty((g.E, K, N), device="cuda")
    M.moe_grouped_gemm_grad_w(g, x, dy, o, total, ws)
    for scale in (1e6, 1.0, 0.0):
        old = torch.randn((g.E, K, N), generator=gen, device="cuda") * scale
        dw = old.clone()
        M.moe_grouped_gemm_grad_w(g, x, dy, o, dw, ws, accumulate=True)
        assert M.moe_check_device_status(ws)[0] == M.MOE_OK
        assert torch.equal(dw, old + total)


# ------------------------------------------------------------------ GELU far below zero
def tail_case(ffn, dtype):
    """Pre-activations from -9 to 1 (exact in bf16), and in float64 Phi, phi, h = p Phi(p) and h' = Phi + p phi of them."""
    p = torch.linspace(-9, 1, ffn).to(dtype)
    q = p.double()
    cdf = 0.5 * torch.special.erfc(-q / math.sqrt(2))
    pdf = torch.exp(-q * q / 2) / math.sqrt(2 * math.pi)
    return p, q, cdf, pdf


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gelu_gradients_in_the_tail(dtype):
    """h and dp where Phi is small keep their own relative precision: one token, one row of dy, so that each gradient
    is a single term.  Phi from an argument rounded once has p^2 u (and 1.6 p^2 u for the scaled argument), its four
    units in the last place 8 u; the exponential of p^2 / 2 as much (bf16: its fast form about 100 u more); the
    products 3 u.  bf16 rounds h and dp to its type once."""
    d, ffn, dt = 64, 128, DT[dtype]
    cfg = M.MoEConfig(T=1, d=d, ffn=ffn, E=1, k=1, dtype=dtype, act="gelu_bias", capacity_factor=0.0)
    p, q, cdf, pdf = tail_case(ffn, dt)
    w1, w2 = torch.zeros(1, d, ffn, dtype=dt), rand((1, ffn, d), 1.0, dt, 3)
    x, dy = torch.zeros(1, d, dtype=dt), torch.zeros(1, d, dtype=dt)
    x[0, 5], dy[0, 9] = 1.5, 0.75
    w = {"w1": w1, "b1": p[None], "w2": w2, "b2": torch.zeros(1, d, dtype=dt)}
    grads = {n: torch.empty(v.shape, device="cuda") for n, v in w.items()}
    ws = M.Workspace(None, nbytes=M.moe_expert_ffn_backward_workspace_size(cfg))
    M.moe_expert_ffn_backward(cfg, {n: v.cuda() for n, v in w.items()}, x.cuda(),
                              torch.tensor([0, 1], dtype=torch.int32).cuda(), dy.cuda(), grads, ws)
    assert M.moe_check_device_status(ws)[0] == M.MOE_OK
    step = 1.01 * HALF[dt] if dtype == "bf16" else 0.0
    rel = (3 * q * q + 20 + (100 if dtype == "bf16" else 0)) * U
    h, dh = q * cdf, 0.75 * w2[0, :, 9].double()
    dp, dp_mag = dh * (cdf + q * pdf), dh.abs() * (cdf + (q * pdf).abs())
    got = {n: v[0].double().cpu() for n, v in grads.items()}
    for name, g, ref, mag in (("h", got["w2"][:, 9], 0.75 * h, (0.75 * h).abs()), ("dp", got["b1"], dp, dp_mag),
                              ("dw1", got["w1"][5], 1.5 * dp, 1.5 * dp_mag)):
        err, tol = (g - ref).abs(), rel * mag + step * ref.abs()
        assert (err <= tol).all(), (name, float((err / tol).max()))


@pytest.mark.parametrize("group", [32, 64, 128])
def test_int4_gelu_in_the_tail(group):
    """The 4-bit FFN's h likewise: codes of 0 before the activation, an identity behind it."""
    d = ffn = 128
    cfg = M.MoEConfig(T=2, d=d, ffn=ffn, E=1, k=1, act="gelu_bias", capacity_factor=0.0, weights=f"int4_g{group}")
    p, q, cdf, _ = tail_case(ffn, torch.bfloat16)
    eye = torch.eye(ffn, dtype=torch.int8)[None].cuda()
    ones = torch.ones(1, -(-d // group), ffn, device="cuda")
    w = {"w1": M.moe_pack_int4(torch.zeros_like(eye)), "w1_scale": ones, "b1": p[None].cuda(),
         "w2": M.moe_pack_int4(eye), "w2_scale": ones, "b2": torch.zeros(1, d, dtype=torch.bfloat16, device="cuda")}
    ws, y = M.Workspace(cfg), torch.empty(2, d, dtype=torch.bfloat16, device="cuda")
    M.moe_expert_ffn(cfg, w, rand((2, d), 1.0, torch.bfloat16, 1).cuda(), torch.tensor([0, 2], dtype=torch.int32).cuda(), y, ws)
    assert M.moe_check_device_status(ws)[0] == M.MOE_OK
    h = q * cdf
    tol = ((3 * q * q + 20) * U + 1.01 * HALF[torch.bfloat16]) * h.abs()
    for r in (0, 1):
        err = (y[r].double().cpu() - h).abs()
        assert (err <= tol).all(), float((err / tol).max())


# ------------------------------------------------------------------ b1's gradient
@pytest.mark.parametrize("counts,behind", [
    ([1], 0), ([5], 3), ([31, 1, 33], 2), ([0, 64, 2, 0, 127, 128, 129], 9), ([300, 255, 257], 0), ([3] * 40, 1),
    ([2100, 0, 3001], 5),                   # the experts' rows in parts
], ids=lambda v: f"E{len(v)}_R{sum(v)}" if isinstance(v, list) else None)
@pytest.mark.parametrize("accumulate", [False, True])
def test_b1_gradient_sums_unrounded_terms(counts, behind, accumulate):
    """bf16 GELU: dp = dh gelu'(p) is rounded to bf16 for the products, but not where b1's gradient sums it.  With x = 0
    p is b1, and with one column of dy dh is one product: a term is off by what test_gelu_gradients_in_the_tail states,
    the fp32 sum of n terms by n u of their absolute values at most."""
    d, ffn, E, dt = 64, 192, len(counts), torch.bfloat16
    off = [0]
    for n in counts:
        off.append(off[-1] + n)
    T = off[-1] + behind
    cfg = M.MoEConfig(T=T, d=d, ffn=ffn, E=E, k=1, act="gelu_bias", capacity_factor=0.0)
    p, q, cdf, pdf = tail_case(ffn, dt)
    w2 = rand((E, ffn, d), 1.0, dt, 3)
    x, dy = torch.zeros(T, d, dtype=dt), torch.zeros(T, d, dtype=dt)
    dy[:, 9] = rand((T,), 1.0, dt, 4)
    x[off[-1]:], dy[off[-1]:] = math.nan, math.nan
    w = {"w1": torch.zeros(E, d, ffn, dtype=dt), "b1": p.expand(E, ffn).contiguous(), "w2": w2,
         "b2": torch.zeros(E, d, dtype=dt)}
    base = rand((E, ffn), 0.5, torch.float32, 5)
    grads = {"b1": base.cuda() if accumulate else torch.full((E, ffn), math.nan, device="cuda")}
    ws = M.Workspace(None, nbytes=M.moe_expert_ffn_backward_workspace_size(cfg))
    wd = {n: v.cuda() for n, v in w.items()}
    M.moe_expert_ffn_backward(cfg, wd, x.cuda(), torch.tensor(off, dtype=torch.int32).cuda(), dy.cuda(), grads, ws,
                              accumulate=accumulate)
    assert M.moe_check_device_status(ws)[0] == M.MOE_OK
    got, rel = grads["b1"].double().cpu(), (3 * q * q + 120) * U
    for e, n in enumerate(counts):
        dh = dy[off[e]:off[e + 1], 9:10].double() * w2[e, :, 9].double()[None]
        b0 = base[e].double() if accumulate else torch.zeros(ffn, dtype=torch.float64)
        ref, mag = (dh * (cdf + q * pdf)).sum(0) + b0, (dh.abs() * (cdf + (q * pdf).abs())).sum(0)
        err, tol = (got[e] - ref).abs(), (rel + (n + 2) * U) * mag + 2 * U * (ref.abs() + b0.abs()) + 1e-37
        assert (err <= tol).all(), (e, float((err / tol).max()))


def test_b1_gradient_with_offsets_that_are_refused():
    """The slabs of the experts that are taken stay apart whatever the others' offsets say."""
    d, ffn, rows, off = 64, 128, 900, [300, 333, 0, 320, 320, 900]
    E, dt = len(off) - 1, torch.bfloat16
    cfg = M.MoEConfig(T=rows, d=d, ffn=ffn, E=E, k=1, act="gelu_bias", capacity_factor=0.0)
    w = {"w1": rand((E, d, ffn), 0.1, dt, 1), "b1": rand((E, ffn), 0.1, dt, 2), "w2": rand((E, ffn, d), 0.1, dt, 3),
         "b2": rand((E, d), 0.1, dt, 4)}
    x, dy = rand((rows, d), 1.0, dt, 5).cuda(), rand((rows, d), 0.5, dt, 6).cuda()
    ws = M.Workspace(None, nbytes=M.moe_expert_ffn_backward_workspace_size(cfg))
    wd = {n: v.cuda() for n, v in w.items()}

    def grads(o):
        g = {"b1": torch.empty(E, ffn, device="cuda"), "w1": torch.empty(E, d, ffn, device="cuda")}
        M.moe_expert_ffn_backward(cfg, wd, x, torch.tensor(o, dtype=torch.int32).cuda(), dy, g, ws)
        return g, M.moe_check_device_status(ws)[0]

    bad, status = grads(off)
    assert status == M.MOE_ERR_RANGE
    taken = accepted(off, rows)
    for e, (a, n) in enumerate(taken):              # each expert by itself, the others empty
        alone, status = grads([a] * (e + 1) + [a + n] * (E - e))
        assert status == M.MOE_OK
        for name in alone:
            assert torch.equal(alone[name][e], bad[name][e]), (e, name)
