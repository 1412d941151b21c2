"""Grouped products over sorted rows, their gradients and the expert FFN's
backward pass, against float64.

Tolerances, per output element, from the arithmetic (u = 2^-24, A = the same
sum over the absolute values of its terms, n its length):
  * fp32 sums of exact products: |err| <= (n + 8) u A for FMA chains; the tensor
    cores add K=16 products per step and may truncate (one ulp, 2 u) where fp32
    rounds (u), so their sums get (n / 4 + 64) u A;
  * an output rounded to bf16 adds half a step, 2^-8 of the value;
  * the backward pass rounds the inner gradients and activations to bf16 once:
    2^-8 of each term, 2^-8 A over the sum; __expf in the sigmoid adds about
    2^-20 relative and is covered by doubling u's share.
"""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import mixture_experts_layer_37_b200 as M

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def offsets_of(counts):
    off = [0]
    for n in counts:
        off.append(off[-1] + n)
    return off


def rand(shape, std, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g, dtype=torch.float64) * std).to(dtype)


def sum_tol(dtype, n):
    return (n + 8) * U if dtype == torch.float32 else (n / 4 + 64) * U


def check(got, ref, absum, n, in_dtype, extra=0.0):
    """got [..] against float64 ref with the sums' absolute values absum."""
    got64 = got.double().cpu()
    tol = (sum_tol(in_dtype, n) + extra) * absum + HALF[got.dtype] * ref.abs() + 1e-37
    bad = ~((got64 - ref).abs() <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}: worst {float(((got64 - ref).abs() / tol).max())} of its tolerance"


# (counts per expert, rows behind the last one, K, N)
SHAPES = [
    ([3], 0, 64, 64),
    ([1], 0, 8, 8),
    ([130, 0, 1, 257], 5, 200, 328),
    ([0, 0, 0], 4, 128, 64),
    ([0, 64, 65, 63, 128, 0], 1, 72, 264),
    ([16, 15, 17, 33, 1, 2, 300], 9, 136, 512),
    ([2] * 64, 0, 256, 128),
    ([0] * 31 + [500] + [0] * 20 + [7] + [0] * 11, 3, 328, 200),
    ([640, 1000], 0, 512, 1024),
    # long sums of few outputs: the experts' rows in parts
    ([5000], 3, 72, 136),
    ([0, 9001, 100, 30], 2, 40, 64),
    ([2100, 2049, 2200], 0, 264, 72),
]


def case(shape, dtype, seed=0):
    counts, behind, K, N = shape
    dt = DT[dtype]
    if dtype == "f32":
        K, N = K + 4, N + 4 * (N > 8)   # multiples of 4 that are none of 8
    E, off = len(counts), offsets_of(counts)
    rows = off[-1] + behind
    x, dy = rand((rows, K), 1.0, dt, seed + 1), rand((rows, N), 0.1, dt, seed + 2)
    x[off[-1]:] = math.nan      # whatever lies behind the last row is not read
    dy[off[-1]:] = math.inf
    w, b = rand((E, K, N), 0.05, dt, seed + 3), rand((E, N), 0.5, dt, seed + 4)
    g = M.GroupedConfig(rows=rows, E=E, K=K, N=N, dtype=dtype)
    ws = M.Workspace(None, nbytes=M.moe_grouped_workspace_size(g))
    return g, off, x, dy, w, b, torch.tensor(off, dtype=torch.int32).cuda(), ws


def ids(s):
    return f"E{len(s[0])}_R{sum(s[0])}_K{s[2]}_N{s[3]}"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=ids)
@pytest.mark.parametrize("with_bias", [False, True])
def test_forward(shape, dtype, with_bias):
    g, off, x, dy, w, b, o, ws = case(shape, dtype)
    y = torch.full((g.rows, g.N), 7.0, dtype=DT[dtype], device="cuda")
    M.moe_grouped_gemm(g, x.cuda(), w.cuda(), o, y, ws, bias=b.cuda() if with_bias else None)
    assert M.moe_check_device_status(ws)[0] == M.MOE_OK
    for e in range(g.E):
        xe, we = x[off[e]:off[e + 1]].double(), w[e].double()
        be = b[e].double() if with_bias else torch.zeros(g.N, dtype=torch.float64)
        check(y[off[e]:off[e + 1]], xe @ we + be, xe.abs() @ we.abs() + be.abs(), g.K, DT[dtype])
    assert (y[off[-1]:] == 7.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=ids)
def test_grad_x(shape, dtype):
    g, off, x, dy, w, b, o, ws = case(shape, dtype)
    dx = torch.full((g.rows, g.K), -3.0, dtype=DT[dtype], device="cuda")
    M.moe_grouped_gemm_grad_x(g, dy.cuda(), w.cuda(), o, dx, ws)
    assert M.moe_check_device_status(ws)[0] == M.MOE_OK
    for e in range(g.E):
        de, we = dy[off[e]:off[e + 1]].double(), w[e].double()
        check(dx[off[e]:off[e + 1]], de @ we.t(), de.abs() @ we.abs().t(), g.N, DT[dtype])
    assert (dx[off[-1]:] == -3.0).all()


@pytest.mark.parametrize("dtype,grad", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=ids)
def test_grad_w(shape, dtype, grad, accumulate):
    g, off, x, dy, w, b, o, ws = case(shape, dtype)
    dw0, db0 = rand((g.E, g.K, g.N), 0.3, DT[grad], 11), rand((g.E, g.N), 0.3, DT[grad], 12)
    if not accumulate:
        dw0[:], db0[:] = math.nan, math.nan   # overwritten, never read
    dw, db = dw0.cuda(), db0.cuda()
    M.moe_grouped_gemm_grad_w(g, x.cuda(), dy.cuda(), o, dw, ws, db=db, accumulate=accumulate)
    assert M.moe_check_device_status(ws)[0] == M.MOE_OK
    for e in range(g.E):
        xe, de = x[off[e]:off[e + 1]].double(), dy[off[e]:off[e + 1]].double()
        n = off[e + 1] - off[e]
        base, bbase = (dw0[e].double(), db0[e].double()) if accumulate else (torch.zeros_like(w[e]).double(),
                                                                            torch.zeros(g.N, dtype=torch.float64))
        check(dw[e], xe.t() @ de + base, xe.abs().t() @ de.abs() + base.abs(), n, DT[dtype])
        check(db[e], de.sum(0) + bbase, de.abs().sum(0) + bbase.abs(), n, torch.float32)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_values_stay_in_their_expert(dtype):
    """Infinities and NaN in one expert's rows or weights reach no other expert, in any form."""
    g, off, x, dy, w, b, o, ws = case(([33, 70, 5], 0, 72, 136), dtype)
    x[off[1]:off[2]] = math.nan
    dy[off[1]:off[2]] = math.inf
    w[1] = math.nan
    dt = DT[dtype]
    y = torch.empty((g.rows, g.N), dtype=dt, device="cuda")
    dx = torch.empty((g.rows, g.K), dtype=dt, device="cuda")
    dw = torch.empty((g.E, g.K, g.N), dtype=dt, device="cuda")
    db = torch.empty((g.E, g.N), dtype=dt, device="cuda")
    xd, dyd, wd = x.cuda(), dy.cuda(), w.cuda()
    M.moe_grouped_gemm(g, xd, wd, o, y, ws)
    M.moe_grouped_gemm_grad_x(g, dyd, wd, o, dx, ws)
    M.moe_grouped_gemm_grad_w(g, xd, dyd, o, dw, ws, db=db)
    for e in (0, 2):
        xe, de, we = x[off[e]:off[e + 1]].double(), dy[off[e]:off[e + 1]].double(), w[e].double()
        check(y[off[e]:off[e + 1]], xe @ we, xe.abs() @ we.abs(), g.K, dt)
        check(dx[off[e]:off[e + 1]], de @ we.t(), de.abs() @ we.abs().t(), g.N, dt)
        check(dw[e], xe.t() @ de, xe.abs().t() @ de.abs(), xe.shape[0], dt)
        check(db[e], de.sum(0), de.abs().sum(0), xe.shape[0], torch.float32)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [[0, 40, 30, 30], [0, -5, 30, 90], [0, 40, 60, 95]])
def test_bad_offsets_are_refused_on_the_device(dtype, bad):
    """An expert whose offsets decrease or leave the buffers is taken as empty; the others are right."""
    g, off, x, dy, w, b, _, ws = case(([30, 30, 30], 0, 64, 72), dtype)
    o = torch.tensor(bad, dtype=torch.int32).cuda()
    y = torch.full((g.rows, g.N), 5.0, dtype=DT[dtype], device="cuda")
    M.moe_grouped_gemm(g, x.cuda(), w.cuda(), o, y, ws)
    assert M.moe_check_device_status(ws) == (M.MOE_ERR_RANGE, 0x501)
    assert M.moe_check_device_status(ws)[0] == M.MOE_OK
    dw = torch.full((g.E, g.K, g.N), 5.0, dtype=DT[dtype], device="cuda")
    M.moe_grouped_gemm_grad_w(g, x.cuda(), dy.cuda(), o, dw, ws)
    assert M.moe_check_device_status(ws)[0] == M.MOE_ERR_RANGE
    written = torch.zeros(g.rows, dtype=torch.bool)
    for e in range(3):
        ok = 0 <= bad[e] <= bad[e + 1] <= g.rows
        lo, hi = (bad[e], bad[e + 1]) if ok else (0, 0)
        written[lo:hi] = True
        xe, de, we = x[lo:hi].double(), dy[lo:hi].double(), w[e].double()
        check(y[lo:hi], xe @ we, xe.abs() @ we.abs(), g.K, DT[dtype])
        check(dw[e], xe.t() @ de, xe.abs().t() @ de.abs(), hi - lo, DT[dtype])
    assert (y.cpu()[~written] == 5.0).all()


def test_no_rows_at_all():
    g = M.GroupedConfig(rows=0, E=3, K=64, N=128)
    ws = M.Workspace(None, nbytes=M.moe_grouped_workspace_size(g))
    e = lambda *s: torch.full(s, 2.0, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    o = torch.zeros(4, dtype=torch.int32, device="cuda")
    M.moe_grouped_gemm(g, e(0, 64), e(3, 64, 128), o, e(0, 128), ws)
    M.moe_grouped_gemm_grad_x(g, e(0, 128), e(3, 64, 128), o, e(0, 64), ws)
    dw, db = e(3, 64, 128), e(3, 128)
    M.moe_grouped_gemm_grad_w(g, e(0, 64), e(0, 128), o, dw, ws, db=db, accumulate=True)
    assert (dw == 2).all() and (db == 2).all()
    M.moe_grouped_gemm_grad_w(g, e(0, 64), e(0, 128), o, dw, ws, db=db)
    assert (dw == 0).all() and (db == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_same_bits_again_captured_and_on_another_stream(dtype):
    g, off, x, dy, w, b, o, ws = case(([130, 0, 1, 257], 5, 200, 328), dtype)
    dt = DT[dtype]
    xd, dyd, wd, bd = x.cuda(), dy.cuda(), w.cuda(), b.cuda()

    def outs():
        return (torch.zeros((g.rows, g.N), dtype=dt, device="cuda"), torch.zeros((g.rows, g.K), dtype=dt, device="cuda"),
                torch.zeros((g.E, g.K, g.N), dtype=torch.float32, device="cuda"),
                torch.zeros((g.E, g.N), dtype=torch.float32, device="cuda"))

    def step(t, space):
        M.moe_grouped_gemm(g, xd, wd, o, t[0], space, bias=bd)
        M.moe_grouped_gemm_grad_x(g, dyd, wd, o, t[1], space)
        M.moe_grouped_gemm_grad_w(g, xd, dyd, o, t[2], space, db=t[3], accumulate=True)

    first, again, other = outs(), outs(), outs()
    step(first, ws)
    step(again, ws)
    ws2 = M.Workspace(None, nbytes=ws.nbytes)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(other, ws2)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    caught = outs()
    with torch.cuda.graph(graph):
        step(caught, ws)
    for t in caught:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, *more in zip(first, again, other, caught):
        for m in more:
            assert torch.equal(a, m)
    graph.replay()   # accumulates once more
    torch.cuda.synchronize()
    assert torch.equal(caught[0], first[0]) and torch.allclose(caught[2], 2 * first[2], rtol=2 * U, atol=0)


def test_offsets_past_32_bits():
    """Element offsets beyond 2^31 in the weights and in their gradients."""
    E, K, N = 24, 8192, 11008
    assert E * K * N > 2 ** 31
    g = M.GroupedConfig(rows=50, E=E, K=K, N=N)
    ws = M.Workspace(None, nbytes=M.moe_grouped_workspace_size(g))
    counts = [0] * E
    counts[0], counts[22], counts[23] = 10, 25, 15
    off = offsets_of(counts)
    o = torch.tensor(off, dtype=torch.int32).cuda()
    x, dy = rand((50, K), 1.0, torch.bfloat16, 1).cuda(), rand((50, N), 0.1, torch.bfloat16, 2).cuda()
    w = torch.empty((E, K, N), dtype=torch.bfloat16, device="cuda").normal_(0, 0.05)
    y = torch.zeros((50, N), dtype=torch.bfloat16, device="cuda")
    dx = torch.zeros((50, K), dtype=torch.bfloat16, device="cuda")
    M.moe_grouped_gemm(g, x, w, o, y, ws)
    M.moe_grouped_gemm_grad_x(g, dy, w, o, dx, ws)
    for e in (0, 22, 23):
        s = slice(off[e], off[e + 1])
        xe, de, we = x[s].double(), dy[s].double(), w[e].double()
        check(y[s], (xe @ we).cpu(), (xe.abs() @ we.abs()).cpu(), K, torch.bfloat16)
        check(dx[s], (de @ we.t()).cpu(), (de.abs() @ we.abs().t()).cpu(), N, torch.bfloat16)
    M.moe_grouped_gemm_grad_w(g, x, dy, o, w, ws)   # into the same memory
    assert (w[1:22] == 0).all()
    for e in (0, 22, 23):
        s = slice(off[e], off[e + 1])
        xe, de = x[s].double(), dy[s].double()
        check(w[e], (xe.t() @ de).cpu(), (xe.abs().t() @ de.abs()).cpu(), counts[e], torch.bfloat16)


# ------------------------------------------------------------------ backward pass of the expert FFN
def ffn_case(act, dtype, counts, behind, d, ffn, seed=0):
    E, off = len(counts), offsets_of(counts)
    T = off[-1] + behind
    cfg = M.MoEConfig(T=T, d=d, ffn=ffn, E=E, k=1, dtype=dtype, act=act, capacity_factor=0.0)
    dt = DT[dtype]
    if act == "swiglu":
        w = {"w_gate": rand((E, d, ffn), 0.1, dt, seed + 1), "w_up": rand((E, d, ffn), 0.1, dt, seed + 2),
             "w_down": rand((E, ffn, d), 0.1, dt, seed + 3)}
    else:
        w = {"w1": rand((E, d, ffn), 0.1, dt, seed + 1), "b1": rand((E, ffn), 0.1, dt, seed + 2),
             "w2": rand((E, ffn, d), 0.1, dt, seed + 3), "b2": rand((E, d), 0.1, dt, seed + 4)}
    x, dy = rand((T, d), 1.0, dt, seed + 5), rand((T, d), 0.5, dt, seed + 6)
    x[off[-1]:] = math.nan
    dy[off[-1]:] = math.nan
    ws = M.Workspace(None, nbytes=M.moe_expert_ffn_backward_workspace_size(cfg))
    return cfg, off, w, x, dy, ws


def ffn_ref(act, w, x, dy, e):
    """Gradients of one expert in float64 by the product and chain rules, and what their
    terms come to in absolute value."""
    D = lambda n: w[n][e].double()  # noqa: E731
    if act == "swiglu":
        wg, wu, wd = D("w_gate"), D("w_up"), D("w_down")
        g, u = x @ wg, x @ wu
        s = torch.sigmoid(g)
        dh = dy @ wd.t()
        dha = dy.abs() @ wd.abs().t()
        dsilu = s * (1 + g * (1 - s))
        h, dg, du = g * s * u, dh * u * dsilu, dh * g * s
        ga, ua = x.abs() @ wg.abs(), x.abs() @ wu.abs()
        # |d silu'| <= 0.5 |dg|, |silu'| <= 1.1: what an error in g or u moves
        ha = (ga * 1.1 * u.abs() + (g * s).abs() * ua) + h.abs()
        dga = dha * u.abs() * 1.1 + dh.abs() * (ua * 1.1 + u.abs() * 0.5 * ga) + dg.abs()
        dua = dha * (g * s).abs() + dh.abs() * 1.1 * ga + du.abs()
        out = {"w_gate": x.t() @ dg, "w_up": x.t() @ du, "w_down": h.t() @ dy, "dx": dg @ wg.t() + du @ wu.t()}
        mag = {"w_gate": x.abs().t() @ dg.abs(), "w_up": x.abs().t() @ du.abs(), "w_down": h.abs().t() @ dy.abs(),
               "dx": dg.abs() @ wg.abs().t() + du.abs() @ wu.abs().t()}
        amp = {"w_gate": x.abs().t() @ dga, "w_up": x.abs().t() @ dua, "w_down": ha.t() @ dy.abs(),
               "dx": dga @ wg.abs().t() + dua @ wu.abs().t()}
    else:
        w1, b1, w2 = D("w1"), D("b1"), D("w2")
        p = x @ w1 + b1
        pa = x.abs() @ w1.abs() + b1.abs()
        cdf = 0.5 * (1 + torch.erf(p / math.sqrt(2)))
        pdf = torch.exp(-p * p / 2) / math.sqrt(2 * math.pi)
        dh, dha = dy @ w2.t(), dy.abs() @ w2.abs().t()
        h, dp = p * cdf, dh * (cdf + p * pdf)
        ha, dpa = 1.13 * pa + h.abs(), dha * 1.13 + dh.abs() * 0.8 * pa + dp.abs()
        out = {"w1": x.t() @ dp, "b1": dp.sum(0), "w2": h.t() @ dy, "b2": dy.sum(0), "dx": dp @ w1.t()}
        mag = {"w1": x.abs().t() @ dp.abs(), "b1": dp.abs().sum(0), "w2": h.abs().t() @ dy.abs(),
               "b2": dy.abs().sum(0), "dx": dp.abs() @ w1.abs().t()}
        amp = {"w1": x.abs().t() @ dpa, "b1": dpa.sum(0), "w2": ha.t() @ dy.abs(), "b2": dy.abs().sum(0),
               "dx": dpa @ w1.abs().t()}
    return out, mag, amp


FFN_CASES = [
    ("swiglu", "bf16", [70, 0, 130, 1], 6, 128, 192),
    ("swiglu", "bf16", [300], 0, 64, 64),
    ("swiglu", "f32", [30, 0, 70], 3, 36, 20),
    ("gelu_bias", "bf16", [70, 0, 130, 1], 6, 192, 320),
    ("gelu_bias", "f32", [33, 1, 0], 2, 68, 100),
    ("gelu_bias", "bf16", [2100, 3000], 2, 64, 128),   # biases and matrices summed in parts
    ("swiglu", "f32", [1200], 0, 32, 64),
]


@pytest.mark.parametrize("act,dtype,counts,behind,d,ffn", FFN_CASES)
@pytest.mark.parametrize("grad,accumulate", [("own", False), ("f32", True)])
def test_ffn_backward(act, dtype, counts, behind, d, ffn, grad, accumulate):
    cfg, off, w, x, dy, ws = ffn_case(act, dtype, counts, behind, d, ffn)
    dt = DT[dtype]
    gdt = dt if grad == "own" else torch.float32
    base = {n: rand(v.shape, 0.2, gdt, 40 + i) for i, (n, v) in enumerate(w.items())}
    grads = {n: v.cuda() for n, v in base.items()}
    grads["dx"] = torch.full(x.shape, 9.0, dtype=dt, device="cuda")
    M.moe_expert_ffn_backward(cfg, {n: v.cuda() for n, v in w.items()}, x.cuda(),
                              torch.tensor(off, dtype=torch.int32).cuda(), dy.cuda(), grads, ws, accumulate=accumulate)
    assert M.moe_check_device_status(ws)[0] == M.MOE_OK
    assert (grads["dx"][off[-1]:] == 9.0).all()
    n = max(d, ffn, max(counts))
    for e in range(cfg.E):
        sl = slice(off[e], off[e + 1])
        ref, mag, amp = ffn_ref(act, w, x[sl].double(), dy[sl].double(), e)
        for name, r in ref.items():
            got = (grads[name][sl] if name == "dx" else grads[name][e]).double().cpu()
            b0 = base[name][e].double() if name != "dx" and accumulate else torch.zeros_like(r)
            stored = grads[name].dtype
            # sums in fp32 at two levels (amp: what an error of the inner sums moves, twice for __expf / erff),
            # the inner values' rounding to the operand type, the output's rounding
            inner = 0.0 if dtype == "f32" else 2.0 ** -8
            tol = 2 * sum_tol(dt, n) * (amp[name] + mag[name] + b0.abs()) + 1.01 * inner * mag[name] + \
                HALF[stored] * 1.01 * (r + b0).abs() + 1e-30
            err = (got - r - b0).abs()
            assert (err <= tol).all(), (name, e, float((err / tol).max()))


@pytest.mark.parametrize("act", ["swiglu", "gelu_bias"])
def test_ffn_backward_against_differences(act):
    """fp32 gradients along a random direction against central differences of the float64 forward."""
    cfg, off, w, x, dy, ws = ffn_case(act, "f32", [40, 25, 0], 0, 32, 48, seed=3)
    grads = {n: torch.zeros(v.shape, dtype=torch.float32, device="cuda") for n, v in w.items()}
    grads["dx"] = torch.zeros(x.shape, dtype=torch.float32, device="cuda")
    M.moe_expert_ffn_backward(cfg, {n: v.cuda() for n, v in w.items()}, x.cuda(),
                              torch.tensor(off, dtype=torch.int32).cuda(), dy.cuda(), grads, ws)

    def loss(w, x):
        total = 0.0
        for e in range(cfg.E):
            xe, de = x[off[e]:off[e + 1]], dy[off[e]:off[e + 1]].double()
            if act == "swiglu":
                g = xe @ w["w_gate"][e]
                y = (g * torch.sigmoid(g) * (xe @ w["w_up"][e])) @ w["w_down"][e]
            else:
                y = torch.nn.functional.gelu(xe @ w["w1"][e] + w["b1"][e]) @ w["w2"][e] + w["b2"][e]
            total += float((y * de).sum())
        return total

    w64, x64 = {n: v.double() for n, v in w.items()}, x.double()
    for name in list(w) + ["dx"]:
        v = x64 if name == "dx" else w64[name]
        step = rand(v.shape, 1.0, torch.float64, 77)
        h = 1e-4

        def at(s):
            return loss(w64, x64 + s * step) if name == "dx" else loss({**w64, name: v + s * step}, x64)

        want = (at(h) - at(-h)) / (2 * h)
        got = float((grads[name].double().cpu() * step).sum())
        size = float((grads[name].double().cpu().abs() * step.abs()).sum())
        # differences: h^2 / 6 of the third derivative along the step; fp32 gradients: 1e-6 of the terms
        assert abs(got - want) <= 1e-4 * abs(want) + 1e-5 * size, (name, got, want)


def test_ffn_backward_parts_left_out():
    """Gradients that are not asked for change none of the others."""
    cfg, off, w, x, dy, ws = ffn_case("gelu_bias", "bf16", [70, 30], 0, 64, 128)
    wd, o, xd, dyd = {n: v.cuda() for n, v in w.items()}, torch.tensor(off, dtype=torch.int32).cuda(), x.cuda(), dy.cuda()
    full = {n: torch.empty_like(v) for n, v in wd.items()}
    full["dx"] = torch.empty_like(xd)
    M.moe_expert_ffn_backward(cfg, wd, xd, o, dyd, full, ws)
    for names in (["dx"], ["w1", "b2"], ["b1"], ["w2"], []):
        part = {n: torch.empty_like(full[n]) for n in names}
        M.moe_expert_ffn_backward(cfg, wd, xd, o, dyd, part, ws)
        for n in names:
            assert torch.equal(part[n], full[n]), n


def test_training_step_through_the_layer():
    """A run of the calls as a training step makes them: dispatch, FFN, combine, then the combine's
    gradient (rows of dout times their weights), the FFN's backward pass and the rows' gradients summed
    per token -- against autograd in float64 on the same routing."""
    T, d, ffn, E, k = 96, 64, 128, 4, 2
    cfg = M.MoEConfig(T=T, d=d, ffn=ffn, E=E, k=k, capacity_factor=0.9)
    w = {"w_gate": rand((E, d, ffn), 0.1, torch.bfloat16, 1), "w_up": rand((E, d, ffn), 0.1, torch.bfloat16, 2),
         "w_down": rand((E, ffn, d), 0.1, torch.bfloat16, 3), "w_router": rand((d, E), 0.3, torch.bfloat16, 4)}
    x, dout = rand((T, d), 1.0, torch.bfloat16, 5), rand((T, d), 1.0, torch.bfloat16, 6)
    wd = {n: v.cuda() for n, v in w.items()}
    layer = M.MoELayer(cfg, wd)
    xd, doutd = x.cuda(), dout.cuda()
    out = layer.forward(xd)
    layer.check()
    R, rows = int(out["offsets"][-1]), M.moe_max_rows(cfg)
    src = out["src_assign"].long()
    held = torch.arange(rows, device="cuda") < R
    src = torch.where(held, src, 0)
    x_perm = xd[src // k]
    dy = (out["topk_w"].flatten()[src][:, None] * doutd[src // k].float()).to(torch.bfloat16)
    ws = M.Workspace(None, nbytes=M.moe_expert_ffn_backward_workspace_size(cfg))
    grads = {n: torch.zeros(v.shape, dtype=torch.float32, device="cuda") for n, v in wd.items() if n != "w_router"}
    grads["dx"] = torch.zeros_like(x_perm)
    M.moe_expert_ffn_backward(cfg, wd, x_perm, out["offsets"], dy, grads, ws, accumulate=True)
    slot = out["slot"].long()
    dx = torch.where((slot >= 0)[..., None], grads["dx"][slot.clamp(min=0)].float(), 0.0).sum(1)
    # float64, by autograd, on the routing of the device
    p = {n: v.double().requires_grad_() for n, v in w.items() if n != "w_router"}
    x64 = x.double().requires_grad_()
    idx, tw, sl = out["topk_idx"].cpu().long(), out["topk_w"].cpu().double(), slot.cpu()
    total = 0.0
    for t in range(T):
        for j in range(k):
            if sl[t, j] >= 0:
                e = idx[t, j]
                g = x64[t] @ p["w_gate"][e]
                y = (g * torch.sigmoid(g) * (x64[t] @ p["w_up"][e])) @ p["w_down"][e]
                total = total + tw[t, j] * (y * dout[t].double()).sum()
    total.backward()
    for n, v in p.items():
        err = float((grads[n].double().cpu() - v.grad).norm() / v.grad.norm())
        assert err <= 3 * 2.0 ** -8, (n, err)   # dy, inner values: each rounded to bf16 once
    err = float((dx.double().cpu() - x64.grad).norm() / x64.grad.norm())
    assert err <= 4 * 2.0 ** -8, err


def test_ffn_backward_captured_and_two_at_once():
    """The same bits from a captured backward pass replayed twice, and from two calls at the same time on two streams
    with workspaces of their own."""
    calls = []
    for act, counts, d, ffn in (("swiglu", [300, 0, 41], 128, 192), ("gelu_bias", [2100, 64], 64, 128)):
        cfg, off, w, x, dy, ws = ffn_case(act, "bf16", counts, 3, d, ffn)
        wd, xd, dyd = {n: v.cuda() for n, v in w.items()}, x.cuda(), dy.cuda()
        o = torch.tensor(off, dtype=torch.int32).cuda()

        def make(cfg=cfg, wd=wd, xd=xd, dyd=dyd, o=o):
            grads = {n: torch.zeros(v.shape, dtype=torch.float32, device="cuda") for n, v in wd.items()}
            grads["dx"] = torch.zeros_like(xd)
            space = M.Workspace(None, nbytes=M.moe_expert_ffn_backward_workspace_size(cfg))
            return grads, lambda: M.moe_expert_ffn_backward(cfg, wd, xd, o, dyd, grads, space, accumulate=True)

        calls.append(make)
    refs = []
    for make in calls:
        grads, run = make()
        run()
        torch.cuda.synchronize()
        refs.append({n: v.clone() for n, v in grads.items()})
    for make, ref in zip(calls, refs):
        grads, run = make()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        for _ in range(2):
            for v in grads.values():
                v.zero_()
            graph.replay()
            torch.cuda.synchronize()
            for n, v in grads.items():
                assert torch.equal(v, ref[n]), n
    streams = [torch.cuda.Stream() for _ in calls]
    made = [make() for make in calls]
    torch.cuda.synchronize()
    for _ in range(5):
        for (grads, run), s in zip(made, streams):
            with torch.cuda.stream(s):
                for v in grads.values():
                    v.zero_()
                run()
    torch.cuda.synchronize()
    for (grads, _), ref in zip(made, refs):
        for n, v in grads.items():
            assert torch.equal(v, ref[n]), n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_tiles_of_ragged_experts(dtype):
    """Many tiles per CTA pair with every kind of edge among them, twice into the same buffers."""
    counts = [0, 1, 63, 64, 65, 127, 128, 129, 255, 256, 257, 383, 511, 512, 513, 700]
    g, off, x, dy, w, b, o, ws = case((counts, 7, 648, 1160), dtype, seed=9)
    xd, dyd, wd, bd = x.cuda(), dy.cuda(), w.cuda(), b.cuda()
    dt = DT[dtype]
    y, dx = torch.zeros((g.rows, g.N), dtype=dt, device="cuda"), torch.zeros((g.rows, g.K), dtype=dt, device="cuda")
    dw, db = torch.empty((g.E, g.K, g.N), dtype=torch.float32, device="cuda"), torch.empty((g.E, g.N), device="cuda")
    for _ in range(2):
        M.moe_grouped_gemm(g, xd, wd, o, y, ws, bias=bd)
        M.moe_grouped_gemm_grad_x(g, dyd, wd, o, dx, ws)
        M.moe_grouped_gemm_grad_w(g, xd, dyd, o, dw, ws, db=db)
    assert M.moe_check_device_status(ws)[0] == M.MOE_OK
    for e in range(g.E):
        sl = slice(off[e], off[e + 1])
        xe, de, we, be = (t.double() for t in (xd[sl], dyd[sl], wd[e], bd[e]))
        n = counts[e]
        check(y[sl], (xe @ we + be).cpu(), (xe.abs() @ we.abs() + be.abs()).cpu(), g.K, dt)
        check(dx[sl], (de @ we.t()).cpu(), (de.abs() @ we.abs().t()).cpu(), g.N, dt)
        check(dw[e], (xe.t() @ de).cpu(), (xe.abs().t() @ de.abs()).cpu(), n, dt)
        check(db[e], de.sum(0).cpu(), de.abs().sum(0).cpu(), n, torch.float32)


def test_long_sums_in_fp32():
    """fp32 weight gradients over many rows keep fp32's precision: the tensor cores' own sums lose 1.9e-5 of the
    value (relative norm) at 16384 rows, 4.4e-6 at 4096; promoted every 512 rows they lose 4.8e-7."""
    g = M.GroupedConfig(rows=16384, E=1, K=2048, N=2048)
    ws = M.Workspace(None, nbytes=M.moe_grouped_workspace_size(g))
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((g.rows, g.K), generator=gen, device="cuda").bfloat16()
    dy = torch.randn((g.rows, g.N), generator=gen, device="cuda").bfloat16()
    dw = torch.empty((1, g.K, g.N), dtype=torch.float32, device="cuda")
    M.moe_grouped_gemm_grad_w(g, x, dy, torch.tensor([0, g.rows], dtype=torch.int32).cuda(), dw, ws)
    ref = x.double().t() @ dy.double()
    assert float((dw[0].double() - ref).norm() / ref.norm()) <= 1e-6


def test_a_workspace_of_another_device_is_refused():
    g = M.GroupedConfig(rows=4, E=2, K=64, N=64)
    d = dict(device="cuda", dtype=torch.bfloat16)
    x, w, y = torch.zeros(4, 64, **d), torch.zeros(2, 64, 64, **d), torch.full((4, 64), 3.0, **d)
    o = torch.tensor([0, 2, 4], device="cuda", dtype=torch.int32)
    host = torch.empty(1 << 20, dtype=torch.uint8)
    ws = type("W", (), {"tensor": host, "ptr": 1 << 20, "nbytes": host.numel()})()
    codes, scale = M.moe_quantize_int4(w, 64)
    cfg = M.MoEConfig(T=4, d=64, ffn=64, E=2, k=1)
    sw = {"w_gate": w, "w_up": w, "w_down": w}
    rows = torch.zeros(M.moe_max_rows(cfg), 64, **d)
    for f in (lambda: M.moe_grouped_gemm(g, x, w, o, y, ws), lambda: M.moe_grouped_gemm_grad_x(g, x, w, o, y, ws),
              lambda: M.moe_grouped_gemm_grad_w(g, x, x, o, w, ws),
              lambda: M.moe_grouped_gemm_int4(g, x, codes, scale, o, y, ws, 64),
              lambda: M.moe_expert_ffn_backward(cfg, sw, rows, o, rows, {"dx": torch.empty_like(rows)}, ws)):
        with pytest.raises(M.MoEError, match="workspace"):
            f()
    assert torch.equal(y, torch.full_like(y, 3.0))
