"""What the expert-product operators are measured on.

Four operators, all over rows sorted by expert (rows [offsets[e], offsets[e+1]) belong to expert e, and rows behind
offsets[E] are left as they were):

  gemm    y = x W[e] (+ b[e]) and its two gradients, dx = dy W[e]^T and dW[e] = x_e^T dy_e (db[e] = sum of dy_e)
  int4    y = x W[e] (+ b[e]) with W stored as 4-bit codes and a float32 scale per group of K and output column
  ffn4    a SwiGLU expert FFN whose three matrices are stored that way (the layer's serving form for single tokens)
  ffn_bwd the backward pass of the SwiGLU or GELU expert FFN: gradients of the rows, the matrices and the biases

``run`` computes them with elementary torch operations in float32 when ``own`` is false, and through the package's
entry points when it is true.
"""
import math

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the first matrix of the 4096-token, top-2, 8-expert layer: its rows after dispatch
        dict(name="fwd_8192x2048x4096_e8", op="gemm", dir="fwd", rows=8192, K=2048, N=4096, E=8, dtype="bf16", skew=0.0,
             slack=37, bias=False),
        # a small ragged batch with sizes that fill no tile, and a bias
        dict(name="fwd_517x200x328_e6", op="gemm", dir="fwd", rows=517, K=200, N=328, E=6, dtype="bf16", skew=0.7,
             slack=5, bias=True),
        # rows of a long context over 32 experts with a skewed router, gradient of the rows
        dict(name="gx_16384x4096x4096_e32", op="gemm", dir="gx", rows=16384, K=4096, N=4096, E=32, dtype="bf16",
             skew=0.5, slack=0, bias=False),
        # gradient of the first matrix, added to float32 gradients over micro-batches
        dict(name="gw_8192x2048x4096_e8_f32", op="gemm", dir="gw", rows=8192, K=2048, N=4096, E=8, dtype="bf16",
             skew=0.3, slack=100, bias=False, grad="f32", accumulate=True),
        # the float32 layer the pages start from: a forward call where latency counts
        dict(name="fwd_128x128x256_e4_f32", op="gemm", dir="fwd", rows=128, K=128, N=256, E=4, dtype="f32", skew=0.2,
             slack=3, bias=True),
        # float32 gradient of the weights and the bias
        dict(name="gw_2048x1024x1024_e8_f32", op="gemm", dir="gw", rows=2048, K=1024, N=1024, E=8, dtype="f32",
             skew=0.3, slack=11, bias=True, grad="f32", accumulate=False),
        # one token, top-2 of 8: two experts stream one matrix each
        dict(name="int4_2x2048x4096_e8", op="int4", rows=2, K=2048, N=4096, E=8, group=128, skew=0.0, slack=0,
             bias=False),
        # 64 tokens, top-2 of 64: nearly every expert streams its matrix for two rows
        dict(name="int4_128x2048x2048_e64", op="int4", rows=128, K=2048, N=2048, E=64, group=64, skew=0.0, slack=0,
             bias=False),
        # a batch with tens of rows per expert, where the products begin to count
        dict(name="int4_500x4096x4096_e8", op="int4", rows=500, K=4096, N=4096, E=8, group=128, skew=0.3, slack=12,
             bias=True),
        # the decode layer's whole expert FFN
        dict(name="ffn4_t64_2048x2048_e64", op="ffn4", T=64, k=2, d=2048, ffn=2048, E=64, group=64, skew=0.0, slack=0),
        # a training step's expert FFNs, 4096 tokens, top-2 of 8
        dict(name="ffn_bwd_swiglu_t4096", op="ffn_bwd", act="swiglu", T=4096, k=2, d=2048, ffn=4096, E=8, dtype="bf16",
             skew=0.2, slack=19),
        # a small GELU layer, top-3 of 5, with biases
        dict(name="ffn_bwd_gelu_t259", op="ffn_bwd", act="gelu_bias", T=259, k=3, d=192, ffn=320, E=5, dtype="bf16",
             skew=0.6, slack=8),
    ]


_MOST_FLOPS = 2.0 * 16384 * 4096 * 4096


def _log_int(rng, lo, hi, step=1):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, min(hi, -(-v // step) * step))


def draw(rng):
    op = rng.choice(["gemm", "gemm", "gemm", "int4", "int4", "ffn4", "ffn_bwd"])
    skew = round(rng.uniform(0.0, 1.0), 3)
    while True:
        E = _log_int(rng, 1, 64)
        if op == "gemm":
            dtype = rng.choice(["bf16", "bf16", "f32"])
            rows = _log_int(rng, 1, 16384 if dtype == "bf16" else 4096)
            K, N = (_log_int(rng, 64, 4096 if dtype == "bf16" else 1024, 8) for _ in range(2))
            c = dict(op="gemm", dir=rng.choice(["fwd", "gx", "gw"]), rows=rows, K=K, N=N, E=E, dtype=dtype, skew=skew,
                     slack=min(rows - 1, rng.randrange(40)), bias=rng.random() < 0.4)
            if c["dir"] == "gx":
                c["bias"] = False
            if c["dir"] == "gw":
                c["grad"] = "f32" if dtype == "f32" else rng.choice(["bf16", "f32"])
                c["accumulate"] = rng.random() < 0.4
            size, weights = 2.0 * rows * K * N, E * K * N
        elif op == "int4":
            rows = _log_int(rng, 1, 1024)
            K, N = _log_int(rng, 64, 4096, 8), _log_int(rng, 64, 4096, 8)
            c = dict(op="int4", rows=rows, K=K, N=N, E=E, group=rng.choice([32, 64, 128]), skew=skew,
                     slack=min(rows - 1, rng.randrange(8)), bias=rng.random() < 0.4)
            size, weights = 2.0 * rows * K * N, E * K * N
        else:
            k = rng.randint(1, min(E, 4))
            d, ffn = _log_int(rng, 64, 2048, 64), _log_int(rng, 64, 4096 if op == "ffn_bwd" else 2048, 64)
            if op == "ffn4":
                T = _log_int(rng, 1, 256)
                c = dict(op="ffn4", T=T, k=k, d=d, ffn=ffn, E=E, group=rng.choice([32, 64, 128]), skew=skew,
                         slack=min(T * k - 1, rng.randrange(4)))
            else:
                T = _log_int(rng, 1, 4096)
                c = dict(op="ffn_bwd", act=rng.choice(["swiglu", "gelu_bias"]), T=T, k=k, d=d, ffn=ffn, E=E,
                         dtype="bf16", skew=skew, slack=min(T * k - 1, rng.randrange(40)))
            size, weights = 16.0 * T * k * d * ffn, 3 * E * d * ffn
        # no dearer than the largest listed case: its products, and its weights
        if size <= _MOST_FLOPS and weights <= 32 * 4096 * 4096 // 2:
            return c


# ------------------------------------------------------------------ inputs
def _counts(case, total, gen):
    """Rows of each expert: a multinomial draw over popularities (e+1)^-skew, shuffled; whole numbers on the host."""
    E = case["E"]
    pop = torch.arange(1, E + 1, dtype=torch.float64).pow(-2.0 * case["skew"])
    pop = pop[torch.randperm(E, generator=gen)]
    pick = torch.multinomial(pop, total, replacement=True, generator=gen) if total else torch.zeros(0, dtype=torch.long)
    return torch.bincount(pick, minlength=E).tolist()


def _rows_of(case):
    return case["rows"] if "rows" in case else case["T"] * case["k"]


def _handles(case, rows):
    """The workspace and the configuration that a program keeps."""
    import mixture_experts_layer_37_b200 as M
    if case["op"] in ("gemm", "int4"):
        g = M.GroupedConfig(rows=rows, E=case["E"], K=case["K"], N=case["N"], dtype=case.get("dtype", "bf16"))
        return dict(M=M, g=g, ws=M.Workspace(None, nbytes=M.moe_grouped_workspace_size(g)))
    weights = "int4_g%d" % case["group"] if case["op"] == "ffn4" else "native"
    cfg = M.MoEConfig(T=case["T"], d=case["d"], ffn=case["ffn"], E=case["E"], k=case["k"], dtype="bf16",
                      act=case.get("act", "swiglu"), capacity_factor=0.0, weights=weights)
    size = M.moe_workspace_size(cfg) if case["op"] == "ffn4" else M.moe_expert_ffn_backward_workspace_size(cfg)
    return dict(M=M, cfg=cfg, ws=M.Workspace(None, nbytes=size))


def prepare(case, seed):
    host = torch.Generator().manual_seed(seed * 7919 + 17)
    gen = torch.Generator(device="cuda").manual_seed(seed * 104729 + 5)
    rows = _rows_of(case)
    counts = _counts(case, rows - case["slack"], host)
    off = [0]
    for n in counts:
        off.append(off[-1] + n)
    st = dict(case=case, most=max(max(counts), 1), offsets=torch.tensor(off, dtype=torch.int32).cuda())

    def normal(shape, std, dtype):
        return torch.randn(shape, generator=gen, device="cuda", dtype=F32).mul_(std).to(dtype)

    def codes(E, K, N, group):
        """4-bit codes as they are stored, [E, N, 64 bytes per 128 of K], and scales [E, groups, N]."""
        st_codes = torch.randint(0, 256, (E, N, -(-K // 128) * 64), generator=gen, device="cuda", dtype=torch.uint8)
        scale = torch.rand((E, -(-K // group), N), generator=gen, device="cuda") * 0.006 + 0.002
        return st_codes, scale

    E = case["E"]
    if case["op"] == "gemm":
        dt = BF16 if case["dtype"] == "bf16" else F32
        K, N = case["K"], case["N"]
        if case["dir"] != "gx":
            st["x"] = normal((rows, K), 1.0, dt)
        if case["dir"] != "fwd":
            st["dy"] = normal((rows, N), 0.01, dt)
        if case["dir"] != "gw":
            st["w"] = normal((E, K, N), 0.02, dt)
            st["b"] = normal((E, N), 0.01, dt) if case["bias"] else None
            st["out"] = torch.zeros((rows, N if case["dir"] == "fwd" else K), dtype=dt, device="cuda")
        else:
            gdt = F32 if case["grad"] == "f32" else BF16
            st["dw"] = normal((E, K, N), 0.3, gdt)
            st["db"] = normal((E, N), 0.3, gdt) if case["bias"] else None
    elif case["op"] == "int4":
        K, N = case["K"], case["N"]
        st["x"] = normal((rows, K), 1.0, BF16)
        st["q"], st["s"] = codes(E, K, N, case["group"])
        st["b"] = normal((E, N), 0.01, BF16) if case["bias"] else None
        st["out"] = torch.zeros((rows, N), dtype=BF16, device="cuda")
    else:
        d, ffn = case["d"], case["ffn"]
        st["x"] = normal((rows, d), 1.0, BF16)
        if case["op"] == "ffn4":
            w = {}
            for n, K, N in (("w_gate", d, ffn), ("w_up", d, ffn), ("w_down", ffn, d)):
                w[n], w[n + "_scale"] = codes(E, K, N, case["group"])
            st["weights"] = w
            st["out"] = torch.zeros((rows, d), dtype=BF16, device="cuda")
        else:
            st["dy"] = normal((rows, d), 0.01, BF16)
            if case["act"] == "swiglu":
                w = {"w_gate": normal((E, d, ffn), 0.02, BF16), "w_up": normal((E, d, ffn), 0.02, BF16),
                     "w_down": normal((E, ffn, d), 0.02, BF16)}
            else:
                w = {"w1": normal((E, d, ffn), 0.02, BF16), "b1": normal((E, ffn), 0.01, BF16),
                     "w2": normal((E, ffn, d), 0.02, BF16), "b2": normal((E, d), 0.01, BF16)}
            st["weights"] = w
            st["grads"] = {n: torch.empty_like(v) for n, v in w.items()}
            st["grads"]["dx"] = torch.zeros_like(st["x"])
    if own:
        st.update(_handles(case, rows))
    return st


# ------------------------------------------------------------------ plain forms
def _index(offsets, rows, most):
    """(row of each place of a padded [E, most] layout, whether it holds one; expert and place of each row, whether it has one)."""
    off = offsets.long()
    at = off[:-1, None] + torch.arange(most, device=off.device)[None]
    held = at < off[1:, None]
    r = torch.arange(rows, device=off.device)
    e = torch.searchsorted(off[1:].contiguous(), r, right=True).clamp(max=off.numel() - 2)
    return at.clamp(max=rows - 1), held, e, (r - off[e]).clamp(min=0, max=most - 1), r < off[-1]


def _padded(t, ix):
    return torch.where(ix[1][..., None], t[ix[0]].float(), 0.0)


def _sorted(t, ix, like):
    return torch.where(ix[4][:, None], t[ix[2], ix[3]], like.float()).to(like.dtype)


def _dequantised(q, s, K, group):
    """float32 [E, K, N] of stored codes.  A byte holds two codes, the low four bits first; a code c stands for c - 8.
    Along K a row is stored in blocks of 128 (64 bytes): the block's 32-bit word 4 t + i holds the eight codes of
    k = 32 i + 8 t .. + 7 in the order k, k+2, k+4, k+6, k+1, k+3, k+5, k+7."""
    E, N, B = q.shape
    c = torch.stack((q & 15, q >> 4), dim=-1).reshape(E, N, B // 64, 4, 4, 2, 4)  # block, t, i, odd, pair
    c = c.permute(0, 1, 2, 4, 3, 6, 5).reshape(E, N, 2 * B)[..., :K]              # block, i, t, pair, odd
    w = c.transpose(1, 2).to(F32) - 8.0
    return w * torch.repeat_interleave(s, group, dim=1)[:, :K]


def _plain_gemm(st, case):
    rows = case["rows"]
    ix = _index(st["offsets"], rows, st["most"])
    if case["dir"] == "fwd":
        y = torch.bmm(_padded(st["x"], ix), st["w"].float())
        if st["b"] is not None:
            y = y + st["b"].float()[:, None]
        return _sorted(y, ix, st["out"])
    dy = _padded(st["dy"], ix)
    if case["dir"] == "gx":
        return _sorted(torch.bmm(dy, st["w"].float().transpose(1, 2)), ix, st["out"])
    dw = torch.bmm(_padded(st["x"], ix).transpose(1, 2), dy)
    db = dy.sum(1)
    if case["accumulate"]:
        dw, db = dw + st["dw"].float(), (db + st["db"].float() if st["db"] is not None else None)
    st["dw"].copy_(dw)
    if st["db"] is not None:
        st["db"].copy_(db)
        return st["dw"], st["db"]
    return st["dw"]


def _plain_ffn_bwd(st, case):
    w, rows = st["weights"], _rows_of(case)
    ix = _index(st["offsets"], rows, st["most"])
    x, dy = _padded(st["x"], ix), _padded(st["dy"], ix)
    t = lambda v: v.transpose(1, 2)  # noqa: E731
    if case["act"] == "swiglu":
        wg, wu, wd = (w[n].float() for n in ("w_gate", "w_up", "w_down"))
        g, u = torch.bmm(x, wg), torch.bmm(x, wu)
        s = torch.sigmoid(g)
        dh = torch.bmm(dy, t(wd))
        dg, du = dh * u * s * (1 + g * (1 - s)), dh * g * s
        out = {"w_gate": torch.bmm(t(x), dg), "w_up": torch.bmm(t(x), du), "w_down": torch.bmm(t(g * s * u), dy)}
        dx = torch.bmm(dg, t(wg)) + torch.bmm(du, t(wu))
    else:
        w1, w2 = w["w1"].float(), w["w2"].float()
        p = torch.bmm(x, w1) + w["b1"].float()[:, None]
        cdf = 0.5 * (1 + torch.erf(p * math.sqrt(0.5)))
        pdf = torch.exp(-0.5 * p * p) / math.sqrt(2 * math.pi)
        # places that hold no row have dh = 0, so they add nothing to a sum
        dp = torch.bmm(dy, t(w2)) * (cdf + p * pdf)
        out = {"w1": torch.bmm(t(x), dp), "b1": dp.sum(1), "w2": torch.bmm(t(p * cdf), dy), "b2": dy.sum(1)}
        dx = torch.bmm(dp, t(w1))
    out = {n: v.to(BF16) for n, v in out.items()}
    out["dx"] = _sorted(dx, ix, torch.zeros_like(st["x"]))
    return out


def _plain(st):
    case = st["case"]
    if case["op"] == "gemm":
        return _plain_gemm(st, case)
    if case["op"] == "ffn_bwd":
        return _plain_ffn_bwd(st, case)
    ix = _index(st["offsets"], _rows_of(case), st["most"])
    x = _padded(st["x"], ix)
    if case["op"] == "int4":
        y = torch.bmm(x, _dequantised(st["q"], st["s"], case["K"], case["group"]))
        if st["b"] is not None:
            y = y + st["b"].float()[:, None]
        return _sorted(y, ix, st["out"])
    w = st["weights"]
    wg, wu, wd = (_dequantised(w[n], w[n + "_scale"], K, case["group"]) for n, K in
                  (("w_gate", case["d"]), ("w_up", case["d"]), ("w_down", case["ffn"])))
    g = torch.bmm(x, wg)
    return _sorted(torch.bmm(g * torch.sigmoid(g) * torch.bmm(x, wu), wd), ix, st["out"])


def run(st):
    if not own:
        return _plain(st)
    case, M = st["case"], st["M"]
    if case["op"] == "gemm":
        if case["dir"] == "fwd":
            M.moe_grouped_gemm(st["g"], st["x"], st["w"], st["offsets"], st["out"], st["ws"], bias=st["b"])
        elif case["dir"] == "gx":
            M.moe_grouped_gemm_grad_x(st["g"], st["dy"], st["w"], st["offsets"], st["out"], st["ws"])
        else:
            M.moe_grouped_gemm_grad_w(st["g"], st["x"], st["dy"], st["offsets"], st["dw"], st["ws"], db=st["db"],
                                      accumulate=case["accumulate"])
            return (st["dw"], st["db"]) if st["db"] is not None else st["dw"]
        return st["out"]
    if case["op"] == "int4":
        M.moe_grouped_gemm_int4(st["g"], st["x"], st["q"], st["s"], st["offsets"], st["out"], st["ws"],
                                group=case["group"], bias=st["b"])
        return st["out"]
    if case["op"] == "ffn4":
        M.moe_expert_ffn(st["cfg"], st["weights"], st["x"], st["offsets"], st["out"], st["ws"])
        return st["out"]
    M.moe_expert_ffn_backward(st["cfg"], st["weights"], st["x"], st["offsets"], st["dy"], st["grads"], st["ws"])
    return st["grads"]


# ------------------------------------------------------------------ work
def _busy(case):
    """Experts that are expected to hold a row: those whose weights a pass has to read."""
    E, n = case["E"], _rows_of(case) - case["slack"]
    pop = [(e + 1) ** (-2.0 * case["skew"]) for e in range(E)]
    total = sum(pop)
    return sum(1 - (1 - p / total) ** n for p in pop)


def work(case):
    rows, busy, E = _rows_of(case) - case["slack"], _busy(case), case["E"]
    if case["op"] == "gemm":
        es = 2 if case["dtype"] == "bf16" else 4
        K, N = case["K"], case["N"]
        if case["dir"] == "gw":
            gs = (4 if case["grad"] == "f32" else 2) * (2 if case["accumulate"] else 1)
            nbytes = rows * (K + N) * es + E * (K + (1 if case["bias"] else 0)) * N * gs
        else:
            nbytes = rows * (K + N) * es + busy * (K + (1 if case["bias"] else 0)) * N * es
        return {"bytes": nbytes, "flops": 2.0 * rows * K * N}
    if case["op"] == "int4":
        K, N = case["K"], case["N"]
        return {"bytes": rows * (K + N) * 2 + busy * N * (K / 2 + 4 * -(-K // case["group"]) + (2 if case["bias"] else 0)),
                "flops": 2.0 * rows * K * N}
    d, ffn = case["d"], case["ffn"]
    if case["op"] == "ffn4":
        g = case["group"]
        per = 2 * ffn * (d / 2 + 4 * -(-d // g)) + d * (ffn / 2 + 4 * -(-ffn // g))
        return {"bytes": rows * 2 * d * 2 + busy * per, "flops": 6.0 * rows * d * ffn}
    mats = 3 if case["act"] == "swiglu" else 2
    # the inner activations are formed again, then two products for each matrix, and dh
    return {"bytes": rows * 3 * d * 2 + (busy + E) * mats * d * ffn * 2, "flops": 2.0 * rows * d * ffn * (3 * mats - 1)}


# ------------------------------------------------------------------ exact values
def exact(case, seed):
    """The operator's definition in float64, expert by expert."""
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    off, E = st["offsets"].tolist(), case["E"]
    D = torch.float64

    def weight(q, s, K, group):
        """One expert's [K, N] from its stored codes, code by code."""
        kk = torch.arange(K, device="cuda")
        block, rest = kk // 128, kk % 128
        i, t, j = rest // 32, rest % 32 // 8, rest % 8
        place = (j // 2) + 4 * (j % 2)                     # which four bits of the word
        byte = block * 64 + (4 * t + i) * 4 + place // 2
        c = (q[:, byte].int() >> (4 * (place % 2))) & 15   # [N, K]
        return (c.to(D) - 8).t() * s.to(D)[kk // group]

    if case["op"] == "gemm" and case["dir"] == "gw":
        dw = st["dw"].to(D) if case["accumulate"] else torch.zeros(st["dw"].shape, dtype=D, device="cuda")
        db = None
        if st["db"] is not None:
            db = st["db"].to(D) if case["accumulate"] else torch.zeros(st["db"].shape, dtype=D, device="cuda")
        for e in range(E):
            xe, de = st["x"][off[e]:off[e + 1]].to(D), st["dy"][off[e]:off[e + 1]].to(D)
            dw[e] += xe.t() @ de
            if db is not None:
                db[e] += de.sum(0)
        return (dw, db) if db is not None else dw
    if case["op"] == "ffn_bwd":
        w = {n: v for n, v in st["weights"].items()}
        out = {n: torch.zeros(v.shape, dtype=D, device="cuda") for n, v in w.items()}
        out["dx"] = torch.zeros(st["x"].shape, dtype=D, device="cuda")
        for e in range(E):
            sl = slice(off[e], off[e + 1])
            x, dy = st["x"][sl].to(D), st["dy"][sl].to(D)
            if case["act"] == "swiglu":
                wg, wu, wd = w["w_gate"][e].to(D), w["w_up"][e].to(D), w["w_down"][e].to(D)
                g, u = x @ wg, x @ wu
                sg = 1 / (1 + torch.exp(-g))
                dh = dy @ wd.t()
                dg = dh * u * (sg + g * sg * (1 - sg))
                du = dh * (g * sg)
                out["w_gate"][e], out["w_up"][e], out["w_down"][e] = x.t() @ dg, x.t() @ du, (g * sg * u).t() @ dy
                out["dx"][sl] = dg @ wg.t() + du @ wu.t()
            else:
                w1, w2 = w["w1"][e].to(D), w["w2"][e].to(D)
                p = x @ w1 + w["b1"][e].to(D)
                cdf = 0.5 * torch.erfc(-p / math.sqrt(2.0))
                dp = (dy @ w2.t()) * (cdf + p * torch.exp(-p * p / 2) / math.sqrt(2 * math.pi))
                out["w1"][e], out["b1"][e], out["w2"][e], out["b2"][e] = x.t() @ dp, dp.sum(0), (p * cdf).t() @ dy, dy.sum(0)
                out["dx"][sl] = dp @ w1.t()
        return out
    y = torch.zeros(st["out"].shape, dtype=D, device="cuda")
    for e in range(E):
        sl = slice(off[e], off[e + 1])
        if off[e] == off[e + 1]:
            continue
        if case["op"] == "gemm":
            we = st["w"][e].to(D)
            y[sl] = st["x"][sl].to(D) @ we if case["dir"] == "fwd" else st["dy"][sl].to(D) @ we.t()
        elif case["op"] == "int4":
            y[sl] = st["x"][sl].to(D) @ weight(st["q"][e], st["s"][e], case["K"], case["group"])
        else:
            w = st["weights"]
            wg, wu, wd = (weight(w[n][e], w[n + "_scale"][e], K, case["group"]) for n, K in
                          (("w_gate", case["d"]), ("w_up", case["d"]), ("w_down", case["ffn"])))
            g = st["x"][sl].to(D) @ wg
            y[sl] = (g / (1 + torch.exp(-g)) * (st["x"][sl].to(D) @ wu)) @ wd
        if st.get("b") is not None:
            y[sl] += st["b"][e].to(D)
    return y
