"""Refusals of the grouped products, the 4-bit weights and the FFN's backward
pass, on the host before any launch: no GPU is needed (pointers are never
dereferenced)."""
from __future__ import annotations

import copy
import ctypes
import dataclasses
import pickle

import pytest
import torch

import mixture_experts_layer_37_b200 as M

A = 1 << 20          # an aligned address that nothing reads
OK, INVALID, UNSUPPORTED, WORKSPACE = M.MOE_OK, M.MOE_ERR_INVALID_ARG, M.MOE_ERR_UNSUPPORTED, M.MOE_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    from mixture_experts_layer_37_b200 import build
    build.build()
    return M.lib()


def g(rows=100, E=4, K=64, N=128, dtype=M.MOE_DT_BF16):
    return M.MoEGroupedConfigC(rows, E, K, N, dtype)


def size_of(lib, c):
    v = ctypes.c_size_t()
    f = lib.moe_grouped_workspace_size
    f.argtypes = [ctypes.POINTER(M.MoEGroupedConfigC), ctypes.POINTER(ctypes.c_size_t)]
    return f(ctypes.byref(c), ctypes.byref(v)), v.value


@pytest.mark.parametrize("kw,want", [
    (dict(), OK), (dict(rows=0), OK), (dict(E=64), OK), (dict(K=8, N=8), OK),
    (dict(dtype=M.MOE_DT_F32, K=4, N=12), OK),
    (dict(rows=-1), INVALID), (dict(E=0), INVALID), (dict(K=0), INVALID), (dict(N=-8), INVALID), (dict(dtype=5), INVALID),
    (dict(E=65), UNSUPPORTED), (dict(K=12), UNSUPPORTED), (dict(N=20), UNSUPPORTED),
    (dict(dtype=M.MOE_DT_F32, K=6), UNSUPPORTED), (dict(rows=2 ** 31 - 1024), UNSUPPORTED),
    (dict(K=2 ** 20, N=2 ** 20), UNSUPPORTED),
])
def test_sizes(lib, kw, want):
    st, n = size_of(lib, g(**kw))
    assert st == want
    if want == OK:
        assert n >= 64 * 1024


def test_size_arguments(lib):
    f = lib.moe_grouped_workspace_size
    c = g()
    assert f(ctypes.byref(c), None) == INVALID and f(None, ctypes.byref(ctypes.c_size_t())) == INVALID


def test_workspace_grows_only_where_rows_are_summed_in_parts(lib):
    assert size_of(lib, g(rows=8192, E=8, K=2048, N=4096))[1] == 64 * 1024
    assert size_of(lib, g(rows=8192, E=1, K=80, N=312))[1] > 64 * 1024


P = ctypes.c_void_p


def call(lib, name, *args):
    f = getattr(lib, name)
    f.argtypes = None
    f.restype = ctypes.c_int
    return f(*args)


def test_products_refuse(lib):
    c = g()
    _, n = size_of(lib, c)
    big = ctypes.c_size_t(n)
    ref = ctypes.byref(c)

    def fwd(x=A, w=A, b=None, o=A, y=A, ws=A, nb=big, cfg=ref):
        return call(lib, "moe_grouped_gemm", cfg, P(x), P(w), P(b), P(o), P(y), P(ws), nb, P(0))

    assert fwd(cfg=None) == INVALID
    for k in ("x", "w", "o", "y"):
        assert fwd(**{k: None}) == INVALID, k
    for k in ("x", "w", "b", "y"):
        assert fwd(**{k: A + 8}) == INVALID, k
    assert fwd(ws=None) == WORKSPACE and fwd(nb=ctypes.c_size_t(n - 1)) == WORKSPACE and fwd(ws=A + 512) == INVALID
    zero = g(rows=0)
    assert fwd(x=None, y=None, cfg=ctypes.byref(zero)) == OK      # nothing to do, nothing launched
    assert fwd(w=None, cfg=ctypes.byref(zero)) == INVALID

    def gx(dy=A, w=A, o=A, dx=A, ws=A, nb=big):
        return call(lib, "moe_grouped_gemm_grad_x", ref, P(dy), P(w), P(o), P(dx), P(ws), nb, P(0))

    for k in ("dy", "w", "o", "dx"):
        assert gx(**{k: None}) == INVALID, k
    assert gx(dx=A + 4) == INVALID and gx(ws=None) == WORKSPACE

    def gw(x=A, dy=A, o=A, dw=A, db=None, dt=M.MOE_DT_F32, acc=0, ws=A, nb=big, cfg=ref):
        return call(lib, "moe_grouped_gemm_grad_w", cfg, P(x), P(dy), P(o), P(dw), P(db), ctypes.c_int32(dt),
                    ctypes.c_int32(acc), P(ws), nb, P(0))

    for k in ("x", "dy", "o", "dw"):
        assert gw(**{k: None}) == INVALID, k
    assert gw(dt=7) == INVALID and gw(db=A + 2) == INVALID and gw(ws=None) == WORKSPACE
    f32 = g(dtype=M.MOE_DT_F32)
    assert gw(dt=M.MOE_DT_BF16, cfg=ctypes.byref(f32)) == INVALID   # no gradients narrower than the config's dtype


def test_int4_refuses(lib):
    c = g()
    _, n = size_of(lib, c)
    ref = ctypes.byref(c)

    def prod(x=A, q=A, s=A, group=64, b=None, o=A, y=A, ws=A, nb=n, cfg=ref):
        return call(lib, "moe_grouped_gemm_int4", cfg, P(x), P(q), P(s), ctypes.c_int32(group), P(b), P(o), P(y), P(ws),
                    ctypes.c_size_t(nb), P(0))

    for k in ("x", "q", "s", "o", "y"):
        assert prod(**{k: None}) == INVALID, k
    for bad in (0, 1, 16, 48, 256, -64):
        assert prod(group=bad) == INVALID
    assert prod(q=A + 8) == INVALID and prod(s=A + 4) == INVALID and prod(ws=None) == WORKSPACE
    assert prod(cfg=ctypes.byref(g(dtype=M.MOE_DT_F32))) == UNSUPPORTED
    assert prod(cfg=ctypes.byref(g(K=2 ** 22 + 8))) == UNSUPPORTED

    def quant(w=A, group=64, q=A, s=A, cfg=ref):
        return call(lib, "moe_quantize_int4", cfg, P(w), ctypes.c_int32(group), P(q), P(s), P(0))

    for k in ("w", "q", "s"):
        assert quant(**{k: None}) == INVALID, k
    assert quant(group=100) == INVALID
    assert call(lib, "moe_pack_int4", ref, P(None), P(A), P(0)) == INVALID
    assert call(lib, "moe_pack_int4", ref, P(A), P(A + 8), P(0)) == INVALID


def test_int4_formats_of_the_layer(lib):
    size = ctypes.c_size_t()
    for name in ("int4_g32", "int4_g64", "int4_g128"):
        c = M.MoEConfig(T=8, d=128, ffn=128, E=8, k=2, weights=name).c()
        assert lib.moe_workspace_size(ctypes.byref(c), ctypes.byref(size)) == OK
        c = M.MoEConfig(T=8, d=128, ffn=128, E=8, k=2, dtype="f32", weights=name).c()
        assert lib.moe_workspace_size(ctypes.byref(c), ctypes.byref(size)) == UNSUPPORTED
    for v in (3, 16, 31, 33, 127, 129, 256):
        c = M.MoEConfig(T=8, d=128, ffn=128, E=8, k=2).c()
        c.weight_format = v
        assert lib.moe_workspace_size(ctypes.byref(c), ctypes.byref(size)) == INVALID, v
    # codes without scales
    cfg = M.MoEConfig(T=8, d=128, ffn=128, E=8, k=2, weights="int4_g64")
    w = M.MoEWeightsC(A, None, A, A, A)
    assert lib.moe_workspace_size(ctypes.byref(cfg.c()), ctypes.byref(size)) == OK
    assert call(lib, "moe_expert_ffn", ctypes.byref(cfg.c()), ctypes.byref(w), P(A), P(A), P(A), P(A), size, P(0)) == INVALID


def test_ffn_backward_refuses(lib):
    cfg = M.MoEConfig(T=64, d=128, ffn=128, E=4, k=2, act="gelu_bias")
    n = M.moe_expert_ffn_backward_workspace_size(cfg)

    def back(cfg=cfg, w=None, x=A, o=A, dy=A, dt=M.MOE_DT_BF16, grad=A, ws=A, nb=n, grads=True):
        w = w or M.MoEWeightsC(None, None, A, None, A, A, A)
        gr = M.MoEFfnGradsC(grad, A, None, A, A, A, dt, 0)
        return call(lib, "moe_expert_ffn_backward", ctypes.byref(cfg.c()), ctypes.byref(w), P(x), P(o), P(dy),
                    ctypes.byref(gr) if grads else None, P(ws), ctypes.c_size_t(nb), P(0))

    assert back(x=None) == INVALID and back(o=None) == INVALID and back(dy=None) == INVALID and back(grads=False) == INVALID
    assert back(dt=3) == INVALID and back(grad=A + 8) == INVALID
    assert back(ws=None) == WORKSPACE and back(nb=n - 1) == WORKSPACE
    assert back(w=M.MoEWeightsC(None, None, A, None, A, None, A)) == INVALID     # GELU without b1
    swiglu = M.MoEConfig(T=64, d=128, ffn=128, E=4, k=2)
    assert back(cfg=swiglu, w=M.MoEWeightsC(None, None, A, None, A)) == INVALID  # SwiGLU without W_up
    for weights in ("int8", "int4_g64"):
        c = M.MoEConfig(T=64, d=128, ffn=128, E=4, k=2, act="gelu_bias", weights=weights)
        assert back(cfg=c) == UNSUPPORTED


def test_python_checks_tensors():
    cfg = M.GroupedConfig(rows=4, E=2, K=64, N=64)
    z = torch.zeros
    ws = type("W", (), {"ptr": A, "nbytes": 1 << 20})()
    with pytest.raises(M.MoEError):   # not on a GPU
        M.moe_grouped_gemm(cfg, z(4, 64), z(2, 64, 64), z(3, dtype=torch.int32), z(4, 64), ws)
    with pytest.raises(M.MoEError):
        M.moe_expert_ffn_backward(M.MoEConfig(T=4, d=64, ffn=64, E=2, k=1), {}, z(4, 64), z(3, dtype=torch.int32), z(4, 64),
                                  {"w1": z(2, 64, 64)}, ws)   # a GELU name for SwiGLU experts


def test_config_copies_and_types():
    c = M.GroupedConfig(4, 2, 64, 128, "f32")
    for d in (copy.copy(c), copy.deepcopy(c), pickle.loads(pickle.dumps(c)), dataclasses.replace(c)):
        assert d == c and hash(d) == hash(c) and d is not c
        assert (d.c().rows, d.c().E, d.c().K, d.c().N, d.c().dtype) == (4, 2, 64, 128, M.MOE_DT_F32)
    assert dataclasses.replace(c, rows=9).c().rows == 9
    for dtype in ("fp16", "float32", None):
        with pytest.raises(M.MoEError):
            M.GroupedConfig(4, 2, 64, 128, dtype)


def test_struct_layouts_match_the_header():
    assert ctypes.sizeof(M.MoEGroupedConfigC) == 24 and ctypes.sizeof(M.MoEFfnGradsC) == 56
