"""The package's functions pass their arguments as declared whatever callers of the C ABI do to the handle
that ``lib()`` returns.  No GPU is needed."""
from __future__ import annotations

import ctypes

import pytest

import mixture_experts_layer_37_b200 as M


@pytest.fixture(scope="module", autouse=True)
def built():
    from mixture_experts_layer_37_b200 import build
    build.build()


@pytest.mark.parametrize("name,call", [
    ("moe_max_rows", lambda: M.moe_max_rows(M.MoEConfig(T=8, d=64, ffn=64, E=2, k=1, capacity_factor=0.0))),
    ("moe_grouped_workspace_size", lambda: M.moe_grouped_workspace_size(M.GroupedConfig(rows=3, E=2, K=64, N=64))),
    ("moe_expert_ffn_backward_workspace_size",
     lambda: M.moe_expert_ffn_backward_workspace_size(M.MoEConfig(T=8, d=64, ffn=64, E=2, k=1))),
    ("moe_ep_recv_rows", lambda: M.moe_ep_recv_rows(M.MoEConfig(T=8, d=64, ffn=64, E=2, k=1), 16, 2)),
])
def test_argument_types_of_the_abi_handle_do_not_reach_the_package(name, call):
    want = call()
    f = getattr(M.lib(), name)
    before = f.argtypes
    try:
        f.argtypes = [ctypes.c_int32]          # would refuse the package's pointers
        assert call() == want
    finally:
        f.argtypes = before


def test_addresses_are_passed_whole():
    """Every function that the package has declared still takes pointers after the ABI handle lost its types."""
    names = ("moe_expert_ffn", "moe_forward", "moe_combine")
    before = {n: getattr(M.lib(), n).argtypes for n in names}
    try:
        for n in names:
            getattr(M.lib(), n).argtypes = None
        for n in names:
            assert ctypes.c_void_p in getattr(M._own(), n).argtypes
        f = M._fn("moe_grouped_gemm", M._GCFG, *[ctypes.c_void_p] * 6, ctypes.c_size_t, ctypes.c_void_p)
        M.lib().moe_grouped_gemm.argtypes = None
        assert f.argtypes.count(ctypes.c_void_p) == 7
    finally:
        for n in names:
            getattr(M.lib(), n).argtypes = before[n]
