"""The bench takes every weight format of the layer and counts its bytes as they are stored.  No GPU is needed."""
from __future__ import annotations

import sys

import pytest

import bench
import mixture_experts_layer_37_b200 as M


def test_every_format_can_be_chosen(monkeypatch):
    for fmt in M.WEIGHT_FORMATS:
        monkeypatch.setattr(sys, "argv", ["bench.py", "--weights", fmt])
        assert bench.parse().weights == fmt


@pytest.mark.parametrize("K,N", [(128, 64), (2048, 4096)])
def test_bytes_are_those_of_the_stored_form(K, N):
    for fmt, group in M.WEIGHT_FORMATS.items():
        if not fmt.startswith("int4"):
            continue
        codes, scales = M._int4_shapes(1, K, N, group)
        assert bench.weight_bytes(fmt, 2) * K * N == codes[1] * codes[2] + 4 * scales[1] * scales[2]
    assert bench.weight_bytes("native", 2) == 2 and bench.weight_bytes("native", 4) == 4 and bench.weight_bytes("int8", 2) == 1
