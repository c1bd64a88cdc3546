"""The expert layer's 8-bit handles without a GPU: tensors that a kernel must not get
are refused before the library is called."""
from __future__ import annotations

import gc
import weakref

import pytest
import torch

import weight_only_quantized_mlx_b200 as mq
from test_mx4_host import E, H, I, code_of, moe8


def view(rows, cols, gs=64, **other):
    t = dict(packed=torch.zeros(rows, cols // 4, dtype=torch.int32), scales=torch.zeros(rows, cols // gs, dtype=torch.bfloat16),
             biases=torch.zeros(rows, cols // gs, dtype=torch.bfloat16))
    t.update(other)
    return mq.weight_view(t["packed"], t["scales"], t["biases"], gs)


def shape(name):
    return (E * H, I) if name == "down" else (E * I, H)


@pytest.fixture
def called(monkeypatch):
    """The library's call, noted and not made."""
    calls = []

    class Library:
        mlxq_moe = staticmethod(lambda *a: calls.append(a) or 0)
        mlxq_last_error = staticmethod(lambda: b"")
    monkeypatch.setattr(mq, "lib", lambda: Library)
    return calls


@pytest.mark.parametrize("name", ["gate", "up", "down"])
def test_weights_on_another_device_are_refused(name, monkeypatch, called):
    monkeypatch.setattr(mq, "_current_device", lambda: 0)
    assert code_of(lambda: moe8(**{name: view(*shape(name))})) == mq.MLXQ_ERR_INVALID_ARG
    assert not called


@pytest.mark.parametrize("name", ["gate", "up", "down"])
def test_weights_that_are_not_whole_are_refused(name, monkeypatch, called):
    monkeypatch.setattr(mq, "_current_device", lambda: -1)  # where host tensors are
    N, K = shape(name)
    bf = dict(dtype=torch.bfloat16)
    bad = [dict(packed=torch.zeros(N, K // 2, dtype=torch.int32)[:, ::2]), dict(packed=torch.zeros(N, K // 4, dtype=torch.int64)),
           dict(scales=torch.zeros(1, K // 64, **bf).expand(N, -1)), dict(scales=torch.zeros(N, K // 64)),
           dict(biases=torch.zeros(N - 1, K // 64, **bf)), dict(biases=torch.zeros(N, K // 64, device="meta", **bf))]
    for other in bad:
        assert code_of(lambda: moe8(**{name: view(N, K, **other)})) == mq.MLXQ_ERR_INVALID_ARG, other
    assert not called
    moe8(**{name: view(N, K)})
    assert len(called) == 1


def test_a_view_keeps_its_tensors():
    h = view(8, 64)
    ref = weakref.ref(h.tensors[1])
    gc.collect()
    assert ref() is not None and h.scales == ref().data_ptr()


def test_numbers_past_32_bits_are_refused(called, monkeypatch):
    """The C side's numbers are 32 bits wide: what does not fit must not come out as another number."""
    big = 2 ** 32 + 64
    meta = lambda *s: torch.empty(*s, dtype=torch.int32, device="meta")
    bytes_ = lambda *s: torch.empty(*s, dtype=torch.uint8, device="meta")
    assert code_of(mq.mx4_view, meta(big, 4), bytes_(big, 1)) == mq.MLXQ_ERR_SHAPE
    assert code_of(mq.mx4_view, meta(1, big // 8), bytes_(1, big // 32)) == mq.MLXQ_ERR_SHAPE
    wide = torch.empty(2 ** 32 + 1, 1, dtype=torch.bfloat16, device="meta")
    tall = mq.weight_view(meta(2 ** 32 + 1, 16), wide, wide, 64)
    assert tall.problem is not None
    for kw in (dict(m=2 ** 32 + 3), dict(m=-1), dict(top_k=2 ** 32 + 2), dict(experts=2 ** 32 + E), dict(flags=2 ** 32)):
        assert code_of(lambda: moe8(**kw)) == mq.MLXQ_ERR_INVALID_ARG, kw
    assert not called


def test_mx4_gemm_rows_past_32_bits_are_refused():
    for m in (2 ** 32, 2 ** 32 + 1, -(2 ** 32) + 1):
        assert code_of(mq.mlxq_mx4_gemm, mq.mlxq_mx4(1 << 20, 2 << 20, 64, 64), 4 << 20, 8 << 20, m, 0) == mq.MLXQ_ERR_INVALID_ARG
    for args in ((2 ** 32 + 64, 64, 2, 2), (64, 2 ** 32 + 64, 2, 2), (64, 64, 2 ** 32 + 2, 2), (64, 64, 2, 2 ** 32 + 2), (64, 64, 2, -1)):
        assert mq.mlxq_moe_workspace_bytes(*args) == 0
