"""MX4 and the expert layer without a GPU: pins of the plain reference, and the
calls' refusals (each is returned before any launch)."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

import _mx4_ref as ref
import weight_only_quantized_mlx_b200 as mq
from _helpers import bits_to_f64
from synth import to_bf16_bits

P = 1 << 20  # aligned addresses that nothing reads: every call below fails its checks


def code_of(call, *args):
    with pytest.raises(mq.MlxqError) as e:
        call(*args)
    return e.value.code


# ---- the plain reference ---------------------------------------------------------------
def test_reference_quantizes_the_grid_to_itself():
    row = np.concatenate([ref.GRID, -ref.GRID, ref.GRID, -ref.GRID]) * 2.0 ** -3
    codes, scales = ref.quantize(to_bf16_bits(row[None, :]))
    assert scales.tolist() == [[124]]  # max 6 / 8: floor(log2) - 2 = -3
    assert codes[0, :16].tolist() == list(range(16))
    assert np.array_equal(ref.values(codes, scales)[0], row)


def test_reference_ties_go_to_the_even_code():
    # under scale 1 (max 4): borders .25 .75 1.25 1.75 2.5 3.5 5, and what saturates
    row = np.zeros(32)
    row[:9] = [4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.75]
    codes, scales = ref.quantize(to_bf16_bits(row[None, :]))
    assert scales.tolist() == [[127]]
    assert codes[0, :9].tolist() == [6, 0, 2, 2, 4, 4, 6, 6, 7]


def test_reference_scale_ends():
    rows = np.zeros((4, 32), np.uint16)
    rows[1, 3] = 1          # the smallest subnormal
    rows[2, 3] = 0x7F7F     # the largest BF16
    rows[3, 3] = 0xFF80     # -inf
    codes, scales = ref.quantize(rows)
    assert scales[:, 0].tolist() == [0, 0, 252, 255]
    assert codes[1, 3] == 0 and codes[2, 3] == 7 and not codes[3].any()
    assert np.isnan(ref.values(codes, scales)[3]).all()


def test_reference_packing_is_low_nibble_first():
    assert ref.pack(np.array([[1, 2, 3, 4, 5, 6, 7, 8]], np.uint8))[0, 0] == 0x87654321


def test_reference_layer_of_one_expert_is_a_gated_mlp():
    g = torch.Generator().manual_seed(1)
    x, r = torch.randn(3, 8, generator=g).double(), torch.randn(1, 8, generator=g).double()
    a, b, c = (torch.randn(1, *s, generator=g).double() for s in ((6, 8), (6, 8), (8, 6)))
    y, ids, _ = ref.moe(x, r, a, b, c, 1, True)
    assert ids.tolist() == [[0]] * 3
    want = (torch.nn.functional.silu(x @ a[0].t()) * (x @ b[0].t())) @ c[0].t()
    assert torch.allclose(y, want, rtol=1e-12, atol=1e-12)


# ---- handles ---------------------------------------------------------------------------
def test_handles_check_their_tensors():
    codes, scales = torch.zeros(4, 8, dtype=torch.int32), torch.zeros(4, 2, dtype=torch.uint8)
    h = mq.mx4_view(codes, scales)
    assert (h.rows, h.cols) == (4, 64) and h.tensors[0] is codes
    assert code_of(mq.mx4_view, codes, scales[:, :1]) == mq.MLXQ_ERR_SHAPE
    assert code_of(mq.mx4_view, codes.to(torch.int64), scales) == mq.MLXQ_ERR_SHAPE
    assert code_of(mq.mx4_view, torch.zeros(8, 4, dtype=torch.int32).t(), scales) == mq.MLXQ_ERR_INVALID_ARG
    assert code_of(mq.mx4_empty, 4, 40, "cpu") == mq.MLXQ_ERR_SHAPE


def handle(rows=64, cols=64, codes=P, scales=2 * P):
    return mq.mlxq_mx4(codes, scales, rows, cols)


@pytest.mark.parametrize("call", ["quantize", "dequant", "gemm"])
def test_mx4_calls_check_the_handle(call):
    def run(h):
        if call == "quantize":
            mq.mlxq_mx4_quantize(4 * P, h, 0)
        elif call == "dequant":
            mq.mlxq_mx4_dequant(h, 4 * P, 0)
        else:
            mq.mlxq_mx4_gemm(h, 4 * P, 8 * P, 1, 0)
    assert code_of(run, handle(cols=48)) == mq.MLXQ_ERR_SHAPE
    assert code_of(run, handle(codes=None)) == mq.MLXQ_ERR_INVALID_ARG
    assert code_of(run, handle(scales=None)) == mq.MLXQ_ERR_INVALID_ARG
    assert code_of(run, handle(codes=P + 8)) == mq.MLXQ_ERR_INVALID_ARG
    assert code_of(run, handle(scales=2 * P + 2)) == mq.MLXQ_ERR_INVALID_ARG
    assert code_of(run, handle(rows=0xFFFFFFFF, cols=0xFFFFFFE0)) == mq.MLXQ_ERR_SHAPE


def test_quantize_and_dequant_check_their_buffers():
    bad = mq.MLXQ_ERR_INVALID_ARG
    assert code_of(mq.mlxq_mx4_quantize, None, handle(), 0) == bad
    assert code_of(mq.mlxq_mx4_quantize, 4 * P + 1, handle(), 0) == bad
    assert code_of(mq.mlxq_mx4_quantize, P - 64, handle(), 0) == bad      # x over the codes
    assert code_of(mq.mlxq_mx4_quantize, 2 * P, handle(), 0) == bad       # x over the scales
    assert code_of(mq.mlxq_mx4_quantize, 4 * P, handle(scales=P + 16), 0) == bad  # scales inside the codes
    assert code_of(mq.mlxq_mx4_dequant, handle(), None, 0) == bad
    assert code_of(mq.mlxq_mx4_dequant, handle(), 4 * P + 1, 0) == bad
    assert code_of(mq.mlxq_mx4_dequant, handle(), P + 2, 0) == bad


def test_gemm_checks_its_buffers():
    bad = mq.MLXQ_ERR_INVALID_ARG
    assert code_of(mq.mlxq_mx4_gemm, handle(), 4 * P, 8 * P, 65, 0) == mq.MLXQ_ERR_UNSUPPORTED
    assert code_of(mq.mlxq_mx4_gemm, handle(), None, 8 * P, 1, 0) == bad
    assert code_of(mq.mlxq_mx4_gemm, handle(), 4 * P, None, 1, 0) == bad
    assert code_of(mq.mlxq_mx4_gemm, handle(), 4 * P + 2, 8 * P, 1, 0) == bad   # X not 16-byte aligned
    assert code_of(mq.mlxq_mx4_gemm, handle(), 4 * P, 4 * P + 64, 1, 0) == bad  # Y over X
    assert code_of(mq.mlxq_mx4_gemm, handle(), 4 * P, P, 1, 0) == bad           # Y over the codes
    mq.mlxq_mx4_gemm(handle(), None, None, 0, 0)  # m == 0: nothing to do


def test_matmul_checks_its_buffers():
    bad = mq.MLXQ_ERR_INVALID_ARG
    a = handle(rows=8, codes=16 * P, scales=17 * P)
    c = lambda w, a, y: code_of(mq.mlxq_mx4_matmul, w, a, y, 0)
    assert c(handle(), handle(cols=96, codes=16 * P, scales=17 * P), 8 * P) == mq.MLXQ_ERR_SHAPE
    assert c(handle(cols=40), a, 8 * P) == mq.MLXQ_ERR_SHAPE
    assert c(handle(), handle(codes=None), 8 * P) == bad
    assert c(handle(codes=P + 4), a, 8 * P) == bad
    assert c(handle(), a, None) == bad
    assert c(handle(), a, 8 * P + 1) == bad
    assert c(handle(), a, P + 16) == bad       # Y over the weight
    assert c(handle(), a, 17 * P) == bad       # Y over the activations' scales
    assert c(handle(rows=(1 << 30) + 1, cols=32, codes=1 << 40, scales=1 << 41), handle(8, 32), 8 * P) == mq.MLXQ_ERR_UNSUPPORTED
    mq.mlxq_mx4_matmul(handle(), handle(rows=0), None, 0)


def test_tensor_arguments_must_be_dense_and_typed():
    h = handle(4, 64)
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    assert code_of(mq.mlxq_mx4_quantize, x.float(), h, 0) == mq.MLXQ_ERR_INVALID_ARG
    assert code_of(mq.mlxq_mx4_quantize, torch.zeros(64, 4, dtype=torch.bfloat16).t(), h, 0) == mq.MLXQ_ERR_INVALID_ARG
    assert code_of(mq.mlxq_mx4_quantize, x[:3], h, 0) == mq.MLXQ_ERR_INVALID_ARG
    assert code_of(mq.mlxq_mx4_gemm, h, x[:, ::2], x, 2, 0) == mq.MLXQ_ERR_INVALID_ARG
    assert code_of(mq.mlxq_mx4_dequant, h, x.half(), 0) == mq.MLXQ_ERR_INVALID_ARG


# ---- the expert layer --------------------------------------------------------------------
class Fake:
    """A workspace tensor's face."""
    def __init__(self, ptr, n):
        self.ptr, self.n = ptr, n

    def data_ptr(self):
        return self.ptr

    def is_contiguous(self):
        return True

    def numel(self):
        return self.n

    def element_size(self):
        return 1


E, H, I = 4, 128, 64
A = [i * (1 << 24) for i in range(1, 12)]


def moe8(gs=64, experts=E, top_k=2, m=3, flags=0, hidden=H, inter=I, gate=None, up=None, down=None, router=A[9],
         x=A[7], y=A[8], ws=None):
    w = lambda base, rows, cols: mq.mlxq_weight(base, base + (1 << 20), base + (1 << 21), rows, cols, gs, 0)
    g = gate or w(A[0], E * inter, hidden)
    u = up or w(A[1], E * inter, hidden)
    d = down or w(A[2], E * hidden, inter)
    mq.mlxq_moe(router, g, u, d, experts, top_k, x, y, m, ws or Fake(A[10], 1 << 20), 0, flags)


def moe4(experts=E, top_k=2, m=3, flags=0, hidden=H, inter=I, gate=None, up=None, down=None, router=A[9], x=A[7], y=A[8],
         ws=None):
    w = lambda base, rows, cols: mq.mlxq_mx4(base, base + (1 << 20), rows, cols)
    g = gate or w(A[0], E * inter, hidden)
    u = up or w(A[1], E * inter, hidden)
    d = down or w(A[2], E * hidden, inter)
    mq.mlxq_mx4_moe(router, g, u, d, experts, top_k, x, y, m, ws or Fake(A[10], 1 << 20), 0, flags)


@pytest.mark.parametrize("call", [moe8, moe4])
def test_moe_refusals(call):
    bad, no, shape = mq.MLXQ_ERR_INVALID_ARG, mq.MLXQ_ERR_UNSUPPORTED, mq.MLXQ_ERR_SHAPE
    c = lambda **k: code_of(lambda: call(**k))
    assert c(experts=0) == no and c(experts=257) == no
    assert c(top_k=0) == no and c(top_k=5) == no
    assert c(m=65) == no
    assert c(flags=2) == bad
    assert c(experts=3) == shape
    assert c(hidden=H + 16) in (no, shape, mq.MLXQ_ERR_GROUP_SIZE)
    assert c(router=None) == bad and c(router=A[9] + 2) == bad
    assert c(x=None) == bad and c(x=A[7] + 8) == bad
    assert c(y=None) == bad and c(y=A[8] + 1) == bad
    assert c(y=A[7] + 16) == bad          # y over x
    assert c(y=A[2]) == bad               # y over the down codes
    assert c(ws=Fake(A[10] + 8, 1 << 20)) == bad
    assert c(ws=Fake(A[10], 1024)) == bad  # too small
    assert c(ws=Fake(A[7] - 256, 1 << 20)) == bad  # workspace over x
    assert c(ws=Fake(A[1], 1 << 20)) == bad        # workspace over the up codes
    call(m=0)                              # nothing to do


def test_moe8_refuses_what_its_kernels_do_not_take():
    w = lambda base, rows, cols, gs: mq.mlxq_weight(base, base + (1 << 20), base + (1 << 21), rows, cols, gs, 0)
    c = lambda **k: code_of(lambda: moe8(**k))
    assert c(gs=16) == mq.MLXQ_ERR_UNSUPPORTED
    assert c(hidden=96, gs=32) == mq.MLXQ_ERR_UNSUPPORTED
    assert c(up=w(A[1], E * I, H, 32)) == mq.MLXQ_ERR_GROUP_SIZE
    assert c(up=w(A[1], E * I, 2 * H, 64)) == mq.MLXQ_ERR_SHAPE
    assert c(down=w(A[2], E * H + 1, I, 64)) == mq.MLXQ_ERR_SHAPE
    assert c(gate=w(A[0] + 4, E * I, H, 64)) == mq.MLXQ_ERR_INVALID_ARG


def test_moe_workspace_size():
    n = mq.mlxq_moe_workspace_bytes(H, I, 2, 3)
    assert n >= 256 + 6 * (4 + 4 + 2 * I)
    assert mq.mlxq_moe_workspace_bytes(4096, 14336, 16, 64) >= 64 * 16 * 14336 * 2


def test_moe_workspace_of_sizes_out_of_range_is_nothing():
    top = 0xFFFFFFFF
    for args in ((top, 64, 2, 2), (64, top, 2, 2), (64, 64, top, top), (64, 64, 17, 1), (64, 64, 2, 65)):
        assert mq.mlxq_moe_workspace_bytes(*args) == 0


def test_tensors_of_another_device_are_refused(monkeypatch):
    """Host tensors while the current device is a GPU: refused before anything is launched."""
    monkeypatch.setattr(mq, "_current_device", lambda: 0)
    bad = mq.MLXQ_ERR_INVALID_ARG
    host = mq.mx4_empty(4, 64, "cpu")
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    calls = [lambda h, t: mq.mlxq_mx4_quantize(t, h, 0), lambda h, t: mq.mlxq_mx4_dequant(h, t, 0),
             lambda h, t: mq.mlxq_mx4_gemm(h, t, 8 * P, 1, 0), lambda h, t: mq.mlxq_mx4_gemm(h, 4 * P, t, 1, 0),
             lambda h, t: mq.mlxq_mx4_matmul(h, handle(rows=1, codes=16 * P, scales=17 * P), t, 0),
             lambda h, t: mq.mlxq_mx4_matmul(handle(rows=1, codes=16 * P, scales=17 * P), h, t, 0)]
    for call in calls:
        assert code_of(call, handle(4, 64), x) == bad
        assert code_of(call, host, 4 * P) == bad
    host_ws = Fake(A[10], 1 << 20)
    host_ws.device, host_ws.get_device = "cpu", lambda: -1
    for call in (moe8, moe4):
        for k in ({"router": torch.zeros(E, H, dtype=torch.bfloat16)}, {"x": torch.zeros(3, H, dtype=torch.bfloat16)},
                  {"y": torch.zeros(3, H, dtype=torch.bfloat16)}, {"ws": host_ws}):
            assert code_of(lambda: call(**k)) == bad
    assert code_of(lambda: moe4(gate=mq.mx4_empty(E * I, H, "cpu"))) == bad


def test_struct_layout():
    assert ctypes.sizeof(mq.mlxq_mx4) == 24
