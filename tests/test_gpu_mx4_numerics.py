"""GPU numerics of the MX4 gemm at the documented bound of its activations."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import synth
import weight_only_quantized_mlx_b200 as mq
import _mx4_ref as ref
from _helpers import bits_to_f64, dev, host_bits
from test_gpu_mx4 import bound, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    mq.lib()
    yield
    torch.cuda.synchronize()
    mq.mlxq_device_status()


@pytest.mark.parametrize("least", [24, 31, 36, 44])
@pytest.mark.parametrize("m,K", [(1, 416), (3, 1312), (8, 1312), (4, 36864), (18, 1312), (50, 1312)])
def test_gemm_activations_far_below_their_rows_largest(m, K, least):
    """The largest activations meet zero codes, so that only the small ones are in the sum: values down to 2^-31
    of their row's largest are whole, smaller ones off by at most 2^-39 of it."""
    N = 90
    g, codes, scales, _ = make(40, N, K)
    top = g.choice(K, 5, replace=False)
    codes[:, top] = 0
    h = mq.mx4_view(dev(ref.pack(codes)), dev(scales))
    w = ref.values(codes, scales)
    v = g.uniform(1, 2, (m, K)) * np.sign(g.standard_normal((m, K))) * 2.0 ** -g.integers(least - 8, least + 1, (m, K))
    v[:, top] = g.uniform(-1.9, 1.9, (m, 5))
    v[:, top[0]] = 1.0
    xb = synth.to_bf16_bits(v * 2.0 ** g.integers(-60, 60, (m, 1)))
    x = bits_to_f64(xb)
    y = torch.empty(m, N, dtype=torch.bfloat16, device="cuda")
    mq.mlxq_mx4_gemm(h, dev(xb), y, m)
    want = x @ w.T
    largest = np.abs(x).max(axis=1, keepdims=True)
    # what 2^-39 of the largest may change: nothing in values that are whole
    lost = np.where(np.abs(x) < 2.0 ** -31 * largest, 2.0 ** -39 * largest, 0.0) @ np.abs(w).T
    small = x.copy()
    small[:, top] = 0  # products with zero codes are zero
    err = np.abs(bits_to_f64(host_bits(y)) - want)
    assert np.all(err <= bound(np.abs(w), np.abs(small) + 2.0 ** -39 * largest, want, K) + lost + 2.0 ** -8 * lost)


@pytest.mark.parametrize("m", [1, 8, 20])
@pytest.mark.parametrize("byte", [0, 3, 40])
@pytest.mark.parametrize("top", [127, 60, 20])
def test_gemm_least_scales_with_large_activations(m, byte, top):
    """Scales down to 2^-127 with activations up to 2^127, the largest under zero codes: the small ones' products
    with the scale alone would be fp32 subnormals."""
    N, K = 400, 32  # few terms: the bound leaves little
    g, codes, scales, _ = make(41, N, K)
    codes[:, 7] = 0
    scales[:] = byte + g.integers(0, 2, scales.shape)
    h = mq.mx4_view(dev(ref.pack(codes)), dev(scales))
    w = ref.values(codes, scales)
    v = g.uniform(1, 1.9, (m, K)) * np.sign(g.standard_normal((m, K))) * 2.0 ** (top - 30)
    v[:, 7] = 1.5 * 2.0 ** top
    xb = synth.to_bf16_bits(v)
    x = bits_to_f64(xb)
    y = torch.empty(m, N, dtype=torch.bfloat16, device="cuda")
    mq.mlxq_mx4_gemm(h, dev(xb), y, m)
    want = x @ w.T
    x[:, 7] = 0
    err = np.abs(bits_to_f64(host_bits(y)) - want)
    # (2^-133: the last place of a BF16 result below 2^-126)
    assert np.all(err <= bound(np.abs(w), np.abs(x), want, K) + 2.0 ** -133)


@pytest.mark.parametrize("wlow,alow", [(0, 235), (235, 0), (60, 60), (160, 160), (100, 150)])
@pytest.mark.parametrize("m,N,K", [(20, 300, 544), (300, 520, 512)])
def test_matmul_scales_at_the_ends_of_the_range(m, N, K, wlow, alow):
    """Scales of both operands from 2^-127 to 2^127 whose products fp32 holds."""
    g, wc, ws, w = make(42, N, K, low=wlow, high=wlow + 20)
    ac, as_ = ref.random_weight(g, m, K, low=alow, high=alow + 20)
    y = torch.empty(m, N, dtype=torch.bfloat16, device="cuda")
    mq.mlxq_mx4_matmul(w, mq.mx4_view(dev(ref.pack(ac)), dev(as_)), y)
    wv, av = ref.values(wc, ws), ref.values(ac, as_)
    want = av @ wv.T
    err = np.abs(bits_to_f64(host_bits(y)) - want)
    # (2^-133: the last place of a BF16 result below 2^-126; 2^-149: fp32's)
    assert np.all(err <= bound(np.abs(wv), np.abs(av), want, K) + 2.0 ** -133 + K * 2.0 ** -149)
