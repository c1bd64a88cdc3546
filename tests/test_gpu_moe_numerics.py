"""GPU numerics of the expert layer beyond its parity tests: how h = p silu(g) u is
held between the projections, sums over the experts, ties and ends of the ranges."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import _mx4_ref as ref
import synth
import weight_only_quantized_mlx_b200 as mq
from _helpers import dev
from test_gpu_moe import Layer, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    mq.lib()
    yield
    torch.cuda.synchronize()
    mq.mlxq_device_status()


def layer_of_integers(seed, E, H, I, group):
    """Experts whose gate and up sums over small integers are exact in fp32 in any order."""
    L = Layer(seed, E, H, I, group)
    L.handles, L.values, L.keep = [], [], []
    for rows, cols in ((E * I, H), (E * I, H), (E * H, I)):
        if group:  # (q - 128) 2^-k
            k = 2.0 ** -round(math.log2(74 * math.sqrt(cols)))
            q = L.g.integers(0, 256, (rows, cols)).astype(np.uint32)
            p = (q.reshape(rows, -1, 4) << (8 * np.arange(4, dtype=np.uint32))).sum(axis=-1, dtype=np.uint32)
            s = np.full((rows, cols // group), k)
            L.keep.append((dev(p), dev(synth.to_bf16_bits(s)), dev(synth.to_bf16_bits(-128.0 * s))))
            L.handles.append(mq.weight_view(*L.keep[-1], group))
            v = (q.astype(np.float64) - 128.0) * k
        else:
            e = 127 + round(math.log2(1 / (2.9 * math.sqrt(cols))))
            codes, scales = ref.random_weight(L.g, rows, cols, low=e, high=e + 1)
            L.handles.append(mq.mx4_view(dev(ref.pack(codes)), dev(scales)))
            v = ref.values(codes, scales)
        L.values.append(torch.from_numpy(v).cuda().reshape(E, -1, cols))
    return L


@pytest.mark.parametrize("group", [64, 0], ids=["gs64", "mx4"])
@pytest.mark.parametrize("m,k", [(1, 1), (4, 1), (5, 2), (8, 1), (12, 1), (64, 1), (64, 2)])
def test_h_is_held_to_eleven_bits(m, k, group):
    """Gate and up are exact here, so what is off beside y's own rounding is how h is held."""
    E, H, I = 4, 64, 64
    L = layer_of_integers(50 + m, E, H, I, group)
    xb = synth.to_bf16_bits(L.g.integers(-4, 5, (m, H)).astype(np.float64))
    y = L.run(dev(xb), k).double()
    x = f64(xb)
    gate, up, down = L.values
    logits = x @ f64(L.router_bits).t()
    ids = torch.sort(logits, dim=1, descending=True, stable=True)[1][:, :k]
    want, slack = torch.zeros_like(x), torch.zeros_like(x)
    # fp32 sums on the tensor pipe: each of the MMAs (16 products, h in up to two parts) loses at most 2^-22 of the magnitudes
    gi = (2 * k * I / 16 + 32) * 2.0 ** -22
    for t in range(m):
        w = torch.exp(logits[t] - logits[t].max())
        for e in ids[t].tolist():
            g, u = gate[e] @ x[t], up[e] @ x[t]
            h = w[e] / w[ids[t]].sum() * g / (1 + torch.exp(-g)) * u
            # 2^-11: h as FP16 (as two BF16 parts 2^-16); 2^-39 of the largest: below FP16's normal numbers;
            # 2^-18: expf, the division, p and the products
            dh = (2.0 ** -11 + 2.0 ** -18) * h.abs() + 2.0 ** -39 * h.abs().max()
            want[t] += down[e] @ h
            slack[t] += down[e].abs() @ (dh + gi * h.abs())
    off = (y - want).abs()
    assert (off <= slack + 2.0 ** -8 * (want.abs() + slack)).all()
    # y's rounding: at most 2^-8, 2^-8 / sqrt(3) in the mean; h's the same with 2^-11
    assert float(off.norm() / want.norm()) <= math.hypot(2.0 ** -8, 2.0 ** -11) / math.sqrt(3)


def routed(L, choices):
    """Activations that send token t to the experts choices[t] (the first E columns are the router's)."""
    m, E = len(choices), L.E
    L.router.zero_()
    L.router[:, :E] = 8 * torch.eye(E, device="cuda")
    x = dev(synth.activations(L.g, m, L.H))
    x[:, :E] = 0
    for t, experts in enumerate(choices):
        x[t, list(experts)] = 8.0
    return x


# tokens of the bad expert, of the one behind it, and of all; choices of a token
@pytest.mark.parametrize("bad,behind,m,k", [(9, 16, 16, 2), (11, 32, 64, 1), (17, 32, 64, 1), (20, 32, 64, 1), (24, 31, 64, 1),
                                            (28, 32, 64, 1), (3, 7, 8, 2)])
@pytest.mark.parametrize("group", [64, 0], ids=["gs64", "mx4"])
def test_a_bad_expert_ahead_of_a_fuller_one(bad, behind, m, k, group):
    """A NaN expert whose tokens do not fill its column tiles, followed by one with more: three hit
    experts of 64 steps, so that every warp of the down phase walks through all of them."""
    E, H, I = 3, 64, 4096 if group else 8192
    L = Layer(60, E, H, I, group)
    if k == 1:
        choices = [(0,) if t < bad else (1,) if t < bad + behind else (2,) for t in range(m)]
    else:  # the first tokens choose expert 0, the last ones expert 1, and all that are left expert 2
        choices = [tuple((([0] if t < bad else []) + ([1] if t >= m - behind else []) + [2])[:2]) for t in range(m)]
    x = routed(L, choices)
    clean = L.run(x, k)
    assert torch.isfinite(clean.float()).all()
    if group:
        L.keep[2][1][:H] = float("nan")
    else:
        L.handles[2].tensors[1][:H] = 255
    y = L.run(x, k)
    for t in range(m):
        if 0 in choices[t]:
            assert not torch.isfinite(y[t].float()).any(), t
        else:
            assert torch.equal(y[t], clean[t]), t


@pytest.mark.parametrize("E", [2, 9, 12, 15, 20, 36, 68, 130])
@pytest.mark.parametrize("m", [1, 20, 40])
def test_equal_router_rows_take_the_lowest_experts(E, m):
    """Equal rows that are not zero: an expert's logit does not depend on the block that sums it."""
    H, I, k = 4096, 32, min(E, 3)
    L = Layer(70, 1, H, I, 0)
    g = synth.rng(70 + E)
    weights = [mq.mx4_view(*(torch.cat([t] * E) for t in h.tensors)) for h in L.handles]  # E times the same expert
    weights[2].tensors[1].view(E, -1)[k:] = 255  # but for NaN where another than the lowest k is chosen
    ws = torch.empty(mq.mlxq_moe_workspace_bytes(H, I, k, m), dtype=torch.uint8, device="cuda")
    for _ in range(6):
        router = dev(np.repeat(synth.to_bf16_bits(g.standard_normal((1, H)) / 16), E, axis=0))
        x = dev(synth.activations(g, m, H))
        y = torch.empty(m, H, dtype=torch.bfloat16, device="cuda")
        mq.mlxq_mx4_moe(router, *weights, E, k, x, y, m, ws)
        assert torch.isfinite(y.float()).all()


@pytest.mark.parametrize("low,high", [(250, 255), (0, 255), (124, 134)])
@pytest.mark.parametrize("m", [1, 4, 7, 40])
def test_down_scales_at_the_ends_of_the_range(m, low, high):
    """Down weights up to 6 * 2^127, beyond BF16 and fp32, times an h so small that the products are not."""
    E, H, I, k = 4, 96, 288, 2
    L = Layer(80, E, H, I, 0)
    L.handles, L.values = [], []
    # h near 2^-110: the up weights are that small
    for rows, cols, ends in ((E * I, H, (121, 124)), (E * I, H, (14, 17)), (E * H, I, (low, high))):
        codes, scales = ref.random_weight(L.g, rows, cols, *ends)
        L.handles.append(mq.mx4_view(dev(ref.pack(codes)), dev(scales)))
        L.values.append(torch.from_numpy(ref.values(codes, scales)).cuda().reshape(E, -1, cols))
    xb = synth.activations(L.g, m, H)
    want, _, err = L.reference(xb, k)
    assert torch.isfinite(want).all()
    y = L.run(dev(xb), k).double()
    # (2^-133: the last place of a BF16 result below 2^-126; a BF16 part below it is off by up to 2^-134)
    small = 2.0 ** -133 + sum(2.0 ** -134 * v.abs().sum(-1).amax(0) for v in [L.values[2]]) * k
    assert torch.isfinite(y).all() and ((y - want).abs() <= err + small).all()


@pytest.mark.parametrize("m", [2, 9])
def test_no_product_times_the_largest_scales_is_zero(m):
    """h = 0 times the largest down weights: zero, not NaN."""
    E, H, I, k = 2, 64, 64, 1
    L = Layer(81, E, H, I, 0)
    L.handles[1].tensors[0].zero_()  # up
    L.handles[2].tensors[1].fill_(254)
    assert not L.run(dev(synth.activations(L.g, m, H)), k).any()


@pytest.mark.parametrize("group", [64, 0], ids=["gs64", "mx4"])
@pytest.mark.parametrize("m", [3, 6, 20, 64])
def test_tokens_of_very_different_sizes(m, group):
    """Each slot's h has a size of its own, from 2^-40 to 2^40 of the others."""
    E, H, I, k = 5, 128, 192, 2
    L = Layer(90, E, H, I, group)
    x32 = synth.bf16_bits_to_f32(synth.activations(L.g, m, H)) * np.float32(2.0) ** L.g.integers(-20, 21, (m, 1)).astype(np.float32)
    xb = synth.to_bf16_bits(x32)
    want, _, err = L.reference(xb, k)
    y = L.run(dev(xb), k).double()
    assert torch.isfinite(y).all() and ((y - want).abs() <= err).all()


@pytest.mark.parametrize("m", [6, 24])
@pytest.mark.parametrize("bad", [0x7FC0, 0x7F80])
@pytest.mark.parametrize("group", [64, 0], ids=["gs64", "mx4"])
def test_a_bad_token_leaves_the_others_bits(m, bad, group):
    L = Layer(91, 6, 128, 160 if group == 0 else 128, group)
    xb = synth.activations(L.g, m, 128)
    clean = L.run(dev(xb), 2)
    xb[2, 9] = bad
    y = L.run(dev(xb), 2)
    keep = [t for t in range(m) if t != 2]
    assert torch.equal(y[keep], clean[keep]) and not torch.isfinite(y[2].float()).any()
