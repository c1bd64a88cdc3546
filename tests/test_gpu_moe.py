"""GPU parity of the expert layer against a plain 64-bit form: 8-bit and MX4
experts, from one token and one expert to 64 tokens and 256 experts."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import _mx4_ref as ref
import oracle
import synth
import weight_only_quantized_mlx_b200 as mq
from _helpers import NORM_REL, bits_to_f64, dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    mq.lib()
    yield
    torch.cuda.synchronize()
    mq.mlxq_device_status()


def f64(bits):
    return torch.from_numpy(bits_to_f64(bits)).cuda()


class Layer:
    """Random experts in the 8-bit (group > 0) or the MX4 format, and their values."""

    def __init__(self, seed, E, H, I, group):
        g = synth.rng(seed)
        self.E, self.H, self.I, self.group = E, H, I, group
        self.handles, self.values, self.keep = [], [], []
        for rows, cols in ((E * I, H), (E * I, H), (E * H, I)):
            if group:
                p, s, b = synth.weight(g, rows, cols, group)
                # spread about 1 / sqrt(cols): the draw's is 0.29
                k = 2.0 ** round(math.log2(1 / (0.29 * math.sqrt(cols))))
                s, b = (synth.to_bf16_bits(synth.bf16_bits_to_f32(t) * np.float32(k)) for t in (s, b))
                self.keep.append((dev(p), dev(s), dev(b)))
                self.handles.append(mq.weight_view(*self.keep[-1], group))
                v = f64(oracle.dequant(p, s, b, group))
            else:
                e = 127 + round(math.log2(1 / (2.9 * math.sqrt(cols))))
                codes, scales = ref.random_weight(g, rows, cols, low=e - 1, high=e + 2)
                self.handles.append(mq.mx4_view(dev(ref.pack(codes)), dev(scales)))
                v = torch.from_numpy(ref.values(codes, scales)).cuda()
            self.values.append(v.reshape(E, -1, cols))
        self.router_bits = synth.to_bf16_bits(g.standard_normal((E, H)) * 2 / math.sqrt(H))
        self.router = dev(self.router_bits)
        self.g = g

    def workspace(self, top_k, m, fill=0xFF):
        return torch.full((mq.mlxq_moe_workspace_bytes(self.H, self.I, top_k, m),), fill, dtype=torch.uint8, device="cuda")

    def run(self, x, top_k, renorm=True, ws=None, y=None, stream=None):
        m = x.shape[0]
        ws = self.workspace(top_k, m) if ws is None else ws
        y = torch.full((m, self.H), float("nan"), dtype=torch.bfloat16, device="cuda") if y is None else y
        call = mq.mlxq_moe if self.group else mq.mlxq_mx4_moe
        call(self.router, *self.handles, self.E, top_k, x, y, m, ws, stream, 0 if renorm else mq.MLXQ_MOE_SOFTMAX_ALL)
        return y

    def reference(self, xb, top_k, renorm=True):
        return ref.moe(f64(xb), f64(self.router_bits), *self.values, top_k, renorm)


def check(y, want, err):
    y = y.double()
    assert torch.isfinite(y).all()
    off = (y - want).abs()
    assert (off <= err).all(), f"worst {float((off / err).max())} of the bound"
    # two roundings to BF16 (h, y), each of at most 2^-8 and 2^-8 / sqrt(3) in
    # the mean: sqrt(2) 2^-8 / sqrt(3) = 3.2e-3
    assert float((y - want).norm() / want.norm()) <= NORM_REL


# (m, E, H, I, top_k, renorm)
SHAPES = [(1, 1, 64, 64, 1, True), (1, 8, 512, 1024, 2, True), (1, 64, 256, 192, 8, False), (2, 3, 128, 64, 3, False),
          (7, 16, 320, 128, 4, True), (8, 256, 64, 64, 16, True), (9, 4, 192, 256, 2, True), (16, 32, 256, 448, 4, False),
          (17, 8, 128, 64, 8, True), (33, 130, 256, 64, 8, True), (64, 2, 448, 320, 1, True), (64, 256, 128, 64, 16, False),
          (64, 5, 1024, 640, 3, True)]


@pytest.mark.parametrize("group", [32, 64, 0], ids=["gs32", "gs64", "mx4"])
@pytest.mark.parametrize("m,E,H,I,k,renorm", SHAPES)
def test_layer(m, E, H, I, k, renorm, group):
    L = Layer(m + E, E, H, I, group)
    xb = synth.activations(L.g, m, H)
    want, _, err = L.reference(xb, k, renorm)
    check(L.run(dev(xb), k, renorm), want, err)


@pytest.mark.parametrize("m,E,H,I,k", [(1, 4, 32, 96, 2), (3, 7, 160, 32, 2), (20, 6, 288, 224, 3), (50, 9, 2080, 96, 2)])
def test_layer_mx4_odd_blocks(m, E, H, I, k):
    """hidden and inter that are odd multiples of 32: rows end inside a step, scales start anywhere in a word."""
    L = Layer(m, E, H, I, 0)
    xb = synth.activations(L.g, m, H)
    want, _, err = L.reference(xb, k)
    check(L.run(dev(xb), k), want, err)


@pytest.mark.parametrize("m,E,H,I,k", [(1, 4, 128, 384, 2), (30, 6, 384, 128, 3)])
def test_layer_group_128(m, E, H, I, k):
    L = Layer(m, E, H, I, 128)
    xb = synth.activations(L.g, m, H)
    want, _, err = L.reference(xb, k)
    check(L.run(dev(xb), k), want, err)


@pytest.mark.parametrize("group", [64, 0], ids=["gs64", "mx4"])
def test_layer_decode_sizes(group):
    """One token and a full batch through larger experts, several tiles to a block."""
    L = Layer(3, 8, 2048, 1408, group)
    for m in (1, 64):
        xb = synth.activations(L.g, m, 2048)
        want, _, err = L.reference(xb, 2)
        check(L.run(dev(xb), 2), want, err)


@pytest.mark.parametrize("group", [64, 0], ids=["gs64", "mx4"])
@pytest.mark.parametrize("m,H", [(3, 32768), (24, 16384)])
def test_layer_wide_hidden(m, H, group):
    """More activations than shared memory holds: several chunks of K, refilled for every round of tiles."""
    L = Layer(m, 2, H, 128, group)
    xb = synth.activations(L.g, m, H)
    # columns whose largest values lie in different chunks
    xb[0, : H // 2] = synth.to_bf16_bits(synth.bf16_bits_to_f32(xb[0, : H // 2]) * np.float32(2.0 ** -12))
    xb[1, H // 2:] = synth.to_bf16_bits(synth.bf16_bits_to_f32(xb[1, H // 2:]) * np.float32(2.0 ** -12))
    want, _, err = L.reference(xb, 1)
    check(L.run(dev(xb), 1), want, err)


@pytest.mark.parametrize("m", [5, 40])
@pytest.mark.parametrize("group", [64, 0], ids=["gs64", "mx4"])
def test_equal_logits_take_the_lowest_experts(m, group):
    L = Layer(11, 40, 128, 64, group)
    L.router_bits[:] = 0
    L.router.zero_()
    xb = synth.activations(L.g, m, 128)
    want, ids, err = L.reference(xb, 3)
    assert ids.tolist() == [[0, 1, 2]] * m
    check(L.run(dev(xb), 3), want, err)  # every token in the same three experts, the others empty


def test_equal_tokens_get_equal_rows():
    L = Layer(12, 16, 256, 128, 0)
    xb = np.repeat(synth.activations(L.g, 1, 256), 64, axis=0)
    y = L.run(dev(xb), 4)
    assert torch.equal(y, y[:1].expand_as(y))


@pytest.mark.parametrize("m", [1, 6, 24, 64])
@pytest.mark.parametrize("group", [64, 0], ids=["gs64", "mx4"])
def test_runs_are_bit_identical(m, group):
    L = Layer(13, 32, 512, 192, group)
    x = dev(synth.activations(L.g, m, 512))
    a = L.run(x, 4)
    ws = L.workspace(4, m, fill=0x33)
    for _ in range(5):
        assert torch.equal(L.run(x, 4, ws=ws), a)  # whatever the workspace held


@pytest.mark.parametrize("m", [3, 40])
@pytest.mark.parametrize("bad", [0x7FC0, 0x7F80])
def test_a_bad_token_stays_alone(m, bad):
    L = Layer(14, 8, 128, 64, 0)
    xb = synth.activations(L.g, m, 128)
    want, _, err = L.reference(xb, 2)
    xb[1, 5] = bad
    y = L.run(dev(xb), 2)
    keep = [t for t in range(m) if t != 1]
    check(y[keep], want[keep], err[keep])
    assert not torch.isfinite(y[1].float()).any()


@pytest.mark.parametrize("m", [1, 3, 8, 12, 40])
@pytest.mark.parametrize("group", [64, 0], ids=["gs64", "mx4"])
def test_a_bad_expert_reaches_only_its_tokens(m, group):
    """Infinite and NaN weights of an expert: tokens that did not choose it get the same bits as before."""
    E, H, I, k = 8, 128, 64, 2
    L = Layer(18, E, H, I, group)
    xb = synth.activations(L.g, m, H)
    _, ids, _ = L.reference(xb, k)
    x = dev(xb)
    clean = L.run(x, k)
    bad = int(ids[0, 0])
    hit = (ids == bad).any(dim=1).tolist()
    for i, per in ((2, H), (0, I), (1, I)):  # down, gate, up
        if group:
            scales = L.keep[i][1]
            scales[bad * per:(bad + 1) * per] = float("nan") if i == 0 else float("inf")
        else:
            L.handles[i].tensors[1][bad * per:(bad + 1) * per] = 255
        y = L.run(x, k)
        for t in range(m):
            if hit[t]:
                assert not torch.isfinite(y[t].float()).any()
            else:
                assert torch.equal(y[t], clean[t])


@pytest.mark.parametrize("m", [2, 30])
def test_activations_of_a_wide_range(m):
    """One activation 2^24 times the others under weights that are zero there (MX4)."""
    E, H, I, k = 4, 128, 96, 2
    L = Layer(19, E, H, I, 0)
    L.router_bits[:, 9] = 0
    L.router = dev(L.router_bits)
    for i in (0, 1):
        L.values[i][:, :, 9] = 0
        L.handles[i].tensors[0][:, 1] &= ~0xF0  # column 9: the second nibble of word 1
    x = synth.bf16_bits_to_f32(synth.activations(L.g, m, H)).astype(np.float32)
    x = np.sign(x) * np.clip(np.abs(x), 2.0 ** -6, None)
    x[:, 9] = 2.0 ** 24
    xb = synth.to_bf16_bits(x)
    want, _, err = L.reference(xb, k)
    check(L.run(dev(xb), k), want, err)


def test_output_is_written_exactly():
    L = Layer(15, 8, 192, 64, 64)
    m = 5
    buf = torch.full((m * 192 + 128,), 7.0, dtype=torch.bfloat16, device="cuda")
    x = dev(synth.activations(L.g, m, 192))
    L.run(x, 2, y=buf[64:64 + m * 192].view(m, 192))
    assert torch.equal(buf[64:-64].view(m, 192), L.run(x, 2))
    assert (buf[:64] == 7).all() and (buf[-64:] == 7).all()


@pytest.mark.parametrize("group", [64, 0], ids=["gs64", "mx4"])
def test_graphs_and_streams(group):
    """Two captured layers on two streams, a workspace each, replayed together."""
    L = Layer(16, 16, 512, 256, group)
    xs = [dev(synth.activations(L.g, m, 512)) for m in (2, 30)]
    want = [L.run(x, 4) for x in xs]
    ys = [torch.zeros_like(w) for w in want]
    wss = [L.workspace(4, x.shape[0]) for x in xs]
    torch.cuda.synchronize()
    graphs, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for x, y, ws, s in zip(xs, ys, wss, streams):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            L.run(x, 4, ws=ws, y=y, stream=s)
            L.run(x, 4, ws=ws, y=y, stream=s)  # the same workspace, in order
        graphs.append(graph)
    for _ in range(4):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(y, w) for y, w in zip(ys, want))


def test_quantized_experts_as_a_program_makes_them():
    """BF16 experts -> MX4 codes -> the layer, against the values that dequantising gives."""
    E, H, I, m, k = 6, 256, 160, 10, 2
    g = synth.rng(17)
    L = Layer(17, E, H, I, 0)
    L.handles, L.values = [], []
    for rows, cols in ((E * I, H), (E * I, H), (E * H, I)):
        w = dev(synth.to_bf16_bits(g.standard_normal((rows, cols)) / math.sqrt(cols)))
        h = mq.mx4_empty(rows, cols)
        mq.mlxq_mx4_quantize(w, h)
        back = torch.empty_like(w)
        mq.mlxq_mx4_dequant(h, back)
        assert float((back.double() - w.double()).norm() / w.double().norm()) < 0.2
        L.handles.append(h)
        L.values.append(back.double().reshape(E, -1, cols))
    xb = synth.activations(g, m, H)
    want, _, err = L.reference(xb, k)
    check(L.run(dev(xb), k), want, err)


def test_equal_tokens_of_many_experts_take_several_entries():
    """Few tokens an expert on average, all 64 on the same sixteen: each expert's weights are streamed several times."""
    L = Layer(21, 256, 128, 64, 0)
    xb = np.repeat(synth.activations(L.g, 1, 128), 64, axis=0)
    want, _, err = L.reference(xb[:1], 16)
    y = L.run(dev(xb), 16)
    assert torch.equal(y, y[:1].expand_as(y))
    check(y[:1], want, err)


@pytest.mark.parametrize("m", [2, 11])
@pytest.mark.parametrize("group", [64, 0], ids=["gs64", "mx4"])
def test_offsets_past_32_bits(m, group):
    """Experts of more than 2^32 bytes of codes per matrix, the last one chosen."""
    E, I, H = 256, 1024, 16512 if group else 33024
    g = torch.Generator("cuda").manual_seed(22)
    handles, values, keep = [], [], []
    for rows, cols in ((E * I, H), (E * I, H), (E * H, I)):
        last = slice(rows - rows // E, rows)
        if group:
            assert rows * cols > 2 ** 32
            p = torch.randint(-2 ** 31, 2 ** 31 - 1, (rows, cols // 4), dtype=torch.int32, device="cuda", generator=g)
            s = torch.full((rows, cols // group), 2.0 ** -7 / math.sqrt(cols), dtype=torch.bfloat16, device="cuda")
            b = torch.full_like(s, -1.0 / math.sqrt(cols))
            keep.append((p, s, b))
            handles.append(mq.weight_view(p, s, b, group))
            q = p[last].contiguous().view(torch.uint8).double().reshape(-1, cols // group, group)
            v = (s[last].double()[:, :, None] * q + b[last].double()[:, :, None]).float().bfloat16().double()
        else:
            assert rows * cols // 2 > 2 ** 32
            codes = torch.randint(-2 ** 31, 2 ** 31 - 1, (rows, cols // 8), dtype=torch.int32, device="cuda", generator=g)
            e = 127 + round(math.log2(1 / (2.9 * math.sqrt(cols))))
            scales = torch.randint(e - 1, e + 2, (rows, cols // 32), dtype=torch.uint8, device="cuda", generator=g)
            handles.append(mq.mx4_view(codes, scales))
            grid = torch.tensor(np.concatenate([ref.GRID, -ref.GRID]), device="cuda")
            c = torch.stack([(codes[last] >> (4 * i)) & 15 for i in range(8)], dim=-1).reshape(-1, cols // 32, 32)
            v = grid[c.long()] * torch.exp2(scales[last].double() - 127)[:, :, None]
        values.append(v.reshape(1, rows // E, cols))
    xb = synth.activations(synth.rng(22), m, H)
    x = dev(xb)
    router = torch.zeros(E, H, dtype=torch.bfloat16, device="cuda")
    y = torch.empty(m, H, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(mq.mlxq_moe_workspace_bytes(H, I, 1, m), dtype=torch.uint8, device="cuda")
    call = mq.mlxq_moe if group else mq.mlxq_mx4_moe
    for t in range(m):  # a row of the router that every token's logit is largest with: one token at a time
        router[E - 1] = x[t]
        call(router, *handles, E, 1, x[t:t + 1], y[t:t + 1], 1, ws)
    want, _, err = ref.moe(f64(xb), torch.ones(1, H, dtype=torch.float64, device="cuda"), *values, 1, True)
    check(y, want, err)
    both = torch.empty_like(y)  # all tokens in one call: those that the last row draws there get the same expert
    router[E - 1] = x.float().mean(dim=0).bfloat16()
    call(router, *handles, E, 1, x, both, m, ws)
    drawn = (x.double() @ router[E - 1].double()) > 0.01
    assert bool(drawn.any())
    check(both[drawn], want[drawn], err[drawn])


@pytest.mark.parametrize("group", [64, 0], ids=["gs64", "mx4"])
def test_layers_on_two_streams_at_once(group):
    """Calls on two streams, a workspace each; and other small sizes in between on a third."""
    L = Layer(23, 16, 1024, 256, group)
    xs = [dev(synth.activations(L.g, m, 1024)) for m in (1, 40, 8)]
    want = [L.run(x, 4) for x in xs]
    ys, wss = [torch.zeros_like(w) for w in want], [L.workspace(4, x.shape[0]) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(20):
        for x, y, ws, s in zip(xs, ys, wss, streams):
            L.run(x, 4, ws=ws, y=y, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(y, w) for y, w in zip(ys, want))
