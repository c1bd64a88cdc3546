"""GPU parity of the MX4 calls against a plain 64-bit reference: quantisation and
dequantisation bit for bit, products within a bound derived from their sums."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import _mx4_ref as ref
import synth
import weight_only_quantized_mlx_b200 as mq
from _helpers import Guarded, bits_to_f64, dev, host_bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    mq.lib()
    yield
    torch.cuda.synchronize()
    mq.mlxq_device_status()


def padded(nbytes):
    """A byte buffer in the middle of guard bytes: (whole, view)."""
    b = torch.full((nbytes + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    return b, b[256:256 + nbytes]


def check_pads(b, nbytes):
    h = b.cpu().numpy()
    assert np.all(h[:256] == 0xA5) and np.all(h[256 + nbytes:] == 0xA5), "write outside the buffer"


def run_quantize(bits, offset=0):
    rows, cols = bits.shape
    src = torch.zeros(rows * cols + offset, dtype=torch.bfloat16, device="cuda")
    src[offset:] = dev(bits).reshape(-1)
    cb, codes = padded(rows * cols // 2)
    sb, scales = padded(rows * cols // 32)
    mq.mlxq_mx4_quantize(src[offset:], mq.mlxq_mx4(codes.data_ptr(), scales.data_ptr(), rows, cols))
    torch.cuda.synchronize()
    check_pads(cb, rows * cols // 2)
    check_pads(sb, rows * cols // 32)
    return codes.cpu().numpy().view(np.uint32).reshape(rows, -1), scales.cpu().numpy().reshape(rows, -1)


def draw(kind, g, rows, cols):
    if kind == "normal":
        return synth.activations(g, rows, cols)
    if kind == "bits":  # every exponent, finite
        b = g.integers(0, 1 << 16, (rows, cols)).astype(np.uint16)
        return np.where((b & 0x7F80) == 0x7F80, b & 0xBFFF, b).astype(np.uint16)
    if kind == "ties":  # borders of the grid at several scales
        v = g.choice([0, .25, .5, .75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 7], (rows, cols)) * g.choice([-1, 1], (rows, cols))
        return synth.to_bf16_bits(v * 2.0 ** g.integers(-140, 120, (rows, 1)))
    if kind == "tiny":  # zeros of both signs, subnormals, the smallest normals
        return (g.choice([0, 0, 1, 2, 3, 0x40, 0x7F, 0x80, 0xC0, 0x17F, 0x1FF], (rows, cols)) | (g.integers(0, 2, (rows, cols)) << 15)).astype(np.uint16)
    b = synth.activations(g, rows, cols)  # "special": some blocks hold infinities and NaN
    b[0, 0], b[-1, -1], b[0, cols // 2] = 0x7F80, 0xFFC0, 0xFF80
    return b


@pytest.mark.parametrize("kind", ["normal", "bits", "ties", "tiny", "special"])
@pytest.mark.parametrize("rows,cols", [(1, 32), (1, 4096), (3, 96), (67, 160), (33, 1056)])
def test_quantize_bit_exact(rows, cols, kind):
    bits = draw(kind, synth.rng(rows + cols), rows, cols)
    want_codes, want_scales = ref.quantize(bits)
    for offset in (0, 1, 8):  # 32-byte aligned, 2-byte, 16-byte
        codes, scales = run_quantize(bits, offset)
        assert np.array_equal(scales, want_scales), offset
        assert np.array_equal(codes, ref.pack(want_codes)), offset


def test_dequant_every_code_and_scale_bit_exact():
    codes = np.tile(np.arange(16, dtype=np.uint8), (256, 4))  # 64 columns: two blocks
    scales = np.stack([np.arange(256), 255 - np.arange(256)], axis=1).astype(np.uint8)
    want = ref.values(codes, scales)
    with np.errstate(over="ignore", invalid="ignore"):
        want_bits = synth.to_bf16_bits(want.astype(np.float32))  # exact, or infinite
    for offset in (0, 1, 8):
        out = Guarded(codes.size, offset_elems=offset)
        h = mq.mx4_view(dev(ref.pack(codes)), dev(scales))
        mq.mlxq_mx4_dequant(h, out.data_ptr())
        torch.cuda.synchronize()
        out.check_guards()
        got = out.value_bits().reshape(codes.shape)
        nan = np.isnan(want)
        assert np.array_equal(np.isnan(bits_to_f64(got)), nan)
        assert np.array_equal(got[~nan], want_bits[~nan])


def bound(absw, absx, y, K):
    """|Y - Y_ref| for an fp32 sum of K exact products on the tensor pipe (each of
    its K / 16 steps loses at most 2^-22 of the sum of magnitudes, the joins of
    partial sums a few more), rounded once to BF16."""
    s = (K / 16 + 32) * 2.0 ** -22 * (absx @ absw.T)
    return s + 2.0 ** -8 * (np.abs(y) + s)


def make(seed, rows, cols, **k):
    g = synth.rng(seed)
    codes, scales = ref.random_weight(g, rows, cols, **k)
    return g, codes, scales, mq.mx4_view(dev(ref.pack(codes)), dev(scales))


GEMM = [(1, 1, 32), (1, 9, 64), (3, 148, 96), (8, 300, 4128), (9, 17, 160), (16, 4099, 544), (17, 1200, 128),
        (33, 2500, 1056), (64, 333, 2080), (61, 64, 32), (1, 4096, 4096), (5, 9000, 256), (40, 5003, 96),
        (8, 200, 8192), (2, 150, 36864), (20, 700, 14336), (64, 4099, 4128), (64, 20, 4096), (30, 2000, 64)]


@pytest.mark.parametrize("m,N,K", GEMM)
def test_gemm(m, N, K):
    g, codes, scales, h = make(m + N, N, K)
    w = ref.values(codes, scales)
    xb = synth.activations(g, m, K)
    x = bits_to_f64(xb)
    y = Guarded(m * N)
    mq.mlxq_mx4_gemm(h, dev(xb), y.data_ptr(), m)
    torch.cuda.synchronize()
    y.check_guards()
    want = x @ w.T
    err = np.abs(bits_to_f64(y.value_bits()).reshape(m, N) - want)
    assert np.all(err <= bound(np.abs(w), np.abs(x), want, K)), float(err.max())


@pytest.mark.parametrize("m", [1, 12])
def test_gemm_extreme_scales(m):
    """Scale bytes from 0 to 254, mixed within rows; x small enough that nothing overflows."""
    N, K = 70, 416
    g, codes, scales, h = make(5, N, K, low=100, high=150)
    scales[:, 0], scales[:, 1], scales[:, 2] = 0, 128, 129
    scales[3, :] = 250
    h = mq.mx4_view(dev(ref.pack(codes)), dev(scales))
    w = ref.values(codes, scales)
    xb = synth.to_bf16_bits(g.standard_normal((m, K)) * 2.0 ** -20)
    x = bits_to_f64(xb)
    y = torch.empty(m, N, dtype=torch.bfloat16, device="cuda")
    mq.mlxq_mx4_gemm(h, dev(xb), y, m)
    want = x @ w.T
    err = np.abs(bits_to_f64(host_bits(y)) - want)
    assert np.all(err <= bound(np.abs(w), np.abs(x), want, K))


@pytest.mark.parametrize("m", [2, 20])
def test_gemm_nan_and_infinity_stay_in_their_rows(m):
    N, K = 40, 224
    g, codes, scales, h = make(6, N, K)
    scales[7, 6] = 255
    h = mq.mx4_view(dev(ref.pack(codes)), dev(scales))
    xb = synth.activations(g, m, K)
    xb[1, K - 1] = 0x7FC0
    y = torch.empty(m, N, dtype=torch.bfloat16, device="cuda")
    mq.mlxq_mx4_gemm(h, dev(xb), y, m)
    nan = np.isnan(bits_to_f64(host_bits(y)))
    want = np.zeros((m, N), bool)
    want[1, :], want[:, 7] = True, True
    assert np.array_equal(nan, want)


@pytest.mark.parametrize("m,K", [(1, 416), (4, 36864), (12, 416), (40, 2080)])
@pytest.mark.parametrize("ratio", [17, 24, 30])
def test_gemm_activations_of_a_wide_range(m, K, ratio):
    """One column of activations 2^ratio times the others, under codes that are zero: what is left
    is the others' sum, as exact as without it (BF16 values down to 2^-31 of the largest are kept whole)."""
    N = 90
    g, codes, scales, h = make(7, N, K)
    codes[:, 5] = 0
    h = mq.mx4_view(dev(ref.pack(codes)), dev(scales))
    w = ref.values(codes, scales)
    x32 = np.sign(g.standard_normal((m, K))) * g.uniform(1, 2, (m, K))
    x32[:, 5] = 1.5 * 2.0 ** ratio
    xb = synth.to_bf16_bits(x32)
    x = bits_to_f64(xb)
    y = torch.empty(m, N, dtype=torch.bfloat16, device="cuda")
    mq.mlxq_mx4_gemm(h, dev(xb), y, m)
    want = x @ w.T
    err = np.abs(bits_to_f64(host_bits(y)) - want)
    assert np.all(err <= bound(np.abs(w), np.abs(x), want, K))


@pytest.mark.parametrize("m", [3, 20])
@pytest.mark.parametrize("e", [-126, -120, -112, 100, 127])
def test_gemm_activations_at_the_ends_of_the_range(m, e):
    """The largest activations near the least and the largest BF16 powers of two."""
    N, K = 50, 160
    g, codes, scales, h = make(8, N, K)
    scales[:] = g.integers(117, 123, scales.shape) if e < 0 else g.integers(100, 110, scales.shape)
    h = mq.mx4_view(dev(ref.pack(codes)), dev(scales))
    w = ref.values(codes, scales)
    xb = synth.to_bf16_bits(g.uniform(-1.9, 1.9, (m, K)) * 2.0 ** e)
    x = bits_to_f64(xb)
    y = torch.empty(m, N, dtype=torch.bfloat16, device="cuda")
    mq.mlxq_mx4_gemm(h, dev(xb), y, m)
    want = x @ w.T
    err = np.abs(bits_to_f64(host_bits(y)) - want)
    # (2^-133: the last place of a BF16 result below 2^-126, half of it for each of two roundings)
    assert np.all(err <= bound(np.abs(w), np.abs(x), want, K) + 2.0 ** -133)


def test_gemm_of_no_columns_is_zero_and_empty_outputs_are_nothing():
    y = torch.full((2, 8), 7.0, dtype=torch.bfloat16, device="cuda")
    mq.mlxq_mx4_gemm(mq.mlxq_mx4(None, None, 8, 0), None, y, 2)
    assert not y.any()
    mq.mlxq_mx4_gemm(mq.mlxq_mx4(None, None, 0, 64), torch.zeros(2, 64, dtype=torch.bfloat16, device="cuda"), None, 2)
    mq.mlxq_mx4_quantize(None, mq.mlxq_mx4(None, None, 0, 64))
    mq.mlxq_mx4_dequant(mq.mlxq_mx4(None, None, 3, 0), None)
    torch.cuda.synchronize()


def test_quantize_then_gemm_on_a_side_stream_and_in_a_graph():
    """The calls in a row as a program makes them, on a stream of its own, captured and replayed."""
    rows, cols, m = 200, 256, 4
    g = synth.rng(9)
    wb, xb = synth.activations(g, rows, cols), synth.activations(g, m, cols)
    w, x = dev(wb), dev(xb)
    q = mq.mx4_empty(rows, cols)
    back = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    y = torch.empty(m, rows, dtype=torch.bfloat16, device="cuda")

    def chain(s):
        mq.mlxq_mx4_quantize(w, q, s)
        mq.mlxq_mx4_dequant(q, back, s)
        mq.mlxq_mx4_gemm(q, x, y, m, s)

    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    chain(s)
    s.synchronize()
    eager, eager_back = host_bits(y), host_bits(back)
    v = ref.values(*ref.quantize(wb))
    assert np.array_equal(bits_to_f64(eager_back), v)
    xv = bits_to_f64(xb)
    assert np.all(np.abs(bits_to_f64(eager) - xv @ v.T) <= bound(np.abs(v), np.abs(xv), xv @ v.T, cols))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        chain(s)
    y.zero_()
    back.zero_()
    q.tensors[0].zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert np.array_equal(host_bits(y), eager) and np.array_equal(host_bits(back), eager_back)


def test_gemm_rows_of_very_different_sizes():
    """Each row of X has its own unit: tiny and huge rows side by side, and values of very different size within a row."""
    N, K = 90, 1312
    g, codes, scales, h = make(10, N, K)
    w = ref.values(codes, scales)
    for m in (3, 18, 50):
        v = g.standard_normal((m, K)) * 2.0 ** g.integers(-100, 100, (m, 1)) * 2.0 ** g.integers(-30, 1, (m, K))
        xb = synth.to_bf16_bits(v)
        x = bits_to_f64(xb)
        y = torch.empty(m, N, dtype=torch.bfloat16, device="cuda")
        mq.mlxq_mx4_gemm(h, dev(xb), y, m)
        want = x @ w.T
        # and each value is off by at most 2^-25 of its row's largest
        extra = 2.0 ** -25 * np.abs(x).max(axis=1, keepdims=True) * np.abs(w).sum(axis=1)[None, :]
        err = np.abs(bits_to_f64(host_bits(y)) - want)
        assert np.all(err <= bound(np.abs(w), np.abs(x), want, K) + extra), m


def test_gemm_graphs_side_by_side():
    """Batches that take scratch from the pool: two captured graphs replayed on two streams at once."""
    N, K = 1500, 2080
    g, codes, scales, h = make(11, N, K)
    w = ref.values(codes, scales)
    xs = [synth.activations(g, m, K) for m in (12, 50)]
    ys = [torch.zeros(x.shape[0], N, dtype=torch.bfloat16, device="cuda") for x in xs]
    keep = [dev(x) for x in xs]
    graphs, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for x, y, s in zip(keep, ys, streams):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            for _ in range(3):
                mq.mlxq_mx4_gemm(h, x, y, x.shape[0], s)
        graphs.append(graph)
    for _ in range(5):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for xb, y in zip(xs, ys):
        x = bits_to_f64(xb)
        err = np.abs(bits_to_f64(host_bits(y)) - x @ w.T)
        assert np.all(err <= bound(np.abs(w), np.abs(x), x @ w.T, K))


def test_calls_repeat_bit_for_bit():
    g, codes, scales, h = make(12, 1000, 4128)
    ac, as_ = ref.random_weight(g, 70, 4128)
    a = mq.mx4_view(dev(ref.pack(ac)), dev(as_))
    first = None
    for _ in range(4):
        out = []
        for m in (1, 7, 20, 64):
            x = dev(synth.activations(synth.rng(m), m, 4128))
            y = torch.empty(m, 1000, dtype=torch.bfloat16, device="cuda")
            mq.mlxq_mx4_gemm(h, x, y, m)
            out.append(host_bits(y))
        y = torch.empty(70, 1000, dtype=torch.bfloat16, device="cuda")
        mq.mlxq_mx4_matmul(h, a, y)
        out.append(host_bits(y))
        if first is None:
            first = out
        assert all(np.array_equal(p, q) for p, q in zip(first, out))


def test_gemm_past_32_bits_of_codes():
    """A weight whose codes pass 2^31 bytes: the last rows are read where they are."""
    N, K = 2 ** 20 + 8, 4224
    codes = torch.zeros(N, K // 8, dtype=torch.int32, device="cuda")
    scales = torch.full((N, K // 32), 127, dtype=torch.uint8, device="cuda")
    codes[-1] = 0x22222222      # ones
    codes[N // 2] = 0x44444444  # twos
    x = torch.ones(1, K, dtype=torch.bfloat16, device="cuda")
    y = torch.empty(1, N, dtype=torch.bfloat16, device="cuda")
    mq.mlxq_mx4_gemm(mq.mx4_view(codes, scales), x, y, 1)
    want = torch.zeros(N, dtype=torch.bfloat16, device="cuda")
    want[-1], want[N // 2] = K, 2 * K
    assert torch.equal(y[0], want)


# (m, N, K): both operands in MX4; tiles are 256 x up to 224, k-blocks 256
MATMUL = [(1, 1, 32), (16, 256, 256), (128, 256, 512), (224, 512, 1024), (5, 300, 96), (130, 260, 288), (300, 1000, 736),
          (225, 257, 4128), (509, 1100, 544), (64, 4097, 1280), (2000, 3100, 256), (17, 5000, 2048), (1, 300, 8192), (250, 600, 14368),
          (40, 2000, 4640)]


@pytest.mark.parametrize("m,N,K", MATMUL)
def test_matmul(m, N, K):
    g, wc, ws, w = make(m + N, N, K)
    ac, as_ = ref.random_weight(g, m, K, low=122, high=130)
    a = mq.mx4_view(dev(ref.pack(ac)), dev(as_))
    y = Guarded(m * N)
    mq.mlxq_mx4_matmul(w, a, y.data_ptr())
    torch.cuda.synchronize()
    y.check_guards()
    wv, av = ref.values(wc, ws), ref.values(ac, as_)
    want = av @ wv.T
    err = np.abs(bits_to_f64(y.value_bits()).reshape(m, N) - want)
    assert np.all(err <= bound(np.abs(wv), np.abs(av), want, K)), float(err.max())


def test_matmul_places_every_code_and_scale():
    """One nonzero activation column at a time: Y is that weight column times a power of two, exactly."""
    N, K, m = 300, 320, 320
    g, wc, ws, w = make(3, N, K, low=110, high=140)
    ac, as_ = np.zeros((m, K), np.uint8), np.full((m, K // 32), 127, np.uint8)
    ac[np.arange(m), np.arange(K)] = 2 + 2 * (np.arange(K) % 3)  # 1, 2, 4
    as_ += g.integers(0, 9, as_.shape).astype(np.uint8)
    y = torch.empty(m, N, dtype=torch.bfloat16, device="cuda")
    mq.mlxq_mx4_matmul(w, mq.mx4_view(dev(ref.pack(ac)), dev(as_)), y)
    want = ref.values(ac, as_) @ ref.values(wc, ws).T
    assert np.array_equal(bits_to_f64(host_bits(y)), want)


def test_matmul_nan_scales_stay_in_their_rows():
    N, K, m = 300, 288, 40
    g, wc, ws, _ = make(4, N, K)
    ac, as_ = ref.random_weight(g, m, K)
    ws[270, 8], as_[33, 0] = 255, 255
    y = torch.empty(m, N, dtype=torch.bfloat16, device="cuda")
    mq.mlxq_mx4_matmul(mq.mx4_view(dev(ref.pack(wc)), dev(ws)), mq.mx4_view(dev(ref.pack(ac)), dev(as_)), y)
    want = np.zeros((m, N), bool)
    want[33, :], want[:, 270] = True, True
    assert np.array_equal(np.isnan(bits_to_f64(host_bits(y))), want)


def test_matmul_unaligned_scales_and_no_columns():
    """Scale tables that are 4-byte but not 8-byte aligned; products of no columns are zero."""
    N, K, m = 70, 512, 20
    g, wc, ws, _ = make(8, N, K)
    ac, as_ = ref.random_weight(g, m, K)
    buf = torch.zeros(ws.size + 4, dtype=torch.uint8, device="cuda")
    buf[4:] = dev(ws).reshape(-1)
    codes = dev(ref.pack(wc))
    y = torch.empty(m, N, dtype=torch.bfloat16, device="cuda")
    mq.mlxq_mx4_matmul(mq.mx4_view(codes, buf[4:].view(N, -1)), mq.mx4_view(dev(ref.pack(ac)), dev(as_)), y)
    wv, av = ref.values(wc, ws), ref.values(ac, as_)
    assert np.all(np.abs(bits_to_f64(host_bits(y)) - av @ wv.T) <= bound(np.abs(wv), np.abs(av), av @ wv.T, K))
    mq.mlxq_mx4_matmul(mq.mlxq_mx4(None, None, N, 0), mq.mlxq_mx4(None, None, m, 0), y)
    assert not y.any()


def test_quantize_then_matmul_in_a_graph():
    """Prefill as a program makes it: activations quantised and multiplied, several times in a row."""
    N, K, m = 500, 1056, 260
    g = synth.rng(21)
    wb, xb = synth.activations(g, N, K), synth.activations(g, m, K)
    w, a, x = mq.mx4_empty(N, K), mq.mx4_empty(m, K), dev(xb)
    mq.mlxq_mx4_quantize(dev(wb), w)
    y = torch.zeros(m, N, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        for _ in range(3):
            mq.mlxq_mx4_quantize(x, a, s)
            mq.mlxq_mx4_matmul(w, a, y, s)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    wv, av = ref.values(*ref.quantize(wb)), ref.values(*ref.quantize(xb))
    want = av @ wv.T
    assert np.all(np.abs(bits_to_f64(host_bits(y)) - want) <= bound(np.abs(wv), np.abs(av), want, K))


def big(rows, cols, seed):
    """A handle over more than 2^32 bytes of random codes; scales near 2^-7."""
    g = torch.Generator("cuda").manual_seed(seed)
    codes = torch.randint(-2 ** 31, 2 ** 31 - 1, (rows, cols // 8), dtype=torch.int32, device="cuda", generator=g)
    scales = torch.randint(118, 123, (rows, cols // 32), dtype=torch.uint8, device="cuda", generator=g)
    return mq.mx4_view(codes, scales)


def rows_of(h, lo, hi):
    """fp64 values of rows [lo, hi)."""
    codes = h.tensors[0][lo:hi].cpu().numpy().view(np.uint32)
    c = ((codes[:, :, None] >> (4 * np.arange(8, dtype=np.uint32))) & 15).astype(np.uint8).reshape(hi - lo, -1)
    return ref.values(c, h.tensors[1][lo:hi].cpu().numpy())


def test_offsets_past_32_bits():
    """More than 2^32 bytes of codes, and more than 2^32 elements on the BF16 side: first, middle and last rows."""
    N, K = 530000, 16416
    assert N * K // 2 > 2 ** 32
    h = big(N, K, 20)
    g = synth.rng(20)
    spans = [(0, 20), (N * 2 // 3, N * 2 // 3 + 20), (N - 37, N)]
    for m in (2, 20):
        xb = synth.activations(g, m, K)
        x = bits_to_f64(xb)
        y = torch.empty(m, N, dtype=torch.bfloat16, device="cuda")
        mq.mlxq_mx4_gemm(h, dev(xb), y, m)
        for lo, hi in spans:
            w = rows_of(h, lo, hi)
            want = x @ w.T
            err = np.abs(bits_to_f64(host_bits(y[:, lo:hi].contiguous())) - want)
            assert np.all(err <= bound(np.abs(w), np.abs(x), want, K))
    out = torch.empty(N, K, dtype=torch.bfloat16, device="cuda")
    mq.mlxq_mx4_dequant(h, out)
    for lo, hi in spans:
        assert np.array_equal(bits_to_f64(host_bits(out[lo:hi])), rows_of(h, lo, hi))
    back = mq.mx4_empty(N, K)
    mq.mlxq_mx4_quantize(out, back)
    again = torch.empty_like(out)
    mq.mlxq_mx4_dequant(back, again)
    assert torch.equal(out, again)  # the values of a block and its largest binade come back
    del out, again, back
    # Y of more than 2^32 elements
    M, N, K = 66000, 66000, 64
    a, w = big(M, K, 21), big(N, K, 22)
    y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    mq.mlxq_mx4_matmul(w, a, y)
    for i in (0, M - 30):
        for j in (0, N - 40):
            va, vw = rows_of(a, i, i + 30), rows_of(w, j, j + 40)
            want = va @ vw.T
            err = np.abs(bits_to_f64(host_bits(y[i:i + 30, j:j + 40].contiguous())) - want)
            assert np.all(err <= bound(np.abs(vw), np.abs(va), want, K))


def test_calls_on_two_streams_at_once():
    """Each call again and again on two streams, other operands on each: the bits of one call alone."""
    jobs = []
    for seed, (m, N, K) in enumerate([(20, 700, 14336), (9, 4100, 4096), (64, 1024, 4128), (3, 3000, 2048)]):
        g, codes, scales, h = make(30 + seed, N, K)
        x = dev(synth.activations(g, m, K))
        a = mq.mx4_empty(m, K)
        jobs.append((h, x, a, m, N))

    def run(job, stream=None):
        h, x, a, m, N = job
        y, z = (torch.full((m, N), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        mq.mlxq_mx4_gemm(h, x, y, m, stream)
        mq.mlxq_mx4_quantize(x, a, stream)
        mq.mlxq_mx4_matmul(h, a, z, stream)
        return y, z

    want = [run(j) for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        got = [run(j, streams[i % 2]) for i, j in enumerate(jobs)]
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for a, b in zip(got, want) for p, q in zip(a, b))
