"""Cases that measure the MX4 (microscaled 4-bit floating point) operators and
the mixture-of-experts layer, with the operators' plain forms.

``kind`` of a case:

* ``roundtrip``  BF16 [rows, cols] -> MX4 codes and scales -> BF16 (quantise, then dequantise)
* ``weight4``    Y = X W^T, W in MX4, X in BF16 (decoding: up to 64 rows)
* ``both4``      Y = X W^T, W in MX4, X quantised to MX4 in the call (prefill)
* ``moe8``       router, top-k, gated experts and their weighted sum; experts as 8-bit group-affine weights
* ``moe4``       the same with MX4 experts
"""
import math

import numpy as np
import torch

own = False

BLOCK = 32          # columns per MX4 scale
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one token's activations on their way into a 4-bit product: latency
        dict(name="roundtrip_token", kind="roundtrip", rows=1, cols=4096),
        # a projection's weight quantised once and checked against its source
        dict(name="roundtrip_weight", kind="roundtrip", rows=14336, cols=4096),
        # decoding, one token through a square projection
        dict(name="weight4_decode", kind="weight4", m=1, n=4096, k=4096),
        # decoding a batch through the widest projection of the benchmark, ragged batch
        dict(name="weight4_batch", kind="weight4", m=13, n=28672, k=8192),
        # the largest batch of decoding, odd output width, k no multiple of 128
        dict(name="weight4_odd", kind="weight4", m=61, n=4099, k=4128),
        # prefill, a long prompt through the up projection
        dict(name="both4_prefill", kind="both4", m=8192, n=14336, k=4096),
        # prefill of a short, odd prompt through a down projection of odd width
        dict(name="both4_odd", kind="both4", m=509, n=4100, k=14368),
        # decoding, one token, few large experts
        dict(name="moe8_token", kind="moe8", m=1, hidden=4096, inter=14336, experts=8, top_k=2, group=64, renorm=True),
        # decoding a batch, many small experts, most of them hit
        dict(name="moe8_batch", kind="moe8", m=32, hidden=2048, inter=1024, experts=64, top_k=8, group=32, renorm=False),
        # decoding, one token, many small experts in 4 bits: the smallest layer
        dict(name="moe4_token", kind="moe4", m=1, hidden=2048, inter=1024, experts=64, top_k=8, renorm=True),
        # the largest batch the layer takes, many experts, odd block counts
        dict(name="moe4_batch", kind="moe4", m=64, hidden=4128, inter=1504, experts=128, top_k=8, renorm=True),
    ]


def _log_int(rng, lo, hi, step=1):
    """An integer in [lo, hi], a multiple of step, spread over its logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return min(hi // step * step, max(step, int(round(v / step)) * step))


def draw(rng):
    kind = rng.choice(["roundtrip", "weight4", "both4", "moe8", "moe4"])
    if kind == "roundtrip":
        cols = _log_int(rng, 32, 16384, 32)
        return dict(kind=kind, rows=_log_int(rng, 1, 14336 * 4096 // cols), cols=cols)
    if kind == "weight4":
        k = _log_int(rng, 64, 28672, 32)
        return dict(kind=kind, m=_log_int(rng, 1, 64), n=_log_int(rng, 64, min(28672, 28672 * 8192 // k)), k=k)
    if kind == "both4":
        k = _log_int(rng, 64, 14336, 32)
        n = _log_int(rng, 64, min(14336, 14336 * 4096 // k))
        return dict(kind=kind, m=_log_int(rng, 1, 8192), n=n, k=k)
    experts = _log_int(rng, 2, 128)
    step = 64 if kind == "moe8" else 32
    c = dict(kind=kind, m=_log_int(rng, 1, 64), hidden=_log_int(rng, 256, 4096, step), inter=_log_int(rng, 256, 2048, step),
             experts=experts, top_k=rng.randint(1, min(8, experts)), renorm=rng.random() < 0.5)
    if kind == "moe8":
        c["group"] = rng.choice([32, 64])
    return c


# ---- inputs ------------------------------------------------------------------------------
def _mx4_weight(gen, rows, cols):
    """Random codes, and scales that give W a spread of about 1 / sqrt(cols)."""
    codes = torch.randint(-2 ** 31, 2 ** 31, (rows, cols // 8), generator=gen, device="cuda", dtype=torch.int64).to(torch.int32)
    base = 127 + round(math.log2(1.0 / (2.9 * math.sqrt(cols))))
    scales = (base + torch.randint(-1, 2, (rows, cols // BLOCK), generator=gen, device="cuda")).to(torch.uint8)
    return codes, scales


def _affine_weight(gen, rows, cols, group):
    """Uniform codes; scales and centred biases that give W a spread of about 1 / sqrt(cols)."""
    packed = torch.randint(-2 ** 31, 2 ** 31, (rows, cols // 4), generator=gen, device="cuda", dtype=torch.int64).to(torch.int32)
    s = (torch.rand(rows, cols // group, generator=gen, device="cuda") + 0.5) / (74.0 * math.sqrt(cols))
    s = s.to(torch.bfloat16)
    b = -128.0 * s.float() + torch.randn(s.shape, generator=gen, device="cuda") * 0.25 * s.float()
    return packed, s, b.to(torch.bfloat16)


def _normal(gen, *shape, scale=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(torch.bfloat16)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case)
    if case["kind"] == "roundtrip":
        # rows of different sizes, as activations of different tokens or a weight's rows have
        spread = torch.exp(torch.randn(case["rows"], 1, generator=gen, device="cuda"))
        s["x"] = (torch.randn(case["rows"], case["cols"], generator=gen, device="cuda") * spread).to(torch.bfloat16)
        s["y"] = torch.empty_like(s["x"])
    elif case["kind"] in ("weight4", "both4"):
        s["w"] = _mx4_weight(gen, case["n"], case["k"])
        s["x"] = _normal(gen, case["m"], case["k"])
        s["y"] = torch.empty(case["m"], case["n"], dtype=torch.bfloat16, device="cuda")
    else:
        E, H, I = case["experts"], case["hidden"], case["inter"]
        make = _mx4_weight if case["kind"] == "moe4" else (lambda g, r, c: _affine_weight(g, r, c, case["group"]))
        s["gate"], s["up"], s["down"] = make(gen, E * I, H), make(gen, E * I, H), make(gen, E * H, I)
        s["router"] = _normal(gen, E, H, scale=2.0 / math.sqrt(H))
        s["x"] = _normal(gen, case["m"], H)
        s["y"] = torch.empty_like(s["x"])
    if own:
        _handles(s)
    return s


def _handles(s):
    """What a program keeps beside its tensors: handles over them and buffers."""
    import weight_only_quantized_mlx_b200 as mq
    if s["kind"] == "roundtrip":
        s["q"] = mq.mx4_empty(s["rows"], s["cols"])
    elif s["kind"] == "weight4":
        s["hw"] = mq.mx4_view(*s["w"])
    elif s["kind"] == "both4":
        s["hw"] = mq.mx4_view(*s["w"])
        s["q"] = mq.mx4_empty(s["m"], s["k"])
    else:
        view = mq.mx4_view if s["kind"] == "moe4" else (lambda p, sc, b: mq.weight_view(p, sc, b, s["group"]))
        s["handles"] = tuple(view(*s[n]) for n in ("gate", "up", "down"))
        nbytes = mq.mlxq_moe_workspace_bytes(s["hidden"], s["inter"], s["top_k"], s["m"])
        s["workspace"] = torch.empty(nbytes, dtype=torch.uint8, device="cuda")


# ---- plain forms ---------------------------------------------------------------------------
def _lut(device, dtype=torch.float32):
    return torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=dtype, device=device)


def _mx4_values(codes, scales):
    """fp32 values [rows, cols] of MX4 codes (eight per int32, low nibble first)."""
    shifts = torch.arange(0, 32, 4, device=codes.device, dtype=torch.int32)
    nib = (codes.unsqueeze(-1) >> shifts) & 15
    v = _lut(codes.device)[nib].reshape(codes.shape[0], -1, BLOCK)
    return torch.ldexp(v, scales.to(torch.int32).unsqueeze(-1) - 127).reshape(codes.shape[0], -1)


def _mx4_rounded(x):
    """The values that x becomes in MX4 (fp32)."""
    v = x.float().reshape(x.shape[0], -1, BLOCK)
    e = (torch.frexp(v.abs().amax(-1, keepdim=True)).exponent - 3).clamp(-127, 127)
    a = torch.ldexp(v.abs(), -e).clamp(max=6.0)
    # spacing of the E2M1 grid: 0.5 below 2, 1 below 4, 2 above; round() takes ties to even
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = torch.round(a / step) * step
    return torch.ldexp(torch.copysign(q, v), e).reshape(x.shape)


def _affine_values(packed, s, b):
    """fp32 values of 8-bit group-affine codes: bf16(s q + b)."""
    shifts = torch.arange(0, 32, 8, device=packed.device, dtype=torch.int32)
    q = ((packed.unsqueeze(-1) >> shifts) & 255).float().reshape(*s.shape, -1)
    return (s.float().unsqueeze(-1) * q + b.float().unsqueeze(-1)).to(torch.bfloat16).float().reshape(packed.shape[0], -1)


def _experts(state, name, ids, rows):
    """fp32 weights of the experts `ids` (a tensor or a slice): [len, rows, cols]."""
    w = [t.reshape(state["experts"], rows, -1)[ids] for t in state[name]]
    n = w[0].shape[0]
    flat = [t.reshape(n * rows, -1) for t in w]
    v = _mx4_values(*flat) if state["kind"] == "moe4" else _affine_values(*flat)
    return v.reshape(n, rows, -1)


def _plain_moe(s):
    E, H, I, k = s["experts"], s["hidden"], s["inter"], s["top_k"]
    x = s["x"].float()
    # the choice of experts is a border: logits in 64 bits
    logits = s["x"].double() @ s["router"].double().t()
    top, ids = torch.sort(logits, dim=-1, descending=True, stable=True)
    ids = ids[:, :k]
    whole = top[:, :k] if s["renorm"] else top
    top = top - top[:, :1]
    p = (torch.exp(top[:, :k]) / torch.exp(whole - whole[:, :1]).sum(-1, keepdim=True)).float()
    y = torch.zeros_like(x)
    if s["m"] * k <= E:  # few slots: the chosen experts alone
        for j in range(k):
            g = torch.bmm(_experts(s, "gate", ids[:, j], I), x.unsqueeze(-1)).squeeze(-1)
            u = torch.bmm(_experts(s, "up", ids[:, j], I), x.unsqueeze(-1)).squeeze(-1)
            h = g / (1 + torch.exp(-g)) * u
            y += p[:, j:j + 1] * torch.bmm(_experts(s, "down", ids[:, j], H), h.unsqueeze(-1)).squeeze(-1)
    else:  # most experts are hit: every expert on every token, weighted by its share (0 where not chosen)
        share = torch.zeros(s["m"], E, device=x.device).scatter_(1, ids, p)
        for e in range(E):
            g = x @ _experts(s, "gate", slice(e, e + 1), I)[0].t()
            u = x @ _experts(s, "up", slice(e, e + 1), I)[0].t()
            h = g / (1 + torch.exp(-g)) * u
            y += share[:, e:e + 1] * (h @ _experts(s, "down", slice(e, e + 1), H)[0].t())
    return y.to(torch.bfloat16)


def _run_own(s):
    import weight_only_quantized_mlx_b200 as mq
    if s["kind"] == "roundtrip":
        mq.mlxq_mx4_quantize(s["x"], s["q"])
        mq.mlxq_mx4_dequant(s["q"], s["y"])
    elif s["kind"] == "weight4":
        mq.mlxq_mx4_gemm(s["hw"], s["x"], s["y"], s["m"])
    elif s["kind"] == "both4":
        mq.mlxq_mx4_quantize(s["x"], s["q"])
        mq.mlxq_mx4_matmul(s["hw"], s["q"], s["y"])
    else:
        call = mq.mlxq_mx4_moe if s["kind"] == "moe4" else mq.mlxq_moe
        flags = 0 if s["renorm"] else mq.MLXQ_MOE_SOFTMAX_ALL
        call(s["router"], *s["handles"], s["experts"], s["top_k"], s["x"], s["y"], s["m"], s["workspace"], flags=flags)
    return s["y"]


def run(state):
    if own:
        return _run_own(state)
    kind = state["kind"]
    if kind == "roundtrip":
        return _mx4_rounded(state["x"]).to(torch.bfloat16)
    if kind == "weight4":
        return (state["x"].float() @ _mx4_values(*state["w"]).t()).to(torch.bfloat16)
    if kind == "both4":
        return (_mx4_rounded(state["x"]) @ _mx4_values(*state["w"]).t()).to(torch.bfloat16)
    return _plain_moe(state)


# ---- what a pass cannot do without -----------------------------------------------------------
def work(case):
    b4 = 0.5 + 1.0 / BLOCK
    kind = case["kind"]
    if kind == "roundtrip":  # read x, write and read the codes and scales, write the values
        n = case["rows"] * case["cols"]
        return {"bytes": n * (2 + b4 + b4 + 2), "flops": 0}
    if kind in ("weight4", "both4"):
        m, n, k = case["m"], case["n"], case["k"]
        quantised = 2 * m * k * b4 if kind == "both4" else 0
        return {"bytes": n * k * b4 + m * k * 2 + quantised + m * n * 2, "flops": 2 * m * n * k}
    m, H, I, E, k = case["m"], case["hidden"], case["inter"], case["experts"], case["top_k"]
    hit = E * (1 - (1 - k / E) ** m)  # experts that at least one token chose, on average
    per = b4 if kind == "moe4" else 1 + 4 / case["group"]
    return {"bytes": hit * 3 * H * I * per + E * H * 2 + 2 * m * H * 2, "flops": 2 * m * (3 * k * H * I + E * H)}


# ---- the definitions in 64 bits ---------------------------------------------------------------
def _exact_mx4(codes, scales):
    c = codes.view(torch.uint8)  # two codes per byte, low nibble first (little-endian words)
    nib = torch.stack((c & 15, c >> 4), dim=-1).reshape(c.shape[0], -1).long()
    e, m = (nib >> 1) & 3, (nib & 1).double()
    mag = torch.where(e == 0, m * 0.5, (1 + m / 2) * torch.exp2((e - 1).double()))
    scale = torch.exp2(scales.double() - 127).repeat_interleave(BLOCK, dim=1)
    return torch.where(nib >= 8, -mag, mag) * scale


def _exact_round4(x):
    """Nearest E2M1 value of each element under its block's scale, ties to the even code."""
    v = x.double().reshape(x.shape[0], -1, BLOCK)
    top = v.abs().amax(-1, keepdim=True)
    exponent = (top.view(torch.int64) >> 52) - 1023  # the exponent field: floor(log2) of a normal number
    scale = torch.exp2((exponent - 2).clamp(-127, 127).double())
    a = v.abs() / scale
    code = torch.zeros_like(a)
    for i in range(7):  # the border between codes i and i + 1 belongs to the even one
        mid = (E2M1[i] + E2M1[i + 1]) / 2
        code += ((a > mid) if i % 2 == 0 else (a >= mid)).double()
    mag = _lut(x.device, torch.float64)[code.long()]
    return (torch.where(torch.signbit(v), -mag, mag) * scale).reshape(x.shape)


def _exact_affine(packed, s, b):
    q = packed.view(torch.uint8).double().reshape(*s.shape, -1)
    return (s.double().unsqueeze(-1) * q + b.double().unsqueeze(-1)).float().to(torch.bfloat16).double().reshape(packed.shape[0], -1)


def _rows(value, tensors, rows, product, chunk):
    """product(value of `chunk` rows at a time), joined along the last axis."""
    return torch.cat([product(value(*[t[r:r + chunk] for t in tensors])) for r in range(0, rows, chunk)], dim=-1)


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "roundtrip":
        return torch.cat([_exact_round4(s["x"][r:r + 2048]) for r in range(0, case["rows"], 2048)])
    if kind in ("weight4", "both4"):
        x = _exact_round4(s["x"]) if kind == "both4" else s["x"].double()
        return _rows(_exact_mx4, s["w"], case["n"], lambda w: x @ w.t(), 4096)
    value = _exact_mx4 if kind == "moe4" else _exact_affine
    H, I, k = case["hidden"], case["inter"], case["top_k"]
    x = s["x"].double()
    logits = (x @ s["router"].double().t()).cpu().numpy()
    y = torch.zeros(case["m"], H, dtype=torch.float64, device="cuda")
    chosen = {}
    for t in range(case["m"]):
        order = np.argsort(-logits[t], kind="stable")
        w = np.exp(logits[t] - logits[t].max())
        total = w[order[:k]].sum() if case["renorm"] else w.sum()
        for e in order[:k]:
            chosen.setdefault(int(e), []).append((t, float(w[e] / total)))
    for e, who in chosen.items():
        rows = torch.tensor([t for t, _ in who], device="cuda")
        p = torch.tensor([v for _, v in who], dtype=torch.float64, device="cuda").unsqueeze(-1)
        xe = x[rows]
        part = lambda name, n: [t[e * n:(e + 1) * n] for t in s[name]]
        g = _rows(value, part("gate", I), I, lambda w: xe @ w.t(), 4096)
        u = _rows(value, part("up", I), I, lambda w: xe @ w.t(), 4096)
        h = g * torch.sigmoid(g) * u
        y[rows] += p * _rows(value, part("down", H), H, lambda w: h @ w.t(), 4096)
    return y
