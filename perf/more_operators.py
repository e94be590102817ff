"""The operators of the 8-bit integer path, as they are measured.

Activations have one scale for each token, weights one for each output channel.
Each case is one pass as a user's program makes it:

  linear   linear_int8: one product of codes
  layer    quantize_int8 (RMSNorm absorbed) -> linear_int8
  mlp      quantize_int8 (RMSNorm absorbed) -> linear_silu_int8 -> linear_int8
  grouped  linear_grouped_int8: the product per expert segment, rows gathered
  experts  moe_route -> quantize_int8 -> linear_grouped_silu_int8 -> linear_grouped_int8 -> moe_combine

With ``own`` false a pass runs in elementary torch operations, with it true
through this package. ``exact`` computes the same in float64, written apart.

An int8 tensor is held as the package lays it out: codes i8 [G, R, 64] with
G = ceil(K / 64) and zeros past K, scales fp32 [R]; an entry is code times scale.
"""

import math

import numpy as np
import torch

own = False

EPS = 1e-5
STAGE = 64
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------
# The cases
# ---------------------------------------------------------------------------


def listed():
    return [
        # one token through the Llama-3.1-70B-shaped down projection: weight streaming, K split
        dict(op="linear", T=1, K=28672, O=8192, out="bf16", bias=False, name="linear decode 1x28672x8192"),
        # a prompt through the Llama-3.1-8B-shaped down projection: matrix rate
        dict(op="linear", T=2048, K=14336, O=4096, out="fp32", bias=False, name="linear prompt 2048x14336x4096"),
        # sizes that fit no tile, odd K and O, a bias
        dict(op="linear", T=333, K=4127, O=1001, out="fp32", bias=True, name="linear odd 333x4127x1001"),
        # one token of a served stream through a square projection behind its norm: launch latency
        dict(op="layer", T=1, K=4096, O=4096, out="bf16", bias=False, name="layer decode 1x4096x4096"),
        # a prompt through a fused query, key and value projection with a bias, Llama-3.1-8B-shaped
        dict(op="layer", T=2048, K=4096, O=6144, out="bf16", bias=True, name="layer prompt 2048x4096x6144"),
        # gated MLP block, eight decoding streams, Llama-3.1-70B-shaped
        dict(op="mlp", T=8, H=8192, I=28672, name="mlp decode 8x8192x28672"),
        # gated MLP block over a prompt, Llama-3.1-8B-shaped
        dict(op="mlp", T=2048, H=4096, I=14336, name="mlp prompt 2048x4096x14336"),
        # ragged expert segments (some empty), sizes that fit no tile
        dict(op="grouped", T=500, E=16, k=3, K=2077, O=1000, out="fp32", name="grouped odd 500x16"),
        # a few large experts over a prompt: matrix rate with ragged segments
        dict(op="grouped", T=1024, E=8, k=2, K=4096, O=14336, out="bf16", name="grouped prompt 1024x8"),
        # one token through a few large experts: two experts' weights are read
        dict(op="experts", T=1, E=8, k=2, H=4096, I=14336, name="experts single 1x8"),
        # expert layer of a few decoding streams, Qwen3-30B-A3B-shaped: nearly every pair has an expert of its own
        dict(op="experts", T=4, E=128, k=8, H=2048, I=768, name="experts decode 4x128"),
        # that layer over a prompt
        dict(op="experts", T=4096, E=128, k=8, H=2048, I=768, name="experts prompt 4096x128"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("linear", "linear", "layer", "mlp", "grouped", "grouped", "experts"))
    if op == "linear":
        return dict(op=op, T=_log_int(rng, 1, 2048), K=_log_int(rng, 200, 14336), O=_log_int(rng, 64, 4096),
                    out=rng.choice(("fp32", "bf16")), bias=rng.random() < 0.3)
    if op == "layer":
        return dict(op=op, T=_log_int(rng, 1, 2048), K=32 * _log_int(rng, 8, 256), O=_log_int(rng, 64, 6144),
                    out=rng.choice(("fp32", "bf16")), bias=rng.random() < 0.3)
    if op == "mlp":
        return dict(op=op, T=_log_int(rng, 1, 2048), H=128 * _log_int(rng, 4, 32), I=16 * _log_int(rng, 32, 896))
    if op == "grouped":
        E = _log_int(rng, 2, 64)
        return dict(op=op, T=_log_int(rng, 1, 2048), E=E, k=rng.randint(1, min(6, E)), K=_log_int(rng, 200, 4096),
                    O=_log_int(rng, 64, 2048), out=rng.choice(("fp32", "bf16")))
    E = _log_int(rng, 4, 128)
    return dict(op=op, T=_log_int(rng, 1, 4096), E=E, k=rng.randint(1, min(8, E)), H=128 * _log_int(rng, 4, 16),
                I=16 * _log_int(rng, 16, 64))


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)


def _rand(gen, *shape):
    return torch.rand(shape, generator=gen, device="cuda", dtype=torch.float32)


def _activation(gen, T, K):
    """Normal entries, 0.5% outlier channels of 20 times the size, a lognormal scale for each token."""
    x = _randn(gen, T, K)
    channels = torch.where(_rand(gen, K) < 0.005, 20.0, 1.0)
    return (x * channels * torch.exp(0.5 * _randn(gen, T, 1))).to(torch.bfloat16)


def _code(x):
    """fp32 [.., K] -> (codes as fp32 [.., K], scales fp32 [..]): the scale is amax / 127, a code the nearest to the
    quotient by it (ties to the even one). 64 bits, for a quotient may lie next to the middle of two codes."""
    scale = (x.abs().amax(-1).double() / 127).float()
    divisor = torch.where(scale > 0, scale, 1.0).double()
    return (x.double() / divisor[..., None]).round().clamp(-127, 127).float(), scale


def _laid_out(code, scale):
    """Codes [.., R, K] in stages of 64 entries, [.., G, R, 64]."""
    lead, R, K = code.shape[:-2], *code.shape[-2:]
    G = -(-K // STAGE)
    padded = torch.zeros((*lead, R, G * STAGE), dtype=torch.int8, device=code.device)
    padded[..., :K] = code.to(torch.int8)
    return padded.reshape(*lead, R, G, STAGE).transpose(-3, -2).contiguous(), scale


def _weight(gen, *shape):
    """An int8 weight [.., O, K] of N(0, 0.02) entries; with a leading dimension, one for each expert."""
    if len(shape) == 2:
        return _laid_out(*_code((0.02 * _randn(gen, *shape)).to(torch.bfloat16).float()))
    parts = [_weight(gen, *shape[1:]) for _ in range(shape[0])]
    return torch.stack([c for c, _ in parts]), torch.stack([s for _, s in parts])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(1000003 * int(seed) + 29)
    op, T = case["op"], case["T"]
    s = dict(case)
    if op in ("linear", "layer"):
        K, O = case["K"], case["O"]
        x = _activation(gen, T, K)
        if op == "linear":
            s["a"] = _laid_out(*_code(x.float()))
        else:
            s["x"] = x
            s["gamma"] = (0.5 + _rand(gen, K)).to(torch.bfloat16)
        s["w"] = _weight(gen, O, K)
        s["b"] = _randn(gen, O) if case["bias"] else None
    elif op == "mlp":
        s["x"] = _activation(gen, T, case["H"])
        s["gamma"] = (0.5 + _rand(gen, case["H"])).to(torch.bfloat16)
        s["gu"] = _weight(gen, 2 * case["I"], case["H"])
        s["dn"] = _weight(gen, case["H"], case["I"])
    elif op == "grouped":
        E, k = case["E"], case["k"]
        s["a"] = _laid_out(*_code(_activation(gen, T, case["K"]).float()))
        s["w"] = _weight(gen, E, case["O"], case["K"])
        favour = _randn(gen, E)  # some experts take most tokens, some hardly any
        chosen = (favour + _randn(gen, T, E)).argsort(1, descending=True)[:, :k]
        order = chosen.reshape(-1).argsort(stable=True)
        s["rows"] = (order // k).to(torch.int32)
        s["seg"] = torch.cat([chosen.new_zeros(1), chosen.reshape(-1).bincount(minlength=E).cumsum(0)]).to(torch.int32)
    else:
        s["x"] = _activation(gen, T, case["H"])
        s["logits"] = _randn(gen, T, case["E"])
        s["gu"] = _weight(gen, case["E"], 2 * case["I"], case["H"])
        s["dn"] = _weight(gen, case["E"], case["H"], case["I"])
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import activation_sparsity_fp4_amd as sq

    op = s["op"]
    if op == "linear":
        return sq.linear_int8(sq.Int8(*s["a"], s["K"]), sq.Int8(*s["w"], s["K"]), dtype=DTYPES[s["out"]], bias=s["b"])
    if op == "layer":
        a = sq.quantize_int8(s["x"], gamma=s["gamma"], rms_eps=EPS)
        return sq.linear_int8(a, sq.Int8(*s["w"], s["K"]), dtype=DTYPES[s["out"]], bias=s["b"])
    if op == "grouped":
        return sq.linear_grouped_int8(sq.Int8(*s["a"], s["K"]), sq.Int8(*s["w"], s["K"]), s["seg"], s["rows"],
                                      dtype=DTYPES[s["out"]])
    H, I = s["H"], s["I"]
    gu, dn = sq.Int8(*s["gu"], H), sq.Int8(*s["dn"], I)
    if op == "mlp":
        a = sq.quantize_int8(s["x"], gamma=s["gamma"], rms_eps=EPS)
        return sq.linear_int8(sq.linear_silu_int8(a, gu), dn, dtype=torch.bfloat16)
    r = sq.moe_route(s["logits"], s["k"])
    a = sq.quantize_int8(s["x"])
    h = sq.linear_grouped_silu_int8(a, gu, r.seg_offsets, r.a_rows)
    y = sq.linear_grouped_int8(h, dn, r.seg_offsets, dtype=torch.bfloat16)
    return sq.moe_combine(y, r.pair_index, r.weight, bf16=True)


def _rows(tensor, K):
    """(codes fp32 [.., R, K], scales [.., R]) of an int8 tensor."""
    code, scale = tensor
    lead, (G, R, _) = code.shape[:-3], code.shape[-3:]
    return code.transpose(-3, -2).reshape(*lead, R, G * STAGE)[..., :K].float(), scale


def _normed(x, gamma):
    """The RMS-normed rows: 1/rms from a sum in 64 bits, the normed entry a bf16, its product with gamma exact."""
    x = x.float()
    r = 1 / torch.sqrt(x.double().square().mean(1, keepdim=True) + EPS)
    return (x * r.float()).to(torch.bfloat16).float() * gamma.float()


def _product(a, w):
    (qa, sa), (qw, sw) = a, w
    return qa @ qw.T * sa[:, None] * sw


def _gated(y):
    """bf16(silu(gate) up) of [gate | up], as fp32."""
    g, u = y.chunk(2, -1)
    return (g / (1 + torch.exp(-g)) * u).to(torch.bfloat16).float()


def _per_expert(a, w, seg):
    """Row p of [P, K] times the weight of the expert whose segment holds it: [P, O]."""
    (qa, sa), (qw, sw) = a, w
    E = qw.shape[0]
    counts = (seg[1:] - seg[:-1]).long()
    place = torch.arange(qa.shape[0], device=qa.device)
    expert = torch.searchsorted(seg[1:].long(), place, right=True)
    inside = place - seg.long()[expert]
    padded = qa.new_zeros((E, qa.shape[1], int(counts.max())))
    padded[expert, :, inside] = qa
    return torch.bmm(qw, padded)[expert, :, inside] * sa[:, None] * sw[expert]


def _route_plain(x, k):
    """The k largest of softmax(x), their weights and the pairs sorted by expert."""
    T, E = x.shape
    s = torch.exp(x.double() - x.double().amax(1, keepdim=True))
    expert = x.sort(dim=1, descending=True, stable=True)[1][:, :k]
    weight = s.gather(1, expert)
    weight = (weight / weight.sum(1, keepdim=True)).float()
    by = expert.reshape(-1)
    order = by.argsort(stable=True)
    seg = torch.cat([by.new_zeros(1), by.bincount(minlength=E).cumsum(0)])
    place = torch.empty_like(order).scatter_(0, order, torch.arange(T * k, device=x.device)).reshape(T, k)
    return weight, order // k, seg, place


def _run_plain(s):
    op = s["op"]
    if op in ("linear", "layer"):
        a = _rows(s["a"], s["K"]) if op == "linear" else _code(_normed(s["x"], s["gamma"]))
        y = _product(a, _rows(s["w"], s["K"]))
        return (y if s["b"] is None else y + s["b"]).to(DTYPES[s["out"]])
    if op == "grouped":
        code, scale = _rows(s["a"], s["K"])
        rows = s["rows"].long()
        return _per_expert((code[rows], scale[rows]), _rows(s["w"], s["K"]), s["seg"]).to(DTYPES[s["out"]])
    H, I = s["H"], s["I"]
    gu, dn = _rows(s["gu"], H), _rows(s["dn"], I)
    if op == "mlp":
        h = _gated(_product(_code(_normed(s["x"], s["gamma"])), gu))
        return _product(_code(h), dn).to(torch.bfloat16)
    weight, rows, seg, place = _route_plain(s["logits"], s["k"])
    code, scale = _code(s["x"].float())
    h = _gated(_per_expert((code[rows], scale[rows]), gu, seg))
    y = _per_expert(_code(h), dn, seg)
    return (y[place] * weight[..., None]).sum(1).to(torch.bfloat16)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------


def work(case):
    op, T = case["op"], case["T"]
    if op in ("linear", "layer"):
        K, O = case["K"], case["O"]
        item = 4 if case["out"] == "fp32" else 2
        a = T * K + 4 * T if op == "linear" else 2 * T * K + 2 * K
        return {"bytes": a + K * O + 4 * O * (1 + case["bias"]) + T * O * item, "flops": 2 * T * O * K}
    if op == "mlp":
        H, I = case["H"], case["I"]
        return {"bytes": 4 * T * H + 2 * H + 3 * H * I + 8 * I + 4 * H, "flops": 6 * T * H * I}
    E, k = case["E"], case["k"]
    used = E * (1 - (1 - k / E) ** T)  # experts that some token chose, on average
    if op == "grouped":
        K, O = case["K"], case["O"]
        return {"bytes": T * (K + 4) + used * O * (K + 4) + T * k * (4 + O * (4 if case["out"] == "fp32" else 2)),
                "flops": 2 * T * k * O * K}
    H, I = case["H"], case["I"]
    return {"bytes": 4 * T * H + 4 * T * E + (3 * H * I + 8 * I + 4 * H) * used, "flops": 6 * T * k * H * I}


# ---------------------------------------------------------------------------
# The same in 64 bits
# ---------------------------------------------------------------------------


def _exact_values(tensor, K):
    codes, scales = tensor
    values = torch.cat(codes.double().unbind(-3), -1)[..., :K]  # the stages of a row, one after the other
    return values * scales.double()[..., None]


def _exact_rounded(x):
    """float64 rows as their codes give them back: the grid value below or above, whichever is nearer."""
    top = torch.maximum(x.amax(-1, keepdim=True), -x.amin(-1, keepdim=True))
    unit = (top / 127).float().double()
    at = x.abs() / unit.clamp(min=2.0 ** -149)
    below = torch.floor(at)
    rest = at - below
    up = (rest > 0.5) | ((rest == 0.5) & (below % 2 == 1))
    return torch.sign(x) * (below + up.double()).clamp(max=127) * unit


def _exact_normed(x, gamma):
    x = x.double()
    r = (1 / torch.sqrt((x * x).sum(1, keepdim=True) / x.shape[1] + EPS)).float().double()
    return (x * r).float().to(torch.bfloat16).double() * gamma.double()


def _exact_gated(y):
    half = y.shape[-1] // 2
    gate, up = y[..., :half], y[..., half:]
    return (gate * torch.sigmoid(gate) * up).to(torch.bfloat16).double()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("linear", "layer"):
        K = case["K"]
        a = _exact_values(s["a"], K) if op == "linear" else _exact_rounded(_exact_normed(s["x"], s["gamma"]))
        y = torch.mm(a, _exact_values(s["w"], K).T.contiguous())
        return y if s["b"] is None else y + s["b"].double()
    if op == "grouped":
        a, seg = _exact_values(s["a"], case["K"]), s["seg"].tolist()
        parts = [a[s["rows"][lo:hi].long()] @ _exact_values((s["w"][0][e], s["w"][1][e]), case["K"]).T.contiguous()
                 for e, (lo, hi) in enumerate(zip(seg[:-1], seg[1:]))]
        return torch.cat(parts)
    H, I = case["H"], case["I"]
    if op == "mlp":
        a = _exact_rounded(_exact_normed(s["x"], s["gamma"]))
        h = _exact_rounded(_exact_gated(a @ _exact_values(s["gu"], H).T.contiguous()))
        return h @ _exact_values(s["dn"], I).T.contiguous()
    logits = s["logits"].double().cpu().numpy()
    expert = np.argsort(-logits, axis=1, kind="stable")[:, :case["k"]]
    e = np.exp(np.take_along_axis(logits, expert, 1) - logits.max(1, keepdims=True))
    weight = e / e.sum(1, keepdims=True)
    a = _exact_rounded(s["x"].double())
    y = torch.zeros_like(a)
    for number in range(case["E"]):
        t, j = np.nonzero(expert == number)
        if t.size:
            rows = torch.as_tensor(t, device="cuda")
            gu = _exact_values((s["gu"][0][number], s["gu"][1][number]), H)
            dn = _exact_values((s["dn"][0][number], s["dn"][1][number]), I)
            h = _exact_rounded(_exact_gated(a[rows] @ gu.T.contiguous()))
            y[rows] += (h @ dn.T.contiguous()) * torch.as_tensor(weight[t, j], device="cuda")[:, None]
    return y
