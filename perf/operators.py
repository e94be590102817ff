"""The operators of the plain MXFP4 path and of expert routing, as they are measured.

Each case is one pass as a user's program makes it:

  route    moe_route: router logits -> chosen experts, weights and the sorted dispatch plan
  linear   linear_mxfp4: one plain MXFP4 product
  grouped  linear_grouped_mxfp4: the product per expert segment, rows gathered
  mlp      quantize_mxfp4 (RMSNorm absorbed) -> linear_silu_mxfp4 -> linear_mxfp4
  experts  moe_route -> quantize_mxfp4 -> linear_grouped_silu_mxfp4 -> linear_grouped_mxfp4 -> moe_combine

With ``own`` false a pass runs in elementary torch operations, with it true
through this package. ``exact`` computes the same in float64, written apart.

MXFP4 tensors are held as the package lays them out: codes u8 [G, R, 64] and
scales u8 [G, R, 4] with G = ceil(K / 128), padding bytes zero.
"""

import math

import numpy as np
import torch

own = False

EPS = 1e-5
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------------------
# The cases
# ---------------------------------------------------------------------------


def _route(T, E, k, score="softmax", logits="fp32", bias=False, groups=1, top_groups=1, group_score="max",
           renormalize=True, scale=1.0, pad=0, masked=0.0):
    return dict(op="route", T=T, E=E, k=k, score=score, logits=logits, bias=bias, groups=groups,
                top_groups=top_groups, group_score=group_score, renormalize=renormalize, scale=scale, pad=pad,
                masked=masked)


def listed():
    cases = [
        # one token of a served stream through a Qwen3-30B-A3B-shaped router: launch latency
        dict(_route(1, 128, 8), name="route decode 1x128"),
        # that router over a prompt, logits as a bf16 gate projection writes them
        dict(_route(4096, 128, 8, logits="bf16"), name="route prompt 4096x128"),
        # sigmoid scores, balance bias, 4 of 8 groups, a large batch of prompts
        dict(_route(16384, 256, 8, score="sigmoid", bias=True, groups=8, top_groups=4, group_score="sum2",
                    scale=2.5), name="route groups 16384x256"),
        # odd sizes, strided rows, masked experts, a padded batch (rows past the last token)
        dict(_route(777, 60, 4, logits="fp16", renormalize=False, pad=57, masked=0.05), name="route ragged 777x60"),
        # one token through the Llama-3.1-70B-shaped down projection: weight streaming, K split
        dict(op="linear", T=1, K=28672, O=8192, out="bf16", name="linear decode 1x28672x8192"),
        # a prompt through the Llama-3.1-8B-shaped down projection: matrix rate
        dict(op="linear", T=2048, K=14336, O=4096, out="fp32", name="linear prompt 2048x14336x4096"),
        # sizes that fit no tile, K a multiple of 32 only
        dict(op="linear", T=333, K=4128, O=1000, out="fp32", name="linear odd 333x4128x1000"),
        # gated MLP block, eight decoding streams, Llama-3.1-70B-shaped
        dict(op="mlp", T=8, H=8192, I=28672, name="mlp decode 8x8192x28672"),
        # gated MLP block over a prompt, Llama-3.1-8B-shaped
        dict(op="mlp", T=2048, H=4096, I=14336, name="mlp prompt 2048x4096x14336"),
        # ragged expert segments (some empty), sizes that fit no tile
        dict(op="grouped", T=500, E=16, k=3, K=2080, O=1000, out="fp32", name="grouped odd 500x16"),
        # expert layer of a few decoding streams, Qwen3-30B-A3B-shaped: nearly every pair has an expert of its own
        dict(op="experts", T=4, E=128, k=8, H=2048, I=768, name="experts decode 4x128"),
        # that layer over a prompt
        dict(op="experts", T=4096, E=128, k=8, H=2048, I=768, name="experts prompt 4096x128"),
    ]
    return cases


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("route", "route", "linear", "linear", "mlp", "grouped", "experts"))
    if op == "route":
        groups = rng.choice((1, 1, 2, 4, 8))
        E = groups * _log_int(rng, 8 // min(groups, 4), 512 // groups)
        E = max(E, 2 * groups)
        top_groups = rng.randint(1, groups)
        k = rng.randint(1, min(10, E // groups * top_groups))
        return _route(_log_int(rng, 1, 16384), E, k, score=rng.choice(("softmax", "sigmoid")),
                      logits=rng.choice(("fp32", "bf16", "fp16")), bias=rng.random() < 0.5, groups=groups,
                      top_groups=top_groups, group_score=rng.choice(("max", "sum2")),
                      renormalize=rng.random() < 0.7, scale=rng.choice((1.0, 2.5)), pad=rng.choice((0, 0, 3, 64)),
                      masked=rng.choice((0.0, 0.0, 0.05)))
    if op == "linear":
        T = _log_int(rng, 1, 2048)
        return dict(op="linear", T=T, K=32 * _log_int(rng, 8, 448), O=_log_int(rng, 64, 4096),
                    out=rng.choice(("fp32", "bf16")))
    if op == "mlp":
        return dict(op="mlp", T=_log_int(rng, 1, 2048), H=128 * _log_int(rng, 4, 32), I=128 * _log_int(rng, 4, 112))
    if op == "grouped":
        E = _log_int(rng, 2, 64)
        return dict(op="grouped", T=_log_int(rng, 1, 2048), E=E, k=rng.randint(1, min(6, E)),
                    K=32 * _log_int(rng, 8, 96), O=_log_int(rng, 64, 2048), out=rng.choice(("fp32", "bf16")))
    E = _log_int(rng, 4, 128)
    return dict(op="experts", T=_log_int(rng, 1, 4096), E=E, k=rng.randint(1, min(8, E)),
                H=128 * _log_int(rng, 4, 16), I=128 * _log_int(rng, 2, 8))


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)


def _rand(gen, *shape):
    return torch.rand(shape, generator=gen, device="cuda", dtype=torch.float32)


def _activation(gen, T, K):
    """Normal entries, 0.5% outlier channels of 50 times the size, a lognormal scale for each token."""
    x = _randn(gen, T, K)
    channels = torch.where(_rand(gen, K) < 0.005, 50.0, 1.0)
    return (x * channels * torch.exp(0.5 * _randn(gen, T, 1))).to(torch.bfloat16)


def _mxfp4(x):
    """fp32 [R, K] -> (codes [G, R, 64], scales [G, R, 4]): E8M0 exponent floor(log2 amax) - 2, E2M1 codes to nearest
    (ties to the even code), saturated at 6."""
    code, exponent = _code(x)
    R, K = x.shape
    G = -(-K // 128)
    sign = torch.signbit(x).to(torch.uint8) << 3
    nibble = torch.zeros((R, G * 128), dtype=torch.uint8, device=x.device)
    nibble[:, :K] = code.to(torch.uint8).reshape(R, K) | sign
    codes = nibble[:, 0::2] | (nibble[:, 1::2] << 4)
    scales = torch.zeros((R, G * 4), dtype=torch.uint8, device=x.device)
    scales[:, :K // 32] = (exponent + 127).to(torch.uint8)
    return (codes.reshape(R, G, 64).permute(1, 0, 2).contiguous(),
            scales.reshape(R, G, 4).permute(1, 0, 2).contiguous())


def _power(e):
    """2^e in fp32 for int32 exponents above -127 (0 at -127, the scale of an all-zero block)."""
    return ((e + 127) << 23).view(torch.float32)


def _code(x):
    """Code index 0..7 of every entry's magnitude [R, K/32, 32] and the exponents [R, K/32] of the blocks' scales."""
    a = x.abs().reshape(x.shape[0], -1, 32)
    amax = a.amax(-1)
    exponent = torch.where(amax > 0, torch.frexp(amax)[1] - 3, -127).clamp(-127, 127).int()
    v = a * _power(-exponent)[..., None]
    code = ((v > 0.25).to(torch.int8) + (v >= 0.75) + (v > 1.25) + (v >= 1.75) + (v > 2.5) + (v >= 3.5) + (v > 5.0))
    return code, exponent


def _weight(gen, *shape):
    """An MXFP4 weight [.., O, K] of N(0, 0.02) entries; with a leading dimension, one tensor for each expert."""
    if len(shape) == 2:
        return _mxfp4((0.02 * _randn(gen, *shape)).to(torch.bfloat16).float())
    E, O, K = shape
    codes, scales = _mxfp4((0.02 * _randn(gen, E * O, K)).to(torch.bfloat16).float())
    G = codes.shape[0]
    return (codes.reshape(G, E, O, 64).transpose(0, 1).contiguous(),
            scales.reshape(G, E, O, 4).transpose(0, 1).contiguous())


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(1000003 * int(seed) + 17)
    op, T = case["op"], case["T"]
    s = dict(case)
    if op == "route":
        E = case["E"]
        rows = T + case["pad"]
        buffer = 1.5 * _randn(gen, rows, E + (8 if case["pad"] else 0))
        if case["masked"]:
            buffer[_rand(gen, *buffer.shape) < case["masked"]] = -math.inf
            buffer[T // 2] = -math.inf  # a row without any expert
        s["x"] = buffer.to(DTYPES[case["logits"]])[:, :E]
        s["b"] = 0.1 * _randn(gen, E) if case["bias"] else None
        s["n"] = torch.tensor([T], dtype=torch.int32, device="cuda") if case["pad"] else None
    elif op == "linear":
        s["a"] = _mxfp4(_activation(gen, T, case["K"]).float())
        s["w"] = _weight(gen, case["O"], case["K"])
    elif op == "mlp":
        s["x"] = _activation(gen, T, case["H"])
        s["gamma"] = (0.5 + _rand(gen, case["H"])).to(torch.bfloat16)
        s["gu"] = _weight(gen, 2 * case["I"], case["H"])
        s["dn"] = _weight(gen, case["H"], case["I"])
    elif op == "grouped":
        E, k = case["E"], case["k"]
        s["a"] = _mxfp4(_activation(gen, T, case["K"]).float())
        s["w"] = _weight(gen, E, case["O"], case["K"])
        favour = 2.0 * _randn(gen, E)  # some experts take most tokens, some none
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
    if op == "route":
        r = sq.moe_route(s["x"], s["k"], score=s["score"], bias=s["b"], groups=s["groups"],
                         top_groups=s["top_groups"], group_score=s["group_score"], renormalize=s["renormalize"],
                         scale=s["scale"], num_tokens=s["n"])
        return {"expert": r.expert, "weight": r.weight, "seg_offsets": r.seg_offsets, "a_rows": r.a_rows,
                "pair_index": r.pair_index}
    if op == "linear":
        return sq.linear_mxfp4(sq.MXFP4(*s["a"], s["K"]), sq.MXFP4(*s["w"], s["K"]), dtype=DTYPES[s["out"]])
    if op == "grouped":
        return sq.linear_grouped_mxfp4(sq.MXFP4(*s["a"], s["K"]), sq.MXFP4(*s["w"], s["K"]), s["seg"], s["rows"],
                                       dtype=DTYPES[s["out"]])
    H, I = s["H"], s["I"]
    gu, dn = sq.MXFP4(*s["gu"], H), sq.MXFP4(*s["dn"], I)
    if op == "mlp":
        a = sq.quantize_mxfp4(s["x"], gamma=s["gamma"], rms_eps=EPS)
        return sq.linear_mxfp4(sq.linear_silu_mxfp4(a, gu), dn, dtype=torch.bfloat16)
    r = sq.moe_route(s["logits"], s["k"])
    a = sq.quantize_mxfp4(s["x"])
    h = sq.linear_grouped_silu_mxfp4(a, gu, r.seg_offsets, r.a_rows)
    y = sq.linear_grouped_mxfp4(h, dn, r.seg_offsets, dtype=torch.bfloat16)
    return sq.moe_combine(y, r.pair_index, r.weight, bf16=True)


def _values(tensor, K):
    """The fp32 values [.., R, K] of an MXFP4 tensor."""
    codes, scales = tensor
    lead = codes.shape[:-3]
    G, R, _ = codes.shape[-3:]
    codes = codes.transpose(-3, -2).reshape(*lead, R, G * 64)[..., :K // 2]
    scales = scales.transpose(-3, -2).reshape(*lead, R, G * 4)[..., :K // 32]
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    v = table[torch.stack([codes & 15, codes >> 4], -1).int()].reshape(*lead, R, K // 32, 32)
    return (v * _power(scales.int() - 127)[..., None]).reshape(*lead, R, K)


def _rounded(x):
    """The values that fp32 rows have in MXFP4."""
    code, exponent = _code(x)
    v = torch.tensor(E2M1, device=x.device)[code.int()]
    return (v * _power(exponent)[..., None]).reshape(x.shape) * torch.where(torch.signbit(x), -1.0, 1.0)


def _gated(y):
    """bf16(silu(gate) up) of [gate | up], as fp32."""
    g, u = y.chunk(2, -1)
    return (g / (1 + torch.exp(-g)) * u).to(torch.bfloat16).float()


def _per_expert(a, w, seg):
    """Row p of a [P, K] times the weight of the expert whose segment holds it: [P, O]."""
    E = w.shape[0]
    counts = (seg[1:] - seg[:-1]).long()
    place = torch.arange(a.shape[0], device=a.device)
    expert = torch.searchsorted(seg[1:].long(), place, right=True)
    inside = place - seg.long()[expert]
    padded = a.new_zeros((E, a.shape[1], int(counts.max())))
    padded[expert, :, inside] = a
    return torch.bmm(w, padded)[expert, :, inside]


def _route_plain(x, k, score, bias, groups, top_groups, group_score, renormalize, scale, n):
    T, E = x.shape
    live = x > -math.inf
    if n is not None:
        live = live & (torch.arange(T, device=x.device) < n)[:, None]
    x = x.double().clamp(max=torch.finfo(torch.float32).max)
    x = torch.where(live, x, -math.inf)
    if score == "softmax":
        top = torch.where(live.any(1, keepdim=True), x.amax(1, keepdim=True), 0.0)
        e = torch.exp(x - top)
        s = e / e.sum(1, keepdim=True).clamp(min=1e-300)
    else:
        s = 1 / (1 + torch.exp(-x))
    key = x if bias is None else torch.where(live, s + bias.double(), -math.inf)
    if groups > 1:
        part = (key if group_score == "max" else torch.where(live, s if bias is None else key, -math.inf))
        best = part.reshape(T, groups, -1).sort(dim=2, descending=True)[0][..., :1 if group_score == "max" else 2]
        total = best[..., 0] + (best[..., 1:].clamp(min=-1e300) * (best[..., 1:] > -math.inf)).sum(2)
        kept = total.sort(dim=1, descending=True, stable=True)[1][:, :top_groups]
        keep = torch.zeros((T, groups), dtype=torch.bool, device=x.device).scatter_(1, kept, True)
        key = torch.where(keep.repeat_interleave(E // groups, 1), key, -math.inf)
    key, expert = key.sort(dim=1, descending=True, stable=True)
    key, expert = key[:, :k], expert[:, :k]
    empty = key == -math.inf
    weight = torch.where(empty, 0.0, s.gather(1, expert))
    if renormalize:
        weight = weight / weight.sum(1, keepdim=True).clamp(min=1e-300)
    expert = torch.where(empty, -1, expert)
    by = torch.where(empty, E, expert).reshape(-1)
    order = by.argsort(stable=True)
    count = by.bincount(minlength=E + 1).cumsum(0)
    seg = torch.cat([count.new_zeros(1), count[:E]])
    rows = torch.where(torch.arange(T * k, device=x.device) < seg[E], order // k, -1)
    place = torch.empty_like(order).scatter_(0, order, torch.arange(T * k, device=x.device))
    place = torch.where(empty, -1, place.reshape(T, k))
    return {"expert": expert.int(), "weight": (scale * weight).float(), "seg_offsets": seg.int(),
            "a_rows": rows.int(), "pair_index": place.int()}


def _run_plain(s):
    op = s["op"]
    if op == "route":
        return _route_plain(s["x"], s["k"], s["score"], s["b"], s["groups"], s["top_groups"], s["group_score"],
                            s["renormalize"], s["scale"], s["n"])
    if op == "linear":
        return (_values(s["a"], s["K"]) @ _values(s["w"], s["K"]).T).to(DTYPES[s["out"]])
    if op == "grouped":
        a = _values(s["a"], s["K"])[s["rows"].long()]
        return _per_expert(a, _values(s["w"], s["K"]), s["seg"]).to(DTYPES[s["out"]])
    x, H, I = s["x"].float(), s["H"], s["I"]
    if op == "mlp":
        r = 1 / torch.sqrt(x.double().square().mean(1, keepdim=True) + EPS)
        a = _rounded((x * r.float()).to(torch.bfloat16).float() * s["gamma"].float())
        h = _rounded(_gated(a @ _values(s["gu"], H).T))
        return (h @ _values(s["dn"], I).T).to(torch.bfloat16)
    r = _route_plain(s["logits"], s["k"], "softmax", None, 1, 1, "max", True, 1.0, None)
    a = _rounded(x)[r["a_rows"].long()]
    h = _rounded(_gated(_per_expert(a, _values(s["gu"], H), r["seg_offsets"])))
    y = _per_expert(h, _values(s["dn"], I), r["seg_offsets"])
    return (y[r["pair_index"].long()] * r["weight"][..., None]).sum(1).to(torch.bfloat16)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------


def work(case):
    op, T = case["op"], case["T"]
    mx = 17 / 32  # bytes of an MXFP4 entry
    if op == "route":
        rows, E, k = T + case["pad"], case["E"], case["k"]
        item = 4 if case["logits"] == "fp32" else 2
        return {"bytes": T * E * item + 4 * E * case["bias"] + 16 * rows * k + 4 * (E + 1), "flops": 4 * T * E}
    if op == "linear":
        K, O = case["K"], case["O"]
        return {"bytes": mx * K * (T + O) + T * O * (4 if case["out"] == "fp32" else 2), "flops": 2 * T * O * K}
    if op == "mlp":
        H, I = case["H"], case["I"]
        return {"bytes": 4 * T * H + 2 * H + 3 * mx * H * I, "flops": 6 * T * H * I}
    E, k = case["E"], case["k"]
    used = E * (1 - (1 - k / E) ** T)  # experts that some token chose, on average
    if op == "grouped":
        K, O = case["K"], case["O"]
        return {"bytes": mx * K * (T + used * O) + T * k * (4 + O * (4 if case["out"] == "fp32" else 2)),
                "flops": 2 * T * k * O * K}
    H, I = case["H"], case["I"]
    return {"bytes": 4 * T * H + 4 * T * E + 3 * mx * H * I * used, "flops": 6 * T * k * H * I}


# ---------------------------------------------------------------------------
# The same in 64 bits
# ---------------------------------------------------------------------------


def _exact_values(tensor, K):
    codes, scales = (t.cpu().numpy() if t.numel() < (1 << 22) else t for t in tensor)
    codes, scales = torch.as_tensor(codes, device="cuda"), torch.as_tensor(scales, device="cuda")
    blocks = codes.reshape(*codes.shape[:-1], 4, 16)  # 4 blocks of 16 bytes in each stage
    nibbles = torch.empty((*blocks.shape[:-1], 32), dtype=torch.uint8, device="cuda")
    nibbles[..., 0::2] = blocks % 16
    nibbles[..., 1::2] = blocks // 16
    magnitude = (nibbles % 8).double()
    # 0, 0.5, then (1 + m / 2) 2^(e - 1) for the two exponent bits e and the mantissa bit m
    e, m = magnitude.div(2, rounding_mode="floor"), magnitude % 2
    value = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * torch.exp2(e - 1))
    value = value * (1 - 2 * (nibbles >= 8).double()) * torch.exp2(scales.double() - 127)[..., None]
    value = value.reshape(*codes.shape[:-1], 128)
    value = torch.cat(value.unbind(-3), -1)  # the stages of a row, one after the other
    return value[..., :K]


def _exact_rounded(x):
    """float64 rows rounded to MXFP4 by their distances to the grid."""
    grid = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    blocks = x.reshape(*x.shape[:-1], -1, 32)
    top = blocks.abs().amax(-1, keepdim=True)
    power = torch.floor(torch.log2(top.clamp(min=2.0 ** -140)))
    power = power - (torch.exp2(power) > top).double() + (torch.exp2(power + 1) <= top).double()
    unit = torch.exp2((power - 2).clamp(-127, 127))
    v = blocks.abs() / unit
    lower = (torch.bucketize(v, grid, right=True) - 1).clamp(0, 7)
    upper = (lower + 1).clamp(max=7)
    down, up = v - grid[lower], grid[upper] - v
    code = torch.where((up < down) | ((up == down) & (lower % 2 == 1)), upper, lower)
    return (torch.sign(blocks) * grid[code] * unit).reshape(x.shape)


def _exact_gated(y):
    half = y.shape[-1] // 2
    gate, up = y[..., :half], y[..., half:]
    return (gate * torch.sigmoid(gate) * up).to(torch.bfloat16).double()


def _exact_route(x, k, score, bias, groups, top_groups, group_score, renormalize, scale, n):
    """Expert ids and weights of each row, in numpy."""
    x = x.double().cpu().numpy()
    T, E = x.shape
    n = T if n is None else int(n)
    x = np.minimum(np.where(np.isnan(x), -np.inf, x), np.finfo(np.float32).max)
    x[n:] = -np.inf
    live = x > -np.inf
    with np.errstate(invalid="ignore", over="ignore"):
        if score == "softmax":
            e = np.where(live, np.exp(x - x.max(1, keepdims=True)), 0)
            s = e / np.maximum(e.sum(1, keepdims=True), 1e-300)
        else:
            s = np.where(live, 1 / (1 + np.exp(-x)), 0)
    key = x if bias is None else np.where(live, s + bias.double().cpu().numpy(), -np.inf)
    if groups > 1:
        size = E // groups
        grouped = (key if bias is not None or group_score == "max" else np.where(live, s, -np.inf)).reshape(T, groups, size)
        ranked = -np.sort(-grouped, axis=2)
        total = ranked[:, :, 0].copy()
        if group_score == "sum2" and size > 1:
            total += np.where(np.isfinite(ranked[:, :, 1]), ranked[:, :, 1], 0)
        best = np.argsort(-total, axis=1, kind="stable")[:, :top_groups]
        out = np.ones((T, groups), bool)
        np.put_along_axis(out, best, False, 1)
        key = np.where(np.repeat(out, size, axis=1), -np.inf, key)
    expert = np.argsort(-key, axis=1, kind="stable")[:, :k]
    gone = np.take_along_axis(key, expert, 1) == -np.inf
    weight = np.where(gone, 0, np.take_along_axis(s, expert, 1))
    if renormalize:
        weight = weight / np.maximum(weight.sum(1, keepdims=True), 1e-300)
    return np.where(gone, -1, expert), scale * weight


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        _, weight = _exact_route(s["x"], s["k"], s["score"], s["b"], s["groups"], s["top_groups"], s["group_score"],
                                 s["renormalize"], s["scale"], s["n"])
        return {"expert": None, "weight": weight, "seg_offsets": None, "a_rows": None, "pair_index": None}
    if op == "linear":
        return torch.mm(_exact_values(s["a"], s["K"]), _exact_values(s["w"], s["K"]).T.contiguous())
    if op == "grouped":
        a, seg = _exact_values(s["a"], s["K"]), s["seg"].tolist()
        parts = [a[s["rows"][lo:hi].long()] @ _exact_values((s["w"][0][e], s["w"][1][e]), s["K"]).T.contiguous()
                 for e, (lo, hi) in enumerate(zip(seg[:-1], seg[1:]))]
        return torch.cat(parts)
    x, H, I = s["x"].double(), s["H"], s["I"]
    if op == "mlp":
        r = (1 / torch.sqrt((x * x).sum(1, keepdim=True) / H + EPS)).float().double()
        normed = (x * r).float().to(torch.bfloat16).double() * s["gamma"].double()
        h = _exact_rounded(_exact_gated(_exact_rounded(normed) @ _exact_values(s["gu"], H).T.contiguous()))
        return h @ _exact_values(s["dn"], I).T.contiguous()
    expert, weight = _exact_route(s["logits"], s["k"], "softmax", None, 1, 1, "max", True, 1.0, None)
    a = _exact_rounded(x)
    y = torch.zeros_like(x)
    for e in range(case["E"]):
        t, j = np.nonzero(expert == e)
        if t.size:
            rows = torch.as_tensor(t, device="cuda")
            gu = _exact_values((s["gu"][0][e], s["gu"][1][e]), H)
            dn = _exact_values((s["dn"][0][e], s["dn"][1][e]), I)
            h = _exact_rounded(_exact_gated(a[rows] @ gu.T.contiguous()))
            y[rows] += (h @ dn.T.contiguous()) * torch.as_tensor(weight[t, j], device="cuda")[:, None]
    return y
