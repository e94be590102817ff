"""GPU parity of the expert routing against the float64 oracle: ids and plan
equal, weights within one rounding to fp32 (2^-24 relative) of float64's and
its own few roundings (2^-45 covers them)."""

import numpy as np
import pytest

from oracle import moe_route_ref
from gpu_util import f32_to_gpu, i32_to_gpu, to_np

pytestmark = pytest.mark.gpu

PLAN = ("expert", "seg_offsets", "a_rows", "pair_index")


@pytest.fixture(scope="module")
def sq():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    import activation_sparsity_fp4_amd as sq
    return sq


def check(r, ref):
    for name in PLAN:
        assert np.array_equal(to_np(getattr(r, name)), ref[name]), name
    w = to_np(r.weight).astype(np.float64)
    tol = np.abs(ref["weight"]) * (2.0 ** -24 + 2.0 ** -45) + 2.0 ** -150  # half the smallest fp32 step
    assert np.all(np.abs(w - ref["weight"]) <= tol), np.abs(w - ref["weight"]).max()


def run(sq, logits, k, dtype="fp32", bias=None, num_tokens=None, **kw):
    import torch
    t = torch.from_numpy(np.asarray(logits, np.float32)).to({"fp32": torch.float32, "bf16": torch.bfloat16,
                                                               "fp16": torch.float16}[dtype]).cuda()
    r = sq.moe_route(t, k, bias=None if bias is None else f32_to_gpu(bias),
                     num_tokens=None if num_tokens is None else i32_to_gpu([num_tokens]), **kw)
    check(r, moe_route_ref(t.float().cpu().numpy(), k, bias=bias, num_tokens=num_tokens, **kw))
    return r


SIZES = [(1, 1, 1), (1, 8, 2), (1, 128, 8), (3, 7, 7), (5, 17, 3), (16, 33, 4), (64, 128, 8), (65, 60, 4),
         (100, 256, 8), (130, 160, 6), (257, 300, 10), (40, 512, 12), (70, 1000, 5), (33, 1024, 64), (1030, 64, 6)]


@pytest.mark.parametrize("T,E,k", SIZES)
@pytest.mark.parametrize("score,bias,renorm", [("softmax", False, True), ("softmax", False, False),
                                               ("softmax", True, True), ("sigmoid", True, True),
                                               ("sigmoid", False, False)])
def test_route(sq, T, E, k, score, bias, renorm):
    print(f"route T={T} E={E} k={k} {score} bias={bias} renorm={renorm}", flush=True)
    rng = np.random.default_rng(T + E)
    run(sq, 2 * rng.standard_normal((T, E)), k, score=score, renormalize=renorm, scale=2.5 if bias else 1.0,
        bias=0.1 * rng.standard_normal(E).astype(np.float32) if bias else None)


@pytest.mark.parametrize("T,E,groups,top,k", [(1, 8, 2, 1, 4), (20, 60, 4, 2, 5), (70, 256, 8, 4, 8), (9, 12, 12, 5, 5),
                                              (130, 160, 8, 3, 6), (33, 1000, 20, 7, 9), (5, 1024, 64, 3, 20),
                                              (6, 300, 300, 40, 8)])
@pytest.mark.parametrize("gscore", ["max", "sum2"])
@pytest.mark.parametrize("score,bias", [("softmax", False), ("softmax", True), ("sigmoid", True), ("sigmoid", False)])
def test_groups(sq, T, E, groups, top, k, gscore, score, bias):
    print(f"groups T={T} E={E} {top}/{groups} k={k} {gscore} {score} bias={bias}", flush=True)
    rng = np.random.default_rng(T + E)
    x = rng.standard_normal((T, E))
    x[rng.random((T, E)) < 0.1] = -np.inf
    x[T // 2, :E // 2] = -np.inf  # whole groups without an expert
    run(sq, x, k, score=score, groups=groups, top_groups=top, group_score=gscore,
        bias=0.1 * rng.standard_normal(E).astype(np.float32) if bias else None)


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("T,E,k", [(50, 24, 5), (200, 130, 8)])
def test_ties_and_masked_rows(sq, dtype, T, E, k):
    """Few distinct values (most choices are ties), -0 and +0, infinities, NaN, rows without an expert or with
    fewer than k."""
    print(f"ties {dtype} T={T} E={E}", flush=True)
    rng = np.random.default_rng(E)
    x = rng.choice([0.0, -0.0, 0.5, 1.0], (T, E))
    x[rng.random((T, E)) < 0.1] = np.nan
    x[rng.random((T, E)) < 0.1] = -np.inf
    x[rng.random((T, E)) < 0.02] = np.inf
    x[0] = -np.inf
    x[1] = np.nan
    x[2] = -np.inf
    x[2, E - 1] = 3.0
    x[3] = 0.0
    x[4] = np.inf
    x[5] = 60000.0
    x[6] = -60000.0
    for score in ("softmax", "sigmoid"):
        run(sq, x, k, dtype=dtype, score=score)
        run(sq, x, k, dtype=dtype, score=score, renormalize=False, bias=np.zeros(E, np.float32))


def test_bias_without_a_number(sq):
    """A NaN or -inf bias takes its expert out, +inf puts it first."""
    rng = np.random.default_rng(3)
    bias = np.zeros(16, np.float32)
    bias[3], bias[5], bias[9] = np.nan, -np.inf, np.inf
    r = run(sq, rng.standard_normal((20, 16)), 14, bias=bias)
    ids = to_np(r.expert)
    assert (ids[:, 0] == 9).all() and not np.isin(ids, [3, 5]).any()


def test_values_that_differ_only_in_64_bits(sq):
    """Scores + bias that are one value in fp32 and two in float64: the order is float64's."""
    E = 32
    x = np.full((4, E), 1.0, np.float32)
    x[:, 1::2] = np.nextafter(np.float32(1.0), np.float32(2.0))  # larger by 2^-23: sigmoid differs by 2.3e-8
    r = run(sq, x, 8, score="sigmoid", bias=np.full(E, 64.0, np.float32))
    assert (to_np(r.expert) == np.arange(1, 17, 2)).all()


@pytest.mark.parametrize("T,n", [(10, 0), (10, 7), (100, 33), (100, 100), (100, 1000), (100, -3)])
def test_padded_batch(sq, T, n):
    rng = np.random.default_rng(T)
    r = run(sq, rng.standard_normal((T, 20)), 4, num_tokens=n)
    live = max(0, min(T, n))
    assert (to_np(r.expert)[live:] == -1).all() and (to_np(r.weight)[live:] == 0).all()


def test_strided_rows_and_no_tokens(sq):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(0)
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        whole = torch.randn(90, 75, device="cuda", generator=gen).to(dtype)
        for part in (whole[:, 3:63], whole[::2, 1:2], whole[:1, 5:50]):
            k = min(4, part.shape[1])
            check(sq.moe_route(part, k), moe_route_ref(part.float().cpu().numpy(), k))
    r = sq.moe_route(torch.empty((0, 12), device="cuda"), 3)
    assert r.expert.shape == (0, 3) and r.a_rows.numel() == 0 and (to_np(r.seg_offsets) == 0).all()


@pytest.mark.parametrize("T", [4096, 20000])
def test_large_batches(sq, T):
    """Many chunks, some of several 64-token parts; the plan against numpy's stable sort of the ids."""
    import torch
    E, k = 96, 6
    print(f"large batch T={T}", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn(T, E, device="cuda", generator=gen)
    n = T - 1000
    r = sq.moe_route(x, k, num_tokens=i32_to_gpu([n]))
    ids = to_np(r.expert)
    want = np.argsort(-to_np(x).astype(np.float64), axis=1, kind="stable")[:, :k]
    assert np.array_equal(ids[:n], want[:n]) and (ids[n:] == -1).all()
    flat = np.where(ids < 0, E, ids).reshape(-1)
    order = np.argsort(flat, kind="stable")
    counts = np.bincount(flat, minlength=E + 1)
    seg = np.concatenate([[0], np.cumsum(counts[:E])])
    assert np.array_equal(to_np(r.seg_offsets), seg)
    rows = np.where(np.arange(T * k) < seg[E], order // k, -1)
    assert np.array_equal(to_np(r.a_rows), rows)
    place = np.empty(T * k, np.int64)
    place[order] = np.arange(T * k)
    assert np.array_equal(to_np(r.pair_index).reshape(-1), np.where(flat == E, -1, place))


@pytest.mark.parametrize("T", [5, 300])
def test_captured_with_a_changing_token_count(sq, T):
    """One graph serves batches of every fill: logits and the count are changed in place between replays."""
    import torch
    E, k = 40, 5
    x = torch.zeros((T, E), device="cuda")
    n = i32_to_gpu([T])
    sq.moe_route(x, k, num_tokens=n)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r = sq.moe_route(x, k, num_tokens=n)
    rng = np.random.default_rng(0)
    for live in (T, 1, T // 2, 0, T):
        logits = rng.standard_normal((T, E)).astype(np.float32)
        x.copy_(torch.from_numpy(logits))
        n.fill_(live)
        for t in r:
            t.fill_(-7)
        g.replay()
        check(r, moe_route_ref(logits, k, num_tokens=live))
        check(sq.moe_route(x, k, num_tokens=n), moe_route_ref(logits, k, num_tokens=live))


@pytest.mark.parametrize("T,k", [(1, 3), (7, 3), (40, 2)])
def test_feeds_the_two_path_grouped_calls(sq, T, k):
    """The plan is what linear_grouped, linear_grouped_silu_prepare and moe_combine of fp32 rows read (with an odd
    number of pairs too); a padded batch leaves the rows behind its pairs alone and combines them to zero."""
    import torch
    from oracle import linear_grouped_ref, moe_combine_ref, prepare_ref, quantize_weight_ref
    from synth import bf16_round
    from gpu_util import assert_y_close, bf16_to_gpu, oracle_prepared, w_to_gpu
    rng = np.random.default_rng(T)
    E, K, O = 5, 128, 256
    x = bf16_round(rng.standard_normal((T, K)).astype(np.float32))
    wq = [quantize_weight_ref(bf16_round((rng.standard_normal((O, K)) * 0.1).astype(np.float32))) for _ in range(E)]
    wc, ws = np.stack([c for c, _ in wq]), np.stack([s for _, s in wq])
    logits = rng.standard_normal((T + 3, E)).astype(np.float32)
    r = sq.moe_route(f32_to_gpu(logits), k, num_tokens=i32_to_gpu([T]))
    ref = moe_route_ref(logits, k, num_tokens=T)
    check(r, ref)
    p = prepare_ref(x, None, 2, 4)
    P = (T + 3) * k
    y = torch.full((P, O), 7.0, device="cuda")
    sq.linear_grouped(oracle_prepared(p), w_to_gpu(wc, ws), r.seg_offsets, r.a_rows, out=y)
    n = int(ref["seg_offsets"][-1])
    want, bound = linear_grouped_ref(p["bb_codes"], p["bb_scales"], p["res_codes"], p["res_scales"],
                                     ref["a_rows"][:n], ref["seg_offsets"], wc, ws)
    assert_y_close(to_np(y)[:n], want, bound)
    assert (y[n:] == 7).all()
    hp, _ = sq.linear_grouped_silu_prepare(oracle_prepared(p), w_to_gpu(wc, ws), r.seg_offsets, r.a_rows)
    assert hp.K == O // 2
    out = to_np(sq.moe_combine(y, r.pair_index, r.weight))
    full, fb = moe_combine_ref(to_np(y), ref["pair_index"], to_np(r.weight))
    assert np.all(np.abs(out - full) <= k * 2.0 ** -24 * fb + 2.0 ** -126) and (out[T:] == 0).all()


def test_refusals(sq):
    import torch
    x = torch.zeros((4, 12), device="cuda")
    for bad in (lambda: sq.moe_route(x.cpu(), 2), lambda: sq.moe_route(x[0], 2), lambda: sq.moe_route(x.t(), 2),
                lambda: sq.moe_route(x, 2, score="tanh"), lambda: sq.moe_route(x, 2, group_score="mean"),
                lambda: sq.moe_route(x, 2, bias=torch.zeros(11, device="cuda")),
                lambda: sq.moe_route(x, 2, bias=torch.zeros(12)),
                lambda: sq.moe_route(x, 2, num_tokens=torch.zeros(2, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: sq.moe_route(x.double(), 2), lambda: sq.moe_route([[0.0]], 1),
                lambda: sq.moe_route(x, 2, bias=torch.zeros(12, dtype=torch.bfloat16, device="cuda")),
                lambda: sq.moe_route(x, 2, num_tokens=torch.zeros(1, device="cuda"))):
        with pytest.raises(TypeError):
            bad()
    for bad in (dict(k=0), dict(k=13), dict(k=2, groups=5), dict(k=2, groups=4, top_groups=5),
                dict(k=7, groups=4, top_groups=2), dict(k=2, scale=float("nan"))):
        with pytest.raises(sq.SharqError):
            sq.moe_route(x, **bad)
    with pytest.raises(sq.SharqError):
        sq.moe_route(x[:1].expand(4, 12), 2)  # rows that overlap


@pytest.mark.parametrize("T,E,groups,top,k", [(22, 128, 128, 40, 40), (41, 64, 64, 64, 64), (300, 128, 128, 64, 64),
                                              (64, 16, 16, 16, 16)])
def test_many_small_groups(sq, T, E, groups, top, k):
    """The most LDS a token takes; token counts whose last wave is partly empty."""
    print(f"small groups T={T} E={E} {top}/{groups} k={k}", flush=True)
    rng = np.random.default_rng(T)
    run(sq, rng.standard_normal((T, E)), k, groups=groups, top_groups=top, group_score="sum2", score="sigmoid",
        bias=0.1 * rng.standard_normal(E).astype(np.float32))


@pytest.mark.parametrize("T,E,k,groups,top", [(200, 32, 5, 1, 1), (300, 128, 8, 1, 1), (300, 128, 15, 1, 1),
                                              (200, 256, 8, 8, 4), (100, 512, 20, 16, 5), (40, 1000, 9, 1, 1),
                                              (100, 64, 40, 1, 1), (50, 16, 16, 1, 1), (300, 60, 4, 12, 3)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("gscore", ["max", "sum2"])
def test_values_closer_than_float32_tells(sq, T, E, k, groups, top, score, gscore):
    """Clusters of one to four logits a last place apart, so that the order inside the first k, the last place and
    the kept groups hang on float64's scores, alone and together."""
    print(f"close values T={T} E={E} k={k} {top}/{groups} {score} {gscore}", flush=True)
    rng = np.random.default_rng(E + k)
    x = np.empty((T, E), np.float32)
    for t in range(T):
        heads = rng.permutation(E).astype(np.float32) * np.float32(4.0 / E) - np.float32(1.0)
        row, at = [], 0
        while len(row) < E:
            v = heads[at]
            for _ in range(rng.integers(1, 5) if rng.random() < 0.3 else 1):
                row.append(v)
                v = np.nextafter(v, np.float32(9.0)) if rng.random() < 0.8 else v
            at += 1
        x[t] = rng.permutation(np.array(row[:E], np.float32))
    bias = np.zeros(E, np.float32)
    run(sq, x, k, score=score, bias=bias, groups=groups, top_groups=top, group_score=gscore)
    bias[rng.random(E) < 0.5] = 0.25
    run(sq, x, k, score=score, bias=bias, groups=groups, top_groups=top, group_score=gscore, renormalize=False)


@pytest.mark.parametrize("scale", [1.1, 0.1, -2.446, 1e-30, 0.0])
def test_scale_is_held_in_float32(sq, scale):
    """The factor is fp32's; the product with the float64 share is rounded once."""
    rng = np.random.default_rng(4)
    x = rng.standard_normal((30, 24)).astype(np.float32)
    check(sq.moe_route(f32_to_gpu(x), 5, scale=scale), moe_route_ref(x, 5, scale=float(np.float32(scale))))
