"""GPU parity of the plain MXFP4 products (dense, fused SiLU, grouped), of the
norming quantiser and of the bf16 combine against the float64 oracle.

Tolerance of a product of K terms: the products of E2M1 entries are exact in
fp32, and each of at most K additions rounds (or truncates) a partial sum of
at most B = sum |a w| by 2^-23 of it, so |Y - ref| <= K 2^-23 B. A bf16 output
adds half a step, 2^-8 of its value. Codes are compared bit for bit."""

import numpy as np
import pytest

from oracle import (f64_to_bf16_bits_rne, linear_mxfp4_ref, moe_combine_ref, moe_route_ref, mxfp4_quantize,
                    pack_nibbles, prepare_ref, quantize_weight_ref, rms_normalize_ref, rms_row_scale_ref)
from synth import adversarial_rows, bf16_round, bf16_to_f32
from gpu_util import (bf16_to_gpu, codes_row_major, codes_stage_major, f32_to_gpu, i32_to_gpu, row_major,
                      stage_major, to_np, u8_to_gpu, w_to_gpu)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sq():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    import activation_sparsity_fp4_amd as sq
    return sq


def _rows(rng, R, K, sigma=1.0):
    x = rng.standard_normal((R, K)) * rng.lognormal(0, 0.5, (R, 1)) * sigma
    x[:, rng.random(K) < 0.01] *= 50
    return quantize_weight_ref(bf16_round(x.astype(np.float32)))


def _mx(sq, q):
    return w_to_gpu(*q)


def _close(y, ref, bound, K, rows=None):
    import torch
    bf16 = y.dtype == torch.bfloat16
    got = y.float().cpu().numpy().astype(np.float64)
    tol = K * 2.0 ** -23 * bound + (2.0 ** -8 * np.abs(ref) if bf16 else 0) + 2.0 ** -126
    err = np.abs(got - ref)
    if rows is not None:
        err, tol = err[rows], tol[rows]
    assert np.all(err <= tol), f"{(err > tol).sum()} of {err.size} outside; worst {(err / tol).max()}"


def _same(a, b):
    import torch
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


SIZES = [(1, 32, 1), (1, 4096, 1000), (2, 96, 31), (7, 160, 257), (31, 2080, 256), (32, 128, 512), (33, 288, 255),
         (64, 1024, 300), (65, 544, 129), (128, 4128, 64), (129, 256, 1027), (200, 96, 96), (257, 640, 513),
         (1, 16384, 256), (40, 8192, 130), (300, 8192, 72), (4100, 128, 4200)]


@pytest.mark.parametrize("T,K,O", SIZES)
@pytest.mark.parametrize("out", ["fp32", "bf16"])
def test_linear(sq, T, K, O, out):
    import torch
    print(f"linear T={T} K={K} O={O} {out}", flush=True)
    rng = np.random.default_rng(T + K + O)
    a, w = _rows(rng, T, K), _rows(rng, O, K, 0.02)
    ref, bound = linear_mxfp4_ref(*a, *w)
    dtype = torch.float32 if out == "fp32" else torch.bfloat16
    A, W = _mx(sq, a), _mx(sq, w)
    y = sq.linear_mxfp4(A, W, dtype=dtype)
    assert y.dtype == dtype
    _close(y, ref, bound, K)
    assert _same(y, sq.linear_mxfp4(A, W, dtype=dtype)), "not deterministic"
    _close(sq.linear_mxfp4(A, W, dtype=dtype, split_k=False), ref, bound, K)


@pytest.mark.parametrize("T,K,O,ld", [(5, 256, 40, 41), (70, 128, 33, 64), (300, 160, 260, 263), (2, 16384, 40, 47),
                                      (260, 128, 500, 512)])
@pytest.mark.parametrize("out", ["fp32", "bf16"])
def test_linear_strided_output_leaves_the_rest(sq, T, K, O, ld, out):
    import torch
    print(f"linear strided T={T} K={K} O={O} ld={ld} {out}", flush=True)
    rng = np.random.default_rng(3)
    a, w = _rows(rng, T, K), _rows(rng, O, K)
    ref, bound = linear_mxfp4_ref(*a, *w)
    dtype = torch.float32 if out == "fp32" else torch.bfloat16
    whole = torch.full((T + 1, ld), 7.0, dtype=dtype, device="cuda")
    sq.linear_mxfp4(_mx(sq, a), _mx(sq, w), out=whole[:T, :O])
    _close(whole[:T, :O], ref, bound, K)
    assert (whole[T] == 7).all() and (whole[:, O:] == 7).all()


def test_empty_sizes(sq):
    import torch
    rng = np.random.default_rng(0)
    w = _mx(sq, _rows(rng, 8, 64))
    none = sq.MXFP4(torch.empty((1, 0, 64), dtype=torch.uint8, device="cuda"),
                    torch.empty((1, 0, 4), dtype=torch.uint8, device="cuda"), 64)
    assert sq.linear_mxfp4(none, w).shape == (0, 8)
    assert sq.linear_mxfp4(w, none).shape == (8, 0)
    assert sq.linear_silu_mxfp4(none, _mx(sq, _rows(rng, 64, 64))).codes.shape == (1, 0, 64)
    assert sq.quantize_mxfp4(torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"), rms_eps=1e-5).codes.shape[1] == 0


def test_zero_and_extreme_scales(sq):
    """Blocks of zeros, of the smallest and of large scales."""
    K, rng = 256, np.random.default_rng(9)
    rows = adversarial_rows(K)[[0, 1, 2, 4, 5, 9]]
    a = quantize_weight_ref(bf16_round(rows))
    w = _rows(rng, 50, K)
    ref, bound = linear_mxfp4_ref(*a, *w)
    _close(sq.linear_mxfp4(_mx(sq, a), _mx(sq, w)), ref, bound, K)


def test_operand_beyond_two_gigabytes(sq):
    """A weight whose codes pass 2^31 bytes (and 2^32 entries): sampled rows."""
    import torch
    G, O = 128, 280000
    K = 128 * G
    assert G * O * 64 > 1 << 31
    gen = torch.Generator(device="cuda").manual_seed(4)
    codes = torch.randint(0, 256, (G, O, 64), dtype=torch.uint8, device="cuda", generator=gen)
    scales = torch.randint(120, 124, (G, O, 4), dtype=torch.uint8, device="cuda", generator=gen)
    rng = np.random.default_rng(4)
    a = _rows(rng, 3, K)
    pick = np.concatenate([[0, O - 1, O - 256, 262143, 262144], rng.integers(0, O, 40)])
    at = torch.from_numpy(pick).cuda()
    wc = to_np(codes[:, at].permute(1, 0, 2).reshape(len(pick), -1))
    ws = to_np(scales[:, at].permute(1, 0, 2).reshape(len(pick), -1))
    print(f"weight of {G * O * 64} bytes", flush=True)
    y = sq.linear_mxfp4(_mx(sq, a), sq.MXFP4(codes, scales, K))
    ref, bound = linear_mxfp4_ref(*a, wc, ws)
    _close(y[:, at], ref, bound, K)


SILU = [(1, 128, 128), (3, 96, 32), (32, 256, 160), (33, 160, 256), (64, 4128, 64), (65, 128, 96), (130, 256, 384),
        (257, 544, 416), (1, 16384, 128), (20, 8192, 224), (2048, 128, 4128)]


@pytest.mark.parametrize("T,K,I", SILU)
@pytest.mark.parametrize("split", [True, False])
def test_silu_equals_the_chain(sq, T, K, I, split):
    import torch
    print(f"silu T={T} K={K} I={I} split={split}", flush=True)
    rng = np.random.default_rng(T + K + I)
    a, w = _mx(sq, _rows(rng, T, K)), _mx(sq, _rows(rng, 2 * I, K, 0.05))
    out = sq.MXFP4(torch.full((sq.stages(I), T, 64), 0xA5, dtype=torch.uint8, device="cuda"),
                   torch.full((sq.stages(I), T, 4), 0xA5, dtype=torch.uint8, device="cuda"), I)
    h = sq.linear_silu_mxfp4(a, w, out=out, split_k=split)
    want = sq.quantize_mxfp4(sq.silu_mul(sq.linear_mxfp4(a, w, split_k=split)))
    assert torch.equal(h.scales, want.scales) and torch.equal(h.codes, want.codes)


def test_silu_against_the_oracle(sq):
    """The chain's own stages are checked elsewhere; here the coded h is, within one code step of float64's h where
    a rounding may fall the other way."""
    T, K, I = 40, 256, 128
    rng = np.random.default_rng(8)
    a, w = _rows(rng, T, K), _rows(rng, 2 * I, K, 0.1)
    y, _ = linear_mxfp4_ref(*a, *w)
    g, u = y[:, :I], y[:, I:]
    h = bf16_to_f32(f64_to_bf16_bits_rne(g / (1 + np.exp(-g)) * u))
    codes, e = mxfp4_quantize(h)
    got = sq.linear_silu_mxfp4(_mx(sq, a), _mx(sq, w))
    gc = codes_row_major(to_np(got.codes), I // 2)
    gs = row_major(to_np(got.scales), I // 32)
    same = (gs == (e + 127).astype(np.uint8))
    assert same.mean() > 0.99
    wantc = pack_nibbles(codes)
    assert (gc == wantc).mean() > 0.98


def _experts(rng, E, O, K):
    q = [_rows(rng, O, K, 0.02) for _ in range(E)]
    return np.stack([c for c, _ in q]), np.stack([s for _, s in q])


def _grouped_ref(a, w, seg, rows, P):
    y = np.zeros((P, w[0].shape[1]))
    b = np.zeros_like(y)
    src = np.arange(P) if rows is None else rows
    for e in range(len(seg) - 1):
        for p in range(seg[e], seg[e + 1]):
            if 0 <= src[p] < a[0].shape[0]:
                y[p:p + 1], b[p:p + 1] = linear_mxfp4_ref(a[0][src[p]:src[p] + 1], a[1][src[p]:src[p] + 1],
                                                          w[0][e], w[1][e])
    return y, b


GROUPED = [
    # E, K, O, seg, gather
    (3, 160, 40, [0, 1, 1, 2], True),
    (5, 256, 300, [0, 0, 40, 41, 200, 200], True),   # empty experts, one row
    (4, 2080, 257, [0, 130, 130, 131, 300], False),
    (2, 96, 33, [0, 0, 0], True),                    # no rows in any segment
    (130, 128, 64, [min(i, 90) for i in range(131)], True),  # more experts than one wave scans
]


@pytest.mark.parametrize("E,K,O,seg,gather", GROUPED)
@pytest.mark.parametrize("out", ["fp32", "bf16"])
def test_grouped(sq, E, K, O, seg, gather, out):
    import torch
    print(f"grouped E={E} K={K} O={O} {out}", flush=True)
    rng = np.random.default_rng(E + K)
    T, P = (50, max(seg[-1], 3)) if gather else (seg[-1], seg[-1])
    a, w = _rows(rng, T, K), _experts(rng, E, O, K)
    rows = rng.integers(0, T, P).astype(np.int32) if gather else None
    ref, bound = _grouped_ref(a, w, seg, rows, P)
    dtype = torch.float32 if out == "fp32" else torch.bfloat16
    y = torch.full((P, O), 7.0, dtype=dtype, device="cuda")
    sq.linear_grouped_mxfp4(_mx(sq, a), _mx(sq, w), i32_to_gpu(seg), None if rows is None else i32_to_gpu(rows), out=y)
    n = seg[-1]
    _close(y, ref, bound, K, rows=slice(0, n))
    assert (y[n:] == 7).all()


@pytest.mark.parametrize("E,K,I,seg", [(3, 160, 32, [0, 1, 1, 2]), (5, 256, 160, [0, 0, 40, 41, 200, 200]),
                                       (2, 544, 128, [0, 300, 429]), (16, 128, 96, [4 * i for i in range(17)])])
def test_grouped_silu_equals_the_chain(sq, E, K, I, seg):
    import torch
    print(f"grouped silu E={E} K={K} I={I}", flush=True)
    rng = np.random.default_rng(E)
    T, P = 60, seg[-1] + 2
    a, w = _mx(sq, _rows(rng, T, K)), _mx(sq, _experts(rng, E, 2 * I, K))
    rows, segs = i32_to_gpu(rng.integers(0, T, P)), i32_to_gpu(seg)
    out = sq.MXFP4(torch.full((sq.stages(I), P, 64), 0xA5, dtype=torch.uint8, device="cuda"),
                   torch.full((sq.stages(I), P, 4), 0xA5, dtype=torch.uint8, device="cuda"), I)
    h = sq.linear_grouped_silu_mxfp4(a, w, segs, rows, out=out)
    want = sq.quantize_mxfp4(sq.silu_mul(sq.linear_grouped_mxfp4(a, w, segs, rows)))
    n = seg[-1]
    assert torch.equal(h.codes[:, :n], want.codes[:, :n]) and torch.equal(h.scales[:, :n], want.scales[:, :n])
    assert (h.codes[:, n:] == 0xA5).all() and (h.scales[:, n:] == 0xA5).all()


def test_grouped_malformed_contents_stay_inside(sq):
    """Gathered rows outside the activation read as zeros; offsets outside [0, P] and reversed ones are clamped."""
    rng = np.random.default_rng(2)
    a, w = _rows(rng, 10, 128), _experts(rng, 3, 40, 128)
    rows = np.array([0, -1, 10, 1 << 30, 9, 3], np.int32)
    y = sq.linear_grouped_mxfp4(_mx(sq, a), _mx(sq, w), i32_to_gpu([0, 2, 4, 6]), i32_to_gpu(rows))
    ref, bound = _grouped_ref(a, w, [0, 2, 4, 6], rows, 6)
    _close(y, ref, bound, 128)
    sq.linear_grouped_mxfp4(_mx(sq, a), _mx(sq, w), i32_to_gpu([-5, 4, 2, 1000]), i32_to_gpu(rows))
    sq.linear_grouped_silu_mxfp4(_mx(sq, a), _mx(sq, _experts(rng, 3, 64, 128)), i32_to_gpu([5, 1, 9, -3]),
                                 i32_to_gpu(rows))


@pytest.mark.parametrize("T,K", [(1, 32), (5, 96), (40, 2048), (33, 2080), (17, 4096), (9, 4128), (3, 14336)])
@pytest.mark.parametrize("gamma", [True, False])
def test_quantize_rms(sq, T, K, gamma):
    """Codes and scales equal the oracle's bit for bit; so does the backbone-free part of prepare(rms_eps)."""
    import torch
    from activation_sparsity_fp4_amd import _lib
    print(f"quantize rms T={T} K={K} gamma={gamma}", flush=True)
    rng = np.random.default_rng(T + K)
    ld = K + 8
    whole = bf16_round((rng.standard_normal((T, ld)) * rng.lognormal(0, 1, (T, 1))).astype(np.float32))
    x = whole[:, :K]
    g = bf16_round(rng.uniform(0.5, 1.5, K).astype(np.float32)) if gamma else None
    xn, r = rms_normalize_ref(x, 1e-5)
    xp = bf16_to_f32(xn) if xn.dtype == np.uint16 else np.asarray(xn, np.float32)
    if gamma:
        xp = xp * bf16_to_f32(g)
    codes, e = mxfp4_quantize(xp)
    X = bf16_to_gpu(whole)[:, :K]
    q = sq.quantize_mxfp4(X, gamma=None if g is None else bf16_to_gpu(g), rms_eps=1e-5)
    assert np.array_equal(codes_row_major(to_np(q.codes), K // 2), pack_nibbles(codes))
    assert np.array_equal(row_major(to_np(q.scales), K // 32), (e + 127).astype(np.uint8))
    scale = torch.empty(T, dtype=torch.float32, device="cuda")
    G = bf16_to_gpu(g) if gamma else None
    st = _lib.call("sharq_quantize_mxfp4_rms", X.data_ptr(), T, K, ld, G.data_ptr() if gamma else 0, 1e-5,
                   scale.data_ptr(), q.codes.data_ptr(), q.scales.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert st == _lib.SHARQ_OK
    assert np.array_equal(to_np(scale), rms_row_scale_ref(x, 1e-5))


@pytest.mark.parametrize("T,k,H", [(1, 1, 4), (5, 2, 12), (33, 8, 2048), (7, 11, 24), (300, 6, 100)])
@pytest.mark.parametrize("bf16", [True, False])
def test_combine_of_bf16_rows(sq, T, k, H, bf16):
    import torch
    print(f"combine T={T} k={k} H={H} bf16={bf16}", flush=True)
    rng = np.random.default_rng(T * k)
    P = max(1, T * k // 2)
    y = bf16_round(rng.standard_normal((P, H)).astype(np.float32))
    idx = rng.integers(-1, P + 1, (T, k)).astype(np.int32)  # empty slots and indices past the pairs
    w = rng.uniform(0, 1, (T, k)).astype(np.float32)
    ref, bound = moe_combine_ref(bf16_to_f32(y), np.where(idx >= P, -1, idx), w)
    out = sq.moe_combine(bf16_to_gpu(y), i32_to_gpu(idx), f32_to_gpu(w), bf16=bf16)
    got = out.float().cpu().numpy().astype(np.float64)
    # k fused multiply-adds, each rounding by half a step of at most the bound
    tol = k * 2.0 ** -24 * bound + (2.0 ** -8 * np.abs(ref) if bf16 else 0) + 2.0 ** -126
    assert np.all(np.abs(got - ref) <= tol)


def test_refusals(sq):
    import torch
    rng = np.random.default_rng(0)
    a, w = _mx(sq, _rows(rng, 6, 128)), _mx(sq, _rows(rng, 64, 128))
    wide = _mx(sq, _rows(rng, 64, 256))
    f = dict(device="cuda")
    for bad in (lambda: sq.linear_mxfp4(a, wide), lambda: sq.linear_mxfp4(a, w._replace(K=256)),
                lambda: sq.linear_mxfp4(a._replace(codes=a.codes[:, ::2]), w),
                lambda: sq.linear_mxfp4(a, w, out=torch.empty(5, 64, **f)),
                lambda: sq.linear_mxfp4(a, w, out=torch.empty(64, 6, **f).t()),
                lambda: sq.linear_mxfp4(a, w._replace(scales=w.scales.cpu())),
                lambda: sq.linear_silu_mxfp4(a, _mx(sq, _rows(rng, 63, 128))),
                lambda: sq.linear_silu_mxfp4(a, w, out=sq.quantize_mxfp4(torch.zeros(6, 64, dtype=torch.bfloat16, **f))),
                lambda: sq.linear_grouped_mxfp4(a, w, i32_to_gpu([0, 6])),
                lambda: sq.quantize_mxfp4(torch.zeros(6, 64, dtype=torch.bfloat16, **f),
                                          gamma=torch.ones(64, dtype=torch.bfloat16, **f)),
                lambda: sq.quantize_mxfp4(torch.zeros(2, 6, 64, dtype=torch.bfloat16, **f), rms_eps=1e-5),
                lambda: sq.quantize_mxfp4(torch.zeros(6, 64, dtype=torch.bfloat16, **f), rms_eps=1e-5,
                                          gamma=torch.ones(32, dtype=torch.bfloat16, **f))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: sq.linear_mxfp4(a, w, dtype=torch.float16),
                lambda: sq.linear_mxfp4(a, w, out=torch.empty(6, 64, **f), dtype=torch.bfloat16),
                lambda: sq.linear_mxfp4(a, w._replace(codes=w.codes.int()))):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(sq.SharqError):
        sq.linear_silu_mxfp4(a, _mx(sq, _rows(rng, 32, 128)))  # I = 16
    with pytest.raises(sq.SharqError):
        sq.quantize_mxfp4(torch.zeros(6, 64, dtype=torch.bfloat16, **f), rms_eps=0.0)


def _mlp(sq, x, gamma, gu, dn):
    import torch
    return sq.linear_mxfp4(sq.linear_silu_mxfp4(sq.quantize_mxfp4(x, gamma=gamma, rms_eps=1e-5), gu), dn,
                           dtype=torch.bfloat16)


@pytest.mark.parametrize("T,H,I", [(1, 2048, 512), (37, 1024, 640), (300, 512, 384)])
def test_captured_mlp_replays(sq, T, H, I):
    """The block captured into two graphs (each with workspaces of its own), replayed in turn with eager work
    between, on a stream other than the default; each replay equals the eager result."""
    import torch
    print(f"captured mlp T={T} H={H} I={I}", flush=True)
    rng = np.random.default_rng(T)
    gu, dn = _mx(sq, _rows(rng, 2 * I, H, 0.05)), _mx(sq, _rows(rng, H, I, 0.05))
    gamma = bf16_to_gpu(bf16_round(rng.uniform(0.5, 1.5, H).astype(np.float32)))
    xs = [bf16_to_gpu(bf16_round(rng.standard_normal((T, H)).astype(np.float32))) for _ in range(2)]
    want = [_mlp(sq, x, gamma, gu, dn) for x in xs]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        assert torch.equal(_mlp(sq, xs[0], gamma, gu, dn), want[0])
    torch.cuda.synchronize()
    graphs, outs = [], []
    for x in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(_mlp(sq, x, gamma, gu, dn))
        graphs.append(g)
    for rep in range(3):
        for o in outs:
            o.fill_(float("nan"))
        for g in graphs:
            g.replay()
        eager = _mlp(sq, xs[1], gamma, gu, dn)
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want)) and torch.equal(eager, want[1]), rep


def test_two_streams_at_once(sq):
    """Split-K calls on two streams have workspaces of their own."""
    import torch
    rng = np.random.default_rng(1)
    w = _mx(sq, _rows(rng, 256, 16384))
    a = [_mx(sq, _rows(rng, 4, 16384)) for _ in range(2)]
    want = [sq.linear_mxfp4(x, w) for x in a]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(sq.linear_mxfp4(a[i], w))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i]) for i in range(2) for y in got[i])


@pytest.mark.parametrize("T,E,k,H,I", [(1, 8, 2, 256, 128), (50, 16, 4, 512, 96), (200, 6, 3, 256, 160)])
def test_expert_layer(sq, T, E, k, H, I):
    """Routing, the experts' products and the combine together, stage by stage against the oracle."""
    import torch
    print(f"expert layer T={T} E={E} k={k}", flush=True)
    rng = np.random.default_rng(T)
    logits = rng.standard_normal((T, E)).astype(np.float32)
    x = bf16_round(rng.standard_normal((T, H)).astype(np.float32))
    gu, dn = _experts(rng, E, 2 * I, H), _experts(rng, E, H, I)
    r = sq.moe_route(f32_to_gpu(logits), k)
    ref = moe_route_ref(logits, k)
    for name in ("expert", "seg_offsets", "a_rows", "pair_index"):
        assert np.array_equal(to_np(getattr(r, name)), ref[name]), name
    a = sq.quantize_mxfp4(bf16_to_gpu(x))
    h = sq.linear_grouped_silu_mxfp4(a, _mx(sq, gu), r.seg_offsets, r.a_rows)
    y = sq.linear_grouped_mxfp4(h, _mx(sq, dn), r.seg_offsets, dtype=torch.bfloat16)
    hc, hs = codes_row_major(to_np(h.codes), I // 2), row_major(to_np(h.scales), I // 32)
    want, bound = _grouped_ref((hc, hs), dn, ref["seg_offsets"], None, T * k)
    _close(y, want, bound, I)
    out = sq.moe_combine(y, r.pair_index, r.weight)
    full, fb = moe_combine_ref(y.float().cpu().numpy(), ref["pair_index"], to_np(r.weight))
    assert np.all(np.abs(to_np(out) - full) <= k * 2.0 ** -24 * fb + 2.0 ** -126)


@pytest.mark.parametrize("T,K,I", [(5, 16384, 128), (40, 256, 96), (200, 544, 160)])
def test_rows_without_a_number_stay_alone(sq, T, K, I):
    """A row whose scales are NaN (0xFF) and one that overflows leave every other row as it is, and the fused forms
    still equal their chains, codes of NaN included."""
    import torch
    print(f"NaN rows T={T} K={K} I={I}", flush=True)
    rng = np.random.default_rng(T)
    codes, scales = _rows(rng, T, K)
    w = _mx(sq, _rows(rng, 2 * I, K, 0.05))
    clean = _mx(sq, (codes, scales))
    bad = scales.copy()
    bad[1], bad[3, ::2] = 0xFF, 254
    a = _mx(sq, (codes, bad))
    keep = [t for t in range(T) if t not in (1, 3)]
    for split in (True, False):
        y = sq.linear_mxfp4(a, w, split_k=split)
        assert torch.equal(y[keep], sq.linear_mxfp4(clean, w, split_k=split)[keep]) and y[1].isnan().all()
        h = sq.linear_silu_mxfp4(a, w, split_k=split)
        want = sq.quantize_mxfp4(sq.silu_mul(y))
        assert torch.equal(h.scales, want.scales) and torch.equal(h.codes, want.codes)


def _random_mx(sq, gen, *shape, K):
    """Random codes and scales near 1, zeros where a partial last stage is padded."""
    import torch
    G, R = sq.stages(K), shape[-1]
    codes = torch.randint(0, 256, (*shape[:-1], G, R, 64), dtype=torch.uint8, device="cuda", generator=gen)
    scales = torch.randint(124, 128, (*shape[:-1], G, R, 4), dtype=torch.uint8, device="cuda", generator=gen)
    left = K - 128 * (G - 1)
    codes[..., G - 1, :, left // 2:] = 0
    scales[..., G - 1, :, left // 32:] = 0
    return sq.MXFP4(codes, scales, K)


def _rows_of(sq, q, at):
    return sq.MXFP4(q.codes[:, at].contiguous(), q.scales[:, at].contiguous(), q.K)


def test_results_beyond_four_gigabytes(sq):
    """Outputs, coded outputs and expert weights whose bytes pass 2^32: sampled rows equal those of small calls (the
    additions of an element do not depend on the tile)."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(6)
    T = O = 33000
    print("fp32 output", flush=True)
    a, w = _random_mx(sq, gen, T, K=32), _random_mx(sq, gen, O, K=32)
    at = torch.tensor([0, 31, T // 2, T - 129, T - 1], device="cuda")
    y = sq.linear_mxfp4(a, w)
    assert y.numel() * 4 > 1 << 32
    assert torch.equal(y[at], sq.linear_mxfp4(_rows_of(sq, a, at), w, split_k=False))
    del y
    T, I = 1 << 20, 8224
    print("coded output", flush=True)
    a, w = _random_mx(sq, gen, T, K=32), _random_mx(sq, gen, 2 * I, K=32)
    at = torch.tensor([0, 77, T // 2, T - 1], device="cuda")
    h = sq.linear_silu_mxfp4(a, w)
    assert h.codes.numel() > 1 << 32
    want = sq.linear_silu_mxfp4(_rows_of(sq, a, at), w, split_k=False)
    assert torch.equal(h.codes[:, at], want.codes) and torch.equal(h.scales[:, at], want.scales)
    del h, a, w
    E, O, K = 64, 131104, 1024
    print("expert weights", flush=True)
    a, w = _random_mx(sq, gen, 9, K=K), _random_mx(sq, gen, E, O, K=K)
    assert w.codes.numel() > 1 << 32
    seg = [0] + [2] * (E - 2) + [5, 9]  # expert 0, and the last two
    y = sq.linear_grouped_mxfp4(a, w, i32_to_gpu(seg))
    for e in (0, E - 2, E - 1):
        one = sq.linear_mxfp4(a, sq.MXFP4(w.codes[e], w.scales[e], K), split_k=False)
        assert torch.equal(y[seg[e]:seg[e + 1]], one[seg[e]:seg[e + 1]])
    del y, w
    P, H = 70000, 32768
    print("combined rows", flush=True)
    y = torch.randn(P, H, device="cuda", generator=gen, dtype=torch.bfloat16)
    idx = torch.tensor([[P - 1, 0], [P - 2, -1]], dtype=torch.int32, device="cuda")
    out = sq.moe_combine(y, idx, torch.tensor([[1.0, 0.0], [1.0, 1.0]], device="cuda"))
    assert torch.equal(out, y[[P - 1, P - 2]].float())


def test_norming_quantiser_of_many_rows(sq):
    """More rows than one grid dimension holds workgroups for."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(2)
    T = (1 << 26) + 3
    x = torch.randn(T, 32, device="cuda", generator=gen, dtype=torch.bfloat16)
    at = torch.tensor([0, (1 << 20) - 1, 1 << 20, 1 << 26, T - 1], device="cuda")
    print(f"{T} rows", flush=True)
    q, want = sq.quantize_mxfp4(x, rms_eps=1e-5), sq.quantize_mxfp4(x[at], rms_eps=1e-5)
    assert torch.equal(q.codes[:, at], want.codes) and torch.equal(q.scales[:, at], want.scales)


@pytest.mark.parametrize("T,E,k,H,I", [(40, 16, 4, 512, 96), (300, 6, 2, 256, 160)])
def test_captured_expert_layer_of_padded_batches(sq, T, E, k, H, I):
    """One graph of the whole expert layer serves batches of every fill. What lies behind the pairs is NaN: it is
    left as it is and reaches no result."""
    import torch
    print(f"captured experts T={T} E={E}", flush=True)
    rng = np.random.default_rng(T)
    gu, dn = _mx(sq, _experts(rng, E, 2 * I, H)), _mx(sq, _experts(rng, E, H, I))
    logits = f32_to_gpu(rng.standard_normal((T, E)).astype(np.float32))
    x = bf16_to_gpu(bf16_round(rng.standard_normal((T, H)).astype(np.float32)))
    h = sq.MXFP4(torch.empty((sq.stages(I), T * k, 64), dtype=torch.uint8, device="cuda"),
                 torch.empty((sq.stages(I), T * k, 4), dtype=torch.uint8, device="cuda"), I)
    y = torch.empty((T * k, H), dtype=torch.bfloat16, device="cuda")
    n = i32_to_gpu([T])

    def layer(logits, x, n=None, h=None, y=None):
        r = sq.moe_route(logits, k, num_tokens=n)
        h = sq.linear_grouped_silu_mxfp4(sq.quantize_mxfp4(x), gu, r.seg_offsets, r.a_rows, out=h)
        y = sq.linear_grouped_mxfp4(h, dn, r.seg_offsets, out=y, dtype=torch.bfloat16)
        return sq.moe_combine(y, r.pair_index, r.weight, bf16=True)

    layer(logits, x, n, h, y)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = layer(logits, x, n, h, y)
    for live in (T, 1, 0, T // 3, T):
        n.fill_(live)
        h.codes.fill_(0xFF), h.scales.fill_(0xFF), y.fill_(float("nan")), out.fill_(float("nan"))
        g.replay()
        assert (out[live:] == 0).all() and y[live * k:].isnan().all() and (h.scales[:, live * k:] == 0xFF).all()
        if live:
            assert torch.equal(out[:live], layer(logits[:live], x[:live])), live


@pytest.mark.parametrize("T,K", [(2, 16416), (3, 28672), (1, 131072)])
def test_quantize_rms_of_long_rows(sq, T, K):
    """Rows of more blocks than a workgroup holds in registers, up to the longest."""
    print(f"quantize rms T={T} K={K}", flush=True)
    rng = np.random.default_rng(K)
    x = bf16_round((rng.standard_normal((T, K)) * rng.lognormal(0, 1, (T, 1))).astype(np.float32))
    g = bf16_round(rng.uniform(0.5, 1.5, K).astype(np.float32))
    xn, _ = rms_normalize_ref(x, 1e-5)
    xp = (bf16_to_f32(xn) if xn.dtype == np.uint16 else np.asarray(xn, np.float32)) * bf16_to_f32(g)
    codes, e = mxfp4_quantize(xp)
    q = sq.quantize_mxfp4(bf16_to_gpu(x), gamma=bf16_to_gpu(g), rms_eps=1e-5)
    assert np.array_equal(codes_row_major(to_np(q.codes), K // 2), pack_nibbles(codes))
    assert np.array_equal(row_major(to_np(q.scales), K // 32), (e + 127).astype(np.uint8))


def test_workspace_too_small_is_no_split(sq):
    """At the C boundary a workspace below the asked size counts as none; a larger one splits."""
    import torch
    from activation_sparsity_fp4_amd import _lib
    T, K, O = 2, 16384, 256
    rng = np.random.default_rng(5)
    a, w = _mx(sq, _rows(rng, T, K)), _mx(sq, _rows(rng, O, K))
    need = _lib.call("sharq_linear_mxfp4_workspace_bytes", T, O, K)
    assert need > 0
    ws = torch.full((2 * need,), 0xFF, dtype=torch.uint8, device="cuda")
    for nbytes, split in ((need - 4, False), (need, True), (2 * need, True)):
        y = torch.empty((T, O), device="cuda")
        st = _lib.call("sharq_linear_mxfp4", a.codes.data_ptr(), a.scales.data_ptr(), w.codes.data_ptr(),
                       w.scales.data_ptr(), T, O, K, y.data_ptr(), O, 0, ws.data_ptr(), nbytes,
                       torch.cuda.current_stream().cuda_stream)
        assert st == _lib.SHARQ_OK
        assert torch.equal(y, sq.linear_mxfp4(a, w, split_k=split))
        assert (ws[need:] == 0xFF).all() and (split or (ws == 0xFF).all())


# Shapes for which the library takes its larger tiles (128 x 256, 128 x 128, 64 x 128, 32 x 256), whole and split.
LARGE = [(70, 128, 33000), (70, 160, 16416), (1, 128, 16416), (3, 160, 33000), (4100, 96, 4200), (1030, 544, 2500),
         (130, 28672, 4128), (70, 8224, 8200), (1, 8224, 4128), (2, 28672, 16416), (600, 14336, 4096)]


@pytest.mark.parametrize("T,K,O", LARGE)
@pytest.mark.parametrize("out", ["fp32", "bf16"])
def test_linear_of_large_shapes(sq, T, K, O, out):
    """Sampled rows and columns, the ends of tiles among them, against the oracle."""
    import torch
    print(f"large linear T={T} K={K} O={O} {out}", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(T + O)
    a, w = _random_mx(sq, gen, T, K=K), _random_mx(sq, gen, O, K=K)
    rng = np.random.default_rng(T + K)

    def pick(n):
        edges = [0, 31, 32, 63, 64, 127, 128, 255, 256, n // 2, n - 65, n - 2, n - 1]
        return np.unique([i for i in edges + list(rng.integers(0, n, 20)) if 0 <= i < n])

    def sample(q, at):
        i = torch.from_numpy(at).cuda()
        rows = lambda x, n: to_np(x[:, i].permute(1, 0, 2).reshape(len(at), -1))[:, :n]  # noqa: E731
        return rows(q.codes, K // 2), rows(q.scales, K // 32)

    t, o = pick(T), pick(O)
    ref, bound = linear_mxfp4_ref(*sample(a, t), *sample(w, o))
    for split in (True, False):
        y = sq.linear_mxfp4(a, w, dtype=torch.float32 if out == "fp32" else torch.bfloat16, split_k=split)
        assert y.isfinite().all()
        _close(y[torch.from_numpy(t).cuda()][:, torch.from_numpy(o).cuda()], ref, bound, K)


@pytest.mark.parametrize("T,K,I", [(8, 8192, 28672), (64, 4096, 14336), (128, 4096, 14336), (300, 4096, 14336),
                                   (515, 2048, 4128), (8200, 160, 288), (4100, 96, 256)])
def test_silu_of_large_shapes_equals_the_chain(sq, T, K, I):
    import torch
    print(f"large silu T={T} K={K} I={I}", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(T)
    a, w = _random_mx(sq, gen, T, K=K), _random_mx(sq, gen, 2 * I, K=K)
    w.scales[w.scales > 0] -= 8  # gate and up of order 1 and 10
    for split in (True, False):
        h = sq.linear_silu_mxfp4(a, w, split_k=split)
        want = sq.quantize_mxfp4(sq.silu_mul(sq.linear_mxfp4(a, w, split_k=split)))
        assert torch.equal(h.scales, want.scales) and torch.equal(h.codes, want.codes)


@pytest.mark.parametrize("T,E,P,K,I", [(90, 16, 700, 128, 2080), (500, 70, 4100, 160, 256), (3, 3, 3, 128, 4096),
                                       (20, 70, 71, 160, 512), (64, 128, 512, 2048, 768), (1, 128, 8, 2048, 768),
                                       (256, 8, 512, 1024, 4128), (1000, 128, 8000, 544, 768)])
@pytest.mark.parametrize("out", ["fp32", "bf16"])
def test_grouped_of_large_shapes(sq, T, E, P, K, I, out):
    """Every expert's rows equal those of a dense call of their own; the fused form equals its chain. Some experts
    are empty, some rows behind the last segment."""
    import torch
    print(f"large grouped T={T} E={E} P={P} K={K} I={I} {out}", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(E + P)
    rng = np.random.default_rng(P)
    share = rng.dirichlet(np.where(rng.random(E) < 0.2, 1e-3, 3.0))
    seg = np.concatenate([[0], np.cumsum(rng.multinomial(P - min(3, P - 1), share))]).astype(np.int32)
    rows = rng.integers(0, T, P).astype(np.int32)
    a, w = _random_mx(sq, gen, T, K=K), _random_mx(sq, gen, E, 2 * I, K=K)
    w.scales[w.scales > 0] -= 8
    dtype = torch.float32 if out == "fp32" else torch.bfloat16
    y = torch.full((P, 2 * I), 7.0, dtype=dtype, device="cuda")
    sq.linear_grouped_mxfp4(a, w, i32_to_gpu(seg), i32_to_gpu(rows), out=y)
    n = int(seg[-1])
    for e in np.unique([int(np.argmax(np.diff(seg))), *np.flatnonzero(np.diff(seg))[[0, -1]]]):
        at = torch.from_numpy(rows[seg[e]:seg[e + 1]]).long().cuda()
        one = sq.linear_mxfp4(_rows_of(sq, a, at), sq.MXFP4(w.codes[e], w.scales[e], K), dtype=dtype, split_k=False)
        assert torch.equal(y[seg[e]:seg[e + 1]], one), e
    assert (y[n:] == 7).all()
    ordered = _rows_of(sq, a, torch.from_numpy(rows).long().cuda())
    plain = torch.full((P, 2 * I), 7.0, dtype=dtype, device="cuda")
    sq.linear_grouped_mxfp4(ordered, w, i32_to_gpu(seg), out=plain)
    assert torch.equal(plain, y)
    if out == "fp32":
        for act, gather in ((a, i32_to_gpu(rows)), (ordered, None)):
            h = sq.linear_grouped_silu_mxfp4(act, w, i32_to_gpu(seg), gather)
            want = sq.quantize_mxfp4(sq.silu_mul(y))
            assert torch.equal(h.scales[:, :n], want.scales[:, :n]) and torch.equal(h.codes[:, :n], want.codes[:, :n])


@pytest.mark.parametrize("E,P", [(127, 300), (128, 300), (129, 300), (300, 900), (1000, 70)])
def test_grouped_over_many_experts(sq, E, P):
    """More experts than a workgroup holds of the segments at once; tiles of every one of them."""
    import torch
    print(f"many experts E={E} P={P}", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(E)
    rng = np.random.default_rng(E)
    K, I, T = 96, 64, 40
    seg = np.concatenate([[0], np.cumsum(rng.multinomial(P - 2, np.full(E, 1 / E)))]).astype(np.int32)
    rows = rng.integers(0, T, P).astype(np.int32)
    a, w = _random_mx(sq, gen, T, K=K), _random_mx(sq, gen, E, 2 * I, K=K)
    y = torch.full((P, 2 * I), 7.0, device="cuda")
    sq.linear_grouped_mxfp4(a, w, i32_to_gpu(seg), i32_to_gpu(rows), out=y)
    for e in np.flatnonzero(np.diff(seg)):
        at = torch.from_numpy(rows[seg[e]:seg[e + 1]]).long().cuda()
        one = sq.linear_mxfp4(_rows_of(sq, a, at), sq.MXFP4(w.codes[e], w.scales[e], K), split_k=False)
        assert torch.equal(y[seg[e]:seg[e + 1]], one), e
    n = int(seg[-1])
    assert (y[n:] == 7).all()
    h = sq.linear_grouped_silu_mxfp4(a, w, i32_to_gpu(seg), i32_to_gpu(rows))
    want = sq.quantize_mxfp4(sq.silu_mul(y))
    assert torch.equal(h.scales[:, :n], want.scales[:, :n]) and torch.equal(h.codes[:, :n], want.codes[:, :n])


def test_one_row_of_any_stride(sq):
    """A single row has no leading dimension: whatever stride its tensor reports, and rows of a wider tensor."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(1, 320, device="cuda", generator=gen, dtype=torch.bfloat16)
    column = x.reshape(320, 1).t()
    assert column.shape == (1, 320) and column.stride(0) != 320
    want = sq.quantize_mxfp4(x, rms_eps=1e-5)
    got = sq.quantize_mxfp4(column, rms_eps=1e-5)
    assert torch.equal(got.codes, want.codes) and torch.equal(got.scales, want.scales)
    w = _random_mx(sq, gen, 40, K=320)
    y = torch.full((40, 3), 7.0, device="cuda").t()[:1]  # one row, unit column stride refused
    with pytest.raises(ValueError):
        sq.linear_mxfp4(want, w, out=y)
    y = torch.zeros((1, 40), device="cuda").expand(1, 40)
    sq.linear_mxfp4(want, w, out=y)
    assert torch.equal(y, sq.linear_mxfp4(want, w))
    logits = torch.randn(24, 1, device="cuda", generator=gen).t()
    r, s = sq.moe_route(logits, 3), sq.moe_route(logits.contiguous(), 3)
    assert all(torch.equal(a, b) for a, b in zip(r, s))
