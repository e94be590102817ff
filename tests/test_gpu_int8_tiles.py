"""GPU parity of the 8-bit products on every tile and in every kind of output: the
sizes of int8_tiles.py, of which test_int8_tiles.py shows that they reach them.

The sums of codes are exact in float64 (below 2^53), so that a result differs from
the float64 one by the two roundings of its scales' products, one of the result,
and one to bfloat16: |Y - ref| <= 2^-24 (2.01 |Y - bias| + 1.01 |Y|) + 2^-149
(+ 2^-8 |Y| + 2^-134). The gate|up product equals its chain bit for bit."""

import pytest

from int8_tiles import BEHIND, BF16, DENSE, FP32, GROUPED, SILU, tile, weight_rows

pytestmark = pytest.mark.gpu

GUARD = 7.0


@pytest.fixture(scope="module")
def sq():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    import activation_sparsity_fp4_amd as sq
    return sq


def random_int8(sq, gen, *shape):
    """(Int8 tensor of random codes from -128 to 127, its codes and scales as float64 rows)."""
    import torch
    q = torch.randint(-128, 128, shape, dtype=torch.int8, device="cuda", generator=gen)
    s = torch.exp(torch.randn(shape[:-1], device="cuda", generator=gen)) * 0.01
    *lead, R, K = shape
    G = -(-K // 64)
    padded = torch.zeros((*lead, R, G * 64), dtype=torch.int8, device="cuda")
    padded[..., :K] = q
    codes = padded.reshape(*lead, R, G, 64).transpose(-3, -2).contiguous()
    return sq.Int8(codes, s, K), q, s


def product(a, w, bias=None):
    """(the float64 product, its size without the bias) of codes and scales."""
    (qa, sa), (qw, sw) = a, w
    p = (qa.double() @ qw.double().T.contiguous()) * sa.double()[:, None] * sw.double()
    return p if bias is None else p + bias.double(), p.abs()


def check(y, ref, size):
    import torch
    tol = 2.0 ** -24 * (2.01 * size + 1.01 * ref.abs()) + 2.0 ** -149
    if y.dtype == torch.bfloat16:
        tol += 2.0 ** -8 * ref.abs() + 2.0 ** -134
    outside = ~((y.double() - ref).abs() <= tol)
    assert not outside.any(), f"{int(outside.sum())} of {outside.numel()} outside, first {outside.nonzero()[0].tolist()}"


def dtype_of(kind):
    import torch
    return torch.bfloat16 if kind == BF16 else torch.float32


def same(a, b):
    import torch
    return torch.equal(a.codes, b.codes) and torch.equal(a.scales.view(torch.int32), b.scales.view(torch.int32))


def chain(sq, y, I):
    """Codes of h from the fp32 gate and up values y [R, 2 I]: silu_mul takes widths in eights, so zeros fill up."""
    import torch
    more = -I % 8
    y = torch.nn.functional.pad(y.reshape(-1, 2, I), (0, more)).reshape(-1, 2 * (I + more)).contiguous()
    return sq.quantize_int8(sq.silu_mul(y)[:, :I])


@pytest.mark.parametrize("T,K,O", DENSE)
@pytest.mark.parametrize("kind", [FP32, BF16], ids=["fp32", "bf16"])
def test_linear(sq, T, K, O, kind):
    import torch
    print(f"linear T={T} K={K} O={O} kind={kind} tile={tile(T, 0, O, K, kind)}", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(T + K + O)
    A, qa, sa = random_int8(sq, gen, T, K)
    W, qw, sw = random_int8(sq, gen, O, K)
    bias = torch.randn(O, device="cuda", generator=gen)
    check(sq.linear_int8(A, W, dtype=dtype_of(kind), bias=bias), *product((qa, sa), (qw, sw), bias))
    # rows on the 16-byte grid, the columns behind them and the row behind the last left alone
    whole = torch.full((T + 1, O + -O % 8 + 8), GUARD, dtype=dtype_of(kind), device="cuda")
    sq.linear_int8(A, W, out=whole[:T, :O])
    check(whole[:T, :O], *product((qa, sa), (qw, sw)))
    assert bool((whole[T] == GUARD).all()) and bool((whole[:, O:] == GUARD).all())


@pytest.mark.parametrize("T,K,O", DENSE)
def test_silu(sq, T, K, O):
    import torch
    I = O // 2
    print(f"silu T={T} K={K} I={I} tile={tile(T, 0, 2 * I, K, SILU)}", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(T + K + O)
    A, W = random_int8(sq, gen, T, K)[0], random_int8(sq, gen, 2 * I, K)[0]
    assert same(sq.linear_silu_int8(A, W), chain(sq, sq.linear_int8(A, W), I))


def grouped_case(sq, sizes, K, O, seed):
    """(activation, weight, offsets, gathered rows, first row, pairs, float64 operands): the segments begin at row 3."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    E, P, first = len(sizes), sum(sizes) + BEHIND, 3
    T = P // 3 + 4
    A, qa, sa = random_int8(sq, gen, T, K)
    W, qw, sw = random_int8(sq, gen, E, O, K)
    seg = torch.tensor([0] + sizes).cumsum(0).add(first).to(torch.int32)
    rows = torch.randint(0, T, (P,), dtype=torch.int32, device="cuda", generator=gen)
    return A, W, seg, rows, P, (qa, sa, qw, sw)


@pytest.mark.parametrize("case", range(len(GROUPED)))
@pytest.mark.parametrize("kind", [FP32, BF16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("eights", [False, True])
def test_grouped(sq, case, kind, eights):
    """Also with O in eights, so that rows lie on the 16-byte grid."""
    import torch
    sizes, K, O = GROUPED[case]
    if eights:
        O += -O % 8
    A, W, seg, rows, P, (qa, sa, qw, sw) = grouped_case(sq, sizes, K, O, case)
    print(f"grouped P={P} E={len(sizes)} K={K} O={O} kind={kind} tile={tile(P, len(sizes), O, K, kind)}", flush=True)
    y = torch.full((P, O), GUARD, dtype=dtype_of(kind), device="cuda")
    sq.linear_grouped_int8(A, W, seg.cuda(), rows, out=y)
    at = seg.tolist()
    for e, (lo, hi) in enumerate(zip(at[:-1], at[1:])):
        src = rows[lo:hi].long()
        if hi > lo:
            check(y[lo:hi], *product((qa[src], sa[src]), (qw[e], sw[e])))
    assert bool((y[:at[0]] == GUARD).all()) and bool((y[at[-1]:] == GUARD).all()), "rows of no segment were written"


@pytest.mark.parametrize("case", range(len(GROUPED)))
def test_grouped_silu(sq, case):
    import torch
    sizes, K, O = GROUPED[case]
    I = O // 2
    A, W, seg, rows, P, _ = grouped_case(sq, sizes, K, weight_rows(O, SILU), case)
    print(f"grouped silu P={P} E={len(sizes)} K={K} I={I} tile={tile(P, len(sizes), 2 * I, K, SILU)}", flush=True)
    out = sq.Int8(torch.full((-(-I // 64), P, 64), 85, dtype=torch.int8, device="cuda"),
                  torch.full((P,), GUARD, device="cuda"), I)
    sq.linear_grouped_silu_int8(A, W, seg.cuda(), rows, out)
    y = torch.zeros((P, 2 * I), device="cuda")
    sq.linear_grouped_int8(A, W, seg.cuda(), rows, out=y)
    want = chain(sq, y, I)
    lo, hi = int(seg[0]), int(seg[-1])
    part = lambda t: sq.Int8(t.codes[:, lo:hi], t.scales[lo:hi], I)  # noqa: E731
    assert same(part(out), part(want))
    for rest in (slice(0, lo), slice(hi, P)):
        assert bool((out.codes[:, rest] == 85).all()) and bool((out.scales[rest] == GUARD).all())
