"""GPU parity of the 8-bit integer path against the NumPy oracle.

Codes and scales are compared bit for bit. A product's sum is exact; its value
is fma(fl(fl(sum) sa), sw, bias): two roundings of 2^-24 before the last
operation, and one of 2^-24 of the result (plus half the smallest subnormal
where it underflows), so |Y - ref| <= 2^-24 (2.01 |Y - bias| + 1.01 |Y|) +
2^-149. A bf16 output adds half a step, 2^-8 of its value."""

import numpy as np
import pytest

from oracle import (linear_grouped_int8_ref, linear_int8_ref, moe_route_ref, quantize_int8_ref, rms_row_scale_ref)
from synth import bf16_round, bf16_to_f32
from gpu_util import bf16_to_gpu, f32_to_gpu, i32_to_gpu, to_np

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sq():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    import activation_sparsity_fp4_amd as sq
    return sq


def i8_to_gpu(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, np.int8)).cuda()


def staged(q):
    """Row-major codes [.., R, K] -> [.., ceil(K / 64), R, 64] (data movement only)."""
    *lead, R, K = q.shape
    G = -(-K // 64)
    pad = np.zeros((*lead, R, G * 64), np.int8)
    pad[..., :K] = q
    return np.ascontiguousarray(np.swapaxes(pad.reshape(*lead, R, G, 64), -3, -2))


def to_gpu(sq, q, s):
    return sq.Int8(i8_to_gpu(staged(q)), f32_to_gpu(s), q.shape[-1])


def row_major(t):
    c = to_np(t.codes)
    *lead, G, R, _ = c.shape
    flat = np.swapaxes(c, -3, -2).reshape(*lead, R, G * 64)
    assert not flat[..., t.K:].any(), "bytes past K must be zero"
    return flat[..., :t.K]


def check_codes(t, x, rows=None):
    """An Int8 tensor against the oracle's codes of the values x (on the rows given)."""
    q, s = quantize_int8_ref(x)
    got, gs = row_major(t), to_np(t.scales)
    if rows is not None:
        got, gs = got[rows], gs[rows]
    assert np.array_equal(gs, s, equal_nan=True), (gs[gs != s][:4], s[gs != s][:4])
    bad = np.argwhere(got != q)
    assert not len(bad), (len(bad), bad[0], got[tuple(bad[0])], q[tuple(bad[0])])


def close(y, ref, size, rows=None):
    import torch
    got = y.double().cpu().numpy()
    tol = 2.0 ** -24 * (2.01 * size + 1.01 * np.abs(ref)) + 2.0 ** -149
    if y.dtype == torch.bfloat16:
        tol += 2.0 ** -8 * np.abs(ref) + 2.0 ** -134
    err = np.abs(got - ref)
    if rows is not None:
        err, tol = err[rows], tol[rows]
    assert np.all(err <= tol), f"{(~(err <= tol)).sum()} of {err.size} outside; worst {np.nanmax(err / tol)}"


def random_int8(rng, *shape, full=False):
    """Codes [.., R, K] and scales [.., R]; with full every code from -128 to 127."""
    q = rng.integers(-128, 128, shape) if full else np.clip(np.rint(rng.standard_normal(shape) * 30), -127, 127)
    return q.astype(np.int8), (rng.lognormal(0, 1, shape[:-1]) * 0.01).astype(np.float32)


def same(a, b):
    import torch
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def same_int8(a, b):
    return same(a.codes, b.codes) and same(a.scales, b.scales)


# ---------------------------------------------------------------------------
# Coding
# ---------------------------------------------------------------------------

TYPES = ["bf16", "fp16", "fp32"]


def typed(x, kind):
    """(the values of x in the type, as float32; a GPU tensor of them)."""
    import torch
    x = np.asarray(x, np.float32)
    if kind == "bf16":
        b = bf16_round(x)
        return bf16_to_f32(b), bf16_to_gpu(b)
    with np.errstate(over="ignore"):
        h = x.astype(np.float16 if kind == "fp16" else np.float32)
    return h.astype(np.float32), torch.from_numpy(h).cuda()


CODED = [(1, 1), (2, 7), (3, 64), (5, 1000), (17, 4096), (2, 28672), (1, 131071), (1, 131064), (4, 513), (1030, 520),
         (1025, 8), (1100, 2051), (1024, 9000)]


@pytest.mark.parametrize("R,K", CODED)
@pytest.mark.parametrize("kind", TYPES)
def test_quantize(sq, R, K, kind):
    print(f"quantize {kind} R={R} K={K}", flush=True)
    rng = np.random.default_rng(R + K)
    x = rng.standard_normal((R, K)) * rng.lognormal(0, 0.5, (R, 1))
    x[:, rng.random(K) < 0.01] *= 20
    v, t = typed(x, kind)
    check_codes(sq.quantize_int8(t), v)


def border_rows(K):
    """Rows of entries at and right beside the middles of two codes, and rows of the types' limits."""
    rng = np.random.default_rng(5)
    rows = []
    for s in (1.0, 0.0371, 3e-5, 1e30, 2.0 ** -110):
        s = np.float32(s)
        k = rng.integers(-127, 127, K) + 0.5
        x = (k * np.float64(s)).astype(np.float32)
        x[1::3] = np.nextafter(x[1::3], np.float32(0))
        x[2::3] = np.nextafter(x[2::3], np.float32(np.inf))
        x[0] = np.float32(127) * s
        rows.append(x)
    for top in (2.0 ** -149, 3 * 2.0 ** -149, 300 * 2.0 ** -149, 2.0 ** -133, 2.0 ** -126, 2.0 ** -119, 3e38, 65504.0):
        rows.append((rng.uniform(-1, 1, K) * top).astype(np.float32))
        rows[-1][K // 2] = top
    rows += [np.zeros(K, np.float32), -np.zeros(K, np.float32)]
    for bad in (np.nan, np.inf, -np.inf):
        rows.append(rng.standard_normal(K).astype(np.float32))
        rows[-1][K - 1] = bad
    one = np.zeros(K, np.float32)
    one[K - 1] = -2.5
    half = np.where(np.arange(K) % 2, 1.0, 0.5).astype(np.float32)  # amax / 2 is next to code 63.5
    return np.stack(rows + [one, half])


@pytest.mark.parametrize("K", [24, 1001])
@pytest.mark.parametrize("kind", TYPES)
def test_quantize_borders(sq, K, kind):
    print(f"quantize borders {kind} K={K}", flush=True)
    v, t = typed(border_rows(K), kind)
    check_codes(sq.quantize_int8(t), v)


@pytest.mark.parametrize("R,K,ld,skip", [(5, 512, 520, 8), (5, 512, 519, 0), (3, 100, 300, 1), (1030, 96, 101, 3),
                                         (1030, 96, 104, 4)])
@pytest.mark.parametrize("kind", TYPES)
def test_quantize_strided(sq, R, K, ld, skip, kind):
    """Rows apart, off the 16-byte grid, and views into a larger tensor."""
    rng = np.random.default_rng(ld)
    v, t = typed(rng.standard_normal((R, ld)), kind)
    k = min(K, ld - skip)
    check_codes(sq.quantize_int8(t[:, skip:skip + k]), v[:, skip:skip + k])


def test_quantize_more_rows_than_a_grid_is_wide(sq):
    import torch
    R, K = (1 << 20) + 5, 16
    x = torch.randn((R, K), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).bfloat16()
    q = sq.quantize_int8(x)
    rows = np.concatenate([np.arange(0, R, 9973), [(1 << 20) - 1, 1 << 20, R - 1]])
    at = torch.from_numpy(rows).cuda()
    check_codes(sq.Int8(q.codes[:, at], q.scales[at], K), x[at].float().cpu().numpy())


def test_quantize_into_and_empty(sq):
    import torch
    v, t = typed(np.random.default_rng(0).standard_normal((9, 130)), "bf16")
    out = sq.Int8(torch.full((3, 9, 64), 85, dtype=torch.int8, device="cuda"), torch.full((9,), 7.0, device="cuda"), 130)
    assert sq.quantize_int8(t, out) is out
    check_codes(out, v)
    none = sq.quantize_int8(t[:0])
    assert none.codes.shape == (3, 0, 64) and none.scales.shape == (0,)
    assert sq.quantize_int8(t[:0], rms_eps=1e-5).codes.shape == (3, 0, 64)


@pytest.mark.parametrize("E,R,K", [(1, 5, 70), (3, 33, 64), (4, 1, 200), (5, 300, 129)])
def test_quantize_expert_stacks(sq, E, R, K):
    rng = np.random.default_rng(E)
    x = rng.standard_normal((E, R, K + 8)).astype(np.float32)
    for view in (lambda a: a[:, :, :K], lambda a: a[::-1][:, :, 3:3 + K] if isinstance(a, np.ndarray) else
                 a.flip(0)[:, :, 3:3 + K]):
        v, t = typed(x, "bf16")
        q = sq.quantize_int8(view(t))
        assert q.codes.shape == (E, -(-K // 64), R, 64)
        for e in range(E):
            check_codes(sq.Int8(q.codes[e], q.scales[e], K), view(v)[e])
    v, t = typed(x.transpose(1, 0, 2), "fp32")
    q = sq.quantize_int8(t.transpose(0, 1))  # experts interleaved
    for e in range(E):
        check_codes(sq.Int8(q.codes[e], q.scales[e], K + 8), v[:, e])


NORMED = [(1, 32), (1, 4096), (3, 1000), (8, 8192), (2, 28672), (1, 100000), (5, 1001), (1026, 4096), (1030, 264),
          (2048, 1000)]


@pytest.mark.parametrize("R,K", NORMED)
@pytest.mark.parametrize("gamma", [False, True])
def test_quantize_norm(sq, R, K, gamma):
    print(f"quantize norm R={R} K={K} gamma={gamma}", flush=True)
    rng = np.random.default_rng(R * K)
    v, t = typed(rng.standard_normal((R, K)) * rng.lognormal(0, 1, (R, 1)), "bf16")
    g, gt = typed(rng.uniform(0.5, 1.5, K), "bf16")
    r = (1 / np.sqrt((v.astype(np.float64) ** 2).mean(1) + np.float64(np.float32(1e-5)))).astype(np.float32)
    x = bf16_to_f32(bf16_round(v * r[:, None]))
    check_codes(sq.quantize_int8(t, gamma=gt if gamma else None, rms_eps=1e-5), x * g if gamma else x)


def test_quantize_norm_is_the_norm_of_prepare(sq):
    """Against the row scale whose sum's order is fixed (equal but for a last bit that these rows do not meet)."""
    rng = np.random.default_rng(2)
    v, t = typed(rng.standard_normal((40, 512)), "bf16")
    r = rms_row_scale_ref(bf16_round(v), 1e-5)
    x = bf16_to_f32(bf16_round(v * np.asarray(r, np.float32).reshape(-1, 1)))
    check_codes(sq.quantize_int8(t, rms_eps=1e-5), x)


def test_norm_of_misaligned_rows_and_gamma(sq):
    rng = np.random.default_rng(3)
    v, t = typed(rng.standard_normal((6, 203)), "bf16")
    g, gt = typed(rng.uniform(0.5, 1.5, 201), "bf16")
    v, t = v[:, 1:201], t[:, 1:201]
    r = (1 / np.sqrt((v.astype(np.float64) ** 2).mean(1) + np.float64(np.float32(1e-6)))).astype(np.float32)
    x = bf16_to_f32(bf16_round(v * r[:, None]))
    check_codes(sq.quantize_int8(t, gamma=gt[1:], rms_eps=1e-6), x * g[1:])


def test_norm_of_rows_without_a_value(sq):
    """Zeros, a NaN and an infinity."""
    import torch
    x = torch.zeros(4, 96, dtype=torch.bfloat16, device="cuda")
    x[1, 3], x[2, 5], x[3, 7] = float("nan"), float("inf"), 3.0
    q = sq.quantize_int8(x, rms_eps=1e-5)
    s = to_np(q.scales)
    assert s[0] == 0 and np.isnan(s[1]) and np.isnan(s[2]) and s[3] > 0
    c = row_major(q)
    assert not c[:3].any() and c[3, 7] == 127


@pytest.mark.parametrize("shape", [(1, 1), (3, 64), (5, 100), (70, 129), (2, 3, 40), (4, 33, 256)])
def test_pack_and_unpack(sq, shape):
    rng = np.random.default_rng(sum(shape))
    q, s = random_int8(rng, *shape, full=True)
    t = sq.pack_int8(i8_to_gpu(q), f32_to_gpu(s))
    assert np.array_equal(to_np(t.codes), staged(q)) and np.array_equal(to_np(t.scales), s)
    assert np.array_equal(to_np(sq.unpack_int8(t)), q)


def test_pack_off_the_grid(sq):
    q, s = random_int8(np.random.default_rng(1), 6, 64, full=True)
    flat = i8_to_gpu(np.concatenate([np.zeros(3, np.int8), q.reshape(-1)]))
    assert np.array_equal(to_np(sq.pack_int8(flat[3:].view(6, 64), f32_to_gpu(s)).codes), staged(q))


# ---------------------------------------------------------------------------
# Products
# ---------------------------------------------------------------------------

SIZES = [(1, 1, 1), (1, 64, 8), (1, 4096, 1000), (2, 96, 31), (7, 161, 257), (16, 4096, 96), (17, 65, 40),
         (31, 2080, 256), (32, 128, 513), (33, 288, 255), (64, 1024, 300), (65, 545, 129), (128, 4127, 64),
         (129, 256, 1027), (200, 97, 96), (257, 640, 513), (1, 16384, 257), (40, 8192, 130), (300, 8192, 72),
         (4100, 128, 4200), (1, 63, 8200), (700, 64, 2100), (1500, 192, 4100), (2048, 320, 6144), (3000, 100, 12000)]


@pytest.mark.parametrize("T,K,O", SIZES)
@pytest.mark.parametrize("out", ["fp32", "bf16"])
def test_linear(sq, T, K, O, out):
    import torch
    print(f"linear T={T} K={K} O={O} {out}", flush=True)
    rng = np.random.default_rng(T + K + O)
    a, w = random_int8(rng, T, K), random_int8(rng, O, K, full=True)
    dtype = torch.float32 if out == "fp32" else torch.bfloat16
    A, W = to_gpu(sq, *a), to_gpu(sq, *w)
    y = sq.linear_int8(A, W, dtype=dtype)
    assert y.dtype == dtype and y.shape == (T, O)
    qa, qw = torch.from_numpy(a[0]).cuda().double(), torch.from_numpy(w[0]).cuda().double()
    p = ((qa @ qw.T).cpu().numpy() * a[1].astype(np.float64)[:, None]) * w[1].astype(np.float64)  # sums below 2^53
    close(y, p, np.abs(p))
    assert same(y, sq.linear_int8(A, W, dtype=dtype)), "not deterministic"
    bias = rng.standard_normal(O).astype(np.float32)
    close(sq.linear_int8(A, W, dtype=dtype, bias=f32_to_gpu(bias)), p + bias, np.abs(p))


@pytest.mark.parametrize("T,O", [(3, 20), (40, 33), (130, 70)])
def test_linear_against_the_oracle(sq, T, O):
    rng = np.random.default_rng(T)
    a, w = random_int8(rng, T, 333, full=True), random_int8(rng, O, 333, full=True)
    close(sq.linear_int8(to_gpu(sq, *a), to_gpu(sq, *w)), *linear_int8_ref(*a, *w))


@pytest.mark.parametrize("T", [1, 40, 300])
def test_largest_sums(sq, T):
    """K = 131071 entries of -128 times -128 (2^31 - 2^14, the largest sum) and of 127 times -128."""
    K = 131071
    q = np.full((T, K), -128, np.int8)
    q[::2] = 127
    w = np.full((3, K), -128, np.int8)
    w[1] = 127
    one = np.ones
    y = sq.linear_int8(to_gpu(sq, q, one(T, np.float32)), to_gpu(sq, w, one(3, np.float32)))
    close(y, *linear_int8_ref(q, one(T), w, one(3)))


@pytest.mark.parametrize("T,K,O,ld", [(5, 256, 40, 41), (70, 128, 33, 64), (300, 160, 260, 263), (2, 16384, 40, 47),
                                      (260, 128, 500, 512), (600, 64, 4000, 4001), (20, 100, 36, 36)])
@pytest.mark.parametrize("out", ["fp32", "bf16"])
def test_linear_strided_output_leaves_the_rest(sq, T, K, O, ld, out):
    import torch
    print(f"linear strided T={T} K={K} O={O} ld={ld} {out}", flush=True)
    rng = np.random.default_rng(3)
    a, w = random_int8(rng, T, K), random_int8(rng, O, K)
    dtype = torch.float32 if out == "fp32" else torch.bfloat16
    whole = torch.full((T + 1, ld), 7.0, dtype=dtype, device="cuda")
    sq.linear_int8(to_gpu(sq, *a), to_gpu(sq, *w), out=whole[:T, :O])
    close(whole[:T, :O], *linear_int8_ref(*a, *w))
    assert (whole[T] == 7).all() and (whole[:, O:] == 7).all()


def test_empty_sizes(sq):
    import torch
    rng = np.random.default_rng(0)
    w = to_gpu(sq, *random_int8(rng, 8, 64))
    none = sq.Int8(torch.empty((1, 0, 64), dtype=torch.int8, device="cuda"), torch.empty(0, device="cuda"), 64)
    assert sq.linear_int8(none, w).shape == (0, 8)
    assert sq.linear_int8(w, none).shape == (8, 0)
    assert sq.linear_silu_int8(none, w).codes.shape == (1, 0, 64)


@pytest.mark.parametrize("T", [1, 20, 100, 700])
def test_scales_without_a_value(sq, T):
    """A scale of NaN or zero belongs to its row or column alone."""
    rng = np.random.default_rng(T)
    a, w = random_int8(rng, T, 100), random_int8(rng, 70, 100)
    a[1][T // 2] = np.nan
    w[1][3], w[1][7] = np.nan, 0
    y = to_np(sq.linear_int8(to_gpu(sq, *a), to_gpu(sq, *w)))
    bad = np.zeros_like(y, bool)
    bad[T // 2], bad[:, 3] = True, True
    assert np.array_equal(np.isnan(y), bad)
    if T > 1:
        assert not y[np.arange(T) != T // 2, 7].any()


def test_operand_beyond_two_gigabytes(sq):
    """A weight whose codes pass 2^31 bytes: sampled rows, few tokens and many."""
    import torch
    K, O = 8192, 280000
    assert K * O > 1 << 31
    gen = torch.Generator(device="cuda").manual_seed(4)
    codes = torch.randint(-128, 128, (K // 64, O, 64), dtype=torch.int8, device="cuda", generator=gen)
    scales = torch.rand(O, device="cuda", generator=gen)
    rng = np.random.default_rng(4)
    pick = np.concatenate([[0, O - 1, O - 256, 262143, 262144], rng.integers(0, O, 40)])
    at = torch.from_numpy(pick).cuda()
    qw = to_np(codes[:, at].permute(1, 0, 2).reshape(len(pick), -1))
    for T in (3, 70):
        print(f"weight of {K * O} bytes, T={T}", flush=True)
        a = random_int8(rng, T, K)
        y = sq.linear_int8(to_gpu(sq, *a), sq.Int8(codes, scales, K))
        close(y[:, at], *linear_int8_ref(*a, qw, to_np(scales[at])))


def test_result_beyond_four_gigabytes(sq):
    import torch
    T, K, O = 40000, 64, 30000
    assert T * O * 4 > 1 << 32
    rng = np.random.default_rng(6)
    a, w = random_int8(rng, T, K), random_int8(rng, O, K)
    print(f"result of {T * O * 4} bytes", flush=True)
    y = sq.linear_int8(to_gpu(sq, *a), to_gpu(sq, *w))
    rows = np.concatenate([[0, T - 1], rng.integers(0, T, 20)])
    close(y[torch.from_numpy(rows).cuda()], *linear_int8_ref(a[0][rows], a[1][rows], *w))


# ---------------------------------------------------------------------------
# Gate and up
# ---------------------------------------------------------------------------

SILU = [(1, 128, 128), (3, 97, 32), (16, 4096, 40), (20, 65, 72), (32, 256, 160), (33, 160, 256), (64, 4128, 64),
        (65, 128, 96), (130, 256, 384), (257, 544, 416), (1, 16384, 128), (40, 8192, 224), (1100, 128, 1000),
        (2048, 128, 4128), (2048, 64, 9000)]


@pytest.mark.parametrize("T,K,I", SILU)
def test_silu_equals_the_chain(sq, T, K, I):
    import torch
    print(f"silu T={T} K={K} I={I}", flush=True)
    rng = np.random.default_rng(T + K + I)
    a, w = to_gpu(sq, *random_int8(rng, T, K)), to_gpu(sq, *random_int8(rng, 2 * I, K, full=True))
    out = sq.Int8(torch.full((-(-I // 64), T, 64), 85, dtype=torch.int8, device="cuda"),
                  torch.full((T,), 7.0, device="cuda"), I)
    assert sq.linear_silu_int8(a, w, out) is out
    assert same_int8(out, sq.quantize_int8(sq.silu_mul(sq.linear_int8(a, w))))


@pytest.mark.parametrize("T", [1, 30, 100, 1100])
@pytest.mark.parametrize("I", [1, 5, 37, 203])
def test_silu_of_odd_widths(sq, T, I):
    """Gate and up rows of zeros up to a multiple of 8 change neither scales nor codes."""
    rng = np.random.default_rng(T + I)
    a = to_gpu(sq, *random_int8(rng, T, 70))
    q, s = random_int8(rng, 2 * I, 70, full=True)
    more = -I % 8
    pad = lambda x: np.concatenate([np.concatenate([h, np.zeros((more, *x.shape[1:]), x.dtype)])  # noqa: E731
                                    for h in (x[:I], x[I:])])
    got = sq.linear_silu_int8(a, to_gpu(sq, q, s))
    want = sq.linear_silu_int8(a, to_gpu(sq, pad(q), pad(s)))
    assert same(got.scales, want.scales)
    assert np.array_equal(row_major(got), row_major(want)[:, :I])


def test_silu_against_float64(sq):
    """h within one bf16 step of float64's, so its codes within a code of float64's codes."""
    T, K, I = 40, 256, 128
    rng = np.random.default_rng(8)
    a, w = random_int8(rng, T, K), random_int8(rng, 2 * I, K)
    y, _ = linear_int8_ref(*a, *w)
    h = y[:, :I] / (1 + np.exp(-y[:, :I])) * y[:, I:]
    got = sq.linear_silu_int8(to_gpu(sq, *a), to_gpu(sq, *w))
    s = to_np(got.scales).astype(np.float64)[:, None]
    # half a code, and of h the fp32 product (2^-21 of it covers a few roundings) and its rounding to bf16
    assert np.all(np.abs(row_major(got) * s - h) <= 0.5 * s + (2.0 ** -8 + 2.0 ** -20) * np.abs(h))


# ---------------------------------------------------------------------------
# Experts
# ---------------------------------------------------------------------------

GROUPED = [
    # E, K, O, segments, gathered
    (3, 161, 40, [0, 1, 1, 2], True),
    (5, 256, 300, [0, 0, 40, 41, 200, 200], True),  # empty experts, one row
    (4, 2080, 257, [0, 130, 130, 131, 300], False),
    (2, 96, 33, [0, 0, 0], True),  # no rows in any segment
    (130, 128, 64, [min(i, 90) for i in range(131)], True),  # more experts than one wave scans
    (200, 70, 40, [3 * i for i in range(201)], True),
    (2, 200, 500, [0, 17, 60], True),
    (3, 64, 2100, [0, 700, 1500, 1600], False),
    (4, 100, 200, [5, 20, 60, 60, 90], True),  # rows before the first segment
    (1, 130, 70, [0, 300], True),
    (8, 64, 1100, [300 * i for i in range(9)], True),
    (6, 100, 2048, [0, 500, 500, 513, 900, 1700, 1710], True),  # column tiles in eights, row tiles of every height
    (150, 64, 1024, [40 * i for i in range(151)], True),  # the same with more experts than two passes of a wave
]


def grouped_case(seed, E, K, O, seg, gather, T=None):
    rng = np.random.default_rng(seed)
    P = seg[-1] + 9
    T = T or (max(P // 3, 4) if gather else P)
    a, w = random_int8(rng, T, K), random_int8(rng, E, O, K, full=True)
    rows = rng.integers(0, T, P).astype(np.int32) if gather else None
    return a, w, np.asarray(seg, np.int32), rows, P


def covered(seg, P):
    in_segment = np.zeros(P, bool)
    in_segment[max(seg[0], 0):seg[-1]] = True
    return in_segment


@pytest.mark.parametrize("case", range(len(GROUPED)))
@pytest.mark.parametrize("out", ["fp32", "bf16"])
def test_grouped(sq, case, out):
    import torch
    print(f"grouped {GROUPED[case][:3]} {out}", flush=True)
    a, w, seg, rows, P = grouped_case(case, *GROUPED[case])
    dtype = torch.float32 if out == "fp32" else torch.bfloat16
    y = torch.full((P, w[0].shape[1]), 7.0, dtype=dtype, device="cuda")
    gathered = None if rows is None else i32_to_gpu(rows)
    A, W = to_gpu(sq, *a), to_gpu(sq, *w)
    assert sq.linear_grouped_int8(A, W, i32_to_gpu(seg), gathered, out=y) is y
    ref, size = linear_grouped_int8_ref(*a, *w, seg, rows, P)
    used = covered(seg, P)
    close(y, ref, size, used)
    assert bool((y[torch.from_numpy(~used).cuda()] == 7).all()), "rows of no segment were written"
    again = sq.linear_grouped_int8(A, W, i32_to_gpu(seg), gathered, dtype=dtype)
    assert same(again[torch.from_numpy(used).cuda()], y[torch.from_numpy(used).cuda()])


@pytest.mark.parametrize("case", range(len(GROUPED)))
@pytest.mark.parametrize("I", [16, 104])
def test_grouped_silu_equals_the_chain(sq, case, I):
    import torch
    E, K, _, seg, gather = GROUPED[case]
    print(f"grouped silu {E, K, I}", flush=True)
    a, w, seg, rows, P = grouped_case(case, E, K, 2 * I, seg, gather)
    gathered = None if rows is None else i32_to_gpu(rows)
    A, W, S = to_gpu(sq, *a), to_gpu(sq, *w), i32_to_gpu(seg)
    out = sq.Int8(torch.full((-(-I // 64), P, 64), 85, dtype=torch.int8, device="cuda"),
                  torch.full((P,), 7.0, device="cuda"), I)
    assert sq.linear_grouped_silu_int8(A, W, S, gathered, out) is out
    y = torch.zeros((P, 2 * I), device="cuda")
    sq.linear_grouped_int8(A, W, S, gathered, out=y)
    want = sq.quantize_int8(sq.silu_mul(y))
    used = torch.from_numpy(covered(seg, P)).cuda()
    assert same(out.codes[:, used], want.codes[:, used]) and same(out.scales[used], want.scales[used])
    assert bool((out.codes[:, ~used] == 85).all()) and bool((out.scales[~used] == 7).all())


@pytest.mark.parametrize("E,P", [(3, 40), (2, 300)])
def test_malformed_segments_and_rows(sq, E, P):
    """Offsets outside [0, P] or decreasing and gathered rows outside the activation address no memory outside their
    tensors; a gathered row outside counts as zeros."""
    import torch
    a, w, _, rows, _ = grouped_case(3, E, 90, 50, [0] * E + [P - 9], True, T=P // 3)
    rows[::5], rows[1::7] = -1, P // 3 + 5
    A, W = to_gpu(sq, *a), to_gpu(sq, *w)
    seg = [0] * E + [P + 50]
    y = sq.linear_grouped_int8(A, W, i32_to_gpu(seg), i32_to_gpu(rows))
    close(y, *linear_grouped_int8_ref(*a, *w, seg, rows, P))
    for seg in ([-7] * E + [P + 3], [P] + [0] * E, [P // 2] * E + [0]):
        guard = torch.full((P + 64, 50), 7.0, device="cuda")
        sq.linear_grouped_int8(A, W, i32_to_gpu(seg), i32_to_gpu(rows), out=guard[:P])
        h = sq.linear_grouped_silu_int8(A, W, i32_to_gpu(seg), i32_to_gpu(rows))
        assert h.codes.shape == (1, P, 64)
        torch.cuda.synchronize()
        assert bool((guard[P:] == 7).all())


def _layer(sq, T, E, k, H, I, seed):
    rng = np.random.default_rng(seed)
    x = bf16_round((rng.standard_normal((T, H)) * rng.lognormal(0, 0.5, (T, 1))).astype(np.float32))
    logits = rng.standard_normal((T, E)).astype(np.float32)
    gu = quantize_int8_ref(bf16_to_f32(bf16_round((rng.standard_normal((E * 2 * I, H)) * 0.05).astype(np.float32))))
    dn = quantize_int8_ref(bf16_to_f32(bf16_round((rng.standard_normal((E * H, I)) * 0.05).astype(np.float32))))
    gu = gu[0].reshape(E, 2 * I, H), gu[1].reshape(E, 2 * I)
    dn = dn[0].reshape(E, H, I), dn[1].reshape(E, H)
    return x, logits, gu, dn


def _run_layer(sq, x, logits, k, gu, dn, num_tokens=None):
    import torch
    r = sq.moe_route(logits, k, num_tokens=num_tokens)
    a = sq.quantize_int8(x)
    h = sq.linear_grouped_silu_int8(a, gu, r.seg_offsets, r.a_rows)
    y = sq.linear_grouped_int8(h, dn, r.seg_offsets, dtype=torch.bfloat16)
    return r, a, h, sq.moe_combine(y, r.pair_index, r.weight, bf16=True)


@pytest.mark.parametrize("T,E,k,pad", [(1, 4, 2, 0), (5, 16, 3, 0), (50, 8, 2, 7), (400, 6, 3, 0)])
def test_expert_layer(sq, T, E, k, pad):
    """moe_route -> quantize_int8 -> grouped gate|up -> grouped down -> moe_combine, some tokens padding.

    Codes of x and the routing equal the oracle's. h and y: h = bf16 of a value whose fp32 steps err by less than
    2^-20 of it plus 2^-22 of its factors' products, coded to half a step; the down product of the codes that the GPU
    holds is exact up to its roundings, so the combined row differs from float64's combination of that product by at
    most 2^-8 of each weighted pair (its bf16 rounding), 2^-22 of their sum (fp32 additions) and 2^-8 of the result."""
    import torch
    H, I = 96, 40
    x, logits, gu, dn = _layer(sq, T, E, k, H, I, T)
    n = None if not pad else i32_to_gpu([T - pad])
    r, a, h, out = _run_layer(sq, bf16_to_gpu(x), f32_to_gpu(logits), k, to_gpu(sq, *gu), to_gpu(sq, *dn), n)
    check_codes(a, bf16_to_f32(x))
    ref = moe_route_ref(logits, k, num_tokens=T - pad)
    assert np.array_equal(to_np(r.expert), ref["expert"]) and np.array_equal(to_np(r.a_rows), ref["a_rows"])
    seg, P = ref["seg_offsets"], T * k
    live = int(seg[-1])
    qa, sa = quantize_int8_ref(bf16_to_f32(x))
    gy, _ = linear_grouped_int8_ref(qa, sa, *gu, seg, ref["a_rows"], P)
    g, u = gy[:live, :I], gy[:live, I:]
    want_h = g / (1 + np.exp(-g)) * u
    hq, hs = row_major(h)[:live], to_np(h.scales)[:live].astype(np.float64)[:, None]
    assert np.all(np.abs(hq * hs - want_h) <= 0.5 * hs + (2.0 ** -8 + 2.0 ** -20) * np.abs(want_h))
    y, size = linear_grouped_int8_ref(hq, hs[:, 0], *dn, seg, None, live)
    want, bound = np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        for j in range(k):
            p = ref["pair_index"][t, j]
            if p >= 0:
                want[t] += ref["weight"][t, j] * y[p]
                bound[t] += abs(ref["weight"][t, j]) * np.abs(y[p])
    tol = (2.0 ** -8 + 2.0 ** -20) * bound + 2.0 ** -8 * 1.01 * (np.abs(want) + 2.0 ** -8 * bound)
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= tol)
    if pad:
        assert not out[T - pad:].any()


# ---------------------------------------------------------------------------
# Streams and graphs
# ---------------------------------------------------------------------------


@pytest.mark.parametrize("T", [3, 40, 300])
def test_side_stream(sq, T):
    import torch
    x, logits, gu, dn = _layer(sq, T, 4, 2, 96, 40, 1)
    args = bf16_to_gpu(x), f32_to_gpu(logits), 2, to_gpu(sq, *gu), to_gpu(sq, *dn)
    want = _run_layer(sq, *args)[-1]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = _run_layer(sq, *args)[-1]
    s.synchronize()
    assert same(got, want)


@pytest.mark.parametrize("T,K,I", [(2, 512, 256), (40, 512, 264), (300, 512, 384)])
def test_two_graphs_at_once(sq, T, K, I):
    """An MLP block captured twice on inputs of its own, both replayed at once several times, eager calls between."""
    import torch
    rng = np.random.default_rng(T)
    gu = sq.quantize_int8(bf16_to_gpu(bf16_round((rng.standard_normal((2 * I, K)) * 0.05).astype(np.float32))))
    dn = sq.quantize_int8(bf16_to_gpu(bf16_round((rng.standard_normal((K, I)) * 0.05).astype(np.float32))))
    gamma = bf16_to_gpu(bf16_round(rng.uniform(0.5, 1.5, K).astype(np.float32)))
    xs = [bf16_to_gpu(bf16_round(rng.standard_normal((T, K)).astype(np.float32))) for _ in range(2)]

    def block(x):
        h = sq.linear_silu_int8(sq.quantize_int8(x, gamma=gamma, rms_eps=1e-5), gu)
        return sq.linear_int8(h, dn, dtype=torch.bfloat16)

    want = [block(x) for x in xs]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for x in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append([block(x) for _ in range(10)])
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for rep in range(3):
        for ys in outs:
            for y in ys:
                y.fill_(float("nan"))
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        eager = block(xs[0])
        torch.cuda.synchronize()
        assert same(eager, want[0])
        for i in range(2):
            assert all(same(y, want[i]) for y in outs[i]), (rep, i)


@pytest.mark.parametrize("T,E,k,H,I", [(2, 8, 2, 96, 40), (60, 16, 4, 128, 64), (500, 5, 2, 128, 512)])
def test_captured_expert_layer_with_new_inputs(sq, T, E, k, H, I):
    """A captured expert layer, replayed on inputs and routings that change between the replays."""
    import torch
    xs, ls = [], []
    for seed in range(4):
        x, logits, gu, dn = _layer(sq, T, E, k, H, I, seed)
        xs.append(bf16_to_gpu(x))
        ls.append(f32_to_gpu(logits))
    gu, dn = to_gpu(sq, *gu), to_gpu(sq, *dn)
    counts = torch.tensor([[T], [T - 1], [T // 2], [0]], dtype=torch.int32, device="cuda")
    want = [_run_layer(sq, xs[i], ls[i], k, gu, dn, counts[i])[-1] for i in range(4)]
    x, logits, n = xs[0].clone(), ls[0].clone(), counts[0].clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = _run_layer(sq, x, logits, k, gu, dn, n)[-1]
    for i in (0, 1, 2, 3, 0):
        x.copy_(xs[i])
        logits.copy_(ls[i])
        n.copy_(counts[i])
        out.fill_(float("nan"))
        g.replay()
        live = int(counts[i])
        assert same(out[:live], want[i][:live]) and not out[live:].any()
