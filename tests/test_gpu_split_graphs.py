"""Split-K calls of the two-path method in captured graphs: every graph has a
workspace of its own. Two graphs replayed on two streams at once give the eager
results, and a graph leaves memory alone that was handed out after its capture,
also where a later call on its stream needed a larger workspace."""

import numpy as np
import pytest

from synth import bf16_round
from gpu_util import bf16_to_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sq():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    import activation_sparsity_fp4_amd as sq
    return sq


def _layer(sq, T, K, O, seed):
    from activation_sparsity_fp4_amd import _lib
    rng = np.random.default_rng(seed)
    assert _lib.call("sharq_linear_workspace_bytes", T, O, K) > 0, "the shape must split K"
    w = sq.quantize_mxfp4(bf16_to_gpu(bf16_round((rng.standard_normal((O, K)) * 0.02).astype(np.float32))))
    return [sq.prepare(bf16_to_gpu(bf16_round(rng.standard_normal((T, K)).astype(np.float32)))) for _ in range(2)], w


def _same(a, b):
    import torch
    return torch.equal(a.view(torch.int32), b.view(torch.int32))


@pytest.mark.parametrize("T,K,O", [(4, 8192, 512), (64, 14336, 1024)])
def test_two_graphs_at_once(sq, T, K, O):
    import torch
    print(f"two graphs T={T} K={K} O={O}", flush=True)
    preps, w = _layer(sq, T, K, O, T)
    want = [sq.linear(p, w) for p in preps]
    hidden = [sq.linear_silu_prepare(p, w)[0] for p in preps]
    graphs, outs, hs = [], [], []
    for p in preps:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ys = [sq.linear(p, w) for _ in range(20)]
            hs.append(sq.linear_silu_prepare(p, w)[0])
        graphs.append(g)
        outs.append(ys)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for rep in range(3):
        for ys in outs:
            for y in ys:
                y.fill_(float("nan"))
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        eager = sq.linear(preps[0], w)
        torch.cuda.synchronize()
        assert _same(eager, want[0])
        for i in range(2):
            assert all(_same(y, want[i]) for y in outs[i]), (rep, i)
            for f in ("bb_codes", "bb_scales", "res_codes", "res_scales", "mask"):
                assert torch.equal(getattr(hs[i], f), getattr(hidden[i], f)), (rep, i, f)


def test_a_graph_leaves_later_memory_alone(sq):
    import torch
    (small, _), w = _layer(sq, 4, 8192, 512, 1)
    (large, _), w2 = _layer(sq, 64, 14336, 4096, 2)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        want = sq.linear(small, w)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            y = sq.linear(small, w)
        sq.linear(large, w2)
        others = [torch.full((1 << 18,), 7, dtype=torch.int32, device="cuda") for _ in range(64)]
        torch.cuda.synchronize()
        for _ in range(3):
            y.fill_(float("nan"))
            g.replay()
            torch.cuda.synchronize()
            assert _same(y, want)
            assert all(bool((t == 7).all()) for t in others)
