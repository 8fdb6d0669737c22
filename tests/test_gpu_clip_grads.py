"""GPU tests of the gradients' global norm and their clipping."""
import math

import pytest
import torch

from e4m3_ref import UBF16, U32, within
from gpu_util import log

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def wc():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    from lossless_entropy_coded_amd import wc as mod
    return mod


def _run(wc, grads, outs, max_norm, **kw):
    handle = wc.GradList(grads, outs)
    need = wc.clip_grads_work_bytes(handle)
    work = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    norm = torch.full((3,), -7.0, device="cuda")
    wc.clip_grads_async(handle, max_norm, norm[1:2], work if need else None, need, **kw)
    torch.cuda.synchronize()
    assert bool((work[need:] == 0xFF).all()) and float(norm[0]) == float(norm[2]) == -7.0
    return norm[1].clone()


def _norm64(grads):
    return math.sqrt(sum(float(g.double().square().sum()) for g in grads))


def _check(grads, outs, norm, max_norm):
    """The norm is a sum in double precision, rounded once; the factor is rounded, and the product: 2^-23 in all, before
    the rounding to bf16."""
    want = _norm64(grads)
    assert abs(float(norm) - want) <= (U32 + 1e-12) * want
    for g, out in zip(grads, outs):
        assert out.dtype == g.dtype
        if not want > max_norm:
            assert torch.equal(out.view(torch.int16 if g.dtype == BF16 else torch.int32),
                               g.view(torch.int16 if g.dtype == BF16 else torch.int32))
            continue
        exact = g.cpu().double() * (max_norm / want)
        tol = (2.0 ** -23 + 1e-12) * exact.abs() + 1e-45
        assert within(out, exact, tol + (UBF16 * (exact.abs() + tol) + 1e-40 if g.dtype == BF16 else 0.0))


LISTS = [[1], [7, 0, 1], [8, 16, 4096], [100003], [131, 4583, 131, 17161, 45457, 35], [1 << 20, 5, 1 << 18, 3],
         [64] * 300, [4096 * 3 + k for k in range(97)]]


@pytest.mark.parametrize("max_norm", [0.5, 1e9])
@pytest.mark.parametrize("kinds", ["f32", "bf16", "mixed"])
@pytest.mark.parametrize("sizes", LISTS, ids=lambda s: f"{len(s)}x{s[0]}")
def test_lists(wc, sizes, kinds, max_norm):
    g = torch.Generator().manual_seed(sum(sizes))
    log(f"case: clip_grads {len(sizes)} tensors, {sum(sizes)} elements, {kinds}, max {max_norm}")
    kind = [F32 if kinds == "f32" or (kinds == "mixed" and i % 2) else BF16 for i in range(len(sizes))]
    grads = [torch.randn(n, generator=g).to(k).cuda() for n, k in zip(sizes, kind)]
    kept = [t.clone() for t in grads]
    outs = [torch.full((n + 16,), -7.0, dtype=k, device="cuda") for n, k in zip(sizes, kind)]
    views = [o[:n] for o, n in zip(outs, sizes)]
    norm = _run(wc, grads, views, max_norm)
    _check(grads, views, norm, max_norm)
    assert all(bool((o[n:] == -7.0).all()) for o, n in zip(outs, sizes)), "wrote past the end"
    assert all(torch.equal(a, b) for a, b in zip(grads, kept))
    again = _run(wc, grads, None, max_norm)                     # in place: the same bits
    assert float(again) == float(norm)
    assert all(torch.equal(a, b) for a, b in zip(grads, views))


@pytest.mark.parametrize("kind", [F32, BF16])
@pytest.mark.parametrize("shift_in,shift_out", [(1, 1), (1, 0), (0, 3), (5, 2)])
def test_views_off_alignment(wc, kind, shift_in, shift_out):
    """Gradients that are views at any element of a flat buffer."""
    g = torch.Generator().manual_seed(4)
    log(f"case: clip_grads views {shift_in}, {shift_out} {kind}")
    sizes = [1, 9, 5000, 70001]
    flat = torch.randn(sum(sizes) + 64, generator=g).to(kind).cuda()
    into = torch.full_like(flat, -7.0)
    grads, outs, at = [], [], 0
    for n in sizes:
        grads.append(flat[at + shift_in:at + shift_in + n])
        outs.append(into[at + shift_out:at + shift_out + n])
        at += n
    norm = _run(wc, grads, outs, 1.0)
    _check(grads, outs, norm, 1.0)
    assert bool((into[:shift_out] == -7.0).all()) and bool((into[at + shift_out:] == -7.0).all())


@pytest.mark.parametrize("size", [1e-38, 1e-25, 1e18, 1e30, 3e38])
def test_sizes_of_values(wc, size):
    """Squares far outside fp32's range."""
    grads = [torch.full((1,), size, device="cuda"), torch.full((3,), -size, device="cuda")]
    log(f"case: clip_grads values of {size:g}")
    outs = [torch.empty_like(t) for t in grads]
    norm = _run(wc, grads, outs, size)
    if size < 2e38:
        _check(grads, outs, norm, float(torch.tensor(size)))
    else:      # the norm is past fp32's range: it is infinite, and nothing is changed
        assert math.isinf(float(norm)) and all(torch.equal(a, b) for a, b in zip(grads, outs))


@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("kind", [F32, BF16])
def test_no_numbers(wc, bad, kind):
    """The norm says so and the gradients stay as they are."""
    g = torch.Generator().manual_seed(1)
    grads = [torch.randn(3000, generator=g).to(kind).cuda(), torch.randn(70, generator=g).to(kind).cuda()]
    grads[0][1234] = bad
    log(f"case: clip_grads {bad} {kind}")
    outs = [torch.empty_like(t) for t in grads]
    norm = _run(wc, grads, outs, 1.0)
    assert math.isnan(float(norm)) if math.isnan(bad) else float(norm) == math.inf
    for a, b in zip(grads, outs):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_no_elements_and_infinite_bound(wc):
    log("case: clip_grads of nothing")
    assert float(_run(wc, [], None, 1.0)) == 0.0
    assert float(_run(wc, [torch.empty(0, device="cuda")], None, 1.0)) == 0.0
    many = [torch.empty(0, device="cuda")] * 200 + [torch.full((4,), 3.0, device="cuda")]
    assert float(_run(wc, many, None, math.inf)) == 6.0
    assert bool((many[-1] == 3.0).all())
    assert float(_run(wc, many, None, 0.0)) == 6.0 and bool((many[-1] == 0.0).all())


def test_streams_and_graph(wc):
    """Two lists at once, and a captured call that is replayed with other gradients."""
    g = torch.Generator().manual_seed(6)
    sizes = [50000, 129, 70001] + [33] * 150
    grads = [torch.randn(n, generator=g).cuda() for n in sizes]
    log("case: clip_grads on two streams and captured")
    want = [torch.empty_like(t) for t in grads]
    norm = _run(wc, grads, want, 1.0)
    calls = []
    for _ in range(2):
        outs = [torch.empty_like(t) for t in grads]
        handle = wc.GradList(grads, outs)
        need = wc.clip_grads_work_bytes(handle)
        calls.append((handle, outs, torch.empty(need, dtype=torch.uint8, device="cuda"),
                      torch.empty(1, device="cuda"), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for handle, _, work, into, stream in calls:
        wc.clip_grads_async(handle, 1.0, into, work, work.numel(), stream=stream)
    torch.cuda.synchronize()
    for _, outs, _, into, _ in calls:
        assert float(into) == float(norm) and all(torch.equal(a, b) for a, b in zip(outs, want))
    handle, outs, work, into, _ = calls[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        wc.clip_grads_async(handle, 1.0, into, work, work.numel())
    for seed in range(3):
        for t in grads:
            t.copy_(torch.randn(t.numel(), generator=torch.Generator().manual_seed(seed + t.numel())))
        norm = _run(wc, grads, want, 1.0)
        graph.replay()
        torch.cuda.synchronize()
        assert float(into) == float(norm) and all(torch.equal(a, b) for a, b in zip(outs, want))
