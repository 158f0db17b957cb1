"""The global norm of a gradient set and clipping by it, on the GPU, against
64 bits.  The norm is a float64 sum rounded once: at most 2^-24 of it off, plus
n * 2^-53.  A clipped value is a float32 product rounded to its type: the
factor is off by 2^-24 twice (its division and rounding) and the product by
2^-24, so eps/2 + 2^-22 of the value, and half the smallest subnormal."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env(gpu_available):
    import torch
    import lossless_fp8_weight_b200 as L
    return L, torch


def _tensors(torch, sizes, kinds, seed=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    types = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
    return [(torch.randn(n, generator=g, device="cuda") * scale).to(types[k]) for n, k in zip(sizes, kinds)]


def _norm(grads):
    return math.sqrt(sum(float(t.double().square().sum()) for t in grads))


def _check(env, grads, outs, most, before):
    L, torch = env
    norm = torch.full((1,), -1.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    L.GradSet(grads, outs).clip(most, norm, status=status)
    want = _norm(before)
    assert abs(float(norm) - want) <= 2.0 ** -23 * want
    factor = min(1.0, most / (want + 1e-6))
    for b, o in zip(before, outs if outs is not None else grads):
        exact = b.double() * factor
        tol = (torch.finfo(b.dtype).eps / 2 + 2.0 ** -22) * exact.abs() + torch.finfo(b.dtype).tiny * torch.finfo(b.dtype).eps
        assert bool(((o.double() - exact).abs() <= tol).all())
    assert int(status.item()) == 0


SETS = [
    ([1], ["fp32"]),
    ([0, 1, 0], ["bf16", "fp16", "fp32"]),
    ([7, 8, 9, 8191, 8192, 8193, 0, 3], ["bf16"] * 8),
    ([100_003, 1, 65_536, 33], ["fp32", "bf16", "fp16", "fp32"]),
    ([0, 0, 0, 5000] * 100 + [0, 0], ["bf16", "fp32", "fp16", "fp32"] * 100 + ["bf16", "bf16"]),
    ([3_000_017, 12, 5_000_001], ["fp16", "bf16", "fp32"]),
    ([17 + 3 * i for i in range(1500)], ["bf16", "fp32"] * 750),
]


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("most", [0.25, 1e9])
@pytest.mark.parametrize("k", range(len(SETS)))
def test_clip_equals_the_formula(env, k, most, in_place):
    L, torch = env
    grads = _tensors(torch, *SETS[k], seed=k)
    before = [g.clone() for g in grads]
    outs = None if in_place else [torch.full_like(g, 9.0) for g in grads]
    _check(env, grads, outs, most, before)
    if not in_place:
        assert all(torch.equal(g, b) for g, b in zip(grads, before))


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_views_at_any_offset_of_a_flat_buffer(env, dtype):
    """Packed gradients start at any element; in and out may be offset differently; nothing around them changes."""
    L, torch = env
    (flat,) = _tensors(torch, [100_000], [dtype], seed=3)
    out = torch.full_like(flat, 5.0)
    spans = [(1, 3), (3, 20), (20, 21), (25, 9000), (9001, 40_003), (40_010, 99_999)]
    for shift in (0, 1, 3):
        out.fill_(5.0)
        grads = [flat[a:b] for a, b in spans]
        outs = [out[a - (a > 20) * shift:b - (a > 20) * shift] for a, b in spans]
        _check(env, grads, outs, 0.5, [g.clone() for g in grads])
        covered = torch.zeros(flat.numel(), dtype=torch.bool, device="cuda")
        for a, b in spans:
            covered[a - (a > 20) * shift:b - (a > 20) * shift] = True
        assert bool((out[~covered] == 5).all())


def test_norm_alone_needs_no_outputs_and_changes_nothing(env):
    L, torch = env
    grads = _tensors(torch, [1000, 70_001], ["bf16", "fp32"], seed=4)
    before = [g.clone() for g in grads]
    norm = torch.zeros(1, device="cuda")
    L.GradSet(grads).norm(norm)
    assert abs(float(norm) - _norm(grads)) <= 2.0 ** -23 * _norm(grads)
    assert all(torch.equal(g, b) for g, b in zip(grads, before))


def test_empty_sets(env):
    L, torch = env
    for grads in ([], [torch.empty(0, device="cuda")], [torch.empty(0, device="cuda", dtype=torch.bfloat16)] * 5):
        norm = torch.full((1,), 3.0, device="cuda")
        L.GradSet(grads).clip(1.0, norm)
        assert float(norm) == 0.0


@pytest.mark.parametrize("scale", [1e-25, 1e-38, 1e18, 1e30])
def test_squares_outside_float32_are_summed(env, scale):
    L, torch = env
    grads = _tensors(torch, [5000, 123], ["fp32", "bf16"], seed=5, scale=scale)
    norm = torch.zeros(1, device="cuda")
    L.GradSet(grads).norm(norm)
    want = _norm(grads)
    assert abs(float(norm) - want) <= 2.0 ** -23 * want + 2.0 ** -149


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("in_place", [True, False])
def test_a_norm_that_is_not_finite_leaves_the_gradients(env, bad, in_place):
    L, torch = env
    grads = _tensors(torch, [100, 50_000, 3], ["bf16", "fp32", "fp16"], seed=6)
    grads[1][49_999] = bad
    before = [g.clone() for g in grads]
    outs = None if in_place else [torch.full_like(g, 9.0) for g in grads]
    norm, status = torch.zeros(1, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    s = L.GradSet(grads, outs)
    s.clip(1.0, norm, status=status)
    assert int(status.item()) == L.STATUS_NONFINITE and not math.isfinite(float(norm))
    for g, b in zip(outs if outs else grads, before):
        assert torch.equal(g.view(torch.uint8), b.view(torch.uint8))


def test_limits_of_zero_and_infinity(env):
    L, torch = env
    grads = _tensors(torch, [1000], ["fp32"], seed=7)
    norm = torch.zeros(1, device="cuda")
    out = [torch.full_like(grads[0], 9.0)]
    L.GradSet(grads, out).clip(float("inf"), norm)
    assert torch.equal(out[0], grads[0])
    L.GradSet(grads, out).clip(0.0, norm)
    assert float(out[0].abs().max()) == 0.0


def test_repeated_and_captured_calls(env):
    L, torch = env
    grads = _tensors(torch, [1_000_003, 77, 400_000], ["bf16", "fp32", "fp16"], seed=8)
    outs = [torch.zeros_like(g) for g in grads]
    norm = torch.zeros(1, device="cuda")
    s = L.GradSet(grads, outs)
    s.clip(1.0, norm)
    first = (norm.clone(), [o.clone() for o in outs])
    for _ in range(5):
        s.clip(1.0, norm)
        assert torch.equal(norm, first[0]) and all(torch.equal(o, f) for o, f in zip(outs, first[1]))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.clip(1.0, norm)
    for g in grads:
        g.mul_(3)
    graph.replay()
    want = _norm(grads)
    assert abs(float(norm) - want) <= 2.0 ** -23 * want
    # a set on another stream, with its own workspace, beside it
    other = _tensors(torch, [200_000], ["fp32"], seed=9)
    norm2 = torch.zeros(1, device="cuda")
    torch.cuda.synchronize()
    s2, side = L.GradSet(other), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        s.norm(norm)
        s2.norm(norm2, stream=side)
    torch.cuda.synchronize()
    assert abs(float(norm2) - _norm(other)) <= 2.0 ** -23 * _norm(other)
    assert abs(float(norm) - want) <= 2.0 ** -23 * want
