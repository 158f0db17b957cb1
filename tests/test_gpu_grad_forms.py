"""Gradient sets on the GPU: norms past float32, and sets of which only the norm is wanted."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env(gpu_available):
    import torch
    import lossless_fp8_weight_b200 as L
    return L, torch


@pytest.mark.parametrize("values,finite", [([3e38, 3e38], False), ([3e38, 1e38], True), ([-3.4e38] * 9, False)])
@pytest.mark.parametrize("in_place", [True, False])
def test_the_status_tells_what_the_norm_shows(env, values, finite, in_place):
    """A norm of finite values that float32 does not hold is shown as infinite: then the status says so, and the
    gradients stay as they are; one that it holds is clipped by."""
    L, torch = env
    grads = [torch.tensor(values, device="cuda"), torch.ones(1000, device="cuda", dtype=torch.bfloat16)]
    before = [g.clone() for g in grads]
    outs = None if in_place else [torch.full_like(g, 9.0) for g in grads]
    norm, status = torch.zeros(1, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    L.GradSet(grads, outs).clip(1.0, norm, status=status)
    got = grads if in_place else outs
    assert bool(norm.isfinite()) == finite
    assert int(status.item()) == (0 if finite else L.STATUS_NONFINITE)
    want = float(sum((b.double() ** 2).sum() for b in before).sqrt())
    for g, b in zip(got, before):
        if finite:  # a factor and a product in float32, rounded to the type
            exact = b.double() / want
            most = (torch.finfo(b.dtype).eps / 2 + 2.0 ** -22) * exact.abs() + 2.0 ** -133
            assert bool(((g.double() - exact).abs() <= most).all())
        else:
            assert torch.equal(g, b)


def test_sets_of_which_only_the_norm_is_wanted(env):
    """Without outputs a tensor may be listed twice, or lie in another; such a set is not clipped."""
    L, torch = env
    g = torch.randn(5000, device="cuda")
    grads = [g, g[100:700], g, g[3:4], g.to(torch.bfloat16)]
    before, norm = g.clone(), torch.zeros(1, device="cuda")
    s = L.GradSet(grads, [None] * 5)
    s.norm(norm)
    want = float(sum((t.double() ** 2).sum() for t in grads).sqrt())
    assert abs(float(norm) - want) <= 2.0 ** -23 * want and torch.equal(g, before)
    with pytest.raises(L.Ecf8Error) as e:
        s.clip(1.0, norm)
    assert e.value.code == -1
    # one output missing is one too few
    with pytest.raises(L.Ecf8Error):
        L.GradSet([g, g.clone()], [torch.empty_like(g), None]).clip(1.0, norm)
    torch.cuda.synchronize()
    assert torch.equal(g, before)
