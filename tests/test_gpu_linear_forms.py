"""Linear layers on the GPU in the forms that large and unusual calls take,
against the formula in 64 bits."""
import pytest

from test_gpu_linear import Case, env  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,k", [(128, 512), (600, 3328)])
def test_a_scaled_weight_is_not_rounded_before_the_product(env, rows, k, dtype):
    """One term a sum: dx[t] = s[t] W[t] dy[t][t], with scales over 2^-10 of the largest.  It is rounded to its type
    once (eps/2); before that a term loses 2^-17 (BF16) or 2^-23 (FP16), or 2^-31 of the largest scale's, and three
    float32 roundings.  A product of s W rounded to the type would lose another eps/2."""
    L, torch = env
    c = Case(env, rows, rows, k, 1, 0, [rows], [-1], dtype, "row", seed=rows)
    c.scale.copy_(2.0 ** (torch.arange(rows, device="cuda") % 11 - 8) * (1 + torch.rand(rows, device="cuda")))
    c.dy = torch.diag((0.5 + torch.rand(rows, device="cuda"))).to(c.dtype)
    dx, _, _ = c.backward(None)
    w, s = c.wide()
    want = w * (s * c.dy.double().diag())[:, None]
    kinds = torch.finfo(c.dtype)
    lost = 2.0 ** -17 if dtype == "bf16" else 2.0 ** -23
    most = (kinds.eps / 2 * (1 + lost) + lost + 2.0 ** -22) * want.abs() + kinds.smallest_normal * kinds.eps / 2
    if dtype == "fp16":
        most += 2.0 ** -31 * float(s.max()) * c.dy.double().diag()[:, None]
    err = (dx.double() - want).abs()
    assert bool((err <= most).all()), float((err / most).max())
