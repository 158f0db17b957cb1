"""Linear layers on the GPU in the forms that large and unusual calls take,
against the formula in 64 bits."""
import ctypes

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


@pytest.mark.parametrize("rows,n,k,rank", [(64, 256, 4096, 128), (64, 144, 2048, 16), (300, 272, 512, 96)])
def test_requests_that_overlap_leave_the_other_rows(env, rows, n, k, rank):
    """Offsets that go back and forth, each request with an adapter of its own: rows of one request only are as they
    should be, the others get the same values in every call, and the status tells."""
    L, torch = env
    # rows 0-7 and 40- belong to one request; 8-39 to up to four
    ends = [v for i in range(11) for v in (8 + 2 * i, 16 + 2 * i)]
    offsets = [0, *ends, 40, rows]
    c = Case(env, rows, n, k, rank, len(offsets) - 1, [1] * (len(offsets) - 1), range(len(offsets) - 1), "bf16", 1,
             seed=31)
    c.requests.offsets.copy_(torch.tensor(offsets, dtype=torch.int32))
    y, u = c.forward()
    assert int(c.status.item()) == L.STATUS_BAD_REQUEST
    grads = c.backward(u)
    for _ in range(5):
        y2, u2 = c.forward()
        assert torch.equal(y, y2) and torch.equal(u, u2)
        assert all(torch.equal(p, q) for p, q in zip(grads, c.backward(u)))
    # the formula for the rows of one request
    c.offsets, c.ids = [0, 8, 40, rows], [0, -1, len(offsets) - 2]
    want, wu, size, pairs = c.exact_forward()
    wdx, _, _, sizex, pairsx, _, _ = c.exact_backward(u)
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[8:40] = False
    c.near(y[keep], want[keep], size[keep], k + rank, pairs[keep])
    c.near(grads[0][keep], wdx[keep], sizex[keep], n + rank, pairsx[keep])


class Checked:
    """Forward and backward of a case through the bounds-checked build, beside the library itself."""

    def __init__(self, c):
        L, torch = c.env
        from lossless_fp8_weight_b200 import _build
        self.c, self.so = c, ctypes.CDLL(_build.build(checked=True))
        self.so.ecf8_linear_forward.argtypes = L._lib.ecf8_linear_forward.argtypes
        self.so.ecf8_linear_backward.argtypes = L._lib.ecf8_linear_backward.argtypes

    def run(self):
        """[y, u, dx, da, db] and the status."""
        c, torch = self.c, self.c.env[1]
        y = torch.zeros(c.rows, c.n, dtype=c.dtype, device="cuda")
        u = torch.zeros(c.rows, c.rank, device="cuda")
        grads = [torch.zeros_like(t) for t in (c.x, c.a, c.b)]
        q, s = c.linear._requests(c.requests), torch.cuda.current_stream().cuda_stream
        rest = (c.ws.data_ptr(), c.ws.numel(), c.status.data_ptr(), s)
        assert self.so.ecf8_linear_forward(c.linear._ref, q, c.x.data_ptr(), c.k, y.data_ptr(), c.n, c.rows,
                                           u.data_ptr(), *rest) == 0
        assert self.so.ecf8_linear_backward(c.linear._ref, q, c.x.data_ptr(), c.k, c.dy.data_ptr(), c.n, u.data_ptr(),
                                            grads[0].data_ptr(), c.k, grads[1].data_ptr(), grads[2].data_ptr(), c.rows,
                                            *rest) == 0
        torch.cuda.synchronize()
        status = int(c.status.item())
        c.status.zero_()
        return [y, u, *grads], status


@pytest.mark.parametrize("rows,n,k", [(40, 256, 4096), (600, 3328, 512)])
def test_two_copies_of_the_library_in_one_process(env, rows, n, k):
    """The checked build beside the other one: the same bits, whichever ran first."""
    L, torch = env
    c = Case(env, rows, n, k, 16, 2, [rows - 9], [1], "bf16", "row", seed=32)
    y, u = c.forward()
    want = [y, u, *c.backward(u)]
    got, status = Checked(c).run()
    assert status == 0 and all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("kernel", [0, 1, 2], ids=["projection", "first product", "gradients"])
@pytest.mark.parametrize("rows,n,k", [(40, 256, 4096), (600, 3328, 512)])
def test_a_wait_that_runs_out_is_reported(env, rows, n, k, kernel):
    """A barrier that waits for an arrival too many, with a limit of a millisecond: the calls end, say so, and leave the
    device as it was.  The bounds-checked build alone can be told to."""
    L, torch = env
    c = Case(env, rows, n, k, 16, 2, [rows - 9], [1], "bf16", "row", seed=32)
    checked = Checked(c)
    want, status = checked.run()
    assert status == 0
    limits = checked.so.ecf8_checked_limits
    limits.argtypes = [ctypes.c_int, ctypes.c_longlong, ctypes.c_uint32]
    limits(kernel, 2_000_000, 1)
    try:
        assert checked.run()[1] == L.STATUS_TIMEOUT
    finally:
        limits(kernel, 0, 0)
    got, status = checked.run()
    assert status == 0 and all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("at", [0, 100, 127, 128, 200, 255, 256, 300])
def test_a_row_that_is_not_finite_in_either_half_of_a_tile(env, at):
    """Tiles of a pair of CTAs, each of which reads half of the rows: an infinity of one row's A x is in all of its
    columns, and in no other row.  (x and W x are finite.)"""
    L, torch = env
    c = Case(env, 310, 4864, 128, 16, 2, [310], [1], "bf16", 1, seed=33)
    c.x[at, 3:5] = 3e38
    c.a[1, :, 3:5] = 1.0
    c.w[:, 3:5] = 0
    y, u = c.forward()
    assert bool(u[at].isinf().all())
    assert not bool(y[at].isfinite().any())
    rest = torch.arange(310, device="cuda") != at
    assert bool(y[rest].isfinite().all())
    want, _, size, pairs = c.exact_forward()
    c.near(y[rest], want[rest], size[rest], 128 + 16, pairs[rest])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,n,k,shift", [(70, 256, 512, 0), (70, 256, 512, 3), (2100, 256, 128, 0)])
def test_adapters_without_rows_get_zeros_whatever_their_alpha(env, rows, n, k, shift, dtype):
    """By both kinds of kernel: x and dy whose rows start off 16-byte bounds (shift) take the plain ones."""
    L, torch = env
    alpha = torch.tensor([float("nan"), 0.5, float("inf"), float("-inf")], device="cuda")
    c = Case(env, rows, n, k, 16, 4, [rows, 0], [1, 2], dtype, 1, seed=34, alpha=alpha)
    _, u = c.forward()
    if shift:
        c.x, c.dy = (torch.nn.functional.pad(t, (shift, 2))[:, shift:-2] for t in (c.x, c.dy))
    _, da, db = c.backward(u)
    for i in (0, 2, 3):
        assert bool((da[i] == 0).all()) and bool((db[i] == 0).all())
    _, wda, wdb, _, _, sa, sb = c.exact_backward(u)
    c.near(da[1], wda[1], sa[1], rows + n, sa[1])
    c.near(db[1], wdb[1], sb[1], rows, sb[1])
    assert int(c.status.item()) == 0
