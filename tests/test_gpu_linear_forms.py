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


# ---- the form of large calls: two CTAs to a tile ----

def pairs(c, backward):
    """Fails where a size no longer takes that form."""
    assert c.linear.tile_ctas(c.rows, backward) == 2


BACK = [
    # rows, n, k, rank, adapters, lengths, ids; dx has 256 columns and 256 rows a tile
    (1300, 512, 4096, 16, 3, [700, 0, 500, 90], [2, 1, 0, -1]),
    (150, 264, 9472, 24, 2, [70, 80], [1, 0]),
    (700, 333, 3335, 12, 5, [100, 250, 0, 300], [4, 0, 1, 4]),
    (257, 64, 5120, 128, 2, [256], [1]),
    (1030, 2064, 2100, 64, 9, [100] * 10, [8, 7, 6, 5, 4, 3, 2, 1, 0, 8]),
    (600, 72, 3328, 1, 1, [600], [0]),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("n_scale", [0, 1, "row"])
@pytest.mark.parametrize("size", BACK, ids=lambda s: "x".join(map(str, s[:4])))
def test_large_input_gradients_equal_the_formula(env, size, n_scale, dtype):
    c = Case(env, *size, dtype, n_scale, seed=size[0])
    pairs(c, True)
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("n_scale", [0, 1, "row"])
@pytest.mark.parametrize("size", BACK, ids=lambda s: "x".join(map(str, s[:4])))
def test_large_projections_equal_the_formula(env, size, n_scale, dtype):
    rows, n, k, *rest = size
    c = Case(env, rows, k, n, *rest, dtype, n_scale, seed=size[0] + 1)
    pairs(c, False)
    c.check(backward=False)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("backward", [False, True])
def test_large_calls_without_adapters(env, backward, dtype):
    L, torch = env
    for n_scale in (0, 1, "row"):
        n, k = (520, 4864) if backward else (4864, 520)
        c = Case(env, 300, n, k, 1, 0, [300], [-1], dtype, n_scale, seed=41)
        pairs(c, backward)
        c.check()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("backward", [False, True])
def test_one_requests_infinities_and_nans_stay_in_its_rows_of_large_calls(env, backward, dtype):
    L, torch = env
    rows, rank = 500, 32
    n, k = (144, 4864) if backward else (4864, 144)
    lengths, ids = [100, 60, 140, 40, 150], [0, 1, -1, 2, 1]

    def case():
        c = Case(env, rows, n, k, rank, 3, lengths, ids, dtype, "row", seed=42)
        pairs(c, backward)
        return c

    c = case()
    y0, u0 = c.forward()
    dx0, da0, db0 = c.backward(u0)
    bad = torch.from_numpy(c.row_ids() == 1).cuda()
    # an adapter
    c.a[1, 0, 3], c.b[1, 5, 0], c.b[1, 6, rank - 1], c.alpha[1] = float("inf"), float("nan"), float("-inf"), 2.0
    y, u = c.forward()
    dx, _, _ = c.backward(u0)
    assert torch.equal(y[~bad], y0[~bad]) and torch.equal(u[~bad], u0[~bad])
    assert torch.equal(dx[~bad], dx0[~bad])
    assert torch.equal(y[bad].isnan(), c.exact_forward()[0][bad].isnan()) and bool(y[bad].isnan().any())
    assert torch.equal(dx[bad].isnan(), c.exact_backward(u0)[0][bad].isnan()) and bool(dx[bad].isnan().any())
    # its alpha
    c = case()
    c.alpha[1] = float("nan")
    y, u = c.forward()
    dx, da, db = c.backward(u)
    assert torch.equal(y[~bad], y0[~bad]) and bool(y[bad].isnan().all())
    assert torch.equal(dx[~bad], dx0[~bad]) and bool(dx[bad].isnan().all())
    # rows of x and of dy spoil themselves, and their adapter's gradients
    c = case()
    c.x[100, 0], c.x[255, 1], c.dy[256, 1], c.dy[400, 2] = float("nan"), float("inf"), float("nan"), float("-inf")
    y, u = c.forward()
    dx, da, db = c.backward(u)
    hit = torch.zeros(rows, dtype=torch.bool, device="cuda")
    hit[100] = hit[255] = True
    assert torch.equal(y[~hit], y0[~hit]) and bool(y[100].isnan().all()) and not bool(y[255].isfinite().any())
    hit = torch.zeros(rows, dtype=torch.bool, device="cuda")
    hit[256] = hit[400] = True
    assert torch.equal(dx[~hit], dx0[~hit]) and bool(dx[256].isnan().all()) and not bool(dx[400].isfinite().any())
    for i in (0, 2):
        assert torch.equal(da[i], da0[i]) and torch.equal(db[i], db0[i])
    assert bool(da[1].isnan().any()) and bool(db[1].isnan().any())


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("scale", [0.0, 1e-30, 1e30, -0.5, float("inf")])
def test_rows_of_unusual_scale_in_large_calls(env, scale, dtype):
    L, torch = env
    c = Case(env, 300, 4864, 264, 16, 2, [130, 170], [1, 0], dtype, "row", seed=43)
    pairs(c, False)
    c.scale[5], c.scale[4863] = scale, -scale
    c.make()
    y, _ = c.forward()
    want, _, size, pair = c.exact_forward()
    keep = torch.ones(4864, dtype=torch.bool, device="cuda")
    if scale > 1:
        for i in (5, 4863):
            keep[i] = False
            if dtype == "fp16" or scale == float("inf"):
                assert torch.equal(y[:, i], want[:, i].to(c.dtype))  # infinities
    c.near(y[:, keep], want[:, keep], size[:, keep], 264 + 16, pair[:, keep])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,n,k", [(300, 264, 4864), (60, 264, 512)])
@pytest.mark.parametrize("scale", [0.0, 1e-30, -0.5, float("inf")])
def test_rows_of_unusual_scale_in_input_gradients(env, scale, rows, n, k, dtype):
    L, torch = env
    c = Case(env, rows, n, k, 16, 2, [rows - 20, 20], [1, 0], dtype, "row", seed=44)
    if rows == 300:
        pairs(c, True)
    c.scale[5] = scale
    c.make()
    u = c.forward()[1]
    dx, _, _ = c.backward(u)
    want, _, _, size, pair, _, _ = c.exact_backward(u)
    if scale == float("inf"):
        assert torch.equal(dx.isnan(), want.isnan())
        assert torch.equal(dx.double()[~want.isnan()], want[~want.isnan()]) and not bool(dx.isfinite().any())
    else:
        c.near(dx, want, size, n + 16, pair)


@pytest.mark.parametrize("backward", [False, True])
def test_nan_weights_reach_the_outputs_of_large_calls_that_read_them(env, backward):
    L, torch = env
    n, k = (144, 4864) if backward else (4864, 144)
    for n_scale in (1, "row"):
        c = Case(env, 300, n, k, 8, 1, [300], [0], "bf16", n_scale, seed=45)
        pairs(c, backward)
        c.w[3, 7], c.w[n - 1, k - 1] = 0x7F, 0xFF
        y, u = c.forward()
        dx, _, _ = c.backward(u)
        for got, size, at in ((y, n, (3, n - 1)), (dx, k, (7, k - 1))):
            nan = torch.zeros(size, dtype=torch.bool, device="cuda")
            nan[list(at)] = True
            assert torch.equal(got.isnan(), nan.expand(300, size))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("backward", [False, True])
def test_large_calls_repeated_captured_and_on_another_stream(env, backward, dtype):
    L, torch = env
    n, k = (272, 4864) if backward else (4864, 272)
    c = Case(env, 400, n, k, 40, 3, [130, 0, 200, 1], [1, 2, 0, 1], dtype, "row", seed=46)
    pairs(c, backward)
    y, u = c.forward()
    grads = c.backward(u)
    first = [t.clone() for t in (y, u, *grads)]

    def same(now):
        assert all(torch.equal(a, b) for a, b in zip(now, first))

    for _ in range(5):
        c.ws.random_(0, 256)
        y2, u2 = c.forward()
        same([y2, u2, *c.backward(u2)])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        y2, u2 = c.forward()
        grads2 = c.backward(u2)
    side.synchronize()
    same([y2, u2, *grads2])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.linear.forward(c.x, y, requests=c.requests, u=u, workspace=c.ws, status=c.status)
        c.linear.backward(c.x, c.dy, u, dx=grads[0], da=grads[1], db=grads[2], requests=c.requests, workspace=c.ws,
                          status=c.status)
    for t in (y, u, *grads):
        t.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    same([y, u, *grads])
    assert int(c.status.item()) == 0


@pytest.mark.parametrize("backward", [False, True])
def test_bad_request_tables_in_large_calls(env, backward):
    L, torch = env
    n, k = (272, 4864) if backward else (4864, 272)
    rows = 300
    c = Case(env, rows, n, k, 16, 2, [rows], [1], "bf16", 1, seed=47)
    pairs(c, backward)
    for offsets, ids in (([0, rows + 1], [0]), ([0, 10, 5, rows], [0, 1, 1]), ([-3, 5], [1]), ([0, 5], [2]),
                         ([0, 2 ** 31 - 1], [0]), ([5, -2 ** 31], [0])):
        c.requests = L.Requests(torch.tensor(offsets, dtype=torch.int32, device="cuda"),
                                torch.tensor(ids, dtype=torch.int32, device="cuda"))
        c.status.zero_()
        y, u = c.forward()
        assert int(c.status.item()) == L.STATUS_BAD_REQUEST
        c.status.zero_()
        c.backward(u)
        assert int(c.status.item()) == L.STATUS_BAD_REQUEST


def test_large_calls_write_nothing_past_their_outputs(env):
    L, torch = env
    for rows, n, k, rank in ((261, 4880, 4936, 24), (300, 4871, 4867, 7)):
        c = Case(env, rows, n, k, rank, 2, [rows - 1], [1], "bf16", "row", seed=48)
        pairs(c, False)
        pairs(c, True)
        flats = [torch.full((rows * m + 4096,), 5.0, dtype=c.dtype, device="cuda") for m in (n, k)]
        y, dx = (f[2048:2048 + rows * m].view(rows, m) for f, m in zip(flats, (n, k)))
        u = torch.zeros(rows, rank, device="cuda")
        c.linear.forward(c.x, y, requests=c.requests, u=u, workspace=c.ws)
        c.linear.backward(None, c.dy, None, dx=dx, requests=c.requests, workspace=c.ws)
        torch.cuda.synchronize()
        for f in flats:
            assert bool((f[:2048] == 5).all()) and bool((f[-2048:] == 5).all())
        want, _, size, pair = c.exact_forward()
        c.near(y, want, size, k + rank, pair)


# ---- calls at the edges of what the entry points take ----

def test_no_rows_no_requests_no_table(env):
    """No rows: adapters' gradients are zeros.  No table: no row has an adapter."""
    L, torch = env
    c = Case(env, 40, 256, 512, 16, 2, [40], [1], "bf16", "row", seed=51)
    da, db = torch.full_like(c.a, 7.0), torch.full_like(c.b, 7.0)
    u0 = torch.empty(0, 16, device="cuda")
    c.linear.forward(c.x[:0], torch.empty(0, 256, dtype=c.dtype, device="cuda"), requests=c.requests, u=u0,
                     workspace=c.ws, status=c.status)
    c.linear.backward(c.x[:0], c.dy[:0], u0, dx=torch.empty_like(c.x[:0]), da=da, db=db, requests=c.requests,
                      workspace=c.ws, status=c.status)
    assert not bool(da.any()) and not bool(db.any())
    plain = L.Linear(c.w, scale=c.scale, dtype=c.dtype)
    y, want = torch.empty_like(c.dy), torch.empty_like(c.dy)
    dx, wdx = torch.empty_like(c.x), torch.empty_like(c.x)
    u = torch.full((40, 16), 9.0, device="cuda")
    c.linear.forward(c.x, y, u=u, workspace=c.ws, status=c.status)
    plain.forward(c.x, want)
    assert torch.equal(y, want) and not bool(u.any())
    da.fill_(7.0), db.fill_(7.0)
    c.linear.backward(c.x, c.dy, u, dx=dx, da=da, db=db, workspace=c.ws, status=c.status)
    plain.backward(None, c.dy, None, dx=wdx)
    assert torch.equal(dx, wdx) and not bool(da.any()) and not bool(db.any())
    assert int(c.status.item()) == 0


@pytest.mark.parametrize("rows,n,k", [(700, 96, 160), (700, 4864, 96), (700, 96, 4864)])
@pytest.mark.parametrize("adapters,rank", [(700, 3), (300, 16), (65535, 1)])
def test_many_adapters(env, rows, n, k, adapters, rank):
    """A row each of its own adapter, the last one's among them."""
    L, torch = env
    ids = [(adapters - 1 - 7 * i) % adapters for i in range(rows)]
    c = Case(env, rows, n, k, rank, adapters, [1] * rows, ids, "fp16", 1, seed=52)
    y, u = c.forward()
    dx, da, db = c.backward(u)
    # by rows: the reference's loop over requests would take seconds
    w, s = c.wide()
    x, dy, at = c.x.double(), c.dy.double(), torch.tensor(ids, device="cuda")
    a, b, al = c.a.double()[at], c.b.double()[at], c.alpha.double()[at, None]
    wu = torch.einsum("tk,trk->tr", x, a)
    want = (x @ w.T) * s + al * torch.einsum("tr,tnr->tn", wu, b)
    pair = al * torch.einsum("tr,tnr->tn", torch.einsum("tk,trk->tr", x.abs(), a.abs()), b.abs())
    c.near(y, want, (x.abs() @ w.abs().T) * s + pair, k + rank, pair)
    v = al * torch.einsum("tn,tnr->tr", dy, b)
    pair = al * torch.einsum("tr,trk->tk", torch.einsum("tn,tnr->tr", dy.abs(), b.abs()), a.abs())
    c.near(dx, (dy * s) @ w + torch.einsum("tr,trk->tk", v, a), (dy.abs() * s) @ w.abs() + pair, n + rank, pair)
    wda, wdb = torch.zeros_like(c.a, dtype=torch.float64), torch.zeros_like(c.b, dtype=torch.float64)
    wda.index_add_(0, at, torch.einsum("tr,tk->trk", v, x))
    wdb.index_add_(0, at, al[:, :, None] * torch.einsum("tn,tr->tnr", dy, u.double()))
    sa, sb = torch.zeros_like(wda), torch.zeros_like(wdb)
    va = al * torch.einsum("tn,tnr->tr", dy.abs(), b.abs())
    sa.index_add_(0, at, torch.einsum("tr,tk->trk", va, x.abs()))
    sb.index_add_(0, at, al[:, :, None] * torch.einsum("tn,tr->tnr", dy.abs(), u.double().abs()))
    c.near(da, wda, sa, rows + n, sa)
    c.near(db, wdb, sb, rows, sb)
    assert int(c.status.item()) == 0
