"""Linear layers over decoded weights on the GPU, forward and backward, against
the formula in 64 bits.

Tolerances.  An output is one rounding to its type of a float32 sum, so the
2-norm of its error is at most eps/2 times its own, eps = finfo(type).eps,
and where the input type rounds once more (s * W with one scale per row, in
the input gradient; hi/lo pairs of 16-bit parts, 2^-16, in the adapters' part)
at most another eps/2 of the terms' norm: 1.05 * eps/2 and 2.1 * eps/2 with
the float32 sums' share.  Element by element a sum of m terms in float32, in
any order, is off by at most (m + 64) * 2^-23 of the terms' absolute sum (2^-23:
an add that truncates), and the pairs by 2^-15 of theirs."""
import math

import numpy as np
import pytest

import ecf8_synth as synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env(gpu_available):
    import torch
    import lossless_fp8_weight_b200 as L
    return L, torch


class Case:
    """One projection with its adapters, requests and gradients, and the same in 64 bits."""

    def __init__(self, env, rows, n, k, rank, adapters, lengths, ids, dtype, n_scale=1, seed=0, w=None, alpha=None):
        L, torch = env
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.env, self.rows, self.n, self.k, self.rank = env, rows, n, k, rank
        self.dtype = torch.bfloat16 if dtype == "bf16" else torch.float16
        self.n_scale = {0: 0, 1: 1, "row": n}[n_scale]

        def normal(*shape):
            return torch.randn(*shape, generator=g, device="cuda")

        if w is None:
            w = (normal(n, k) * 16).to(torch.float8_e4m3fn).view(torch.uint8)
        self.w = w
        self.scale = None if not self.n_scale else (0.25 + torch.rand(self.n_scale, generator=g, device="cuda")) / (
            16 * math.sqrt(k))
        self.x = normal(rows, k).to(self.dtype)
        self.dy = normal(rows, n).to(self.dtype)
        self.a = (normal(adapters, rank, k) / math.sqrt(k)).to(self.dtype)
        self.b = normal(adapters, n, rank).to(self.dtype)
        self.alpha = alpha if alpha is not None else 0.5 + torch.rand(adapters, generator=g, device="cuda")
        self.offsets = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
        self.ids = np.asarray(ids, np.int32)
        self.requests = L.Requests(torch.from_numpy(self.offsets).cuda(), torch.from_numpy(self.ids).cuda())
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.make()

    def make(self):
        L, torch = self.env
        ad = L.Adapters(self.a, self.b, self.alpha) if self.a.shape[0] else None
        self.linear = L.Linear(self.w, scale=self.scale, adapters=ad, dtype=self.dtype)
        self.ws = torch.zeros(max(16, self.linear.workspace_size(self.rows)), dtype=torch.uint8, device="cuda")

    def row_ids(self):
        out = np.full(self.rows, -1)
        for i, a in enumerate(self.ids):
            out[max(0, self.offsets[i]):max(0, self.offsets[i + 1])] = max(-1, a)
        return out

    def forward(self, x=None, keep_u=True, **kw):
        L, torch = self.env
        x = self.x if x is None else x
        y = torch.full((self.rows, self.n), 7.0, dtype=self.dtype, device="cuda")
        u = torch.full((self.rows, self.rank), 9.0, device="cuda") if keep_u and self.a.shape[0] else None
        self.linear.forward(x, y, requests=self.requests, u=u, workspace=self.ws, status=self.status, **kw)
        return y, u

    def backward(self, u, **kw):
        L, torch = self.env
        dx = torch.full((self.rows, self.k), 7.0, dtype=self.dtype, device="cuda")
        da, db = torch.full_like(self.a, 7.0), torch.full_like(self.b, 7.0)
        if not self.a.shape[0]:
            self.linear.backward(None, self.dy, None, dx=dx, requests=self.requests, workspace=self.ws,
                                 status=self.status, **kw)
        else:
            self.linear.backward(self.x, self.dy, u, dx=dx, da=da, db=db, requests=self.requests, workspace=self.ws,
                                 status=self.status, **kw)
        return dx, da, db

    # the formula in 64 bits, and the sums of absolute terms

    def wide(self):
        torch = self.env[1]
        w = self.w.view(torch.float8_e4m3fn).double()
        s = torch.ones(1, device="cuda").double() if self.scale is None else self.scale.double()
        return w, s

    def exact_forward(self):
        w, s = self.wide()
        x, a, b = self.x.double(), self.a.double(), self.b.double()
        y, size = (x @ w.T) * s, (x.abs() @ w.abs().T) * s.abs()
        pairs = size * 0
        u = x.new_zeros(self.rows, self.rank)
        for i, ad in enumerate(self.ids):
            lo, hi = int(self.offsets[i]), int(self.offsets[i + 1])
            if ad < 0 or hi <= lo:
                continue
            u[lo:hi] = x[lo:hi] @ a[ad].T
            al = self.alpha[ad].double()
            y[lo:hi] += al * (u[lo:hi] @ b[ad].T)
            part = al.abs() * ((x[lo:hi].abs() @ a[ad].abs().T) @ b[ad].abs().T)
            pairs[lo:hi] += part
        return y, u, size + pairs, pairs

    def exact_backward(self, u):
        w, s = self.wide()
        x, dy, a, b, u = self.x.double(), self.dy.double(), self.a.double(), self.b.double(), u.double()
        dx, size = (dy * s) @ w, (dy * s).abs() @ w.abs()
        pairs = size * 0
        da, db = a * 0, b * 0
        sa, sb = a * 0, b * 0
        for i, ad in enumerate(self.ids):
            lo, hi = int(self.offsets[i]), int(self.offsets[i + 1])
            if ad < 0 or hi <= lo:
                continue
            al = self.alpha[ad].double()
            v, va = al * (dy[lo:hi] @ b[ad]), al.abs() * (dy[lo:hi].abs() @ b[ad].abs())
            dx[lo:hi] += v @ a[ad]
            pairs[lo:hi] += va @ a[ad].abs()
            da[ad] += v.T @ x[lo:hi]
            sa[ad] += va.T @ x[lo:hi].abs()
            db[ad] += al * (dy[lo:hi].T @ u[lo:hi])
            sb[ad] += al.abs() * (dy[lo:hi].T.abs() @ u[lo:hi].abs())
        return dx, da, db, size + pairs, pairs, sa, sb

    def near(self, got, want, size, terms, pairs=None, twice=False):
        torch = self.env[1]
        half = torch.finfo(self.dtype).eps / 2
        tiny = torch.finfo(self.dtype).smallest_normal
        err = (got.double() - want).abs()
        most = half * want.abs() + (terms + 64) * 2.0 ** -23 * size + tiny
        if pairs is not None:
            most = most + 2.0 ** -15 * pairs
        if twice:
            most = most + half * size
        assert bool((err <= most).all()), float((err - most).max())
        if want.numel() >= 64 and float(want.norm()) > 0:
            assert float(err.norm()) <= (2.1 if twice else 1.05) * half * float(want.norm()) + tiny * want.numel() ** 0.5

    def check(self, backward=True):
        y, u = self.forward()
        want, wu, size, pairs = self.exact_forward()
        self.near(y, want, size, self.k + self.rank, pairs)
        if u is not None:
            bound = (self.k + 64) * 2.0 ** -23 * (self.x.double().abs() @ self.a.double().abs().amax(dim=0).T) + 1e-30
            assert bool(((u.double() - wu).abs() <= bound).all())
        if backward:
            u = u if u is not None else wu.float()
            dx, da, db = self.backward(u)
            wdx, wda, wdb, size, pairs, sa, sb = self.exact_backward(u)
            self.near(dx, wdx, size, self.n + self.rank, pairs, twice=self.n_scale > 1)
            if self.a.shape[0]:
                self.near(da, wda, sa, self.rows + self.n, sa)
                self.near(db, wdb, sb, self.rows, sb)
        assert int(self.status.item()) == 0


SIZES = [
    # rows, n, k, rank, adapters, lengths, ids
    (1, 1024, 4096, 16, 1, [1], [0]),
    (1, 16, 16, 1, 1, [1], [0]),
    (2, 128, 64, 8, 3, [1, 1], [2, 2]),
    (17, 256, 512, 16, 5, [1] * 15, [0, 1, 2, 3, 4, -1, 4, 4, 0, 1, -1, 2, 3, 0, 0]),
    (64, 512, 1024, 64, 3, [1] * 64, [i % 4 - 1 for i in range(64)]),
    (100, 1024, 512, 16, 90, [1] * 100, [(7 * i) % 90 for i in range(100)]),
    (129, 144, 272, 32, 4, [0, 40, 1, 0, 60, 28], [0, 3, 1, 2, -1, 3]),
    (257, 1040, 528, 128, 2, [100, 157], [1, 0]),
    (300, 640, 2064, 24, 3, [130, 3, 90], [2, 0, 2]),
    (1000, 384, 256, 4, 2, [999], [1]),
    (1537, 768, 640, 48, 6, [600, 500, 0, 437], [5, 0, 1, 5]),
    (333, 1001, 1999, 12, 5, [100, 50, 0, 150, 33], [4, 0, 1, -1, 4]),
    (5, 7, 3, 3, 2, [2, 1], [1, 0]),
    (1, 1, 1, 1, 1, [1], [0]),
    (70, 129, 130, 127, 1, [70], [0]),
    (400, 520, 264, 20, 3, [150, 0, 250], [1, 0, 2]),
    # more tiles than pairs of SMs
    (1777, 4096, 1056, 24, 3, [700, 900, 100], [1, 2, 0]),
    (1280, 4608, 1024, 8, 2, [1270], [1]),
    (1250, 4096, 1552, 40, 2, [620, 1, 600], [0, 1, 1]),
    (150, 1000, 1001, 33, 4, [31, 64, 1, 54], [3, 0, 1, 3]),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("n_scale", [1, "row"])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s[:4])))
def test_forward_and_backward_equal_the_formula(env, size, n_scale, dtype):
    Case(env, *size, dtype, n_scale, seed=size[0] + size[1]).check()


@pytest.mark.parametrize("rows,n,k", [(1, 256, 512), (33, 272, 528), (200, 1024, 256), (515, 400, 1040), (9, 33, 17),
                                      (40, 264, 520), (300, 130, 1000)])
def test_without_adapters(env, rows, n, k):
    for n_scale in (0, 1, "row"):
        c = Case(env, rows, n, k, 1, 0, [rows], [-1], "bf16", n_scale, seed=rows)
        c.check()
        # without a workspace nothing is copied: odd sizes take the plain kernels
        y, _ = c.forward()
        dx, _, _ = c.backward(None)
        c.ws = None
        want, _, size, pairs = c.exact_forward()
        c.near(c.forward()[0], want, size, k, pairs)
        wdx, _, _, size, pairs, _, _ = c.exact_backward(torch_zeros(c))
        c.near(c.backward(None)[0], wdx, size, n, pairs, twice=c.n_scale > 1)


def torch_zeros(c):
    return c.env[1].zeros(c.rows, 1, device="cuda")


@pytest.mark.parametrize("rows", [40, 600])
def test_all_rows_without_an_adapter_equal_the_plain_projection(env, rows):
    """Ids of -1, requests of no rows and no requests at all: the same bits as a projection without adapters."""
    L, torch = env
    c = Case(env, rows, 272, 528, 16, 2, [rows // 2, rows - rows // 2], [-1, -1], "bf16", "row", seed=1)
    y, u = c.forward()
    plain = Case(env, rows, 272, 528, 16, 0, [rows], [-1], "bf16", "row", seed=1)
    plain.w, plain.x, plain.scale = c.w, c.x, c.scale
    plain.make()
    want, _ = plain.forward()
    assert torch.equal(y, want) and float(u.abs().max()) == 0
    dx, da, db = c.backward(u)
    assert float(da.abs().max()) == 0 and float(db.abs().max()) == 0
    for offsets, ids in (([0], []), ([0, 0, 0], [0, 1]), ([rows, rows], [1])):
        c.requests = L.Requests(torch.tensor(offsets, dtype=torch.int32, device="cuda"),
                                torch.tensor(ids, dtype=torch.int32, device="cuda"))
        y, u = c.forward()
        assert torch.equal(y, want) and float(u.abs().max()) == 0
        _, da, db = c.backward(u)
        assert float(da.abs().max()) == 0 and float(db.abs().max()) == 0
    assert int(c.status.item()) == 0


@pytest.mark.parametrize("rows,n,k,rank", [(60, 256, 512, 16), (300, 256, 528, 32), (50, 101, 99, 5)])
def test_one_requests_infinities_and_nans_stay_in_its_rows(env, rows, n, k, rank):
    L, torch = env
    per = rows // 5
    lengths, ids = [per, per, per, per, rows - 4 * per], [0, 1, -1, 2, 1]
    c = Case(env, rows, n, k, rank, 3, lengths, ids, "bf16", "row", seed=3)
    c.forward()
    y0, u0 = c.forward()
    _, da0, db0 = c.backward(u0)
    bad = torch.from_numpy(c.row_ids() == 1).cuda()
    c.a[1, 0, 3], c.b[1, 5, 0], c.b[1, 6, rank - 1] = float("inf"), float("nan"), float("-inf")
    y, u = c.forward()
    assert torch.equal(y[~bad], y0[~bad]) and torch.equal(u[~bad], u0[~bad])
    want, _, _, _ = c.exact_forward()
    assert torch.equal(y[bad].isnan(), want[bad].isnan())
    assert bool(y[bad].isnan().any())
    # a row of x that is not finite spoils itself only
    c = Case(env, rows, n, k, rank, 3, lengths, ids, "bf16", "row", seed=3)
    c.x[per, 0], c.x[2 * per, 1] = float("nan"), float("inf")
    y, u = c.forward()
    hit = torch.zeros(rows, dtype=torch.bool, device="cuda")
    hit[per] = hit[2 * per] = True
    assert torch.equal(y[~hit], y0[~hit]) and bool(y[per].isnan().all()) and not bool(y[2 * per].isfinite().any())
    # and its adapter's gradients only
    _, da, db = c.backward(u)
    for i in (0, 2):
        assert torch.equal(da[i], da0[i]) and torch.equal(db[i], db0[i])
    assert bool(da[1].isnan().any()) and bool(db[1].isnan().any())


@pytest.mark.parametrize("rows,n,k", [(20, 256, 512), (400, 144, 256), (20, 37, 50)])
def test_nan_weights_reach_the_outputs_that_read_them(env, rows, n, k):
    L, torch = env
    c = Case(env, rows, n, k, 8, 1, [rows], [0], "bf16", 1, seed=4)
    c.w[3, 7], c.w[n - 1, k - 1] = 0x7F, 0xFF
    c.make()
    y, u = c.forward()
    nan = torch.zeros(n, dtype=torch.bool, device="cuda")
    nan[3] = nan[n - 1] = True
    assert torch.equal(y.isnan(), nan.expand(rows, n))
    dx, _, _ = c.backward(u)
    nan = torch.zeros(k, dtype=torch.bool, device="cuda")
    nan[7] = nan[k - 1] = True
    assert torch.equal(dx.isnan(), nan.expand(rows, k))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_every_weight_byte_is_read_exactly(env, dtype):
    """One-hot rows of x pick single weights: y is the E4M3 value itself."""
    L, torch = env
    w = torch.arange(256, dtype=torch.int32, device="cuda").to(torch.uint8).repeat(16, 1)
    c = Case(env, 256, 16, 256, 1, 0, [256], [-1], dtype, 0, w=w.contiguous())
    c.x = torch.eye(256, device="cuda").to(c.dtype)
    c.w[:, 0x7F] = c.w[:, 0xFF] = 0
    y, _ = c.forward()
    assert torch.equal(y.float(), c.w.view(torch.float8_e4m3fn).float().T)
    c.dy = torch.eye(256, 16, device="cuda").to(c.dtype)
    dx, _, _ = c.backward(None)
    assert torch.equal(dx[:16].float(), c.w.view(torch.float8_e4m3fn).float())


@pytest.mark.parametrize("scale", [0.0, 1e-30, 1e30, -0.5, float("inf")])
def test_rows_of_unusual_scale(env, scale):
    """A scale of zero leaves the adapter's part; very small and large ones do not lose it."""
    L, torch = env
    c = Case(env, 70, 256, 512, 16, 2, [30, 40], [1, 0], "bf16", "row", seed=6)
    c.scale[5] = scale
    c.make()
    if math.isinf(scale):
        y, _ = c.forward()
        assert not bool(y[:, 5].isfinite().any())
        keep = [i for i in range(256) if i != 5]
        want, _, size, pairs = c.exact_forward()
        c.near(y[:, keep], want[:, keep], size[:, keep], 528, pairs[:, keep])
    else:
        y, _ = c.forward()
        want, _, size, pairs = c.exact_forward()
        c.near(y, want, size, 528, pairs)


@pytest.mark.parametrize("rows,n,k", [(3, 256, 512), (150, 272, 256), (40, 50, 70)])
def test_strided_rows_and_views(env, rows, n, k):
    L, torch = env
    c = Case(env, rows, n, k, 16, 2, [rows], [1], "bf16", "row", seed=7)
    y0, u0 = c.forward()
    dx0, _, _ = c.backward(u0)
    for pad, shift in ((16, 8), (5, 3), (64, 0)):
        wide_w = torch.full((n, k + pad * 16), 0x33, dtype=torch.uint8, device="cuda")
        wide_w[:, shift * 2:shift * 2 + k] = c.w
        wide_x = torch.full((rows, k + pad), 3.0, dtype=c.dtype, device="cuda")
        wide_x[:, shift:shift + k] = c.x
        wide_y = torch.full((rows, n + pad), 5.0, dtype=c.dtype, device="cuda")
        lin = L.Linear(wide_w[:, shift * 2:shift * 2 + k], scale=c.scale, adapters=L.Adapters(c.a, c.b, c.alpha))
        ws = torch.zeros(lin.workspace_size(rows), dtype=torch.uint8, device="cuda")
        y = wide_y[:, shift:shift + n]
        lin.forward(wide_x[:, shift:shift + k], y, requests=c.requests, workspace=ws, status=c.status)
        want, _, size, pairs = c.exact_forward()
        c.near(y, want, size, k + 16, pairs)
        assert bool((wide_y[:, :shift] == 5).all()) and bool((wide_y[:, shift + n:] == 5).all())
        wide_dx = torch.full((rows, k + pad), 5.0, dtype=c.dtype, device="cuda")
        dx = wide_dx[:, shift:shift + k]
        wide_dy = torch.full((rows, n + pad), 3.0, dtype=c.dtype, device="cuda")
        wide_dy[:, shift:shift + n] = c.dy
        lin.backward(wide_x[:, shift:shift + k], wide_dy[:, shift:shift + n], u0, dx=dx, requests=c.requests,
                     workspace=ws)
        wdx, _, _, size, pairs, _, _ = c.exact_backward(u0)
        c.near(dx, wdx, size, n + 16, pairs, twice=True)
        assert bool((wide_dx[:, :shift] == 5).all()) and bool((wide_dx[:, shift + k:] == 5).all())
    assert int(c.status.item()) == 0


def test_outputs_end_where_they_end(env):
    """Nothing is written past y, dx, da, db and u."""
    L, torch = env
    for rows, n, k, rank in ((5, 144, 272, 24), (261, 144, 272, 24), (5, 7, 9, 3)):
        c = Case(env, rows, n, k, rank, 2, [rows - 1], [1], "bf16", 1, seed=8)

        def guarded(*shape, dtype=c.dtype):
            size = math.prod(shape)
            flat = torch.full((size + 4096,), 5.0, dtype=dtype, device="cuda")
            return flat, flat[2048:2048 + size].view(*shape)

        bufs = [guarded(rows, n), guarded(rows, rank, dtype=torch.float32), guarded(rows, k), guarded(2, rank, k),
                guarded(2, n, rank)]
        c.linear.forward(c.x, bufs[0][1], requests=c.requests, u=bufs[1][1], workspace=c.ws)
        c.linear.backward(c.x, c.dy, bufs[1][1], dx=bufs[2][1], da=bufs[3][1], db=bufs[4][1], requests=c.requests,
                          workspace=c.ws)
        torch.cuda.synchronize()
        for flat, view in bufs:
            assert bool((flat[:2048] == 5).all()) and bool((flat[2048 + view.numel():] == 5).all())


@pytest.mark.parametrize("rows", [24, 300])
def test_bad_request_tables_set_the_status_and_touch_nothing_else(env, rows):
    L, torch = env
    c = Case(env, rows, 256, 512, 16, 2, [rows], [1], "bf16", 1, seed=9)
    for offsets, ids in (([0, rows + 1], [0]), ([0, 10, 5, rows], [0, 1, 0]), ([-3, 5], [1]), ([0, 5], [2]),
                         ([0, 2 ** 31 - 1], [0]), ([5, -2 ** 31], [0]), ([0, 5], [2 ** 31 - 1])):
        c.requests = L.Requests(torch.tensor(offsets, dtype=torch.int32, device="cuda"),
                                torch.tensor(ids, dtype=torch.int32, device="cuda"))
        c.status.zero_()
        y, u = c.forward()
        assert int(c.status.item()) == L.STATUS_BAD_REQUEST
        c.status.zero_()
        c.backward(u)
        assert int(c.status.item()) == L.STATUS_BAD_REQUEST
    c.status.zero_()


@pytest.mark.parametrize("outputs", [("dx",), ("da",), ("db",), ("da", "db"), ("dx", "db")])
def test_gradients_may_be_left_out(env, outputs):
    L, torch = env
    for rows, n, k in ((90, 256, 512), (30, 33, 21)):
        c = Case(env, rows, n, k, 16, 2, [rows], [1], "bf16", 1, seed=10)
        _, u = c.forward()
        full = dict(zip(("dx", "da", "db"), c.backward(u)))
        some = {q: torch.full_like(full[q], 3.0) for q in outputs}
        c.linear.backward(c.x if "da" in outputs else None, c.dy, u if "db" in outputs else None,
                          requests=c.requests, workspace=c.ws, **some)
        for q in outputs:
            assert torch.equal(some[q], full[q]), q


def test_the_workspace_keeps_u_where_none_is_given(env):
    L, torch = env
    c = Case(env, 50, 256, 512, 16, 2, [20, 30], [1, 0], "fp16", 1, seed=11)
    y, _ = c.forward()
    c.ws.random_(0, 256)
    assert torch.equal(c.forward(keep_u=False)[0], y)


@pytest.mark.parametrize("rows,n,k", [(9, 2048, 2048), (700, 512, 512)])
def test_repeated_calls_give_the_same_bits(env, rows, n, k):
    L, torch = env
    c = Case(env, rows, n, k, 16, 3, [rows // 3, rows // 3, 1], [1, 0, 1], "bf16", "row", seed=12)
    y, u = c.forward()
    g = c.backward(u)
    for _ in range(5):
        c.ws.random_(0, 256)
        y2, u2 = c.forward()
        assert torch.equal(y, y2) and torch.equal(u, u2)
        assert all(torch.equal(p, q) for p, q in zip(g, c.backward(u)))


def test_a_captured_call_follows_its_inputs(env):
    """Forward and backward in one graph: replays follow new activations, request
    tables and adapter values."""
    L, torch = env
    c = Case(env, 40, 256, 512, 16, 3, [1] * 40, [i % 4 - 1 for i in range(40)], "bf16", 1, seed=13)
    y, u = c.forward()
    dx, da, db = c.backward(u)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.linear.forward(c.x, y, requests=c.requests, u=u, workspace=c.ws, status=c.status)
        c.linear.backward(c.x, c.dy, u, dx=dx, da=da, db=db, requests=c.requests, workspace=c.ws, status=c.status)
    other = Case(env, 40, 256, 512, 16, 3, [30] + [0] * 38 + [5], [2] + [-1] * 38 + [0], "bf16", 1, seed=14)
    for q in ("x", "dy", "a", "b", "alpha"):
        getattr(c, q).copy_(getattr(other, q))
    c.w.copy_(other.w)
    c.scale.copy_(other.scale)
    c.requests.offsets.copy_(other.requests.offsets)
    c.requests.ids.copy_(other.requests.ids)
    graph.replay()
    torch.cuda.synchronize()
    y1, u1 = other.forward()
    assert torch.equal(y, y1) and torch.equal(u, u1)
    for got, want in zip((dx, da, db), other.backward(u1)):
        assert torch.equal(got, want)
    assert int(c.status.item()) == 0


def test_calls_on_other_streams(env):
    L, torch = env
    cases = [Case(env, 30 + i, 512, 1024, 16, 2, [30 + i], [i % 2], "bf16", 1, seed=20 + i) for i in range(4)]
    want = [c.forward()[0] for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = []
    for c, s in zip(cases, streams):
        with torch.cuda.stream(s):
            got.append(c.forward()[0])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_gradients_equal_differences(env):
    """y is linear in x, in A and in B: a central difference of any step is the
    derivative, up to the rounding of the two outputs."""
    L, torch = env
    c = Case(env, 96, 256, 128, 16, 2, [50, 30], [1, 0], "bf16", "row", seed=15)
    _, u = c.forward()
    grads = dict(zip(("x", "a", "b"), c.backward(u)))
    g = torch.Generator(device="cuda").manual_seed(5)
    half = torch.finfo(c.dtype).eps / 2
    for name in ("x", "a", "b"):
        base = getattr(c, name).clone()
        step = (torch.randint(0, 2, base.shape, generator=g, device="cuda") * 2 - 1).to(c.dtype) * 2 ** -2
        ends = []
        for sign in (1, -1):
            t = getattr(c, name)
            t.copy_((base.double() + sign * step.double()).to(c.dtype))
            ends.append((t.double().clone(), c.forward()[0].double()))
            t.copy_(base)
        moved = ends[0][0] - ends[1][0]
        change = float((c.dy.double() * (ends[0][1] - ends[1][1])).sum())
        want = float((grads[name].double() * moved).sum())
        # roundings of both outputs and of the gradient, each at most eps/2 of its value, add up at random: six
        # standard deviations of the sum, with one more for s * W rounded in dx
        noise = half * (float((c.dy.double() * ends[0][1]).norm()) + float((c.dy.double() * ends[1][1]).norm())
                        + 3 * float((grads[name].double() * moved).norm()))
        assert abs(change - want) <= 6 * noise, (name, change, want, noise)


def test_offsets_past_32_bits(env):
    """Rows that lie more than 2^31 elements from the first (a long activation buffer), read and written in place."""
    L, torch = env
    k, n = 512, 256
    stride = 3 * 2 ** 28 + 16
    c = Case(env, 4, n, k, 16, 2, [2, 2], [1, 0], "bf16", 1, seed=16)
    big = torch.empty(3 * stride + 4096, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(big, (4, k), (stride, 1))
    x.copy_(c.x)
    assert torch.equal(c.forward(x=x)[0], c.forward()[0])
    y = torch.as_strided(big, (4, n), (stride, 1), 1024)
    big2 = torch.as_strided(big, (4, n), (stride, 1), 2048)
    big2.fill_(3.0)
    c.linear.forward(c.x, y, requests=c.requests, workspace=c.ws)
    assert torch.equal(y, c.forward()[0]) and bool((big2 == 3).all())


def test_a_layer_from_blobs_through_the_pipeline(env):
    """The operators as they are used together: blobs decoded on use, the layer's
    projections with adapters forward and backward, and the adapters' gradients
    clipped; equal, bit for bit, to the same over the source weights."""
    L, torch = env
    n, k, rank, rows, layers = 256, 512, 16, 70, 3
    spec = synth.alpha_sweep_point(1.7, 448.0).tensors[0]
    src = [[spec.generate(begin=1000 * l + 7 * i, count=n * k) for i in range(2)] for l in range(layers)]
    blobs = [[L.encode(x) for x in xs] for xs in src]
    table = [[L.PipelineTensor(L.blob_info(b), torch.from_numpy(b).cuda(), i * n * k) for i, b in enumerate(bs)]
             for bs in blobs]
    slots = [torch.empty(2 * n * k, dtype=torch.uint8, device="cuda") for _ in range(2)]
    compute, decode = torch.cuda.Stream(), torch.cuda.Stream()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    P = L.Pipeline(table, slots, 2 * n * k, depth=1, status=status, decode_stream=decode)
    c = Case(env, rows, n, k, rank, 2, [30, 30], [1, 0], "bf16", 1, seed=17)
    adapters = L.Adapters(c.a, c.b, c.alpha)

    def one_layer(weights):
        """[y, dx, da, db] of the layer's two projections; `weights`: tensors, or addresses."""
        out = []
        for w in weights:
            lin = L.Linear(w, shape=(n, k), scale=c.scale, adapters=adapters)
            y = torch.empty(rows, n, dtype=c.dtype, device="cuda")
            u = torch.empty(rows, rank, device="cuda")
            dx, da, db = torch.empty_like(c.x), torch.empty_like(c.a), torch.empty_like(c.b)
            lin.forward(c.x, y, requests=c.requests, u=u, workspace=c.ws, status=c.status)
            lin.backward(c.x, c.dy, u, dx=dx, da=da, db=db, requests=c.requests, workspace=c.ws, status=c.status)
            out += [y, dx, da, db]
        return out

    def clipped(results):
        grads = [t for r in results for t in (r[2], r[3], r[6], r[7])]
        norm = torch.zeros(1, device="cuda")
        L.GradSet(grads).clip(0.5, norm, status=c.status)
        return norm, grads

    torch.cuda.synchronize()
    with torch.cuda.stream(compute):
        got = []
        for l in range(layers):
            at = P.acquire(l, compute)
            got.append(one_layer([at, at + n * k]))
            P.release(l, compute)
        norm, grads = clipped(got)
    torch.cuda.synchronize()
    want = [one_layer([torch.from_numpy(x).cuda().view(n, k) for x in xs]) for xs in src]
    total = math.sqrt(sum(float(t.double().square().sum()) for r in want for t in (r[2], r[3], r[6], r[7])))
    norm1, grads1 = clipped(want)
    P.close()
    assert int(status.item()) == 0 and int(c.status.item()) == 0
    assert torch.equal(norm, norm1) and abs(float(norm) - total) <= 2.0 ** -23 * total and total > 0.5
    for r, q in zip(got, want):
        assert all(torch.equal(a, b) for a, b in zip(r, q))
    assert all(torch.equal(a, b) for a, b in zip(grads, grads1))
