"""Argument errors of the linear and gradient-set entry points, on CPU: every
one is decided before the library touches the device, so these calls never
reach CUDA.  Device pointers are fake aligned addresses that are never
dereferenced."""
import ctypes

import numpy as np
import pytest

FAKE = 1 << 20
ARG, ALIGN, WORKSPACE = -1, -5, -8


@pytest.fixture(scope="module")
def L():
    import lossless_fp8_weight_b200 as lib
    return lib


def _desc(L, n=64, k=96, adapters=2, rank=8, dtype=0, **over):
    d = L.LinearDesc(FAKE, n, k, k, FAKE, 1, FAKE, FAKE, FAKE, adapters, rank, dtype)
    for key, v in over.items():
        setattr(d, key, v)
    return d


def _forward(L, d, rows=5, x=FAKE, xs=None, y=FAKE, ys=None, u=0, ws=FAKE, ws_bytes=1 << 20, status=0, count=3,
             offsets=FAKE, ids=FAKE):
    q = L.RequestsDesc(offsets, ids, count)
    return L._lib.ecf8_linear_forward(ctypes.byref(d) if d is not None else None, ctypes.byref(q), x,
                                      d.k_in if xs is None and d is not None else xs or 0, y,
                                      d.n_out if ys is None and d is not None else ys or 0, rows, u, ws, ws_bytes,
                                      status, 0)


def _backward(L, d, rows=5, x=FAKE, xs=None, dy=FAKE, ds=None, u=FAKE, dx=FAKE, gs=None, da=FAKE, db=FAKE, ws=FAKE,
              ws_bytes=1 << 20):
    q = L.RequestsDesc(FAKE, FAKE, 3)
    return L._lib.ecf8_linear_backward(ctypes.byref(d), ctypes.byref(q), x, d.k_in if xs is None else xs, dy,
                                       d.n_out if ds is None else ds, u, dx, d.k_in if gs is None else gs, da, db,
                                       rows, ws, ws_bytes, 0, 0)


def test_forward_refuses_null_pointers(L):
    assert _forward(L, None) == ARG
    for key in ("d_w", "d_scale", "d_a", "d_b", "d_alpha"):
        assert _forward(L, _desc(L, **{key: None})) == ARG, key
    assert _forward(L, _desc(L), x=0) == ARG
    assert _forward(L, _desc(L), y=0) == ARG
    assert _forward(L, _desc(L), offsets=0) == ARG
    assert _forward(L, _desc(L), ids=0) == ARG


@pytest.mark.parametrize("over", [dict(n_out=0), dict(k_in=0), dict(n_out=1 << 31), dict(k_in=1 << 31, w_stride=1 << 31),
                                  dict(w_stride=95), dict(n_scale=2), dict(n_scale=63), dict(rank=0), dict(rank=129),
                                  dict(dtype=2), dict(dtype=-1), dict(n_adapters=65536)])
def test_bad_sizes_and_types_are_refused(L, over):
    assert _forward(L, _desc(L, **over)) == ARG
    assert _backward(L, _desc(L, **over)) == ARG


def test_bad_strides_and_rows_are_refused(L):
    d = _desc(L)
    assert _forward(L, d, xs=95) == ARG
    assert _forward(L, d, ys=63) == ARG
    assert _forward(L, d, rows=1 << 31) == ARG
    assert _backward(L, d, xs=95) == ARG
    assert _backward(L, d, ds=63) == ARG
    assert _backward(L, d, gs=95) == ARG


def test_misaligned_pointers_are_refused(L):
    assert _forward(L, _desc(L), x=FAKE + 1) == ALIGN
    assert _forward(L, _desc(L), y=FAKE + 1) == ALIGN
    assert _forward(L, _desc(L), u=FAKE + 2) == ALIGN
    assert _forward(L, _desc(L), ws=FAKE + 8) == ALIGN
    assert _forward(L, _desc(L), status=FAKE + 2) == ALIGN
    assert _forward(L, _desc(L), offsets=FAKE + 2) == ALIGN
    assert _forward(L, _desc(L, d_scale=FAKE + 2)) == ALIGN
    assert _forward(L, _desc(L, d_a=FAKE + 1)) == ALIGN
    assert _forward(L, _desc(L, d_b=FAKE + 1)) == ALIGN
    assert _forward(L, _desc(L, d_alpha=FAKE + 2)) == ALIGN
    for key in ("x", "dy", "dx", "da", "db"):
        assert _backward(L, _desc(L), **{key: FAKE + 1}) == ALIGN, key
    assert _backward(L, _desc(L), u=FAKE + 2) == ALIGN


def test_the_workspace_must_hold_what_the_call_needs(L):
    d = _desc(L)
    need = L._lib.ecf8_linear_workspace_size(ctypes.byref(d), 5)
    assert need > 0
    assert _forward(L, d, ws=0) == WORKSPACE
    assert _forward(L, d, ws_bytes=need - 1) == WORKSPACE
    assert _backward(L, d, ws_bytes=need - 1) == WORKSPACE
    assert L._lib.ecf8_linear_workspace_size(ctypes.byref(_desc(L, adapters=0)), 5) == 0
    assert L._lib.ecf8_linear_workspace_size(None, 5) == 0
    # more rows never need less
    sizes = [L._lib.ecf8_linear_workspace_size(ctypes.byref(d), r) for r in (0, 1, 5, 64, 1000, 100_000)]
    assert sizes == sorted(sizes)


def test_backward_refuses_missing_inputs(L):
    d = _desc(L)
    assert _backward(L, d, dy=0) == ARG
    assert _backward(L, d, x=0) == ARG            # da needs x
    assert _backward(L, d, u=0) == ARG            # db needs u
    assert _backward(L, _desc(L, adapters=0)) == ARG  # adapter gradients without adapters


def test_no_rows_is_nothing_to_do(L):
    assert _forward(L, _desc(L), rows=0, x=0, y=0) == 0


def test_python_checks_shapes_types_and_strides(L):
    import torch
    w = torch.zeros(64, 96, dtype=torch.uint8)
    a = torch.zeros(2, 8, 96, dtype=torch.bfloat16)
    b = torch.zeros(2, 64, 8, dtype=torch.bfloat16)
    alpha = torch.ones(2)
    bad = [dict(weight=w.float()), dict(weight=w.view(-1)), dict(weight=w.t()), dict(weight=FAKE),
           dict(weight=w, dtype=torch.float32), dict(weight=w, scale=torch.ones(2)),
           dict(weight=w, scale=torch.ones(64, dtype=torch.float64)), dict(weight=w, shape=(64, 95)),
           dict(weight=w, adapters=L.Adapters(a, b[:1], alpha)), dict(weight=w, adapters=L.Adapters(a.half(), b, alpha)),
           dict(weight=w, adapters=L.Adapters(a, b.transpose(1, 2), alpha)),
           dict(weight=w, adapters=L.Adapters(a, b, alpha.double()))]
    for args in bad:
        with pytest.raises(L.Ecf8Error) as e:
            L.Linear(**args)
        assert e.value.code == ARG, args
    lin = L.Linear(w, adapters=L.Adapters(a, b, alpha))
    x, y = torch.zeros(5, 96, dtype=torch.bfloat16), torch.zeros(5, 64, dtype=torch.bfloat16)
    for args in [dict(x=x.half(), y=y), dict(x=x[:, :95], y=y), dict(x=x, y=y[:4]), dict(x=x, y=y.t().contiguous().t()),
                 dict(x=x, y=y, u=torch.zeros(5, 7)), dict(x=x, y=y, u=torch.zeros(5, 8).half()),
                 dict(x=x, y=y, requests=L.Requests(torch.zeros(3, dtype=torch.int32), torch.zeros(3, dtype=torch.int32))),
                 dict(x=x, y=y, requests=L.Requests(torch.zeros(4, dtype=torch.int64), torch.zeros(3, dtype=torch.int32)))]:
        with pytest.raises(L.Ecf8Error) as e:
            lin.forward(**args, stream=0)
        assert e.value.code == ARG
    with pytest.raises(L.Ecf8Error):
        lin.backward(x, y, torch.zeros(5, 8), da=torch.zeros(2, 8, 95, dtype=torch.bfloat16), stream=0)
    with pytest.raises(L.Ecf8Error):  # a broadcast gradient has no row stride of its own
        lin.backward(x, y[:1].expand(5, 64), torch.zeros(5, 8), dx=x.clone(), stream=0)
    with pytest.raises(L.Ecf8Error):
        L.Linear(w).backward(x, y, None, da=a.clone(), stream=0)


def _grads(L, entries):
    arr = (L.Grad * max(1, len(entries)))()
    for i, e in enumerate(entries):
        arr[i] = L.Grad(*e)
    table = np.zeros(L._lib.ecf8_grad_table_bytes(len(entries)), np.uint8)
    return L._lib.ecf8_grad_build_table(arr, len(entries), table.ctypes.data), table


def test_gradient_tables_are_checked(L):
    assert _grads(L, [(FAKE, FAKE, 10, 0), (0, 0, 0, 2), (FAKE + 66, 0, 1, 1)])[0] == 0
    assert _grads(L, [(FAKE, FAKE, 10, 3)])[0] == ARG
    assert _grads(L, [(0, FAKE, 10, 0)])[0] == ARG
    assert _grads(L, [(FAKE, FAKE, 1 << 60, 0)])[0] == ARG
    assert _grads(L, [(FAKE + 1, FAKE, 10, 0)])[0] == ALIGN
    assert _grads(L, [(FAKE, FAKE + 2, 10, 2)])[0] == ALIGN
    assert L._lib.ecf8_grad_build_table(None, 1, FAKE) == ARG
    assert L._lib.ecf8_grad_build_table(None, 0, None) == ARG
    assert L._lib.ecf8_grad_table_bytes(-1) == 0


def test_outputs_of_a_set_may_not_share_memory(L):
    far = FAKE + (1 << 16)
    assert _grads(L, [(FAKE, FAKE, 10, 0), (FAKE, FAKE, 10, 0)])[0] == ARG        # listed twice, in place
    assert _grads(L, [(FAKE, far, 10, 0), (FAKE, far + 18, 10, 0)])[0] == ARG     # outputs overlap by a value
    assert _grads(L, [(FAKE, far, 10, 0), (FAKE, far + 20, 10, 0)])[0] == 0       # and lie next to each other
    assert _grads(L, [(FAKE, far, 10, 0), (far + 18, 0, 10, 0)])[0] == ARG        # an output over another's input
    assert _grads(L, [(FAKE, FAKE + 2, 10, 0)])[0] == ARG                         # shifted in place
    assert _grads(L, [(FAKE, 0, 10, 0), (FAKE, 0, 10, 0), (FAKE + 4, 0, 3, 2)])[0] == 0  # inputs may: norm only
    many = [(FAKE + 64 * i, FAKE + 64 * i, 16, 2) for i in range(300)]
    assert _grads(L, many)[0] == 0
    assert _grads(L, many + [(FAKE + 64 * 299, far + (1 << 20), 17, 2)])[0] == ARG  # reads what another writes


def test_tensors_off_the_gpu_are_refused(L):
    import torch
    w = torch.zeros(64, 96, dtype=torch.uint8)
    x, y = torch.zeros(5, 96, dtype=torch.bfloat16), torch.zeros(5, 64, dtype=torch.bfloat16)
    lin = L.Linear(w)
    for call in (lambda: lin.forward(x, y, stream=0), lambda: lin.backward(None, y, None, dx=x, stream=0),
                 lambda: L.GradSet([x])):
        with pytest.raises(L.Ecf8Error) as e:
            call()
        assert e.value.code == ARG


def test_gradient_calls_are_checked(L):
    _, table = _grads(L, [(FAKE, FAKE, 10, 0)])
    _, half = _grads(L, [(FAKE, FAKE, 10, 0), (FAKE + 64, 0, 10, 0)])
    h, ws = table.ctypes.data, L._lib.ecf8_grad_workspace_size()

    def clip(h=h, d=FAKE, most=1.0, norm=FAKE, w=FAKE, ws_bytes=ws, status=0):
        return L._lib.ecf8_grad_clip(h, d, most, norm, w, ws_bytes, status, 0)

    assert clip(h=0) == ARG and clip(d=0) == ARG and clip(norm=0) == ARG
    assert clip(h=np.zeros(64, np.uint8).ctypes.data) == ARG  # not a table
    assert clip(h=half.ctypes.data) == ARG                    # a tensor without an output
    assert clip(most=-1.0) == ARG and clip(most=float("nan")) == ARG
    assert clip(d=FAKE + 8) == ALIGN and clip(norm=FAKE + 2) == ALIGN and clip(status=FAKE + 1) == ALIGN
    assert clip(w=FAKE + 4) == ALIGN
    assert clip(w=0) == WORKSPACE and clip(ws_bytes=ws - 1) == WORKSPACE


def test_gradient_sets_refuse_what_they_cannot_hold(L):
    import torch
    g = torch.zeros(8, 8)
    for args in [([g], [g, g]), ([g.t()[1:]], None), ([g], [g.half()]), ([g], [g[:4]]), ([g.double()], None),
                 ([g.int()], None)]:
        with pytest.raises(L.Ecf8Error) as e:
            L.GradSet(*args)
        assert e.value.code == ARG
