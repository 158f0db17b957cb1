"""Calls on a stream that is not the current one: what the binding allocates,
copies and lets go of on the caller's behalf follows the call's stream."""
import numpy as np
import pytest

import ecf8_synth as synth
import oracle

pytestmark = pytest.mark.gpu

BUSY = 100_000_000  # clock cycles, some 50 ms


@pytest.fixture(scope="module")
def env(gpu_available):
    import torch
    import lossless_fp8_weight_b200 as L
    return L, torch


def _as(stream, raw):
    return stream.cuda_stream if raw else stream


@pytest.mark.parametrize("raw", [False, True])
def test_a_histogram_waits_for_its_own_stream(env, raw):
    L, torch = env
    side = torch.cuda.Stream()
    for i in range(4):
        x = synth.single_normal_1k().tensors[0].generate(begin=i, count=100_003 + i)
        d = torch.from_numpy(x).cuda()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(BUSY)
        h = L.histogram_device(d, stream=_as(side, raw))
        assert np.array_equal(h, np.bincount((x >> 3) & 15, minlength=16).astype(np.uint64))


def test_a_vector_with_gaps_is_counted_and_encoded_by_its_values(env):
    L, torch = env
    x = synth.single_normal_1k().tensors[0].generate(count=70_001)
    d = torch.from_numpy(np.stack([x, np.zeros_like(x)], axis=1)).cuda()[:, 0]
    assert np.array_equal(L.histogram_device(d), np.bincount((x >> 3) & 15, minlength=16).astype(np.uint64))
    assert np.array_equal(L.encode_device(d).cpu().numpy(), oracle.encode(x))


@pytest.mark.parametrize("raw", [False, True])
def test_an_encoders_workspace_outlives_the_call(env, raw):
    """Memory that the current stream gets right after the call is none that the encoder still has to use."""
    L, torch = env
    x = synth.single_normal_1k().tensors[0].generate(count=3_000_001)
    want = oracle.encode(x)
    d, side = torch.from_numpy(np.stack([x, x], axis=1)).cuda()[:, 0], torch.cuda.Stream()  # with gaps: it is copied
    h = L.histogram(x)
    size = L._lib.ecf8_encode_device_workspace_size(x.size)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    blob = L.encode_device(d, hist=h, stream=_as(side, raw))
    junk = [torch.full((m,), 0xFF, dtype=torch.uint8, device="cuda") for m in (size, size, x.size, x.size)]
    torch.cuda.synchronize()
    assert np.array_equal(blob.cpu().numpy(), want)
    assert all(bool((j == 0xFF).all()) for j in junk)


@pytest.mark.parametrize("how", ["stream", "current", "norm"])
def test_a_gradient_set_may_be_dropped_before_its_call_runs(env, how):
    """Its table and workspace are no memory that the stream it was made on hands out meanwhile."""
    L, torch = env
    grads = [torch.randn(1000 + i, device="cuda") for i in range(300)]
    want = float(torch.stack([g.double().square().sum() for g in grads]).sum().sqrt())
    before = [g.clone() for g in grads]
    norm, side = torch.zeros(1, device="cuda"), torch.cuda.Stream()
    L.GradSet(before, [torch.empty_like(b) for b in before]).clip(1.0, norm)  # the first launch loads the kernels
    s = L.GradSet(grads)
    torch.cuda.synchronize()
    own = {t.data_ptr(): t.numel() for t in (s._d, s._ws)}
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
        if how == "current":
            s.clip(1.0, norm)
    if how == "stream":
        s.clip(1.0, norm, stream=side)
    elif how == "norm":
        s.norm(norm, stream=side)
    del s
    junk = [torch.full((m,), 0, dtype=torch.uint8, device="cuda") for _ in range(4) for m in own.values()]
    assert not own.keys() & {j.data_ptr() for j in junk}
    torch.cuda.synchronize()
    assert abs(float(norm) - want) <= 2.0 ** -23 * want
    factor = 1.0 if how == "norm" else 1.0 / (want + 1e-6)
    assert all(bool(((g - b * factor).abs() <= 2.0 ** -21 * b.abs()).all()) for g, b in zip(grads, before))
