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
