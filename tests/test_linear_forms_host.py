"""What the linear layers' entry points answer and refuse before any device work, on CPU."""
import ctypes

import pytest

FAKE = 1 << 20


@pytest.fixture(scope="module")
def L():
    import lossless_fp8_weight_b200 as lib
    return lib


@pytest.mark.parametrize("dtype", ["float8_e5m2", "float8_e4m3fnuz", "float8_e5m2fnuz", "float8_e8m0fnu", "int8", "bool"])
def test_bytes_of_another_type_are_no_weights(L, dtype):
    import torch
    w = torch.zeros(64, 96, dtype=torch.uint8)
    with pytest.raises(L.Ecf8Error) as e:
        L.Linear(w.view(getattr(torch, dtype)))
    assert e.value.code == -1
    for held in (w, w.view(torch.float8_e4m3fn)):
        assert L.Linear(held).k_in == 96


def test_the_form_of_a_call(L):
    """Two CTAs to a tile from 37 tiles of 256 x 256 on, and never in small batches."""
    def ctas(rows, n, k, backward=False):
        return L.Linear(FAKE, shape=(n, k)).tile_ctas(rows, backward)

    assert ctas(128, 1 << 20, 64) == 1 and ctas(129, 36 * 256, 64) == 1 and ctas(129, 36 * 256 + 1, 64) == 2
    assert ctas(8192, 256, 256) == 1 and ctas(8192, 512, 64) == 2
    assert ctas(8192, 64, 512) == 1 and ctas(8192, 64, 512, backward=True) == 2
    assert ctas(0, 64, 64) == 0 and L._lib.ecf8_linear_tile_ctas(None, 5, 0) == 0
    d = L.LinearDesc(FAKE, 64, 64, 64)
    assert L._lib.ecf8_linear_tile_ctas(ctypes.byref(d), 1 << 31, 0) == 0
