"""Numbers that the parameters' fields cannot hold are refused, not cut to fit; on the CPU."""
import ctypes

import pytest
import torch

import free_block_sparse_means_b200 as spr
from free_block_sparse_means_b200 import _binding as bind
from free_block_sparse_means_b200 import build as spr_build

BF = torch.bfloat16
P = 4096  # an aligned address that is never read


@pytest.fixture(scope="module", autouse=True)
def built():
    spr_build.build()


def meta(*shape):
    return torch.empty(*shape, dtype=BF, device="meta")


@pytest.mark.parametrize("N", [2 ** 31, 2 ** 32 + 5])
def test_dimensions_past_32_bits(N):
    """2^32 + 5 tokens are not 5 tokens."""
    t, w = meta(1, 1, N, 64), meta(64, 64)
    for make in (lambda: spr.make_norm_rotate(t, None, t, None), lambda: spr.make_masked(t, t, t, t),
                 lambda: spr.make_project(t, w, t)):
        with pytest.raises(ValueError, match="2\\^31"):
            make()


def test_positions_and_channels_past_their_ranges():
    q = meta(1, 2, 8, 64)
    for start in (-2 ** 31, 2 ** 31, 2 ** 32, 2 ** 30 + 1, -2 ** 30 - 1):
        with pytest.raises(ValueError, match="q_start"):
            spr.make_masked(q, q, q, q, q_start=start)
    assert spr.make_masked(q, q, q, q, q_start=-2 ** 30).q_start == -2 ** 30
    assert spr.make_masked(q, q, q, q).q_start == -2 ** 31  # aligned to the end
    for rot in (2 ** 32, -8, 72):
        with pytest.raises(ValueError, match="rot"):
            spr.make_norm_rotate(q, None, q, None, rot=rot)
    assert spr.make_norm_rotate(q, None, q, None, rot=0).rot == 0


def test_scales_and_caps_that_are_zero_in_fp32():
    """0 selects the usual scale and no cap; a number that only rounds to it does not."""
    q = meta(1, 2, 8, 64)
    for kw in (dict(scale=1e-50), dict(softcap=1e-50)):
        with pytest.raises(ValueError, match="fp32"):
            spr.make_masked(q, q, q, q, **kw)
    assert spr.make_masked(q, q, q, q, scale=1e-30, softcap=1e-30).softcap > 0


def test_tokens_past_what_a_grid_numbers():
    q = meta(1, 1, 8, 64)
    prm = spr.make_norm_rotate(q, q, q, q, rot=0)
    lib = spr.load_library()
    for field in ("Nq", "Nk"):
        setattr(prm, field, 2 ** 31 - 8)
        assert lib.sparsepr_norm_rotate(ctypes.byref(prm), P, P, None, None, None, None, 0, None,
                                        None, P, P, None, None) == bind.SPR_EUNSUPPORTED
        setattr(prm, field, 8)
