"""The rotation's arguments in Python: the ends of a scaling by bands or on a ramp where none are given, as their methods have them, and
frequencies and a factor of the caller's own."""
import ctypes

import numpy as np
import pytest
import torch

import lossless_bf16_weight_exponent_gb300 as uw


@pytest.fixture
def on_host(monkeypatch):
    """Frequencies stay in host memory, where the test reads them by the structure's address."""
    monkeypatch.setattr(torch.Tensor, "cuda", lambda t: t.clone())


def held(r):
    return np.ctypeslib.as_array((ctypes.c_double * (r.desc.dim // 2)).from_address(r.desc.freq)).copy()


@pytest.mark.parametrize("scaling,low,high", [(uw.ROTARY_BANDS, 1.0, 4.0), (uw.ROTARY_RAMP, 1.0, 32.0)])
def test_ends(on_host, scaling, low, high):
    kw = dict(factor=16.0, original=4096)
    want, s = uw.rotary_frequencies(128, 1e4, scaling, low=low, high=high, **kw)
    for a in ({}, dict(low=low), dict(high=high)):
        got, t = uw.rotary_frequencies(128, 1e4, scaling, **a, **kw)
        assert np.array_equal(got, want) and s == t
        r = uw.Rotary(128, 1e4, scaling=scaling, **a, **kw)
        assert np.array_equal(held(r), want) and r.scale == s and r.desc.scale == s
    other, _ = uw.rotary_frequencies(128, 1e4, scaling, low=2.0, high=8.0, **kw)
    assert not np.array_equal(other, want)
    assert np.array_equal(held(uw.Rotary(128, 1e4, scaling=scaling, low=2.0, high=8.0, **kw)), other)
