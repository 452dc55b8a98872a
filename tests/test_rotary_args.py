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


@pytest.mark.parametrize("kind", [list, np.array, torch.tensor, lambda x: torch.tensor(x, dtype=torch.float32), lambda x: np.array(x, np.float32)])
def test_own_frequencies(on_host, kind):
    """A model's list of frequencies, as its configuration's factors for each pair give them, and its own factor on cos and sin."""
    f = [1.0 / (1 + i) ** 2 for i in range(32)]
    r = uw.Rotary(64, layout=uw.ROTARY_INTERLEAVED, freq=kind(f))
    assert np.array_equal(held(r), np.asarray([float(x) for x in kind(f)])) and np.array_equal(r.freq, held(r))
    assert r.desc.dim == 64 and r.desc.layout == uw.ROTARY_INTERLEAVED and r.scale == 1.0 == r.desc.scale
    assert uw.Rotary(64, freq=kind(f), scale=1.25).desc.scale == 1.25


def test_own_factor(on_host):
    r = uw.Rotary(64, 1e4, scaling=uw.ROTARY_RAMP, factor=16.0, original=4096, scale=0.75)
    want, s = uw.rotary_frequencies(64, 1e4, uw.ROTARY_RAMP, factor=16.0, original=4096)
    assert s != 0.75 and r.scale == 0.75 == r.desc.scale and np.array_equal(held(r), want)


def test_refusals(on_host):
    f = np.ones(32)
    for bad in (np.ones(31), np.ones(64), np.ones((1, 32)), np.ones(0), np.full(32, np.nan), np.full(32, np.inf)):
        with pytest.raises(ValueError):
            uw.Rotary(64, freq=bad)
    for scale in (float("nan"), float("inf")):
        with pytest.raises(ValueError):
            uw.Rotary(64, freq=f, scale=scale)


@pytest.mark.gpu
def test_append_with_own_frequencies():
    """The same frequencies, made here or by the library, turn a key alike."""
    k, v = (torch.zeros(2, 16, 1, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    cache, batch = uw.KVCache(k, v), uw.KVBatch(i32([0, 5]), i32([25]), i32([[0, 1]]))
    x = torch.randn(5, 1, 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    got = []
    for r in (uw.Rotary(64, 5e5), uw.Rotary(64, freq=5e5 ** (-np.arange(0, 64, 2) / 64.0)), uw.Rotary(64, 5e5, scale=2.0)):
        cache.append(batch, 5, x, x, rotary=r)
        torch.cuda.synchronize()
        got.append(k.flatten(0, 1)[20:25].clone())
    assert torch.equal(got[0], got[1]) and torch.equal(got[2], 2 * got[0]) and got[0].abs().max() > 0
