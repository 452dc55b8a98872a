"""What the calls on a paged cache and the edits of logits take from tensors: rows that share memory are refused, as a row
stride of 0 is the library's word for dense rows, and a broadcast tensor would be read, or written, past its end.

CPU tensors stand in for the device's: the calls' device is set to theirs, and no call here gets as far as a kernel."""
import pytest
import torch

import lossless_bf16_weight_exponent_gb300 as uw

BF16, I32 = torch.bfloat16, torch.int32
H, D = 2, 64


class OnDevice(torch.Tensor):
    is_cuda = True


def dev(*shape, dtype=BF16):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnDevice)


@pytest.fixture
def cache(monkeypatch):
    monkeypatch.setattr(uw, "_device", lambda: -1)
    c = uw.KVCache.__new__(uw.KVCache)
    c._h, c._device, c.head_dim, c.kv_heads, c._scale = None, -1, D, H, D ** -0.5
    return c


def batch(S=2, pages=3):
    return uw.KVBatch(dev(S + 1, dtype=I32), dev(S, dtype=I32), dev(S, pages, dtype=I32))


def refused(f, *a, **kw):
    with pytest.raises(ValueError):
        f(*a, **kw)


def reaches_the_library(f, *a, **kw):
    with pytest.raises(uw.UwError) as e:
        f(*a, **kw)
    assert e.value.status == uw.ERR_INVALID_ARG and "NULL" in e.value.message


def rows(heads, n=4, flat=False):
    return dev(n, heads * D) if flat else dev(n, heads, D)


@pytest.mark.parametrize("flat", [False, True])
@pytest.mark.parametrize("name", ["q", "q_out", "k", "v"])
def test_append(cache, name, flat):
    t = dict(q=rows(8), q_out=rows(8), k=rows(H), v=rows(H))
    reaches_the_library(cache.append, batch(), 4, stream=1, **t)
    one = rows(8 if name[0] == "q" else H, 1, flat)
    t[name] = one.expand(4, *one.shape[1:])
    refused(cache.append, batch(), 4, stream=1, **t)
    reaches_the_library(cache.append, batch(), 1, stream=1, **t)     # one row: nothing is read past it
    wide = 2 * rows(8 if name[0] == "q" else H, 4, True).shape[1]
    t[name] = dev(4, wide)[:, :wide // 2]
    reaches_the_library(cache.append, batch(), 4, stream=1, **t)


@pytest.mark.parametrize("flat", [False, True])
@pytest.mark.parametrize("name", ["q", "out"])
def test_attend(cache, name, flat):
    t = dict(q=rows(8), out=rows(8))
    one = rows(8, 1, flat)
    t[name] = one.expand(4, *one.shape[1:])
    refused(cache.attend, batch(), 4, stream=1, **t)
    reaches_the_library(cache.attend, batch(), 1, stream=1, **t)


def test_page_table():
    starts, lengths = dev(5, dtype=I32), dev(4, dtype=I32)
    one = dev(1, 3, dtype=I32)
    refused(uw.KVBatch, starts, lengths, one.expand(4, 3))
    refused(uw.KVBatch, starts, lengths, dev(1, 1, dtype=I32).expand(4, 1))
    assert uw.KVBatch(starts[:2], lengths[:1], one).desc.ld_pages == 0
    assert uw.KVBatch(starts, lengths, dev(4, 7, dtype=I32)[:, :3]).desc.ld_pages == 7
    assert uw.KVBatch(starts, lengths, dev(4, 1, dtype=I32)).desc.ld_pages == 1


def edit(R=4, V=100, **kw):
    t = dict(logits=dev(R, V, dtype=torch.float32), out=dev(R, V, dtype=torch.float32))
    t.update(kw)
    logits, out = t.pop("logits"), t.pop("out")
    uw.edit_logits(logits, R, V, out, stream=1, dtype=uw.OUT_F32, **t)


@pytest.fixture
def stopped(monkeypatch):
    """The library's call of the edits, which would launch: it notes its structure and reports NULL."""
    real, seen = uw.lib(), []

    class Lib:
        def __getattr__(self, name):
            if name == "uw_edit_logits":
                return lambda ref, *a: (seen.append((ref._obj, a)), real.uw_edit_logits(None, *[0] * 9))[1]
            return getattr(real, name)

    monkeypatch.setattr(uw, "_device", lambda: -1)
    monkeypatch.setattr(uw, "lib", lambda: Lib())
    return seen


@pytest.mark.parametrize("name,kw", [
    ("logits", {}), ("out", {}), ("tokens", dict(lengths=4)), ("allowed", {})])
def test_edits(stopped, name, kw):
    kw = {k: dev(n, dtype=I32) for k, n in kw.items()}
    width, dtype = (100, torch.float32) if name in ("logits", "out") else (6 if name == "tokens" else 4, I32)
    reaches_the_library(edit, **{name: dev(4, width, dtype=dtype)}, **kw)
    one = dev(1, width, dtype=dtype).expand(4, width)
    assert one.stride(0) == 0
    n = len(stopped)
    refused(edit, **{name: one}, **kw)
    assert len(stopped) == n
    reaches_the_library(edit, **{name: dev(4, 2 * width, dtype=dtype)[:, :width]}, **kw)
    if name != "allowed":
        # a call of one row reads one row
        kw1 = {k: v[:1] for k, v in kw.items()}
        t = dict(logits=dev(1, 100, dtype=torch.float32), out=dev(1, 100, dtype=torch.float32))
        t[name] = one
        reaches_the_library(edit, R=1, **t, **kw1)


def test_edits_without_a_history(stopped):
    """A history of no tokens has no rows to share."""
    for tokens in (dev(4, 0, dtype=I32), dev(1, 0, dtype=I32).expand(4, 0)):
        reaches_the_library(edit, tokens=tokens, lengths=dev(4, dtype=I32), repetition=dev(4, dtype=torch.float32))
        assert not stopped[-1][0].tokens


# ------------------------------------------------------------------------------------------------ the workspace
def attend(cache, ws, n, **kw):
    return cache.attend(batch(), 4, rows(8), rows(8), workspace=ws, ws_bytes=n, stream=1, **kw)


def test_workspace(cache):
    """Its type does not matter, its device and its bytes do: the kernels write as many as the call says."""
    for ws in (dev(4096, dtype=torch.uint8), dev(1024, dtype=torch.float32), dev(2, 2048, dtype=torch.uint8), dev(5000, dtype=torch.uint8), 16, None):
        reaches_the_library(attend, cache, ws, 4096)
    refused(attend, cache, dev(4095, dtype=torch.uint8), 4096)
    refused(attend, cache, dev(1023, dtype=torch.float32), 4096)
    refused(attend, cache, dev(1, dtype=torch.uint8).expand(4096), 4096)
    refused(attend, cache, dev(8192, dtype=torch.uint8)[::2], 4096)
    reaches_the_library(attend, cache, dev(0, dtype=torch.uint8), 0)


def test_workspace_on_another_device(cache):
    t = dict(q=rows(8), out=rows(8))
    cache._device = 1
    for x in t.values():
        x.get_device = lambda: 1
    b = batch()
    b.device = 1
    refused(cache.attend, b, 4, workspace=dev(4096, dtype=torch.uint8), ws_bytes=4096, stream=1, **t)
    reaches_the_library(cache.attend, b, 4, workspace=16, ws_bytes=4096, stream=1, **t)
