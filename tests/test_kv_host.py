"""What the attention and logits operators decide on the host: frequencies, refusals, structures."""
import ctypes
import math
import os
import subprocess

import numpy as np
import pytest

import lossless_bf16_weight_exponent_gb300 as uw

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("dim", [16, 64, 96, 128])
@pytest.mark.parametrize("base", [10000.0, 500000.0])
def test_frequencies(dim, base):
    i = np.arange(dim // 2)
    f = base ** (-2.0 * i / dim)
    close = dict(rtol=1e-12, atol=0)

    def got(scaling, **kw):
        return uw.rotary_frequencies(dim, base, scaling, **kw)

    a, s = got(uw.ROTARY_PLAIN)
    assert s == 1.0 and np.allclose(a, f, **close)
    a, s = got(uw.ROTARY_LINEAR, factor=4.0)
    assert s == 1.0 and np.allclose(a, f / 4, **close)
    a, s = got(uw.ROTARY_STRETCHED, factor=4.0)
    assert s == 1.0 and a[0] == 1.0 and math.isclose(a[-1], f[-1] / 4, rel_tol=1e-12)
    a, s = got(uw.ROTARY_BANDS, factor=8.0, low=1.0, high=4.0, original=8192)
    turns = 8192 * f / (2 * math.pi)
    assert np.allclose(a[turns >= 4], f[turns >= 4], **close) and np.allclose(a[turns <= 1], f[turns <= 1] / 8, **close)
    mid = (turns > 1) & (turns < 4)
    w = (turns[mid] - 1) / 3
    assert np.allclose(a[mid], w * f[mid] + (1 - w) * f[mid] / 8, **close)
    a, s = got(uw.ROTARY_RAMP, factor=16.0, low=1.0, high=32.0, original=4096)
    assert math.isclose(s, 0.1 * math.log(16) + 1, rel_tol=1e-6)
    lo = max(math.floor(dim * math.log(4096 / (32 * 2 * math.pi)) / (2 * math.log(base))), 0)
    hi = min(math.ceil(dim * math.log(4096 / (2 * math.pi)) / (2 * math.log(base))), dim - 1)
    w = 1 - np.clip((i - lo) / max(hi - lo, 0.001), 0, 1)
    assert np.allclose(a, w * f + (1 - w) * f / 16, **close)


def refused(status, f, *a, **kw):
    with pytest.raises(uw.UwError) as e:
        f(*a, **kw)
    assert e.value.status == status, str(e.value)


def test_frequency_refusals():
    r = uw.rotary_frequencies
    for dim in (0, 8, 15, 24, 136, 144, -16):
        refused(uw.ERR_SHAPE, r, dim)
    for base in (1.0, 0.0, -5.0, math.inf, math.nan):
        refused(uw.ERR_INVALID_ARG, r, 64, base)
    for factor in (0.5, 0.0, math.nan, math.inf):
        for scaling in (1, 2, 3, 4):
            refused(uw.ERR_INVALID_ARG, r, 64, 1e4, scaling, factor)
    for low, high, original in ((2.0, 2.0, 10), (3.0, 2.0, 10), (-1.0, 2.0, 10), (1.0, 2.0, 0), (math.nan, 2.0, 10), (1.0, math.inf, 10)):
        for scaling in (3, 4):
            refused(uw.ERR_INVALID_ARG, r, 64, 1e4, scaling, 2.0, low, high, original)
    refused(uw.ERR_INVALID_ARG, r, 64, 1e4, 4, 2.0, 0.0, 2.0, 10)
    refused(uw.ERR_INVALID_ARG, r, 64, 1e4, 5, 2.0)
    refused(uw.ERR_INVALID_ARG, r, 64, 1e4, -1, 2.0)
    assert uw.lib().uw_rotary_frequencies(64, 1e4, 0, 1.0, 1.0, 4.0, 1, None, None) == uw.ERR_INVALID_ARG


def kv(**kw):
    d = dict(k=4096, v=8192, pages=4, page_stride=2048, slot_stride=128, head_stride=64, page_size=16, kv_heads=2, head_dim=64)
    d.update(kw)
    out = ctypes.c_void_p()
    return uw.lib().uw_kv_create(ctypes.byref(uw.KVDesc(**d)), ctypes.byref(out))


@pytest.mark.parametrize("status,kw", [
    (uw.ERR_INVALID_ARG, dict(k=0)), (uw.ERR_INVALID_ARG, dict(v=0)), (uw.ERR_INVALID_ARG, dict(k=4104)), (uw.ERR_INVALID_ARG, dict(v=8194)),
    (uw.ERR_UNSUPPORTED, dict(head_dim=96)), (uw.ERR_UNSUPPORTED, dict(head_dim=256)), (uw.ERR_UNSUPPORTED, dict(head_dim=0)),
    (uw.ERR_SHAPE, dict(pages=0)), (uw.ERR_SHAPE, dict(pages=1 << 31)), (uw.ERR_SHAPE, dict(page_size=0)), (uw.ERR_SHAPE, dict(page_size=12)),
    (uw.ERR_SHAPE, dict(page_size=-8)), (uw.ERR_SHAPE, dict(page_size=65544)), (uw.ERR_SHAPE, dict(kv_heads=0)), (uw.ERR_SHAPE, dict(kv_heads=1025)),
    (uw.ERR_INVALID_ARG, dict(slot_stride=132)), (uw.ERR_INVALID_ARG, dict(slot_stride=0)), (uw.ERR_INVALID_ARG, dict(head_stride=32)),
    (uw.ERR_INVALID_ARG, dict(page_stride=-2048)), (uw.ERR_INVALID_ARG, dict(page_stride=1 << 39))])
def test_cache_refusals(status, kw):
    assert kv(**kw) == status


def test_null():
    L = uw.lib()
    n = ctypes.c_size_t(0)
    assert L.uw_kv_create(None, None) == uw.ERR_INVALID_ARG
    assert L.uw_kv_check(None, None) == uw.ERR_INVALID_ARG
    assert L.uw_kv_attend_workspace_size(None, 1, 1, 1, ctypes.byref(n)) == uw.ERR_INVALID_ARG
    assert L.uw_kv_attend(None, None, 1, None, 0, 1, 1.0, 1, 0, None, 0, None, None, 0, None) == uw.ERR_INVALID_ARG
    assert L.uw_kv_append(None, None, None, 1, 0, None, 0, 1, None, 0, None, 0, None, None, 0, None) == uw.ERR_INVALID_ARG
    assert L.uw_edit_logits(None, None, 0, 1, 1, 0, None, 0, 0, None) == uw.ERR_INVALID_ARG
    L.uw_kv_free(None)


def edit(rows=2, vocab=64, ld=0, ld_out=0, dtype=0, out_dtype=0, logits=4096, out=1 << 20, **kw):
    d = uw.LogitEditsDesc(**kw)
    return uw.lib().uw_edit_logits(ctypes.byref(d), logits, dtype, rows, vocab, ld, out, out_dtype, ld_out, None)


@pytest.mark.parametrize("status,kw", [
    (uw.ERR_SHAPE, dict(rows=-1)), (uw.ERR_SHAPE, dict(vocab=0)), (uw.ERR_SHAPE, dict(vocab=(1 << 24) + 1)), (uw.ERR_SHAPE, dict(ld=63)),
    (uw.ERR_SHAPE, dict(ld_out=63)), (uw.ERR_INVALID_ARG, dict(dtype=2)), (uw.ERR_INVALID_ARG, dict(out_dtype=-1)),
    (uw.ERR_INVALID_ARG, dict(logits=0)), (uw.ERR_INVALID_ARG, dict(out=0)), (uw.ERR_INVALID_ARG, dict(logits=4098)),
    (uw.ERR_INVALID_ARG, dict(out=(1 << 20) + 1, out_dtype=1)), (uw.ERR_INVALID_ARG, dict(logits=4097, dtype=1)),
    (uw.ERR_INVALID_ARG, dict(tokens=4096, max_tokens=4)), (uw.ERR_SHAPE, dict(tokens=4096, lengths=4096, max_tokens=-1)),
    (uw.ERR_SHAPE, dict(tokens=4096, lengths=4096, max_tokens=1 << 24)), (uw.ERR_SHAPE, dict(tokens=4096, lengths=4096, max_tokens=8, ld_tokens=7)),
    (uw.ERR_INVALID_ARG, dict(repetition=4096)), (uw.ERR_INVALID_ARG, dict(frequency=4096)), (uw.ERR_INVALID_ARG, dict(presence=4096)),
    (uw.ERR_INVALID_ARG, dict(bias=4096)), (uw.ERR_INVALID_ARG, dict(bias_ids=4096)), (uw.ERR_SHAPE, dict(max_bias=-1)), (uw.ERR_SHAPE, dict(max_bias=65537)),
    (uw.ERR_SHAPE, dict(allowed=4096, ld_allowed=1, mask_count=1)), (uw.ERR_SHAPE, dict(allowed=4096, mask_count=-1)),
    (uw.ERR_INVALID_ARG, dict(allowed=4098, mask_count=1)),
    # out overlaps logits: shifted by some elements, another type, another stride, rows into one another
    (uw.ERR_INVALID_ARG, dict(out=4096 + 16)), (uw.ERR_INVALID_ARG, dict(out=4096, out_dtype=1)), (uw.ERR_INVALID_ARG, dict(out=4096, ld_out=80)),
    (uw.ERR_INVALID_ARG, dict(out=4096 + 4 * 70, ld=128, ld_out=128)), (uw.ERR_INVALID_ARG, dict(out=4096 - 4 * 70, ld=128, ld_out=128))])
def test_edit_refusals(status, kw):
    assert edit(**kw) == status


def test_nothing_to_do():
    assert edit(rows=0) == uw.OK
    assert edit(out=4096) == uw.OK  # in place without an edit


def test_structures(tmp_path):
    structs = [("uw_rotary", uw.RotaryDesc), ("uw_kv_desc", uw.KVDesc), ("uw_kv_batch", uw.KVBatchDesc), ("uw_logit_edits", uw.LogitEditsDesc)]
    names = ("UW_ROTARY_HALF", "UW_ROTARY_INTERLEAVED", "UW_ROTARY_PLAIN", "UW_ROTARY_LINEAR", "UW_ROTARY_STRETCHED", "UW_ROTARY_BANDS", "UW_ROTARY_RAMP")
    lines = [f'printf("{n} %zu\\n", (size_t){n});' for n in names]
    for name, cls in structs:
        lines.append(f'printf("{name} %zu\\n", sizeof({name}));')
        lines += [f'printf("{name}.{f[0]} %zu\\n", offsetof({name}, {f[0]}));' for f in cls._fields_]
    (tmp_path / "l.c").write_text('#include <stddef.h>\n#include <stdio.h>\n#include "uw.h"\nint main(void) {\n' + "\n".join(lines) + "\nreturn 0; }\n")
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), "-o", str(tmp_path / "l"), str(tmp_path / "l.c")], check=True)
    out = subprocess.run([str(tmp_path / "l")], check=True, capture_output=True, text=True).stdout
    at = {k: int(v) for k, v in (line.split() for line in out.splitlines())}
    for name, cls in structs:
        assert ctypes.sizeof(cls) == at[name]
        for f in cls._fields_:
            assert getattr(cls, f[0]).offset == at[f"{name}.{f[0]}"], f[0]
    for n in names:
        assert getattr(uw, n[3:]) == at[n]
