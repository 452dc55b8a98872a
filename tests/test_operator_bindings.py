"""The binding's structures and constants of the operators against the C header, as the C compiler lays them out."""
import ctypes
import os
import subprocess

import pytest

import lossless_bf16_weight_exponent_gb300 as uw

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
STRUCTS = [("uw_group_info", uw.GroupInfo), ("uw_router", uw.RouterDesc), ("uw_norm", uw.NormDesc)]


@pytest.fixture(scope="module")
def layout(tmp_path_factory):
    d = tmp_path_factory.mktemp("layout")
    lines = []
    for name, cls in STRUCTS:
        lines.append(f'printf("{name} %zu\\n", sizeof({name}));')
        lines += [f'printf("{name}.{f[0]} %zu\\n", offsetof({name}, {f[0]}));' for f in cls._fields_]
    lines += [f'printf("{n} %zu\\n", (size_t){n});' for n in ("UW_SCORE_SOFTMAX", "UW_SCORE_SIGMOID", "UW_OUT_F32", "UW_OUT_BF16")]
    (d / "l.c").write_text('#include <stddef.h>\n#include <stdio.h>\n#include "uw.h"\nint main(void) {\n' + "\n".join(lines) + "\nreturn 0; }\n")
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), "-o", str(d / "l"), str(d / "l.c")], check=True)
    out = subprocess.run([str(d / "l")], check=True, capture_output=True, text=True).stdout
    return {k: int(v) for k, v in (line.split() for line in out.splitlines())}


@pytest.mark.parametrize("name,cls", STRUCTS)
def test_structures(layout, name, cls):
    assert ctypes.sizeof(cls) == layout[name]
    for f in cls._fields_:
        assert getattr(cls, f[0]).offset == layout[f"{name}.{f[0]}"], f[0]


def test_constants(layout):
    assert (uw.SCORE_SOFTMAX, uw.SCORE_SIGMOID) == (layout["UW_SCORE_SOFTMAX"], layout["UW_SCORE_SIGMOID"])
    assert (uw.OUT_F32, uw.OUT_BF16) == (layout["UW_OUT_F32"], layout["UW_OUT_BF16"])


def test_added_score(tmp_path):
    (tmp_path / "c.c").write_text('#include <stdio.h>\n#include "uw.h"\nint main(void) { printf("%d\\n", UW_SCORE_CHOOSES); return 0; }\n')
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), "-o", str(tmp_path / "c"), str(tmp_path / "c.c")], check=True)
    assert int(subprocess.run([str(tmp_path / "c")], check=True, capture_output=True, text=True).stdout) == uw.SCORE_CHOOSES
