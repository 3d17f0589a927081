"""The package around the 8-bit cache's native module, without a GPU."""
import decimal
import importlib.util
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "kv_cache_embedding_b200")


def copy_of_the_package(tmp_path, leave_out):
    """Links to the package's files but one."""
    pkg = tmp_path / "kv_cache_embedding_b200"
    pkg.mkdir()
    for name in os.listdir(PKG):
        if name.endswith((".py", ".so")) and name != leave_out:
            os.symlink(os.path.join(PKG, name), pkg / name)
    return pkg


def run(tmp_path, code):
    p = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, capture_output=True, text=True)
    assert p.returncode == 0, p.stderr


def test_the_package_needs_the_native_module_for_the_8_bit_cache_alone(tq_lib, tmp_path):
    copy_of_the_package(tmp_path, "_kv8.so")
    run(tmp_path, """
import kv_cache_embedding_b200 as tq
assert tq.TurboQuant and tq.tq_encode and tq.KV8Cache
for make in (lambda: tq.Rope(64), lambda: tq.KV8Cache.empty(1, 1, 1, 64, 1, 1, device="cpu")):
    try:
        make()
    except ImportError as e:
        assert "build.py" in str(e)
    else:
        raise SystemExit("no error")
""")


def test_a_native_module_of_another_torch(tq_lib, tmp_path):
    """Refused by name when it is used, and built again."""
    copy_of_the_package(tmp_path, None)
    run(tmp_path, """
import torch
torch.__version__ = "0.0.1"
import kv_cache_embedding_b200 as tq
try:
    tq.Rope(64)
except ImportError as e:
    assert "0.0.1" in str(e) and "build.py" in str(e)
else:
    raise SystemExit("no error")
""")
    spec = importlib.util.spec_from_file_location("_tq_build_again", os.path.join(PKG, "build.py"))
    kb = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(kb)
    assert not kb._stale()
    kb._torch_version = lambda: "0.0.1"
    assert kb._stale()


@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "parts"])
@pytest.mark.parametrize("d,rot,base", [(128, 128, 1e4), (128, 64, 5e5), (256, 256, 1e6), (8, 6, 3.0)])
def test_rope_frequencies_of_far_positions(tq_lib, scaling, d, rot, base):
    """turns[i] against f / 2 pi in 60 digits.  The host computes it with 64 bits of
    mantissa: a handful of roundings (pow within a unit, the rule's products, the
    division by 2 pi, the rounding to the fraction) of 2^-64 of at most 0.16 turn and
    half a unit of 2^-64: 2 units, so an angle at position p is within |p| 2^-63 turn."""
    r = tq_lib.Rope(d, rot, base=base, scaling=scaling, factor=4.0, ctx=4096, low=1.0, high=32.0)
    with decimal.localcontext() as ctx:
        ctx.prec = 60
        D = decimal.Decimal
        pi = D("3.14159265358979323846264338327950288419716939937510582097494")
        b = D(base) * D(4) ** (D(rot) / D(rot - 2)) if scaling == "ntk" else D(base)
        for i in range(rot // 2):
            f = (b.ln() * D(-2 * i) / D(rot)).exp()
            if scaling == "linear":
                f /= 4
            if scaling == "parts":
                g = min(D(1), max(D(0), (D(4096) * f / (2 * pi) - 1) / 31))
                f = f * g + f / 4 * (1 - g)
            assert abs(D(r.params.turns[i]) - f / (2 * pi) * 2 ** 64) <= 2, i
