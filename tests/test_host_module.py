"""The C++ half of the binding, _host.so: without it the entry points that need
libgbw.so alone work and the others say what is missing; it is rebuilt for
another torch or Python.  CPU only."""
import importlib.util
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "grouped_bit_weight_b200")

pytest.importorskip("grouped_bit_weight_b200")

CALLS = """
import torch
import grouped_bit_weight_b200 as gbw
assert gbw.lib.gbw_version() >= 100
try:
    gbw.gnf4_quantize(torch.zeros((2, 65)))
except ValueError as e:
    print("quantize:", e)
for call in (lambda: gbw.gmoe_route(torch.zeros((2, 4)), 1),
             lambda: gbw.gmxfp4_quantize_rows(torch.zeros((2, 32), dtype=torch.bfloat16))):
    try:
        call()
    except ImportError as e:
        print("host:", e)
"""


@pytest.mark.parametrize("broken", [False, True], ids=["missing", "unloadable"])
def test_package_imports_without_the_host_module(tmp_path, broken):
    to = tmp_path / "grouped_bit_weight_b200"
    to.mkdir()
    for name in os.listdir(PKG):
        if name.endswith(".py"):
            shutil.copy(os.path.join(PKG, name), to / name)
    os.symlink(os.path.join(PKG, "libgbw.so"), to / "libgbw.so")
    if broken:
        (to / "_host.so").write_bytes(b"no shared object")
    r = subprocess.run([sys.executable, "-c", CALLS], cwd=tmp_path, capture_output=True, text=True,
                       env={**os.environ, "PYTHONPATH": str(tmp_path)}, timeout=300)
    assert r.returncode == 0, r.stderr
    lines = r.stdout.splitlines()
    assert len(lines) == 3 and lines[0].startswith("quantize:")
    for line in lines[1:]:
        assert line.startswith("host:") and "_host.so does not load" in line and "no fallback" in line


def test_host_module_is_rebuilt_for_another_torch_or_python(tmp_path, monkeypatch):
    spec = importlib.util.spec_from_file_location("_build_under_test", os.path.join(PKG, "build.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    host, stamp = tmp_path / "_host.so", tmp_path / "host.txt"
    monkeypatch.setattr(b, "HOST", str(host))
    monkeypatch.setattr(b, "HOST_STAMP", str(stamp))
    assert not b.host_up_to_date()
    host.write_bytes(b"")
    assert not b.host_up_to_date()  # nothing says what it was built against
    stamp.write_text(b._host_stamp())
    assert b.host_up_to_date()
    stamp.write_text(b._host_stamp().replace("torch ", "torch 1."))
    assert not b.host_up_to_date()
    stamp.write_text(b._host_stamp())
    os.utime(host, (1, 1))          # older than its source
    assert not b.host_up_to_date()
