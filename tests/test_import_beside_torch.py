"""CPU: the package imports whatever stands in for torch, as it did when it loaded the system's HIP runtime only."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

STUB = "import sys, types; sys.modules['torch'] = types.ModuleType('torch')"  # without a spec, as mocked modules are
BROKEN = """import importlib.util, types
real = importlib.util.find_spec
importlib.util.find_spec = lambda n, *a: types.SimpleNamespace(origin={origin!r}) if n == 'torch' else real(n, *a)"""


def imports(first):
    code = first + "\nimport persistent_tile_scheduling_macro_amd as pg; print(pg.pgemm_status_string(0))"
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert "PGEMM_OK" in r.stdout


@pytest.mark.parametrize("first", [STUB, BROKEN.format(origin=None)])
def test_without_a_real_torch(first):
    imports(first)


def test_with_a_runtime_that_does_not_load(tmp_path):
    (tmp_path / "lib").mkdir()
    (tmp_path / "lib" / "libamdhip64.so").write_text("not a library")
    imports(BROKEN.format(origin=str(tmp_path / "__init__.py")))
