"""CPU: one HIP runtime in the process, whichever of torch and the package is imported first."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("imports", ["import torch; from persistent_tile_scheduling_macro_amd import moe",
                                     "from persistent_tile_scheduling_macro_amd import moe, w4",
                                     "import persistent_tile_scheduling_macro_amd; import torch"])
def test_one_hip_runtime(imports):
    code = imports + "; print(len({l.split()[-1] for l in open('/proc/self/maps') if 'libamdhip64' in l}))"
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert r.stdout.split()[-1] == "1", r.stdout
