"""CPU: the library builds where torch for ROCm is missing; the torch binding is then left out, with a word about it."""
import importlib.util
import os
import types

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def build(monkeypatch, tmp_path):
    """The build script with its compilers replaced by ones that write empty files, in a folder of its own."""
    spec = importlib.util.spec_from_file_location("build_under_test",
                                                  os.path.join(ROOT, "persistent_tile_scheduling_macro_amd", "build.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    for name, value in (("LIB", "lib.so"), ("OPS", "ops.so"), ("BUILD_DIR", "build"), ("RESOURCES", "resources.txt")):
        monkeypatch.setattr(b, name, str(tmp_path / value))
    monkeypatch.setattr(b, "_compile", lambda src: (src + ".o", []))
    b.commands = []

    def run(cmd, **_):
        b.commands.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(b.subprocess, "run", run)
    return b


def fake_torch(monkeypatch, b, origin):
    real = importlib.util.find_spec
    found = None if origin is None else types.SimpleNamespace(origin=str(origin))
    monkeypatch.setattr(b.importlib.util, "find_spec", lambda name, *a: found if name == "torch" else real(name, *a))


def torch_tree(tmp_path, *files):
    root = tmp_path / "torch"
    for f in ("__init__.py",) + files:
        (root / f).parent.mkdir(parents=True, exist_ok=True)
        (root / f).touch()
    return root / "__init__.py"


ROCM = ("lib/libc10_hip.so", "lib/libtorch_hip.so", "include/c10/hip/HIPStream.h", "include/ATen/core/Tensor.h")


@pytest.mark.parametrize("files", [None, (), ("lib/libc10_cuda.so",), ROCM[:2]])
def test_the_library_builds_without(build, monkeypatch, tmp_path, capsys, files):
    fake_torch(monkeypatch, build, None if files is None else torch_tree(tmp_path, *files))
    open(build.OPS, "w").close()  # one that an earlier build linked to an earlier library
    assert build.build(verbose=True) == build.LIB and os.path.exists(build.LIB)
    assert not os.path.exists(build.OPS) and len(build.commands) == 1
    assert "torch for ROCm" in capsys.readouterr().out


def test_the_binding_is_built_with(build, monkeypatch, tmp_path, capsys):
    fake_torch(monkeypatch, build, torch_tree(tmp_path, *ROCM))
    assert build.build(verbose=True) == build.LIB
    assert os.path.exists(build.LIB) and os.path.exists(build.OPS) and len(build.commands) == 2
    assert "torch for ROCm" not in capsys.readouterr().out
