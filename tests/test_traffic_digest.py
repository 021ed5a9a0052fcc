"""CPU: the digest that ties HBM counters to code follows the kernels and the launch planner, and nothing else."""
import importlib.util
import os
import shutil

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def bench(monkeypatch, tmp_path):
    spec = importlib.util.spec_from_file_location("bench_under_test", os.path.join(ROOT, "bench.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    monkeypatch.setattr(b, "CSRC", shutil.copytree(b.CSRC, tmp_path / "csrc"))
    return b


def change(bench, name, text):
    with open(os.path.join(bench.CSRC, name), "a", encoding="utf-8") as f:
        f.write(text)


@pytest.mark.parametrize("name", ["context.h", "launch.h", "moe.hip", "moe_rows.h", "grouped.hip", "grouped_pp.h", "w4.h", "binding.cpp"])
def test_other_sources_leave_it(bench, name):
    before = bench.source_digest()
    change(bench, name, "\nint another;\n")
    assert bench.source_digest() == before


@pytest.mark.parametrize("name", ["gemm_fast.h", "gemm_pingpong.h", "gemm_generic.h", "device_common.h", "kernels.h", "pgemm.hip",
                                  "kernels_f16.hip"])
def test_kernels_and_planner_change_it_and_comments_do_not(bench, name):
    before = bench.source_digest()
    change(bench, name, "\n// a remark\n/* another */\n")
    assert bench.source_digest() == before
    change(bench, name, "\nint another;\n")
    assert bench.source_digest() != before
