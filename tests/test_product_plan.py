"""The integer products' choice of kernel (product_plan.hpp, compiled here for the host): some size
takes every kernel that is built, and every size one of them."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
QUERY = os.path.join(ROOT, "tests", "host", "product_plan_query.cpp")


@pytest.fixture(scope="module")
def chosen(tmp_path_factory):
    """sizes -> (kernels built, the one that each (M, N) takes)"""
    cxx = shutil.which("g++") or shutil.which("clang++")
    if cxx is None:
        pytest.skip("no host compiler")
    exe = str(tmp_path_factory.mktemp("plan") / "query")
    subprocess.run([cxx, "-O1", "-std=c++17", QUERY, "-o", exe], check=True, capture_output=True)

    def ask(sizes):
        r = subprocess.run([exe], input="".join("%d %d\n" % s for s in sizes), check=True,
                           capture_output=True, text=True)
        count, *kinds = map(int, r.stdout.split())
        assert len(kinds) == len(sizes)
        return count, kinds
    return ask


def test_every_kernel_has_its_sizes(chosen):
    sides = sorted({v for e in range(25) for v in (2 ** e - 1, 2 ** e, 2 ** e + 1, 2 ** e * 5 // 4) if v > 0})
    sides += [14400, 25100, 2 ** 31 - 1]
    count, kinds = chosen([(m, n) for m in sides for n in sides])
    assert set(kinds) == set(range(count))


def test_gpu_cases_reach_every_kernel(chosen):
    """The sizes that tests/test_gpu_product_kernels.py runs."""
    from test_gpu_product_kernels import CASES
    count, kinds = chosen([(m, n) for m, n, _ in CASES])
    assert set(kinds) == set(range(count))
