"""The sizes under which the 4-bit products are compared with their references reach every kernel that the rule of
sizes chooses (csrc/w4_plan.h, compiled here for the host)."""
import os
import shutil
import subprocess
import tempfile

import pytest

from layers_shapes import GATED, LINEAR

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def kernels():
    cxx = shutil.which("g++") or shutil.which("c++") or shutil.which("hipcc")
    if cxx is None:
        pytest.skip("no C++ compiler")
    d = tempfile.mkdtemp(prefix="w4_plan_")
    exe = os.path.join(d, "w4_plan_print")
    subprocess.check_call([cxx, "-std=c++17", "-O1", "-I", os.path.join(os.path.dirname(HERE), "include"), "-o", exe,
                           os.path.join(HERE, "w4_plan_print.cpp")])

    def ask(sizes):
        text = "".join("%d %d %d %d\n" % s for s in sizes)
        lines = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.splitlines()
        assert len(lines) == len(sizes)
        words = [line.split() for line in lines]
        return [("few", *map(int, w[1:])) if w[0] == "few" else ("many", int(w[1]), w[2] == "1") for w in words]

    yield ask
    shutil.rmtree(d, ignore_errors=True)


@pytest.mark.parametrize("mats,table", [(1, LINEAR), (2, GATED)])
def test_each_size_reaches_the_kernel_that_it_stands_for(kernels, mats, table):
    got = kernels([(*s, mats) for s in table.values()])
    assert got == list(table), [(s, g, w) for s, g, w in zip(table.values(), got, table) if g != w]


@pytest.mark.parametrize("mats,table", [(1, LINEAR), (2, GATED)])
def test_no_kernel_is_left_out(kernels, mats, table):
    """All that the rule chooses over rows, outputs and inputs from small to large."""
    rows = [1, 4, 5, 9, 16, 17, 24, 32, 33, 48, 64, 65, 90, 128, 200, 300, 450, 576, 801, 1200, 1601, 2048, 4096, 8000]
    ns = [2 ** i * j // 4 for i in range(4, 16) for j in (4, 5, 6, 7)] + [1, 40, 1003, 6133, 12277, 49152, 151936]
    ks = [32, 416, 4096, 8064, 8192, 8224, 12288, 16384, 65536]
    sizes = [(r, n, k, mats) for r in rows for n in ns for k in ks]
    assert set(kernels(sizes)) == set(table)
