"""What a group of the residual norm has on its way to shared memory, checked on the host: `native/row_slots_check.cc`
runs the kernel's own bookkeeping (csrc/row_slots.cuh) for every row whose arrival may be given up."""
import os
import shutil
import subprocess

import pytest

from tests.conftest import ROOT

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
CSRC = os.path.join(ROOT, "nvfp4_block_scaled_gather_gb300", "csrc")


def run(tmp_path, *defines):
    exe = tmp_path / ("check" + "".join(defines))
    subprocess.run(["g++", "-std=c++17", "-O1", *[f"-D{d}" for d in defines], "-I", CSRC, "-o", str(exe),
                    os.path.join(ROOT, "tests", "native", "row_slots_check.cc")], check=True)
    return subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)


def test_a_group_that_gives_up_ends_with_nothing_in_flight(tmp_path):
    done = run(tmp_path)
    assert done.returncode == 0 and done.stdout.endswith(" 0 failures\n"), done.stdout


def test_the_check_sees_groups_that_go_on(tmp_path):
    """Going on after a wait that gave up asks for a slot that is in use."""
    done = run(tmp_path, "WITHOUT_LEAVING")
    assert done.returncode == 1 and "a slot that is in use" in done.stdout and "in flight at the end" in done.stdout, done.stdout


def test_the_kernel_keeps_its_books_there():
    source = open(os.path.join(CSRC, "residual_norm.cu")).read()
    for call in ("on_way.start(first, bring)", "on_way.again(row, bring)", "on_way.leave(row,", "on_way.next()"):
        assert source.count(call) == 1, call
