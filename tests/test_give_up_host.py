"""The give-up decision of a row team (csrc/give_up.h) over every interleaving of its
warps, on the host: no interleaving leaves a warp at a barrier that another will not
reach, and all warps leave at the same row. A single flag for all rows fails it.
"""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "memory_bound_normalization_fwd_gb300", "csrc")
GXX = shutil.which("g++")

pytestmark = pytest.mark.skipif(GXX is None, reason="no g++")


def _model(tmp, header_dir):
    exe = os.path.join(tmp, "give_up_model")
    subprocess.run([GXX, "-std=c++17", "-O2", "-I", header_dir, os.path.join(HERE, "give_up_model.cpp"), "-o", exe],
                   check=True)
    return exe


@pytest.fixture(scope="module")
def model(tmp_path_factory):
    return _model(str(tmp_path_factory.mktemp("give_up")), CSRC)


@pytest.mark.parametrize("warps,rows", [(1, 3), (2, 2), (2, 5), (3, 4)])
@pytest.mark.parametrize("marks_the_next_row", [0, 1])
def test_every_interleaving_ends(model, warps, rows, marks_the_next_row):
    p = subprocess.run([model, str(warps), str(rows), str(marks_the_next_row)], capture_output=True, text=True)
    assert p.returncode == 0, p.stdout + p.stderr


def test_one_flag_for_all_rows_is_found_out(tmp_path):
    # The model's own check: with one flag a warp leaves a row that another has passed.
    text = open(os.path.join(CSRC, "give_up.h")).read()
    assert text.count("late[row & 1]") == 2
    (tmp_path / "give_up.h").write_text(text.replace("late[row & 1]", "late[0]"))
    p = subprocess.run([_model(str(tmp_path), str(tmp_path)), "2", "2", "0"], capture_output=True, text=True)
    assert p.returncode == 1 and "hangs" in p.stdout
