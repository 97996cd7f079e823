"""The split of attention's work, as far as it can run without a GPU: its host
parts compiled for the host."""

from __future__ import annotations

import os
import shutil
import subprocess

import pytest

from activation_sparse_predictor_amd import build as B


def host_program(tmp_path, body):
    if not os.path.exists(B.HIPCC) and shutil.which("hipcc") is None:
        pytest.skip("hipcc not available")
    src, exe = tmp_path / "plan.hip", tmp_path / "plan"
    src.write_text('#include <cstdio>\n#include "attend.hpp"\nusing namespace pi;\nint main() {\n' + body + "\n}\n")
    flags = [f for f in B.CFLAGS if f != "-fPIC"]
    res = subprocess.run([B.HIPCC, *flags, str(src), "-o", str(exe)], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-2000:]
    return subprocess.run([str(exe)], capture_output=True, text=True, check=True, timeout=60).stdout.split()


def test_pieces_stay_in_range(tmp_path):
    """Whatever the lengths add up to (row ranges that overlap, tables that repeat
    pages), a piece is between the least and the longest context's tiles."""
    wants = ["0.0f", "3.9f", "4.0f", "100.7f", "16777214.0f", "16777216.0f", "2147483520.0f", "2147483648.0f", "3.6e16f"]
    out = host_program(tmp_path, "\n".join(f'printf("%d\\n", att_piece({w}, 4));' for w in wants))
    assert [int(v) for v in out] == [4, 4, 5, 101, 16777215] + [16777216] * 4
