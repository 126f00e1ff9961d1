"""Overlaps of the norm's and the beam search's arrays (tests/step_overlaps.cu): those that are
refused, and those that only look like overlaps."""

import os
import subprocess

import pytest

from tp_vocab_logits_gb300 import _build

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.mark.parametrize("kind", ["norm", "beam"])
def test_overlaps(kind, tmp_path):
    exe = str(tmp_path / kind)
    subprocess.run([_build.nvcc(), "-gencode", "arch=compute_103a,code=compute_103a", "-std=c++20",
                    f"-I{_build.INCLUDE}", f"-I{_build.CSRC}",
                    *(["-DBEAM"] if kind == "beam" else []),
                    os.path.join(HERE, "step_overlaps.cu"), "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.splitlines()
    ours = [x for x in out if " on device " not in x and x not in ("wait for device 1", "free")]
    assert ours == ["done"]
