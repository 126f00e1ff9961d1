"""The vocabulary operators' host side with two devices, on a fake CUDA runtime
(tests/vocab_devices.cu): a handle made on device 1, then used and freed."""

import os
import subprocess

import pytest

from tp_vocab_logits_gb300 import _build, hg

HERE = os.path.dirname(os.path.abspath(__file__))
CALLS = ("embed", "embed_grad", "loss", "loss_grad")


@pytest.fixture(scope="module")
def events(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("vocab_devices") / "devices")
    subprocess.run([_build.nvcc(), "-gencode", "arch=compute_103a,code=compute_103a", "-std=c++17",
                    f"-I{_build.INCLUDE}", f"-I{_build.CSRC}",
                    os.path.join(HERE, "vocab_devices.cu"), "-o", exe], check=True)
    return subprocess.run([exe], capture_output=True, text=True, check=True).stdout.splitlines()


def test_calls_run_on_the_handles_device_alone(events):
    want = ["wait for device 1", f"create {hg.HG_OK}", "current 0"]
    want += [f"{c} {hg.HG_ERR_ARG}" for c in CALLS]
    want += ["current 1"]
    for c in CALLS:
        want += [f"{c} on device 1", f"{c} {hg.HG_OK}"]
    assert events[:len(want)] == want


def test_destroy_waits_for_the_handles_device(events):
    """And leaves the caller's current."""
    assert events[-4:] == ["wait for device 1", "free", f"destroy {hg.HG_OK}", "current 0"]
