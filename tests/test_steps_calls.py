"""The C entry points of the norm and the beam search on a fake CUDA runtime of two
devices (tests/step_calls.cu): which calls they refuse, which reach the kernels, and on
which device."""

import os
import subprocess

import pytest

from tp_vocab_logits_gb300 import _build, hg

HERE = os.path.dirname(os.path.abspath(__file__))
KERNELS = {"norm": ("rows", "grad"), "beam": ("select", "reorder")}


@pytest.fixture(scope="module", params=["norm", "beam"])
def events(request, tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("step_calls") / request.param)
    subprocess.run([_build.nvcc(), "-gencode", "arch=compute_103a,code=compute_103a", "-std=c++20",
                    f"-I{_build.INCLUDE}", f"-I{_build.CSRC}",
                    *(["-DBEAM"] if request.param == "beam" else []),
                    os.path.join(HERE, "step_calls.cu"), "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.splitlines()
    return request.param, out


def between(lines, first, last):
    return lines[lines.index(first) + 1:lines.index(last)]


def test_calls_run_on_the_handles_device_alone(events):
    kind, lines = events
    assert [x for x in lines[:2] if x != "wait for device 1"][0] == f"create {hg.HG_OK}"
    assert between(lines, "current 0", "current 1") == [f"{k} {hg.HG_ERR_ARG}"
                                                        for k in KERNELS[kind]]
    assert between(lines, "current 1", "refused") == [
        line for k in KERNELS[kind] for line in (f"{k} on device 1", f"{k} {hg.HG_OK}")]
    assert lines[-4:] == ["wait for device 1", "free", f"destroy {hg.HG_OK}", "current 0"]


def test_refusals(events):
    kind, lines = events
    first = "too many " + ("rows" if kind == "norm" else "items")
    refused = between(lines, "refused", first)
    assert len(refused) > 20
    assert [x for x in refused if not x.endswith(f" {hg.HG_ERR_ARG}")] == []
    assert between(lines, first, "served") == [f"{k} {hg.HG_ERR_ROWS}" for k in KERNELS[kind]]


def test_what_is_served(events):
    """Calls with nothing in them launch nothing, unless a gradient is to be cleared."""
    kind, lines = events
    served = between(lines, "served", "workspaces" if kind == "beam" else "end")
    ok = [x for x in served if " on device " not in x]
    assert [x for x in ok if not x.endswith(f" {hg.HG_OK}")] == []
    launched = [served[i + 1].rsplit(" ", 1)[0] for i, x in enumerate(served)
                if " on device 1" in x]
    want = {"norm": ["no rows", "in place", "one row, other distance", "8 bits", "in place"],
            "beam": ["all", "rows outside the layers", "nothing in it"]}[kind]
    assert launched == want


def test_workspaces_are_aligned(events):
    kind, lines = events
    if kind == "beam":
        made = [x for x in between(lines, "workspaces", "end") if x.startswith("aligned")]
        assert made == ["aligned 1"] * 9
