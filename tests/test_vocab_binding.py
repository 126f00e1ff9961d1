"""The binding's checks of the vocabulary operators' tensors, without a device:
stand-ins for CUDA tensors, and entry points that record that they were reached."""

import ctypes

import pytest
import torch

from tp_vocab_logits_gb300 import _build, hg


class Tensor:
    """What the binding asks of a CUDA tensor."""

    is_cuda = True

    def __init__(self, shape, dtype, device=1):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, torch.device("cuda", device)

    def dim(self):
        return len(self.shape)

    def stride(self, i=None):
        s = torch.empty(self.shape, device="meta").stride()
        return s if i is None else s[i]

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 4096

    def get_device(self):
        return self.device.index


@pytest.fixture
def reached():
    """Names of the entry points that calls reach."""
    _build.build()
    names, keep = [], []
    mod = hg._vocab_call()

    def entry(name):
        def record(*_):
            names.append(name)
            return hg.HG_OK
        # The library's arguments are of no interest here; none are read.
        keep.append(ctypes.CFUNCTYPE(ctypes.c_int)(record))
        return ctypes.cast(keep[-1], ctypes.c_void_p).value

    mod.bind_vocab(entry("embed"), entry("embed_grad"), entry("loss"), entry("loss_grad"),
                   torch.int32, torch.int64, torch.float32, lambda device: 0)
    yield names
    hg._VOCAB_CALL = None  # bound to the library again by the next call


TP, W, K, N = 2, 8, 16, 3


def arguments(call):
    """The call's tensors by name, all on device 1."""
    bf16 = torch.bfloat16

    def shards():
        return [Tensor((W, K), bf16) for _ in range(TP)]

    ids, rows = Tensor((N,), torch.int64), Tensor((N, K), bf16)

    def floats():
        return Tensor((N,), torch.float32)

    return {"embed": {"tokens": ids, "table": shards(), "out": rows},
            "embed_grad": {"tokens": ids, "grad_out": rows, "grad_table": shards()},
            "loss": {"hidden": rows, "weight": shards(), "targets": ids, "loss": floats(),
                     "lse": floats()},
            "loss_grad": {"hidden": rows, "weight": shards(), "targets": ids, "lse": floats(),
                          "grad_loss": floats(), "grad_hidden": Tensor((N, K), bf16),
                          "grad_weight": shards()}}[call]


CALLS = {"embed": hg.hg_vocab_embed, "embed_grad": hg.hg_vocab_embed_grad,
         "loss": hg.hg_vocab_loss, "loss_grad": hg.hg_vocab_loss_grad}


def handle(device):
    h = hg.VocabHandle(0, TP, W, TP * W, K, N, torch.bfloat16)
    h.device = torch.device("cuda", device)
    if hasattr(h, "_describe"):
        h._describe()
    return h


@pytest.mark.parametrize("call", CALLS)
def test_tensors_of_the_handles_device_are_served(reached, call):
    CALLS[call](handle(1), **arguments(call))
    assert reached == [call]


@pytest.mark.parametrize("call,name", [(c, n) for c in CALLS for n in arguments(c)])
def test_a_tensor_of_another_device_is_refused(reached, call, name):
    args = arguments(call)
    t = args[name][-1] if isinstance(args[name], list) else args[name]
    t.device = torch.device("cuda", 0)
    with pytest.raises(ValueError, match=f"{name}: need a tensor on cuda:1, got one on cuda:0"):
        CALLS[call](handle(1), **args)
    assert reached == []


@pytest.mark.parametrize("call", CALLS)
def test_ids_without_a_length_are_named(reached, call):
    """A scalar of ids: the binding says so before it asks for its length."""
    args = arguments(call)
    what = "tokens" if "tokens" in args else "targets"
    args[what] = Tensor((), torch.int64)
    with pytest.raises(ValueError, match=f"{what}: need a contiguous 1-D"):
        CALLS[call](handle(1), **args)
    assert reached == []
