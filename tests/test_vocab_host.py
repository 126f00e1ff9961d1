"""Refusals of the vocabulary operators that need no GPU: the C entry points'
checks before any device work, and the binding's checks of its tensors."""

import ctypes

import pytest
import torch

from tp_vocab_logits_gb300 import _build, hg


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return hg.load()


ALL = 15  # every HG_VOCAB_* bit


@pytest.mark.parametrize("args", [
    (0, 64, 0, 64, 4, 0, ALL, 0),            # no shard
    (hg.HG_MAX_TP + 1, 64, 0, 64, 4, 0, ALL, 0),
    (2, 0, 0, 64, 4, 0, ALL, 0),             # empty shards
    (2, 64, 129, 64, 4, 0, ALL, 0),          # vocabulary beyond the shards
    (2, 64, -1, 64, 4, 0, ALL, 0),
    (2, 64, 0, 0, 4, 0, ALL, 0),             # no width
    (2, 64, 0, 64, 0, 0, ALL, 0),            # no rows
    (2, 64, 0, 64, 4, 3, ALL, 0),            # unknown type
    (2, 64, 0, 64, 4, 0, 0, 0),              # no operator
    (2, 64, 0, 64, 4, 0, 16, 0),             # unknown operator
    (2, 64, 0, 68, 4, 0, 4, 0),              # the loss needs K % 8 == 0
    (2, 64, 0, 64, 4, 2, 8, 0),              # the loss is not made for fp32
    (32, 1 << 30, 0, 64, 4, 0, 1, 0),        # columns beyond int
    (1, 64, 0, 64, 1 << 30, 0, 1, 0),        # rows beyond int
])
def test_create_refuses(lib, args):
    out = ctypes.c_void_p(1)
    assert lib.hg_vocab_create(*args, ctypes.byref(out)) == hg.HG_ERR_ARG
    assert out.value is None


def test_calls_refuse_a_null_handle(lib):
    assert lib.hg_vocab_create(2, 64, 0, 64, 4, 0, ALL, 0, None) == hg.HG_ERR_ARG
    assert lib.hg_vocab_destroy(None) == hg.HG_OK
    assert lib.hg_vocab_workspace_bytes(None) == 0
    assert lib.hg_vocab_sync(None, None) == hg.HG_ERR_ARG
    assert lib.hg_vocab_embed(None, None, 8, 0, None, 1.0, None, 64, None) == hg.HG_ERR_ARG
    assert lib.hg_vocab_embed_grad(None, None, 8, 0, None, 64, None, 1.0, 0, None) == hg.HG_ERR_ARG
    assert lib.hg_vocab_loss(None, None, 64, None, None, 8, 0, 1.0, None, None,
                             None) == hg.HG_ERR_ARG
    assert lib.hg_vocab_loss_grad(None, None, 64, None, None, 8, None, None, 0, 1.0, None, 64,
                                  None, 0, None) == hg.HG_ERR_ARG


def test_binding_refuses_before_the_library():
    h = hg.VocabHandle(0, 2, 8, 16, 8, 4, torch.bfloat16)  # never handed to the library here
    ids = torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError, match="tokens"):
        hg.hg_vocab_embed(h, ids, [], torch.zeros(2, 8))
    with pytest.raises(ValueError, match="targets"):
        hg.hg_vocab_loss(h, torch.zeros(2, 8), [], ids, None, None)
    with pytest.raises(ValueError, match="dtype"):
        hg.hg_vocab_create(2, 8, 8, 4, dtype=torch.float64)
    with pytest.raises(ValueError, match="unknown operator"):
        hg.hg_vocab_create(2, 8, 8, 4, ops=("gather",))
