"""GB300-native vocab-parallel LM-head logits gather on a two-parity Lamport
mailbox, for TP virtual ranks on one GPU, with the operators at both ends of the
sharded vocabulary: embedding, softmax cross entropy, and their gradients; the norm
in front of the head with its gradient, and a beam search's step behind it.

The library is libhg.so (C ABI in include/hg.h, CUDA kernels for sm_103a);
``hg`` is its Python binding and ``synth`` makes seeded synthetic inputs.
"""

from . import hg, synth  # noqa: F401
from .hg import (GatherCall, HGError, Handle, hg_beam_create, hg_beam_destroy,  # noqa: F401
                 hg_beam_reorder, hg_beam_select, hg_create, hg_debug_skip_push,
                 hg_destroy, hg_gather, hg_gather_fused, hg_gather_host, hg_gather_static,
                 hg_gather_stats, hg_launch_shape, hg_mailbox, hg_norm_create,
                 hg_norm_destroy, hg_norm_rows, hg_norm_rows_grad, hg_parity, hg_rearm,
                 hg_stock_gather, hg_sync, hg_vocab_create, hg_vocab_destroy, hg_vocab_embed,
                 hg_vocab_embed_grad, hg_vocab_loss, hg_vocab_loss_grad, hg_vocab_sync,
                 mailbox_words, new_row_stats, unpack_row_stats)
