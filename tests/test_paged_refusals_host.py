"""Refusals of the paged-attention C entries that would otherwise reach the GPU as bad addresses.  No GPU: every call is
refused for its argument alone (one that is not would be told apart by LI_ERR_CUDA)."""
import ctypes

import pytest
import torch

from sparse_attention_lightning_score_b200 import _lib

P, ODD = ctypes.c_void_p(256), ctypes.c_void_p(258)
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: an accepted call would be launched")


def _desc():
    return _lib.AttnDesc(2, 64, 2, 8, 16, 4, _lib.LI_DTYPE_E2M1, 0.1)


@pytest.mark.parametrize("which", ["block_table", "requests_of", "sel"])
def test_selection_refuses_misaligned_integers(which):
    at = dict(block_table=P, requests_of=P, sel=P)
    at[which] = ODD
    assert _lib.load().li_paged_sparse_attention(P, P, at["block_table"], at["requests_of"], at["sel"], 8, _desc(), P, P,
                                                 1 << 40, None) == _lib.LI_ERR_INVALID_ARG


@pytest.mark.parametrize("which", ["block_table", "requests_of", "positions"])
def test_window_refuses_misaligned_integers(which):
    at = dict(block_table=P, requests_of=P, positions=P)
    at[which] = ODD
    assert _lib.load().li_window_attention(P, P, at["block_table"], at["requests_of"], at["positions"], 8, 1, 64, _desc(), P,
                                           P, 1 << 40, None) == _lib.LI_ERR_INVALID_ARG
