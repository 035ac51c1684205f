"""Paged-cache operators at edges: tensors that share a buffer.  Definitions: oracle.paged."""
import pytest
import torch

from sparse_attention_lightning_score_b200 import api
from sparse_attention_lightning_score_b200._lib import LI_OK
from tests.test_gpu_paged import DEV, _i32

pytestmark = pytest.mark.gpu


def test_rope_tensors_of_a_call_that_share_a_buffer():
    """The two halves of one fused buffer, both in place, turn as they do apart; a tensor that reads or writes what
    another one writes is refused, and nothing changes."""
    g = torch.Generator().manual_seed(4)
    pos, table = _i32([3, 70000, 12]), api.li_rope_table(64)
    fused = torch.randn(3, 4 * 128, generator=g).to(torch.bfloat16).to(DEV)
    old = fused.clone()
    halves = lambda b: [b[:, :256].view(3, 2, 128), b[:, 256:].view(3, 2, 128)]  # noqa: E731
    want = [api.li_rope(h, pos, table) for h in halves(old)]
    got = api.li_rope(halves(fused), pos, table, out=halves(fused))
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and api.li_get_last_error() == LI_OK
    fused.copy_(old)
    heads = fused.view(3, 4, 128)
    for xs in [[heads[:, :2], heads[:, 1:3]], [heads[:, :2], heads[:, :2]]]:    # the first one's second head; the same
        with pytest.raises(api.LiError):
            api.li_rope(xs, pos, table, out=xs)
    with pytest.raises(api.LiError):                  # reads past its half, into what the other writes
        api.li_rope([heads[:, 2:], heads[:, :3]], pos, table, out=[heads[:, 2:], torch.empty(3, 3, 128, device=DEV,
                                                                                             dtype=torch.bfloat16)])
    assert torch.equal(fused, old)
