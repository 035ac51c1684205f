"""Order of a kernel's first steps, by reading its source: nothing that a GPU run could show without hanging."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_attention_lightning_score_b200",
                    "csrc")


def kernels():
    """(file, body) of every __global__ function, from its signature to the next one."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        src = re.sub(r"//[^\n]*", "", open(path).read())
        at = [m.start() for m in re.finditer(r"__global__", src)]
        for a, b in zip(at, at[1:] + [len(src)]):
            yield os.path.basename(path), src[a:b]


WAITING = [(f, k) for f, k in kernels() if "tmem_alloc(" in k and "pdl_wait()" in k]
SCORERS = {"score_stream.cu", "score_latent8.cu"}    # (asserted in the source never to lack tensor memory)


def test_kernels_that_wait_and_hold_tensor_memory_are_found():
    assert {f for f, _ in WAITING} >= {"paged_attn.cu", "sparse_attn.cu"} | SCORERS


@pytest.mark.parametrize("name,kernel", WAITING, ids=[f for f, _ in WAITING])
def test_tensor_memory_is_taken_behind_the_wait(name, kernel):
    """A kernel that holds tensor memory while it waits for the kernels before it could hold what one of them still
    needs: the allocation stands behind the wait, and no dependent is let in before it."""
    if name in SCORERS:
        src = open(os.path.join(CSRC, name)).read()
        assert re.search(r"static_assert\([^;]*>= kScorerSmem &&[^;]*<= kScorerTmem", src)
        return
    held = kernel.index("tmem_alloc(")
    assert held > kernel.index("pdl_wait()") and "pdl_trigger()" not in kernel[:held]
