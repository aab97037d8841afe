"""Limits of the vocabulary-end calls: a size that no launch takes is refused as
unsupported before anything is enqueued (a launch takes fewer than 2^32 threads).
Runs without a GPU: the pointers are never dereferenced."""
import os

import pytest

from chunked_kl_loss_seq_amd import binding as B

pytestmark = pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="libckl.so not built")

EUNSUPPORTED = -5
G = 1 << 20  # an aligned address that is never used


@pytest.mark.parametrize("dt,d", [(0, 264), (0, 2880), (1, 136), (1, 1 << 20)])
@pytest.mark.parametrize("N", [(1 << 26) - 3, (1 << 26) - 1])
def test_embed_refuses_more_workgroups_than_a_launch_takes(dt, d, N):
    # rows of more than 32 chunks of 16 bytes: four rows a workgroup of 256 threads
    assert B.lib().ckl_embed(dt, G, G, 1.0, N, d, 1000, G, None) == EUNSUPPORTED
