"""dH's tiles stay within what their copies of G can address, on the CPU: the library's own choices, for the loss and for
the log-probabilities from hidden states.

A tile addresses the gradient's tiles by 32-bit byte offsets from its first row, in a buffer of 2^31 - 16 bytes; blocks
of 64 rows of V ids lie ceil(V / 64) x 64 x 64 elements apart, and the last block's own 64 x 64 elements count too."""
import ctypes

import pytest

from chunked_kl_loss_seq_amd import binding

REACH = 2 ** 31 - 16
EDGES = (256, 128, 64)
MOST = 1 << 26


def span(esz, rows, V, edge):
    blocks = (min(rows, edge) + 63) // 64
    return ((blocks - 1) * -(-V // 64) * 4096 + 4096) * esz


def head_edge(dt, rows, d, V):
    f = binding.lib()._ZN3ckl13head_dh_splitENS_5DtypeElll
    f.restype, f.argtypes = ctypes.c_uint64, [ctypes.c_int] + [ctypes.c_int64] * 3
    return EDGES[f(dt, rows, d, V) & 0xFFFFFFFF]


def loss_edge(dt, rows, V):
    f = binding.lib()._ZN3ckl12dh_tile_rowsENS_5DtypeEll
    f.restype, f.argtypes = ctypes.c_int, [ctypes.c_int] + [ctypes.c_int64] * 2
    return f(dt, rows, V)


VS = [1, 1000, 201088, 2796160, 2796161, 5592320, 5592321, 6_000_000, 8388544, 8388545, 8388608, 11_200_000, 16777152,
      16777216, 33_554_432, MOST]


@pytest.mark.parametrize("dt,esz", [(0, 2), (1, 4)])
@pytest.mark.parametrize("V", VS)
def test_tiles_reach_their_rows(dt, esz, V):
    for rows in (1, 64, 65, 128, 129, 192, 193, 256, 300, 4096):
        edge = loss_edge(dt, rows, V)
        assert span(esz, rows, V, edge) <= REACH, (rows, edge)
        # and the most rows that do: the tiles of before wherever those reach
        assert edge == max(e for e in EDGES if span(esz, rows, V, e) <= REACH)
        for d in (8, 64, 512, 1024, 2048, 8192):
            e = head_edge(dt, rows, d, V)
            assert span(esz, rows, V, e) <= REACH, (rows, d, e)
