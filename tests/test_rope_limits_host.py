"""How many channels of a token gn_rope_nd takes, without a GPU: the kernel
counts a token's pieces in 32 bits."""
import ctypes

import pytest

from channels_last_groupnorm_gb300 import build as gnbuild
from channels_last_groupnorm_gb300 import gnsilu as gs

A, B, C, D = (0x10000000000 * n for n in range(1, 5))


@pytest.fixture(scope="module", autouse=True)
def built():
    gnbuild.build()


def rope(heads, kv_heads, dim, interleaved=1):
    # (refused in any case, before it reaches a device: the positions lie on an output)
    strides = (ctypes.c_int64 * 8)(heads * dim, dim, kv_heads * dim, dim, heads * dim, dim, kv_heads * dim, dim)
    return gs.lib().gn_rope_nd(A, B, C, D, strides, 3, heads, kv_heads, dim, C, 0, 1, (ctypes.c_int64 * 1)(64), 1e4, interleaved,
                               0, 0, None)


@pytest.mark.parametrize("heads,kv_heads,dim", [(65536, 65536, 65536), (65536, 1, 65536), (1, 65536, 65536), (32768, 1, 32768),
                                                (16384, 16385, 32768)])
@pytest.mark.parametrize("interleaved", [0, 1])
def test_more_pieces_than_are_counted(heads, kv_heads, dim, interleaved):
    assert rope(heads, kv_heads, dim, interleaved) == gs.GN_ERR_SHAPE


@pytest.mark.parametrize("heads,kv_heads,dim", [(16384, 16384, 32768), (65536, 65536, 8192), (8191, 8193, 65536), (48, 8, 128)])
def test_as_many_as_are_counted(heads, kv_heads, dim):
    assert rope(heads, kv_heads, dim) == gs.GN_ERR_ALIAS
