"""What gn_rope_nd refuses of sizes and output strides, without a GPU: the kernel
counts a token's pieces in 32 bits, and no two heads of its outputs may lie on
one another."""
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


def lies(token, head, tokens=3, heads=3, dim=64):
    """The status for outputs with these strides (refused in any case: the positions lie on an output)."""
    far = 1 << 20
    strides = (ctypes.c_int64 * 8)(far, dim, far, dim, token, head, token, head)
    return gs.lib().gn_rope_nd(A, B, C, D, strides, tokens, heads, heads, dim, C, 0, 1, (ctypes.c_int64 * 1)(64), 1e4, 1, 0, 0, None)


@pytest.mark.parametrize("token,head", [(64, 64), (128, 64), (64, 128), (100, 200), (128, 250), (65, 130), (191, 65), (0, 64), (64, 0)])
def test_output_heads_on_one_another(token, head):
    assert lies(token, head) == gs.GN_ERR_SHAPE


@pytest.mark.parametrize("token,head", [(192, 64), (64, 192), (256, 128), (80, 224), (192, 128), (224, 80), (128, 193)])
def test_output_heads_beside_one_another(token, head):
    spots = sorted(t * token + h * head for t in range(3) for h in range(3))
    assert all(b - a >= 64 for a, b in zip(spots, spots[1:])) == (lies(token, head) == gs.GN_ERR_ALIAS)
