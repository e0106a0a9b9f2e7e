"""Row strides of layer norm's tensors, without a GPU: what the binding makes
of broadcast, sliced and single rows, and what the C entry takes of it.  A
stride that reaches past a tensor's storage must never be made up."""
import ctypes

import pytest
import torch

from channels_last_groupnorm_gb300 import block
from channels_last_groupnorm_gb300 import build as gnbuild
from channels_last_groupnorm_gb300 import gnsilu as gs

A, B, C, D, E, F, G, H = (0x1000000000 * n for n in range(1, 9))


@pytest.fixture(scope="module", autouse=True)
def built():
    gnbuild.build()


def views(cols):
    row, rows, cube = torch.arange(float(cols)), torch.arange(6.0 * cols).view(6, cols), torch.arange(20.0 * cols).view(4, 5, cols)
    return {
        "one row over many": row.expand(6, cols), "one row over two axes": row.expand(4, 5, cols),
        "rows over documents": rows[:5].expand(4, 5, cols), "a row of each document": rows[:4, None].expand(4, 5, cols),
        "a row over an axis and an axis of one": row.expand(6, 1, cols), "an axis of one and a row over an axis": row.expand(1, 6, cols),
        "one row": row[None], "one row, two axes": row[None, None], "one row of many": rows[3:4], "rows": rows, "cube": cube,
        "every other row": rows[::2], "heads of a projection": cube[:, 1:4], "a column slice": rows[:, : cols - 1], "a single axis": row,
    }


@pytest.mark.parametrize("name", list(views(8)))
@pytest.mark.parametrize("cols", [2, 8])
def test_row_strides_address_the_rows(name, cols):
    """Every row that the strides found address is the tensor's row."""
    t = views(cols)[name]
    packed = torch.empty(t.shape)
    found = block._row_strides(t.shape, (t.stride(), packed.stride()))
    assert found is not None
    inner, (outer, stride, _, _) = found
    flat, storage, width = t.reshape(-1, t.shape[-1]), t.storage_offset(), t.shape[-1]
    whole = torch.as_strided(t, (t.untyped_storage().nbytes() // 4,), (1,), 0)
    for n in range(len(flat)):
        at = storage + (n * stride if inner == 0 or inner >= len(flat) else n // inner * outer + n % inner * stride)
        assert at + width <= len(whole), "a row past the end of the storage"
        assert torch.equal(whole[at:at + width], flat[n]), n


# (every call is refused before it reaches a device: where the strides are
# accepted, by two outputs that lie on one another)
def norm(x, y, rows=16, inner=1 << 40, x_at=A, y_at=D):
    return gs.lib().gn_layer_norm(x_at, None, None, y_at, E, E, rows, 64, inner, (ctypes.c_int64 * 4)(*x, *y), 1e-6, 0, 0, None)


def norm_grad(dy, x, dx, rows=16, inner=1 << 40):
    return gs.lib().gn_layer_norm_backward(A, B, C, D, E, F, G, G, rows, 64, inner, (ctypes.c_int64 * 6)(*dy, *x, *dx), 0, 2,
                                           H, 1 << 30, None)


def test_outputs_are_not_broadcast_and_inputs_may_be():
    for y in ((0, 0), (0, 63), (-64, -64)):
        assert norm((0, 64), y) == gs.GN_ERR_SHAPE
        assert norm_grad((0, 64), (0, 64), y) == gs.GN_ERR_SHAPE
    assert norm((0, 64), (0, 64), inner=4) == gs.GN_ERR_SHAPE         # outer 0: groups of rows on one another
    assert norm_grad((256, 64), (256, 64), (0, 64), inner=4) == gs.GN_ERR_SHAPE
    for broadcast in ((0, 0), (0, 64), (64, 0)):
        assert norm(broadcast, (256, 64), inner=4) == gs.GN_ERR_ALIAS
        assert norm_grad(broadcast, broadcast, (256, 64), inner=4) == gs.GN_ERR_ALIAS
    # still refused: a broadcast row normed in place, rows that run into one another, groups of rows that do
    assert gs.lib().gn_layer_norm(A, None, None, A, E, F, 16, 64, 16, (ctypes.c_int64 * 4)(0, 0, 0, 64), 1e-6, 0, 0,
                                  None) == gs.GN_ERR_ALIAS
    assert norm((0, 1), (0, 64)) == gs.GN_ERR_SHAPE
    assert norm((63, 0), (256, 64), inner=4) == gs.GN_ERR_SHAPE
    assert norm((1, 64), (256, 64), inner=4) == gs.GN_ERR_SHAPE
