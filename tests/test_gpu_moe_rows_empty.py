"""Rows by expert and back without tokens, without rows, or with all slots dropped."""
import pytest
import torch

from nvfp4_w4a4_moe_permute_gb300 import minite as M

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
H, K = 24, 3


def tensors(T, m, dtype, dest):
    return (torch.ones(T, H, dtype=dtype, device=DEV), torch.full((m, H), 2.0, dtype=dtype, device=DEV),
            torch.full((T, K), dest, dtype=I32, device=DEV), torch.ones(T, K, device=DEV))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("m", [0, 5])
def test_no_tokens(dtype, m):
    dy, rows, dest, w = tensors(0, m, dtype, -1)
    assert M.combine_rows(rows, dest, w).shape == (0, H)
    drows, dw = M.combine_rows_backward(dy, rows, dest, w, out=rows)
    assert drows is rows and (rows == 2).all() and dw.shape == (0, K)
    assert M.combine_rows_backward(dy, None, dest, w, out=rows)[1] is None
    assert M.spread_rows(dy, dest, rows) is rows and (rows == 2).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [1, 7, 900])
def test_no_rows(dtype, T):
    """A rank that has received nothing: all slots are skipped, forward and backward."""
    dy, rows, dest, w = tensors(T, 0, dtype, -1)
    status = torch.zeros(1, dtype=I32, device=DEV)
    y = M.combine_rows(rows, dest, w, status=status)
    assert y.shape == (T, H) and not y.any()
    for out in (None, rows, torch.empty(0, H, dtype=dtype, device=DEV)):
        drows, dw = M.combine_rows_backward(dy, rows, dest, w, out=out, status=status)
        assert drows.shape == (0, H) and dw.shape == (T, K) and not dw.any()
    assert M.combine_rows_backward(dy, None, dest, w, out=rows, status=status)[1] is None
    assert not M.permute_rows_backward(rows, dest, status=status).any()
    M.spread_rows(dy, dest, rows, status=status)
    assert int(status) == 0


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_that_are_not_there_are_reported(dtype):
    dy, rows, dest, w = tensors(6, 0, dtype, -1)
    dest[4, 1] = 0                            # the first row of none
    for call in (lambda s: M.combine_rows(rows, dest, w, status=s),
                 lambda s: M.combine_rows_backward(dy, rows, dest, w, status=s)[1],
                 lambda s: M.combine_rows_backward(dy, None, dest, w, out=rows, status=s)[0],
                 lambda s: M.spread_rows(dy, dest, rows, status=s)):
        status = torch.zeros(1, dtype=I32, device=DEV)
        assert not call(status).any() and int(status) == 1 << M.ERR_BAD_ROUTING


@pytest.mark.parametrize("dtype", [BF, F32])
def test_every_slot_dropped(dtype):
    """The way of an empty rank through all calls, from the sort on."""
    x, ids, w = torch.randn(50, H, device=DEV).to(dtype), torch.full((50, K), -1, dtype=I32, device=DEV), torch.ones(50, K, device=DEV)
    r = M.permute_rows(x, ids, 4)
    n = int(r["offsets"][-1])
    assert n == 0 and (r["dest_row"] == -1).all() and (r["perm_src"] == -1).all()
    own = r["rows"][:n]
    assert not M.combine_rows(own, r["dest_row"], w).any()
    drows, dw = M.combine_rows_backward(x, own, r["dest_row"], w)
    assert drows.shape == (0, H) and not dw.any()
    assert not M.permute_rows_backward(drows, r["dest_row"]).any()
