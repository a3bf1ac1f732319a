"""Rows by expert, the gradient norm and the verification of drafts refuse bad
arguments on the host, before anything is enqueued (no GPU: every call here fails
its checks first, or has nothing to do)."""
import ctypes
import math

import numpy as np
import pytest
import torch

from nvfp4_w4a4_moe_permute_gb300 import build as B
from nvfp4_w4a4_moe_permute_gb300 import minite as M
from test_operand_devices import On, calls, refused_elsewhere   # noqa: F401

INVALID, SHAPE = 1, 2
FAKE = ctypes.c_void_p(1 << 12)     # never dereferenced
ODD = ctypes.c_void_p((1 << 12) + 2)
ODDEST = ctypes.c_void_p((1 << 12) + 1)
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module")
def lib():
    B.build()
    return M.load()


PERMUTE = dict(x=FAKE, dtype=0, xs=64, ids=FAKE, T=100000, H=64, E=8, k=2, rows=FAKE, rs=64, off=FAKE, src=FAKE,
               dest=FAKE, ws=FAKE, wsn=1 << 30, status=None, stream=None)


@pytest.mark.parametrize("change,rc", [
    (dict(x=None), INVALID), (dict(ids=None), INVALID), (dict(rows=None), INVALID), (dict(off=None), INVALID),
    (dict(src=None), INVALID), (dict(dest=None), INVALID), (dict(ws=None), INVALID), (dict(wsn=64), INVALID),
    (dict(dtype=2), INVALID), (dict(x=ODDEST), INVALID), (dict(dtype=1, x=ODD), INVALID), (dict(ids=ODD), INVALID),
    (dict(ws=ODD), INVALID), (dict(status=ODD), INVALID), (dict(T=-1), SHAPE), (dict(T=1 << 31), SHAPE),
    (dict(T=1 << 30), SHAPE), (dict(H=0), SHAPE), (dict(H=(1 << 24) + 1, xs=1 << 25, rs=1 << 25), SHAPE),
    (dict(E=0), SHAPE), (dict(E=1025), SHAPE), (dict(k=0), SHAPE), (dict(k=33), SHAPE), (dict(xs=63), SHAPE),
    (dict(rs=63), SHAPE), (dict(rs=1 << 31), SHAPE)])
def test_permute_rows(lib, change, rc):
    assert lib.minite_moe_permute_rows(*{**PERMUTE, **change}.values()) == rc


SPREAD = dict(x=FAKE, dtype=0, xs=64, dest=FAKE, T=8, M=16, H=64, k=2, rows=FAKE, rs=64, status=None, stream=None)
COMBINE = dict(rows=FAKE, dtype=0, rs=64, dest=FAKE, w=FAKE, T=8, M=16, H=64, k=2, y=FAKE, ys=64, status=None,
               stream=None)
BACK = dict(dy=FAKE, dtype=0, dys=64, rows=FAKE, rs=64, dest=FAKE, w=FAKE, T=8, M=16, H=64, k=2,
            drows=ctypes.c_void_p(1 << 20), drs=64, dw=FAKE, status=None, stream=None)


@pytest.mark.parametrize("change,rc", [
    (dict(x=None), INVALID), (dict(dest=None), INVALID), (dict(rows=None), INVALID), (dict(dtype=7), INVALID),
    (dict(rows=ODDEST), INVALID), (dict(M=1 << 31), SHAPE), (dict(M=-1), SHAPE), (dict(xs=5), SHAPE),
    (dict(k=40), SHAPE), (dict(T=0), 0), (dict(M=0), 0)])
def test_spread_rows(lib, change, rc):
    assert lib.minite_moe_spread_rows(*{**SPREAD, **change}.values()) == rc


@pytest.mark.parametrize("change,rc", [
    (dict(rows=None), INVALID), (dict(dest=None), INVALID), (dict(y=None), INVALID), (dict(dtype=-1), INVALID),
    (dict(w=ODD), INVALID), (dict(y=ODDEST), INVALID), (dict(dtype=1, rows=ODD), INVALID), (dict(rs=10), SHAPE),
    (dict(ys=10), SHAPE), (dict(T=-3), SHAPE), (dict(k=0), SHAPE), (dict(T=0), 0)])
def test_combine_rows(lib, change, rc):
    assert lib.minite_moe_combine_rows(*{**COMBINE, **change}.values()) == rc


@pytest.mark.parametrize("change,rc", [
    (dict(dy=None), INVALID), (dict(dest=None), INVALID), (dict(w=None), INVALID), (dict(drows=None), INVALID),
    (dict(rows=None), INVALID), (dict(dw=None), INVALID), (dict(dw=ODD), INVALID), (dict(drows=FAKE, drs=72), INVALID),
    (dict(dys=60), SHAPE), (dict(rs=60), SHAPE), (dict(drs=60), SHAPE), (dict(T=0), 0)])
def test_combine_rows_backward(lib, change, rc):
    assert lib.minite_moe_combine_rows_backward(*{**BACK, **change}.values()) == rc


GRAD_TENSOR = np.dtype([("grad", "u8"), ("out", "u8"), ("n", "i8"), ("grad_dtype", "i4"), ("out_dtype", "i4")])


def table(count=3, **change):
    t = np.zeros(count, dtype=GRAD_TENSOR)
    t["grad"] = t["out"] = 1 << 12
    t["n"] = 1 << 20
    for k, v in change.items():
        t[k][-1] = v
    return t


def norm(lib, tensors, **change):
    a = dict(t=tensors.ctypes.data, n=len(tensors), order=0, max_norm=1.0, norm=FAKE, factor=FAKE, ws=FAKE, wsn=1 << 20, stream=None)
    return lib.minite_grad_norm(*{**a, **change}.values())


def test_grad_norm(lib):
    for bad in (dict(t=None), dict(n=-1), dict(order=2), dict(max_norm=-1.0), dict(max_norm=math.nan), dict(norm=ODD),
                dict(factor=ODD), dict(norm=None, factor=None), dict(ws=None), dict(wsn=8), dict(ws=ODD)):
        assert norm(lib, table(), **bad) == INVALID, bad
    for bad in (dict(grad=0), dict(grad=(1 << 12) + 1), dict(grad_dtype=2), dict(grad=(1 << 12) + 2, grad_dtype=1)):
        assert norm(lib, table(**bad)) == INVALID, bad
    for bad in (dict(n=-1), dict(n=1 << 42)):
        assert norm(lib, table(**bad)) == SHAPE, bad
    assert M.minite_workspace_bytes(M.OP_GRAD_NORM, 6, 300001) == 0
    assert M.minite_workspace_bytes(M.OP_GRAD_NORM, 6, 1 << 22) > 0
    assert M.minite_workspace_bytes(M.OP_GRAD_NORM, 3000, 3000) > M.minite_workspace_bytes(M.OP_GRAD_NORM, 40, 40) > 0


def test_clip_grads(lib):
    def clip(t, factor=FAKE):
        return lib.minite_clip_grads(t.ctypes.data, len(t), factor, None)
    for bad in (dict(grad=0), dict(out=0), dict(out=(1 << 12) + 1), dict(out_dtype=2), dict(out_dtype=1)):  # the last: in place
        assert clip(table(**bad)) == INVALID, bad
    assert clip(table(2, grad=1 << 20, grad_dtype=1, out_dtype=1, out=(1 << 12) + 2)) == INVALID
    assert clip(table(), None) == INVALID and clip(table(), ODD) == INVALID
    assert clip(table()[:0]) == 0
    t = table()
    t["n"] = 0
    t["grad"] = 0
    assert clip(t) == 0


VERIFY = dict(target=FAKE, td=0, ts=100, draft=FAKE, dd=0, ds=100, tokens_in=FAKE, u=FAKE, noise=FAKE, ns=100, B=2, S=3,
              V=100, t=1.0, tokens=FAKE, accepted=FAKE, lp=FAKE, ws=FAKE, wsn=1 << 20, status=None, stream=None)


@pytest.mark.parametrize("change,rc", [
    (dict(target=None), INVALID), (dict(tokens_in=None), INVALID), (dict(u=None), INVALID), (dict(noise=None), INVALID),
    (dict(tokens=None), INVALID), (dict(accepted=None), INVALID), (dict(ws=None), INVALID), (dict(wsn=16), INVALID),
    (dict(td=2), INVALID), (dict(dd=3), INVALID), (dict(t=0.0), INVALID), (dict(t=-1.0), INVALID),
    (dict(t=math.nan), INVALID), (dict(t=math.inf), INVALID), (dict(t=1e-45), INVALID), (dict(t=4e-39), INVALID),
    (dict(td=1, target=ODD), INVALID), (dict(noise=ODD), INVALID), (dict(ws=ODD), INVALID), (dict(S=-1), SHAPE),
    (dict(S=32), SHAPE), (dict(B=-1), SHAPE), (dict(B=1 << 24), SHAPE), (dict(V=0), SHAPE),
    (dict(V=(1 << 30) + 1, ts=1 << 31, ds=1 << 31, ns=1 << 31), SHAPE), (dict(ts=99), SHAPE), (dict(ds=99), SHAPE),
    (dict(ns=99), SHAPE), (dict(B=0, target=None), 0)])
def test_verify_drafts(lib, change, rc):
    assert lib.minite_verify_drafts(*{**VERIFY, **change}.values()) == rc


def test_nothing_to_do(lib):
    assert lib.minite_moe_combine_rows_backward(*{**BACK, "T": 0, "dy": None}.values()) == 0
    for op, a, b, e, k in ((M.OP_PERMUTE_ROWS, 1, 0, 128, 8), (M.OP_PERMUTE_ROWS, 0, 0, 8, 8), (M.OP_VERIFY_DRAFTS, 0, 5, 1, 0)):
        assert M.minite_workspace_bytes(op, a, b, e, k) == 0
    assert M.minite_workspace_bytes(M.OP_PERMUTE_ROWS, 1 << 20, 0, 128, 8) > 0


def test_python_calls_refuse_wrong_tensors(calls, monkeypatch):   # noqa: F811
    monkeypatch.setattr(M, "_empty", lambda shape, dtype, like, stream: On(torch.zeros(shape, dtype=dtype)))
    monkeypatch.setattr(M, "_workspace", lambda *a: None)
    x, ids, w = torch.zeros(4, 64, dtype=BF), torch.zeros(4, 2, dtype=I32), torch.zeros(4, 2)
    rows, logits = torch.zeros(8, 64, dtype=BF), torch.zeros(2, 4, 50)
    drafts, u, e = torch.zeros(2, 3, dtype=I32), torch.zeros(2, 3), torch.ones(2, 50)
    for call in (
            lambda: M.permute_rows(x, ids, 4),                                    # not on a GPU
            lambda: M.permute_rows(On(x), On(ids.long()), 4, into=dict(rows=On(rows), offsets=On(torch.zeros(5, dtype=I32)),
                                                                       perm_src=On(torch.zeros(8, dtype=I32)), dest_row=On(ids))),
            lambda: M.permute_rows(On(x), On(ids), 4, into=dict(rows=On(rows[:7]), offsets=On(torch.zeros(5, dtype=I32)),
                                                                perm_src=On(torch.zeros(8, dtype=I32)), dest_row=On(ids))),
            lambda: M.permute_rows(x.view(-1), ids, 4),
            lambda: M.combine_rows(On(rows), On(ids), On(w.double()), out=On(x)),
            lambda: M.combine_rows(On(rows), On(ids), On(w[:3]), out=On(x)),
            lambda: M.combine_rows(On(rows), On(ids), On(w), out=On(x.float())),
            lambda: M.combine_rows(On(rows), On(ids[:3]), None, out=On(x)),
            lambda: M.combine_rows(On(rows.t()), On(ids), None, out=On(x)),
            lambda: M.combine_rows(On(rows[:1].expand(8, 64)), On(ids), None, out=On(x)),   # rows overlap
            lambda: M.combine_rows_backward(On(x), None, On(ids), On(w)),
            lambda: M.minite_moe_combine_rows_backward(On(x), On(rows[:, :32]), On(ids), On(w), On(rows), On(w)),
            lambda: M.spread_rows(On(x), On(ids), On(rows[:, :63])),
            lambda: M.grad_norm([]),
            lambda: M.grad_norm([torch.zeros(3)]),
            lambda: M.grad_norm([On(torch.zeros(3))], order=1.0),
            lambda: M.grad_norm([On(torch.zeros(3, dtype=torch.float16))]),
            lambda: M.grad_norm([On(torch.zeros(4, 4).t()[:2])]),
            lambda: M.clip_grads([On(torch.zeros(3))], 1.0, out=[]),
            lambda: M.clip_grads([On(torch.zeros(3)), On(torch.zeros(3))], 1.0),    # the same tensor twice
            lambda: M.clip_grads([On(torch.zeros(3))], 1.0, out=[On(torch.zeros(4))]),
            lambda: M.clip_grads([On(torch.zeros(3))], 1.0, out=[On(torch.zeros(3).half())]),
            lambda: M.verify_drafts(logits, drafts, u, e),
            lambda: M.minite_verify_drafts(On(logits), None, On(drafts[:, :2]), On(u), On(e), 1.0,
                                           On(torch.zeros(2, 4, dtype=I32)), On(torch.zeros(2, dtype=I32)), None,
                                           On(torch.zeros(4096, dtype=torch.uint8))),
            lambda: M.minite_verify_drafts(On(logits.transpose(0, 1)), None, On(torch.zeros(4, 1, dtype=I32)),
                                           On(torch.zeros(4, 1)), On(torch.ones(4, 50)), 1.0, On(torch.zeros(4, 2, dtype=I32)),
                                           On(torch.zeros(4, dtype=I32)), None, On(torch.zeros(4096, dtype=torch.uint8)))):
        with pytest.raises(M.MiniteError):
            call()
    assert not calls


def test_operands_on_another_device(calls):   # noqa: F811
    x, ids, rows = torch.zeros(4, 64, dtype=BF), torch.zeros(4, 2, dtype=I32), torch.zeros(8, 64, dtype=BF)
    ws = torch.zeros(64, dtype=torch.uint8)
    refused_elsewhere(calls, lambda **k: M.minite_moe_permute_rows(E=4, **k), dict(
        x=x, topk_ids=ids, rows=rows, expert_offsets=torch.zeros(5, dtype=I32), perm_src=torch.zeros(8, dtype=I32),
        dest_row=ids, workspace=ws, status=torch.zeros(1, dtype=I32)))
    calls.clear()
    refused_elsewhere(calls, M.spread_rows, dict(x=x, dest_row=ids, rows=rows, status=torch.zeros(1, dtype=I32)))
    calls.clear()
    refused_elsewhere(calls, M.combine_rows, dict(rows=rows, dest_row=ids, weights=torch.zeros(4, 2), out=x,
                                                  status=torch.zeros(1, dtype=I32)))
    calls.clear()
    refused_elsewhere(calls, M.minite_moe_combine_rows_backward, dict(
        dy=x, rows=rows, dest_row=ids, weights=torch.zeros(4, 2), drows=rows, dweights=torch.zeros(4, 2),
        status=torch.zeros(1, dtype=I32)))
    calls.clear()
    refused_elsewhere(calls, lambda g0, g1, **k: M.minite_grad_norm([g0, g1], 0, 1.0, **k), dict(
        g0=torch.zeros(3), g1=torch.zeros(5, dtype=BF), norm=torch.zeros(1), factor=torch.zeros(1), workspace=ws))
    calls.clear()
    refused_elsewhere(calls, lambda g, o, **k: M.minite_clip_grads([g], [o], **k), dict(
        g=torch.zeros(3), o=torch.zeros(3, dtype=BF), factor=torch.zeros(1)))
    calls.clear()
    refused_elsewhere(calls, lambda **k: M.minite_verify_drafts(temperature=1.0, **k), dict(
        target=torch.zeros(2, 4, 50), draft=torch.zeros(2, 3, 50, dtype=BF), draft_tokens=torch.zeros(2, 3, dtype=I32),
        uniforms=torch.zeros(2, 3), noise=torch.ones(2, 50), tokens=torch.zeros(2, 4, dtype=I32),
        accepted=torch.zeros(2, dtype=I32), logprobs=torch.zeros(2, 4), workspace=ws, status=torch.zeros(1, dtype=I32)))


class At(On):
    """A tensor at an address of its own."""

    def __init__(self, t, at):
        super().__init__(t)
        self.at = at

    def data_ptr(self):
        return self.at


def test_the_gradients_table(calls):   # noqa: F811
    """What a descriptor says: addresses, size, both types."""
    g = [At(torch.zeros(3), 4096), At(torch.zeros(2, 5, dtype=BF), 8192)]
    o = [At(torch.zeros(3, dtype=BF), 12288), At(torch.zeros(10), 16384)]
    t, d, elements = M._grad_table(g, o, "x")
    assert d == 0 and elements == 13
    d = np.frombuffer(t, dtype=GRAD_TENSOR)
    assert d["n"].tolist() == [3, 10] and d["grad_dtype"].tolist() == [1, 0] and d["out_dtype"].tolist() == [0, 1]
    assert d["grad"].tolist() == [4096, 8192] and d["out"].tolist() == [12288, 16384]
    empty = [At(torch.zeros(0), 0), At(torch.zeros(0), 0), g[0]]
    assert M._grad_table(empty, empty, "x")[2] == 3          # no elements: no place of its own
    assert M._grad_table([g[0], g[0]], None, "x")[2] == 6    # read twice: counted twice
