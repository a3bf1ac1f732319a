"""Gradients of the weighted sum of rows against differences, in both types.

Rows, weights and dy are small multiples of powers of two, so that every product and
every sum of three of them is exact in FP32: y is off by its one rounding to the type,
half a step of it, and so is drows. A difference of two sums over y dy is then within the sum
of what the roundings of the y's that change can make of it.
"""
import pytest
import torch

from nvfp4_w4a4_moe_permute_gb300 import minite as M

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,k,H", [(6, 3, 40), (3, 2, 33), (2, 3, 520)])
def test_gradients_against_differences(dtype, T, k, H):
    g = torch.Generator().manual_seed(T + H)
    grid = lambda *s: torch.randint(-24, 25, s, generator=g).float() / 8
    dest = torch.randperm(T * k, generator=g).view(T, k).to(I32)
    dest[1, 0] = -1                               # a slot that is not used
    rows, dy = grid(T * k, H).to(dtype).to(DEV), grid(T, H).to(dtype).to(DEV)
    w = grid(T, k).to(DEV)
    live = (dest >= 0).to(DEV)
    dest = dest.to(DEV)
    drows, dw = M.combine_rows_backward(dy, rows, dest, w, out=torch.zeros_like(rows))
    half = torch.finfo(dtype).eps / 2
    combine = lambda r, v: M.combine_rows(r, dest, v).double()
    y = combine(rows, w)
    f = lambda out: (out * dy.double()).sum()
    may = lambda out, t: float((half * out[t].abs() * dy[t].double().abs()).sum()) + 1e-12

    for t in range(T):
        for j in range(k):
            v = w.clone()
            v[t, j] += 1.0
            out = combine(rows, v)
            # dw is a sum of exact products, which FP32 holds exactly here (multiples of 2^-6 below 2^13)
            assert abs(float(f(out) - f(y)) - float(dw[t, j])) <= may(out, t) + may(y, t), (t, j)
            if not bool(live[t, j]):
                assert float(dw[t, j]) == 0.0
                continue
            r = rows.clone()
            r[dest[t, j].long()] += 1.0           # stays on the grid
            out = combine(r, w)
            want = float(drows[dest[t, j].long()].double().sum())
            rounded = float((half * (w[t, j].double() * dy[t].double()).abs()).sum())
            assert abs(float(f(out) - f(y)) - want) <= may(out, t) + may(y, t) + rounded, (t, j)
