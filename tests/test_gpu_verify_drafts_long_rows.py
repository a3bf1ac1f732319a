"""Draft verification of rows of more segments than a warp has lanes (8192 FP32 or 16384
BF16 logits each), against the definition in 64 bits (tolerances: test_gpu_verify_drafts.py).
"""
import math

import pytest
import torch

from nvfp4_w4a4_moe_permute_gb300 import minite as M
from test_gpu_verify_drafts import check, inputs

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
INF = math.inf
SIZES = [(F32, 300007, 8192), (BF, 600011, 16384)]


def run(x, t=1.0):
    target, draft, tokens, u, e = x
    status = torch.zeros(1, dtype=I32, device=DEV)
    r = M.verify_drafts(target, tokens, u, e, draft_logits=draft, temperature=t, status=status)
    assert int(status) == 0
    return r


@pytest.mark.parametrize("dtype,V,seg", SIZES)
@pytest.mark.parametrize("by_model", [True, False])
@pytest.mark.parametrize("B,S,t,pad,shift", [(2, 1, 1.0, 0, 0), (1, 2, 0.7, 5, 3)])
def test_more_than_32_segments(dtype, V, seg, by_model, B, S, t, pad, shift):
    x = inputs(V + S, B, S, V, dtype, by_model, pad, shift, ragged=False)
    check(*x, t, run(x, t))


@pytest.mark.parametrize("dtype,V,seg", SIZES)
@pytest.mark.parametrize("by_model", [True, False])
@pytest.mark.parametrize("places", [[33], [1, 33], [0, 32], [4, 36], [34, 35], [2, 34, 35]], ids=str)
def test_the_largest_in_late_segments(dtype, V, seg, by_model, places):
    """One maximum, or equal ones, of which one joins a lane's first segment."""
    x = inputs(len(places), 2, 1, V, dtype, by_model, ragged=False)
    for i, s in enumerate(places):
        at = min(s * seg + 17 * i + 5, V - 1)
        x[0][..., at] = 17.0
        if by_model:
            x[1][..., at] = 16.5
    x[2][:] = min(places[-1] * seg + 17 * (len(places) - 1) + 5, V - 1)
    x[3][0] = 0.01
    r = run(x)
    check(*x, 1.0, r)
    assert int(r["accepted"][0]) == 1


@pytest.mark.parametrize("dtype,V,seg", SIZES)
@pytest.mark.parametrize("masked", [(0, 3), (1, 2), (31, 34), (32, 40), (0, 32), (3, 36)], ids=str)
def test_masked_segments(dtype, V, seg, masked):
    x = inputs(3, 2, 1, V, dtype, True, ragged=False)
    a, b = masked[0] * seg, min(masked[1] * seg + 7, V)
    x[0][..., a:b] = -INF
    x[1][1, :, a:b] = -INF
    r = run(x)
    check(*x, 1.0, r)
    assert not ((r["tokens"] >= a) & (r["tokens"] < b)).any()


@pytest.mark.parametrize("dtype,V,seg", SIZES)
@pytest.mark.parametrize("bad", [math.nan, INF])
@pytest.mark.parametrize("at", [0, 33, 36])
def test_no_probabilities_in_a_late_segment(dtype, V, seg, bad, at):
    x = inputs(4, 3, 1, V, dtype, True, ragged=False)
    x[3].zero_()                              # every draft stands that can
    x[0][0, 0, at * seg + 9] = bad
    x[1][1, 0, at * seg + 9] = bad
    r = run(x)
    assert r["accepted"].tolist() == [0, 0, 1]
    for b in (0, 1):
        assert int(r["tokens"][b, 0]) == -1 and math.isnan(float(r["logprobs"][b, 0]))
    assert int(r["tokens"][2, 1]) >= 0


@pytest.mark.parametrize("dtype,V,seg", SIZES)
def test_rows_of_nothing_but_masked_tokens(dtype, V, seg):
    x = inputs(5, 2, 0, V, dtype, False)
    x[0][0] = -INF
    x[0][1, 0] = -INF
    x[0][1, 0, 35 * seg + 3] = -4.0           # a single token, certain
    r = run(x)
    assert r["tokens"][:, 0].tolist() == [-1, 35 * seg + 3]
    assert math.isnan(float(r["logprobs"][0, 0])) and float(r["logprobs"][1, 0]) == 0.0
