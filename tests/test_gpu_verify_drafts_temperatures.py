"""Draft verification at temperatures far from 1 and logits far from 0.

Tolerances. Where the logits lie on a grid whose step over the temperature is above
200, a row's probabilities are 1 / n at its n largest logits and 0 (below 2^-126)
elsewhere, exactly but for log1p(n - 1): 2^-22 of it.
"""
import math

import pytest
import torch

from nvfp4_w4a4_moe_permute_gb300 import minite as M

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def near_log(got, n):
    want = -torch.log(n.double())
    assert ((got.double() - want).abs() <= 2.0 ** -22 * want.abs()).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [3, 100, 9001, 40003])
@pytest.mark.parametrize("t,scale", [(1e-4, 1.0), (1e-6, 1.0), (1e-8, 1.0), (1e-9, 1.0), (1e-10, 1.0), (1e-15, 1.0), (1e-25, 1.0),
                                     (1e-30, 1.0), (1e-37, 1.0), (1.0, 2.0 ** 30), (1.0, 2.0 ** 40), (0.7, 2.0 ** 60),
                                     (1.0, 2.0 ** 90), (1e3, 2.0 ** 100)])
def test_all_but_the_largest_vanish(dtype, V, t, scale):
    """Temperatures near 0, and logits whose differences alone are large: the largest are all
    there is, and a draft stands where it is the only one."""
    B, S = 24, 2
    g = torch.Generator().manual_seed(V)
    # multiples of 1/8 up to 16: exact in BF16, a step of 0.125 scale
    target = (torch.randint(-128, 128, (B, S + 1, V), generator=g).float() / 8 * scale).to(dtype)
    target[: B // 2, :, V // 2] = 17 * scale              # one largest, in half of the sequences
    top = target == target.amax(2, keepdim=True)
    n = top.sum(2)
    tokens = top.to(torch.int8).argmax(2)[:, :S].to(I32)
    tokens[:: 5, 1] = -1
    e = torch.rand(B, V, generator=g) + 0.5
    u = torch.full((B, S), 0.999)
    for draft in (None, target[:, :S].contiguous()):
        r = M.verify_drafts(target.to(DEV), tokens.to(DEV), u.to(DEV), e.to(DEV),
                            draft_logits=None if draft is None else draft.to(DEV), temperature=t)
        got, acc, lp = r["tokens"].cpu(), r["accepted"].cpu(), r["logprobs"].cpu()
        for b in range(B):
            given = 1 if int(tokens[b, 1]) < 0 else S
            stands = 0
            while stands < given and (draft is not None or int(n[b, stands]) == 1):
                stands += 1
            assert int(acc[b]) == stands, b
            w = torch.where(top[b, stands], 1 / e[b], 0.0)
            if stands < given:
                w[tokens[b, stands]] = 0.0                # looked up, fallen: 1 at the draft
            assert int(got[b, stands]) == int(w.argmax()), b
            near_log(lp[b, : stands + 1], n[b, : stands + 1])


@pytest.mark.parametrize("t", [1e4, 1e10, 1e20, 1e37, 3e38])
def test_all_alike(t):
    """Temperatures so high that every token has the same probability."""
    V = 9001
    g = torch.Generator().manual_seed(1)
    target = torch.randn(4, 1, V, generator=g) * 1e-3
    e = torch.rand(4, V, generator=g) + 0.5
    first = e.topk(2, 1, largest=False)
    e.scatter_(1, first.indices[:, :1], 0.25)             # wins beyond any rounding
    r = M.verify_drafts(target.to(DEV), torch.zeros(4, 0, dtype=I32, device=DEV), torch.zeros(4, 0, device=DEV), e.to(DEV),
                        temperature=t)
    assert torch.equal(r["tokens"][:, 0].cpu(), e.argmin(1).to(I32))
    assert ((r["logprobs"][:, 0].cpu().double() + math.log(V)).abs() <= 1e-6 + 2.0 ** -17).all()
