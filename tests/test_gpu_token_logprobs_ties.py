"""Alternatives of long rows with more candidates than are ranked by counting, and
where a row lies in memory.

A row of 131072 logits alone is shared by a cluster of CTAs; three values, or
values that differ in a few places, leave thousands of candidates in each of them,
which sorted lists then rank. The order is exact (larger logit, then lower index),
so ids have to be equal to a stable sort's."""
import math

import pytest
import torch

from nvfp4_w4a4_moe_permute_gb300 import minite as M

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def rows_of(v, dtype):
    i = torch.arange(v)
    g = torch.Generator().manual_seed(v)
    rows = [(i % 3).float(), torch.zeros(v), torch.where(i < v // 2, 1.0, 2.0), torch.where(i > v - 20, 3.0, 1.0),
            torch.where(torch.rand(v, generator=g) < 0.02, 4.0, 0.5), (i // 1000 % 7).float(),
            torch.where(i % 5 == 0, -math.inf, 1.0)]
    return torch.stack(rows).to(dtype).to(DEV)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("v", [131072, 200003, 70001])
@pytest.mark.parametrize("k", [1, 20, 32])
@pytest.mark.parametrize("alone", [True, False])
def test_many_equal_logits(v, dtype, k, alone):
    x = rows_of(v, dtype)
    ids = torch.sort(x.float(), dim=1, descending=True, stable=True).indices[:, :k]
    if alone:   # a cluster for every row
        got = torch.cat([M.token_logprobs(x[i:i + 1], alternatives=k)["alt_ids"] for i in range(x.shape[0])])
        assert torch.equal(got.long(), ids)
    else:       # hundreds of rows: one CTA each
        got = M.token_logprobs(x.repeat(100, 1), alternatives=k)["alt_ids"]
        assert torch.equal(got.long(), ids.repeat(100, 1))


@pytest.mark.parametrize("dtype,unit", [(torch.float32, 8), (torch.bfloat16, 16)])
@pytest.mark.parametrize("v", [1000, 32003, 131072])
def test_where_a_row_lies(dtype, unit, v):
    """The same bits at every address of the same remainder by 32 bytes; at another
    one the sums are cut elsewhere, and both are within the rounding of one (the
    derivation in the tests of log probabilities: 2^-19 and 2^-22 times the span of
    the logits, here 2 * 20, on each side)."""
    g = torch.Generator().manual_seed(1)
    row = (torch.randn(v, generator=g) * 3).to(dtype).to(DEV)
    y = torch.tensor([v // 2], device=DEV)
    keys = ("logprob", "entropy", "stats", "alt_logprobs", "alt_ids")

    def at(offset):
        store = torch.zeros(v + 4 * unit, dtype=dtype, device=DEV)
        store[offset:offset + v] = row
        return M.token_logprobs(store[offset:offset + v][None], y, alternatives=5)

    base = at(0)
    for offset in (0, unit, 3 * unit):
        again = at(offset)
        assert all(torch.equal(again[k], base[k]) for k in keys)
    tol = 2 * (2.0 ** -19 + 2.0 ** -22 * 40)
    for offset in (1, 3, unit - 1, unit + 1):
        other = at(offset)
        assert torch.equal(other["alt_ids"], base["alt_ids"])
        assert (other["logprob"] - base["logprob"]).abs().item() <= tol
        assert (other["entropy"] - base["entropy"]).abs().item() <= tol * (1 + base["entropy"].item())
        again = at(offset)
        assert all(torch.equal(again[k], other[k]) for k in keys)
