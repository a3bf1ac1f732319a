"""Rows sorted by expert and back against plain loops and 64-bit formulas.

Tolerances. Copies are exact. A combined element is a chain of at most k fused
multiply-adds in FP32, each off by 2^-24 of the running sum, which stays below the
sum of magnitudes: k 2^-24 sum |w r|, and one rounding to the output type, half its
step. A gradient row is one FP32 product, rounded: half a step (twice for BF16: of the
product, 2^-24, and of the type). A dot product of H terms: a lane's chain of at most
H / 32 + 16 terms, five steps over the lanes, at most H / 256 + 8 partial sums:
(H / 24 + 40) 2^-24 sum |dy r|. Values near the smallest normal are not used.
"""
import pytest
import torch

from nvfp4_w4a4_moe_permute_gb300 import minite as M

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def route(seed, T, k, E, dropped=0.0, skew=0.0):
    """Experts of every slot (the same one twice in a token among them)."""
    g = torch.Generator().manual_seed(seed)
    p = torch.arange(1, E + 1, dtype=torch.float64) ** -skew
    ids = torch.multinomial(p.expand(max(T, 1), E), k, replacement=True, generator=g).to(I32)[:T]
    ids[torch.rand(T, k, generator=g) < dropped] = -1
    return ids


def sorted_by_expert(ids, E):
    T, k = ids.shape
    flat = ids.reshape(-1).tolist()
    order = [p for e in range(E) for p in range(T * k) if flat[p] == e] if T * k < 2000 else \
        torch.argsort(torch.where((ids.reshape(-1) >= 0) & (ids.reshape(-1) < E), ids.reshape(-1), E), stable=True).tolist()
    order = [p for p in order if 0 <= flat[p] < E]
    dest = torch.full((T * k,), -1, dtype=torch.long)
    dest[order] = torch.arange(len(order))
    counts = torch.tensor([0] + [sum(1 for f in flat if f == e) for e in range(E)]) if T * k < 2000 else \
        torch.cat([torch.zeros(1, dtype=torch.long), torch.bincount(ids[(ids >= 0) & (ids < E)].long(), minlength=E)])
    return torch.tensor(order, dtype=torch.long), dest.view(T, k), counts.cumsum(0)


def matrix(g, rows, cols, dtype, pad=0, shift=0):
    """[rows, cols] with rows cols + pad elements apart, the first one `shift` elements in."""
    flat = torch.randn(rows * (cols + pad) + shift, generator=g).to(dtype).to(DEV)
    return flat[shift:].view(rows, cols + pad)[:, :cols]


# T, k, E, H: one launch up to 65536 slots, clusters of CTAs above 16384, three launches above
SORTS = [(1, 1, 1, 1), (1, 8, 128, 2048), (3, 2, 5, 7), (31, 32, 1024, 16), (152, 3, 9, 33), (153, 8, 7, 64),
         (1024, 8, 128, 24), (2049, 8, 128, 16), (4096, 8, 128, 40), (2100, 31, 3, 8), (65536, 1, 60, 8), (9000, 7, 17, 8),
         (3000, 8, 700, 16), (8193, 8, 128, 8), (70000, 2, 257, 8)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,k,E,H", SORTS)
@pytest.mark.parametrize("dropped,skew,pad,shift", [(0.0, 0.0, 0, 0), (0.4, 1.5, 3, 1), (1.0, 0.0, 8, 8)])
def test_permute(T, k, E, H, dtype, dropped, skew, pad, shift):
    g = torch.Generator().manual_seed(T * k + H)
    ids = route(T + E, T, k, E, dropped, skew)
    x = matrix(g, T, H, dtype, pad, shift)
    out = torch.full((T * k, H + pad), 7.0, dtype=dtype, device=DEV)
    into = dict(rows=out[:, :H], offsets=torch.full((E + 1,), -9, dtype=I32, device=DEV),
                perm_src=torch.full((T * k,), -9, dtype=I32, device=DEV),
                dest_row=torch.full((T, k), -9, dtype=I32, device=DEV))
    status = torch.zeros(1, dtype=I32, device=DEV)
    r = M.permute_rows(x, ids.to(DEV), E, into=into, status=status)
    order, dest, offsets = sorted_by_expert(ids, E)
    n = order.numel()
    assert r is into and int(status) == 0
    assert r["offsets"].tolist() == offsets.tolist()
    assert torch.equal(r["dest_row"].cpu().long(), dest)
    assert torch.equal(r["perm_src"][:n].cpu().long(), order // k) and (r["perm_src"][n:] == -1).all()
    assert torch.equal(out[:n, :H], x[(order // k).to(DEV)])
    assert (out[n:] == 7).all() and (out[:, H:] == 7).all()   # what no slot has stays


# the longest ranges of a CTA: 512 slots, or the last number of tokens below that
@pytest.mark.parametrize("T,k,E,H", [(7680, 8, 5, 8), (7681, 8, 128, 3), (7704, 8, 128, 4), (8192, 8, 256, 8), (1923, 32, 257, 8),
                                     (3850, 16, 60, 1), (30785, 2, 1024, 16), (61441, 1, 9, 2), (2113, 31, 1024, 2),
                                     (16384, 1, 1024, 8), (16385, 1, 2, 8), (512, 32, 700, 3), (513, 32, 3, 8)])
def test_longest_ranges(T, k, E, H):
    test_permute(T, k, E, H, BF, 0.2, 1.0, 0, 0)


@pytest.mark.parametrize("T,k", [(5, 2), (5000, 8), (70000, 1)])
def test_permute_reports_ids_out_of_range(T, k):
    ids = route(1, T, k, 6)
    ids[T // 2, 0], ids[T - 1, k - 1], ids[0, 0] = 6, 2 ** 31 - 1, -5
    x = torch.randn(T, 24, device=DEV)
    status = torch.zeros(1, dtype=I32, device=DEV)
    r = M.permute_rows(x, ids.to(DEV), 6, status=status)
    _, dest, offsets = sorted_by_expert(ids, 6)
    assert int(status) == 1 << M.ERR_BAD_ROUTING
    assert torch.equal(r["dest_row"].cpu().long(), dest) and r["offsets"].tolist() == offsets.tolist()
    ids[ids > 5] = -1
    status.zero_()
    M.permute_rows(x, ids.to(DEV), 6, status=status)
    assert int(status) == 0   # a negative id is a slot that is not used


@pytest.mark.parametrize("T,k", [(777, 3), (5000, 5)])
def test_ids_may_start_anywhere(T, k):
    flat = torch.randint(-1, 9, (T * k + 3,), generator=torch.Generator().manual_seed(T)).to(I32)
    x = torch.randn(T, 16, device=DEV)
    dev = flat.to(DEV)
    for shift in range(4):
        ids = flat[shift: shift + T * k].view(T, k)
        r = M.permute_rows(x, dev[shift: shift + T * k].view(T, k), 9)
        _, dest, offsets = sorted_by_expert(ids, 9)
        assert torch.equal(r["dest_row"].cpu().long(), dest) and r["offsets"].tolist() == offsets.tolist()


def test_permute_of_nothing():
    r = M.permute_rows(torch.empty(0, 8, device=DEV), torch.empty(0, 2, dtype=I32, device=DEV), 3)
    assert r["offsets"].tolist() == [0, 0, 0, 0] and r["rows"].shape == (0, 8)


def case(seed, T, k, E, H, dtype, dropped, pad, shift):
    g = torch.Generator().manual_seed(seed)
    ids = route(seed, T, k, E, dropped, 0.7)
    order, dest, _ = sorted_by_expert(ids, E)
    rows = matrix(g, max(1, T * k), H, dtype, pad, shift)
    rows[order.numel():] = float("nan")   # rows that no slot names are not read
    w = torch.rand(T, k, generator=g).sub_(0.3).to(DEV)
    w[(dest < 0).to(DEV)] = float("inf")      # nor is the weight of a skipped slot
    return dest.to(I32).to(DEV), rows, w, g


SHAPES = [(1, 1, 1), (1, 8, 2048), (5, 3, 7), (2, 32, 8), (40, 8, 520), (300, 9, 256), (77, 1, 1000), (33, 17, 4099),
          (9, 4, 20000), (1500, 8, 264)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,k,H", SHAPES)
@pytest.mark.parametrize("dropped,pad,shift", [(0.0, 0, 0), (0.5, 8, 8), (0.3, 3, 1)])
@pytest.mark.parametrize("weighted", [True, False])
def test_combine(T, k, H, dtype, dropped, pad, shift, weighted):
    dest, rows, w, _ = case(T + H, T, k, 7, H, dtype, dropped, pad, shift)
    out = torch.full((T, H + pad), 5.0, dtype=dtype, device=DEV)
    status = torch.zeros(1, dtype=I32, device=DEV)
    y = M.combine_rows(rows, dest, w if weighted else None, out=out[:, :H], status=status)
    assert int(status) == 0 and (out[:, H:] == 5).all()
    live = dest >= 0
    r = torch.where(live[..., None], rows[dest.long().clamp(min=0)].double(), 0.0)
    wd = torch.where(live, w.double() if weighted else 1.0, 0.0)[..., None]
    want, size = (r * wd).sum(1), (r * wd).abs().sum(1)
    assert ((y.double() - want).abs() <= half_step(dtype) * want.abs() * 1.01 + k * 2.0 ** -24 * size).all()
    if not weighted:
        assert torch.equal(M.permute_rows_backward(rows, dest), y)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,k,H", SHAPES)
@pytest.mark.parametrize("dropped,pad,shift", [(0.0, 0, 0), (0.5, 8, 8), (0.3, 3, 1)])
def test_combine_backward(T, k, H, dtype, dropped, pad, shift):
    dest, rows, w, g = case(T + H, T, k, 7, H, dtype, dropped, pad, shift)
    live = dest >= 0
    dy = matrix(g, T, H, dtype, pad, shift)
    out = torch.full((rows.shape[0], H + pad), 5.0, dtype=dtype, device=DEV)
    status = torch.zeros(1, dtype=I32, device=DEV)
    drows, dw = M.combine_rows_backward(dy, rows, dest, w, out=out[:, :H], status=status)
    assert int(status) == 0 and (out[:, H:] == 5).all() and (out[int(live.sum()):] == 5).all()
    at = dest.long().clamp(min=0)
    t, j = torch.nonzero(live, as_tuple=True)
    want = w.double()[t, j, None] * dy.double()[t]
    assert ((drows[dest[t, j].long()].double() - want).abs() <= (half_step(dtype) + 2.0 ** -24) * 1.01 * want.abs()).all()
    r = torch.where(live[..., None], rows[at].double(), 0.0)
    prod = r * dy.double()[:, None]
    assert ((dw.double() - prod.sum(2)).abs() <= (H / 24 + 40) * 2.0 ** -24 * prod.abs().sum(2)).all()
    assert (dw[~live] == 0).all()
    # a router that is not trained, and gradients over the rows themselves
    only, none = M.combine_rows_backward(dy, None, dest, w, out=torch.full_like(out, 5.0)[:, :H])
    assert none is None and torch.equal(only, drows)
    over, dw2 = M.combine_rows_backward(dy, rows, dest, w, out=rows)
    n = int(live.sum())
    assert over is rows and torch.equal(rows[:n], drows[:n]) and torch.equal(dw2, dw)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_gradients_against_differences(dtype):
    """A linear function of rows and weights: differences of any size are exact but for roundings."""
    T, k, H = 6, 3, 40
    dest, rows, w, g = case(3, T, k, 4, H, F32, 0.3, 0, 0)
    rows, live = torch.nan_to_num(rows), dest >= 0
    w = torch.where(live, w, 0.0)
    dy = torch.randn(T, H, generator=g).to(DEV)
    f = lambda r, v: (M.combine_rows(r, dest, v).double() * dy.double()).sum()
    drows, dw = M.combine_rows_backward(dy, rows, dest, w, out=torch.zeros_like(rows))
    for i in range(T):
        for j in range(k):
            v = w.clone()
            v[i, j] += 1.0
            assert abs(float(f(rows, v) - f(rows, w) - dw[i, j].double())) < 1e-4
    for m in (0, 3, int(live.sum()) - 1):
        r = rows.clone()
        r[m] += 1.0
        assert abs(float(f(r, w) - f(rows, w) - drows[m].double().sum())) < 1e-4


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H,pad,shift", [(64, 0, 0), (7, 2, 1), (2048, 0, 0)])
def test_spread(dtype, H, pad, shift):
    g = torch.Generator().manual_seed(H)
    ids = route(2, 50, 4, 6, 0.4)
    order, dest, _ = sorted_by_expert(ids, 6)
    x, n = matrix(g, 50, H, dtype, pad, shift), order.numel()
    rows = torch.full((220, H), 3.0, dtype=dtype, device=DEV)
    assert M.spread_rows(x, dest.to(I32).to(DEV), rows) is rows
    assert torch.equal(rows[:n], x[(order // 4).to(DEV)]) and (rows[n:] == 3).all()


def test_rows_out_of_range_are_reported_and_skipped():
    dest = torch.tensor([[0, 9], [-1, 2], [3, 2 ** 31 - 1]], dtype=I32, device=DEV)
    rows, w = torch.randn(4, 16, device=DEV), torch.ones(3, 2, device=DEV)
    want = torch.stack([rows[0], rows[2], rows[3]])
    for width in (16, 15):
        r, dy = rows[:, :width], want[:, :width]
        for call in (lambda s: M.combine_rows(r, dest, w, status=s), lambda s: M.combine_rows(r, dest, None, status=s)):
            s = torch.zeros(1, dtype=I32, device=DEV)
            assert torch.equal(call(s), dy) and int(s) == 1 << M.ERR_BAD_ROUTING
        s, out = torch.zeros(1, dtype=I32, device=DEV), torch.full((4, width), 8.0, device=DEV)
        _, dw = M.combine_rows_backward(dy, r, dest, w, out=out, status=s)
        assert int(s) == 1 << M.ERR_BAD_ROUTING and (out[1] == 8).all() and torch.equal(out[[0, 2, 3]], dy)
        assert dw[0, 1] == 0 and dw[2, 1] == 0
        s = torch.zeros(1, dtype=I32, device=DEV)
        M.spread_rows(dy, dest, out.fill_(8.0), status=s)
        assert int(s) == 1 << M.ERR_BAD_ROUTING and (out[1] == 8).all() and torch.equal(out[[0, 2, 3]], dy)


def test_results_do_not_depend_on_the_other_tokens():
    T, k, H = 700, 8, 1032
    dest, rows, w, g = case(11, T, k, 9, H, BF, 0.2, 0, 0)
    dy = matrix(g, T, H, BF)
    y = M.combine_rows(rows, dest, w)
    drows, dw = M.combine_rows_backward(dy, rows, dest, w)
    for t in (0, 5, 699):
        a = M.combine_rows(rows, dest[t: t + 1], w[t: t + 1])
        _, b = M.combine_rows_backward(dy[t: t + 1], rows, dest[t: t + 1], w[t: t + 1])
        assert torch.equal(a[0], y[t]) and torch.equal(b[0], dw[t])


def test_special_values_pass_through():
    dest = torch.tensor([[0, 1], [2, -1]], dtype=I32, device=DEV)
    rows = torch.zeros(3, 8, device=DEV)
    rows[0, 0], rows[1, 1], rows[2, 2] = float("inf"), float("nan"), 3e38
    y = M.combine_rows(rows, dest, torch.tensor([[2.0, 1.0], [2.0, 0.0]], device=DEV))
    assert torch.isinf(y[0, 0]) and torch.isnan(y[0, 1]) and torch.isinf(y[1, 2]) and (y[:, 3:] == 0).all()
    x = torch.tensor([[float("nan"), -0.0, float("inf"), 1e-45] * 2], device=DEV)
    r = M.permute_rows(x, torch.zeros(1, 1, dtype=I32, device=DEV), 1)
    assert torch.equal(r["rows"].view(I32), x.view(I32))   # as bits


def test_streams_and_graphs():
    """Two calls at once on streams of their own, and a captured one with other inputs."""
    T, k, E, H = 5000, 8, 16, 64
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    xs = [torch.randn(T, H, device=DEV) for _ in range(2)]
    ids = [route(i, T, k, E, 0.1).to(DEV) for i in range(2)]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(5):
        for i, s in enumerate((one, two)):
            r = M.permute_rows(xs[i], ids[i], E, stream=s)
            got[i] = (r, M.permute_rows_backward(r["rows"], r["dest_row"], stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        n = (ids[i] >= 0).sum(1, keepdim=True)
        assert torch.equal(got[i][0]["dest_row"].cpu().long(), sorted_by_expert(ids[i].cpu(), E)[1])
        assert torch.allclose(got[i][1], xs[i] * n, rtol=1e-6)
    x, i, w = xs[0].clone(), ids[0].clone(), torch.rand(T, k, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = M.permute_rows(x, i, E)
        y = M.combine_rows(r["rows"], r["dest_row"], w)
        drows, dw = M.combine_rows_backward(x, r["rows"], r["dest_row"], w)
    for s in (1, 0):
        x.copy_(xs[s])
        i.copy_(ids[s])
        graph.replay()
        torch.cuda.synchronize()
        live = i >= 0
        assert torch.allclose(y, x * torch.where(live, w, 0.0).sum(1, keepdim=True), rtol=1e-5, atol=1e-5)
        assert torch.allclose(dw, torch.where(live, (x * x).sum(1, keepdim=True), 0.0), rtol=1e-5)


def test_large_offsets():
    """Rows beyond 2^31 elements."""
    H, T = 1 << 20, 2200
    x = torch.randn(4, H, device=DEV).to(BF)
    dest = torch.full((4, 1), -1, dtype=I32, device=DEV)
    dest[:, 0] = torch.tensor([2199, 0, 2047, 2048])
    rows = torch.zeros(T, H, dtype=BF, device=DEV)
    M.spread_rows(x, dest, rows)
    assert torch.equal(rows[dest[:, 0].long()], x) and int((rows[1:2047] != 0).sum()) == 0
    w = torch.full((4, 1), 2.0, device=DEV)
    assert torch.equal(M.combine_rows(rows, dest, w), (x.float() * 2).to(BF))
    drows, dw = M.combine_rows_backward(x, rows, dest, w, out=rows)
    assert torch.equal(rows[dest[:, 0].long()], (x.float() * 2).to(BF))
    want = (x.double() ** 2).sum(1)
    assert ((dw[:, 0].double() - want).abs() <= (H / 24 + 40) * 2.0 ** -24 * want).all()


def test_permute_of_rows_beyond_two_to_the_31_elements():
    H = 1 << 20
    for T, k in ((2100, 1), (270, 8)):   # x, or the rows in expert order, pass it
        x = torch.zeros(T, H, dtype=BF, device=DEV)
        x[:, 0] = torch.arange(T, device=DEV) % 251
        x[:, -1] = torch.arange(T, device=DEV) % 241
        ids = route(5, T, k, 7)
        r = M.permute_rows(x, ids.to(DEV), 7)
        order, dest, _ = sorted_by_expert(ids, 7)
        assert torch.equal(r["dest_row"].cpu().long(), dest)
        src = (order // k).to(DEV)
        assert torch.equal(r["rows"][:, 0], x[src, 0]) and torch.equal(r["rows"][:, -1], x[src, -1])
        assert not r["rows"][:, 1:-1].any()
        del x, r
    # and by ranking, scan and copies
    T, k, H = 40000, 8, 7168
    x = torch.randn(T, H, device=DEV).to(BF)
    ids = route(6, T, k, 12)
    r = M.permute_rows(x, ids.to(DEV), 12)
    src = (sorted_by_expert(ids, 12)[0] // k).to(DEV)
    for a in range(0, T * k, 32000):
        assert torch.equal(r["rows"][a: a + 32000], x[src[a: a + 32000]])
