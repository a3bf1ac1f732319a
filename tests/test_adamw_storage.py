"""An AdamW step works on parameters, copies and states as they lie at the step:
storage that was replaced since the last one (a reload, ``p.data = ...``) is what
is read and written, and what does not fit is refused. No GPU is needed for the
addresses: CPU tensors that say they are on a GPU, and a library that notes the
descriptors it is given."""
import ctypes

import numpy as np
import pytest
import torch

from nvfp4_w4a4_moe_permute_gb300 import minite as M


class On:
    """A tensor that says that it is on cuda:0; its storage is .t's."""

    is_cuda, device = True, torch.device("cuda", 0)

    def __init__(self, t):
        self.t = t

    def get_device(self):
        return 0

    def __getattr__(self, name):
        return getattr(self.t, name)


class Stream:
    cuda_stream = device_index = 0


SIZES = [7, 300, 256]


@pytest.fixture
def given(monkeypatch):
    """The descriptors of every step so far."""
    seen = []

    class Library:
        @staticmethod
        def minite_adamw_step(address, n, *rest):
            raw = ctypes.string_at(address, n * M.ADAMW_TENSOR.itemsize)
            seen.append(np.frombuffer(raw, dtype=M.ADAMW_TENSOR))
            return 0

    monkeypatch.setattr(M, "load", lambda path=None: Library)
    monkeypatch.setattr(M, "_current_device", lambda: 0)
    return seen


def optimizer(bits):
    kind = torch.float8_e4m3fn if bits == 8 else torch.float32
    state = dict(step=0, exp_avg=On(torch.zeros(1024, dtype=kind)), exp_avg_sq=On(torch.zeros(1024, dtype=kind)))
    if bits == 8:
        state |= dict(exp_avg_scale=On(torch.zeros(4)), exp_avg_sq_scale=On(torch.zeros(4)))
    return M.AdamW([On(torch.zeros(n)) for n in SIZES], copies=[On(torch.zeros(n, dtype=torch.bfloat16)) for n in SIZES],
                   state_bits=bits, state=state)


def step(opt):
    opt.step([On(torch.zeros(n)) for n in SIZES], stream=Stream)


def check(opt, d, bits):
    first = np.array([0, 1, 3])
    assert d["param"].tolist() == [p.t.data_ptr() for p in opt.params]
    assert d["param_bf16"].tolist() == [c.t.data_ptr() for c in opt.copies]
    for name in ("exp_avg", "exp_avg_sq"):
        size = 1 if bits == 8 else 4
        assert d[name].tolist() == (getattr(opt, name).t.data_ptr() + 256 * size * first).tolist()
        scale = getattr(opt, name + "_scale").t.data_ptr() + 4 * first if bits == 8 else 0 * first
        assert d[name + "_scale"].tolist() == scale.tolist()


@pytest.mark.parametrize("bits", [8, 32])
def test_replaced_storage_is_what_a_step_uses(given, bits):
    opt = optimizer(bits)
    step(opt)
    check(opt, given[-1], bits)
    old = []   # kept, so that new storage lies elsewhere
    for t in opt.params + opt.copies + [getattr(opt, k) for k in ("exp_avg", "exp_avg_sq") + (
            ("exp_avg_scale", "exp_avg_sq_scale") if bits == 8 else ())]:
        old.append(t.t)
        t.t = t.t.clone()
        step(opt)
        check(opt, given[-1], bits)
    opt.params[1] = On(torch.zeros(300))
    opt.exp_avg_sq = On(torch.zeros_like(opt.exp_avg_sq.t))
    step(opt)
    check(opt, given[-1], bits)
    assert opt.step_count == len(given)


@pytest.mark.parametrize("bits", [8, 32])
def test_storage_that_does_not_fit_is_refused(given, bits):
    def change(what, to):
        opt = optimizer(bits)
        step(opt)
        what(opt).t = to
        before = len(given)
        with pytest.raises(M.MiniteError):
            step(opt)
        assert len(given) == before and opt.step_count == 1

    change(lambda o: o.params[1], torch.zeros(299))
    change(lambda o: o.params[1], torch.zeros(300, dtype=torch.bfloat16))
    change(lambda o: o.params[1], torch.zeros(600)[::2])
    change(lambda o: o.copies[2], torch.zeros(256))
    change(lambda o: o.exp_avg, torch.zeros(768, dtype=torch.float32))
    change(lambda o: o.exp_avg_sq, torch.zeros(1024, dtype=torch.float64))
    opt = optimizer(bits)
    opt.params.pop()
    with pytest.raises(M.MiniteError):
        step(opt)


@pytest.mark.parametrize("bits", [8, 32])
def test_a_refused_step_leaves_no_address_behind(given, bits):
    """One state is replaced by a good tensor and another by a bad one: refused. With
    the old ones put back, a step uses the old ones."""
    opt = optimizer(bits)
    step(opt)
    old = opt.exp_avg.t, opt.exp_avg_sq.t
    opt.exp_avg.t, opt.exp_avg_sq.t = old[0].clone(), torch.zeros(3)
    with pytest.raises(M.MiniteError):
        step(opt)
    opt.exp_avg.t, opt.exp_avg_sq.t = old
    step(opt)
    check(opt, given[-1], bits)


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [8, 32])
def test_a_run_with_replaced_storage_equals_one_without(bits):
    def tensors(seed):
        g = torch.Generator().manual_seed(seed)
        return [torch.randn(n, generator=g).cuda() for n in SIZES]

    p, q = tensors(1), tensors(1)
    a, b = M.AdamW(p, state_bits=bits), M.AdamW(q, state_bits=bits)
    kept = []
    for s in range(4):
        g = tensors(10 + s)
        a.step(g)
        b.step(g)
        for t in q:
            kept.append(t.data)
            t.data = t.data.clone()
        b.exp_avg, b.exp_avg_sq = b.exp_avg.clone(), b.exp_avg_sq.clone()
    for x, y in zip(p, q):
        assert torch.equal(x, y)
