"""Every call compares the device of each operand, and of its stream, with the
current one before anything is enqueued. No GPU is needed: the tensors here are
CPU tensors that say they are on a GPU, and the library is one that only notes
that it was called."""
import numpy as np
import pytest
import torch

from nvfp4_w4a4_moe_permute_gb300 import minite as M

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


class On:
    """A tensor that says that it is on cuda:`index`."""

    is_cuda = True

    def __init__(self, t, index=0):
        self.t, self.index, self.device = t, index, torch.device("cuda", index)

    def get_device(self):
        return self.index

    def data_ptr(self):
        return 1 << 12

    def __getattr__(self, name):
        return getattr(self.t, name)


class Stream:
    cuda_stream = 0

    def __init__(self, index=0):
        self.device_index = index


@pytest.fixture
def calls(monkeypatch):
    """The entry points that a call reached; cuda:0 is current."""
    seen = []

    class Library:
        def __getattr__(self, name):
            return lambda *a: seen.append(name) or 0

    monkeypatch.setattr(M, "load", lambda path=None: Library())
    monkeypatch.setattr(M, "_current_device", lambda: 0, raising=False)
    return seen


def refused_elsewhere(calls, call, operands):
    """`call` takes operands by name: all on cuda:0 it goes through, with one on
    cuda:1, or all, it does not."""
    call(**{k: On(t) for k, t in operands.items()}, stream=Stream())
    assert len(calls) == 1
    for other in list(operands) + ["stream"]:
        with pytest.raises(M.MiniteError, match="device"):
            call(**{k: On(t, int(k == other)) for k, t in operands.items()}, stream=Stream(int(other == "stream")))
    with pytest.raises(M.MiniteError, match="device"):
        call(**{k: On(t, 1) for k, t in operands.items()}, stream=Stream(1))
    assert len(calls) == 1


def test_products(calls):
    o = dict(x=torch.zeros(4, 64, dtype=BF), w=torch.zeros(2, 32, 64, dtype=BF), expert_offsets=torch.zeros(3, dtype=I32),
             out=torch.zeros(4, 32, dtype=BF), status=torch.zeros(1, dtype=I32))
    refused_elsewhere(calls, M.grouped_gemm_bf16, o)


def test_weight_gradients(calls):
    o = dict(dy=torch.zeros(4, 32, dtype=BF), x=torch.zeros(4, 64, dtype=BF), expert_offsets=torch.zeros(3, dtype=I32),
             out=torch.zeros(2, 32, 64), status=torch.zeros(1, dtype=I32))
    refused_elsewhere(calls, M.grouped_wgrad_bf16, o)


def test_log_probabilities(calls):
    o = dict(logits=torch.zeros(4, 50), targets=torch.zeros(4, dtype=I32), logprob=torch.zeros(4), entropy=torch.zeros(4),
             stats=torch.zeros(4, 2), alt_ids=torch.zeros(4, 3, dtype=I32), alt_logprobs=torch.zeros(4, 3),
             status=torch.zeros(1, dtype=I32))
    refused_elsewhere(calls, M.minite_token_logprobs, o)


def test_log_probabilities_with_new_outputs(calls, monkeypatch):
    monkeypatch.setattr(M, "_empty", lambda shape, dtype, like, stream: On(torch.zeros(shape, dtype=dtype), like.index))
    o = dict(logits=torch.zeros(4, 50), targets=torch.zeros(4, dtype=I32), status=torch.zeros(1, dtype=I32))
    refused_elsewhere(calls, lambda **k: M.token_logprobs(alternatives=3, **k), o)


def test_gradient_of_log_probabilities(calls):
    o = dict(logits=torch.zeros(4, 50), targets=torch.zeros(4, dtype=I32), stats=torch.zeros(4, 2), entropy=torch.zeros(4),
             grad_logprob=torch.zeros(4), grad_entropy=torch.zeros(4), dlogits=torch.zeros(4, 50),
             status=torch.zeros(1, dtype=I32))
    refused_elsewhere(calls, M.minite_token_logprobs_backward, o)


@pytest.mark.parametrize("bits", [8, 32])
def test_adamw(calls, bits):
    state = dict(exp_avg=512, exp_avg_sq=512)
    kind = torch.float8_e4m3fn if bits == 8 else F32
    state = {k: On(torch.zeros(n, dtype=kind)) for k, n in state.items()}
    if bits == 8:
        state |= dict(exp_avg_scale=On(torch.zeros(2)), exp_avg_sq_scale=On(torch.zeros(2)))
    params = [On(torch.zeros(7)), On(torch.zeros(100))]

    def step(g0, g1, grad_scale, stream):
        opt.step([g0, g1], grad_scale=grad_scale, stream=stream)

    opt = M.AdamW(params, state_bits=bits, state=dict(state, step=0))
    refused_elsewhere(calls, step, dict(g0=torch.zeros(7), g1=torch.zeros(100), grad_scale=torch.zeros(1)))
    assert opt.step_count == 1


def test_adamw_of_another_device(calls, monkeypatch):
    """Everything on cuda:0 while cuda:1 is current."""
    state = dict(exp_avg=On(torch.zeros(256)), exp_avg_sq=On(torch.zeros(256)), step=0)
    opt = M.AdamW([On(torch.zeros(7))], state=state)
    monkeypatch.setattr(M, "_current_device", lambda: 1)
    with pytest.raises(M.MiniteError, match="device"):
        opt.step([On(torch.zeros(7))], stream=Stream())
    assert not calls


def test_adamw_by_descriptors(calls):
    t = np.zeros(1, dtype=M.ADAMW_TENSOR)
    args = (t, M.OUT_FP32, M.OUT_FP32, 32, 1e-3, 0.9, 0.99, 1e-8, 0.0, 1)
    refused_elsewhere(calls, lambda **k: M.minite_adamw_step(*args, **k), dict(grad_scale=torch.zeros(1)))


def test_the_older_entry_points(calls):
    """They share two helpers."""
    o = dict(expert_out=torch.zeros(8, 64, dtype=BF), dest_row=torch.zeros(4, 2, dtype=I32), y=torch.zeros(4, 64, dtype=BF),
             status=torch.zeros(1, dtype=I32))
    refused_elsewhere(calls, M.minite_moe_combine, o)
