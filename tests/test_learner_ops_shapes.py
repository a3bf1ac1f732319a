"""Tensors with the wrong number of dimensions, a status of another type and a
negative number of alternatives are refused with MiniteError, like every other
argument that does not fit. No GPU is needed: CPU tensors that say they are on
one, and a library that must not be called."""
import ctypes

import pytest
import torch

from nvfp4_w4a4_moe_permute_gb300 import build as B
from nvfp4_w4a4_moe_permute_gb300 import minite as M

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


class On:
    is_cuda, device = True, torch.device("cuda", 0)

    def __init__(self, t):
        self.t = t

    def get_device(self):
        return 0

    def data_ptr(self):
        return 1 << 12

    def __getattr__(self, name):
        return getattr(self.t, name)


class Stream:
    cuda_stream = device_index = 0


def zeros(*shape, dtype=BF):
    return On(torch.zeros(*shape, dtype=dtype))


CALLS = {
    "product": (M.grouped_gemm_bf16, dict(x=zeros(4, 64), w=zeros(2, 32, 64), expert_offsets=zeros(3, dtype=I32),
                                          out=zeros(4, 32))),
    "product with new output": (M.grouped_gemm_bf16, dict(x=zeros(4, 64), w=zeros(2, 32, 64),
                                                          expert_offsets=zeros(3, dtype=I32))),
    "weight gradient": (M.grouped_wgrad_bf16, dict(dy=zeros(4, 32), x=zeros(4, 64), expert_offsets=zeros(3, dtype=I32),
                                                   out=zeros(2, 32, 64, dtype=F32))),
    "weight gradient with new output": (M.grouped_wgrad_bf16, dict(dy=zeros(4, 32), x=zeros(4, 64),
                                                                   expert_offsets=zeros(3, dtype=I32))),
    "log probabilities": (M.token_logprobs, dict(logits=zeros(4, 50), targets=zeros(4, dtype=I32))),
    "log probabilities into buffers": (M.minite_token_logprobs, dict(
        logits=zeros(4, 50), targets=zeros(4, dtype=I32), logprob=zeros(4, dtype=F32), alt_ids=zeros(4, 3, dtype=I32),
        alt_logprobs=zeros(4, 3, dtype=F32))),
    "gradient": (M.minite_token_logprobs_backward, dict(
        logits=zeros(4, 50), targets=zeros(4, dtype=I32), stats=zeros(4, 2, dtype=F32), entropy=zeros(4, dtype=F32),
        grad_logprob=zeros(4, dtype=F32), grad_entropy=zeros(4, dtype=F32), dlogits=zeros(4, 50))),
}


@pytest.fixture(params=CALLS)
def call(request, monkeypatch):
    seen = []

    class Library:
        def __getattr__(self, name):
            return lambda *a: seen.append(name) or 0

    monkeypatch.setattr(M, "load", lambda path=None: Library())
    monkeypatch.setattr(M, "_current_device", lambda: 0)
    monkeypatch.setattr(M, "_empty", lambda shape, dtype, like, stream: On(torch.empty(shape, dtype=dtype)))
    f, args = CALLS[request.param]
    f(**args, status=zeros(1, dtype=I32), stream=Stream)
    assert len(seen) == 1
    yield f, args
    assert len(seen) == 1


def test_dimensions(call):
    f, args = call
    for name, t in args.items():
        for bad in (On(t.t[None]), On(t.t[0]), On(t.t.reshape(-1)) if t.t.dim() > 1 else On(t.t[:0])):
            with pytest.raises(M.MiniteError):
                f(**{**args, name: bad}, stream=Stream)


def test_status(call):
    f, args = call
    for dtype in (torch.uint8, torch.int64, torch.float32):
        with pytest.raises(M.MiniteError):
            f(**args, status=zeros(1, dtype=dtype), stream=Stream)
    with pytest.raises(M.MiniteError):
        f(**args, status=zeros(0, dtype=I32), stream=Stream)


def test_negative_alternatives():
    with pytest.raises(M.MiniteError):
        M.token_logprobs(zeros(4, 50), zeros(4, dtype=I32), alternatives=-1, stream=Stream)


def test_unaligned_status_in_the_library():
    B.build()
    lib = M.load()
    p, odd = ctypes.c_void_p(1 << 12), ctypes.c_void_p((1 << 12) + 2)
    assert lib.minite_grouped_gemm_bf16(p, 64, p, 0, p, 16, 64, 64, 4, p, 64, 0, odd, None) == 1
    assert lib.minite_grouped_wgrad_bf16(p, 64, p, 64, p, 16, 64, 64, 4, p, 1, 0, odd, None) == 1
    assert lib.minite_token_logprobs(p, 0, 4, 100, 100, p, 0, 1.0, p, p, p, 0, None, None, odd, None) == 1
    d = ctypes.c_void_p(1 << 20)
    assert lib.minite_token_logprobs_backward(p, 0, 4, 100, 100, p, 0, 1.0, p, p, p, p, d, 100, odd, None) == 1
