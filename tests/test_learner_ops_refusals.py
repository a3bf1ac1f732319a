"""The BF16 learner operators refuse bad arguments on the host, before anything
is enqueued (no GPU needed: every call here fails its checks first)."""
import ctypes

import numpy as np
import pytest
import torch

from nvfp4_w4a4_moe_permute_gb300 import build as B
from nvfp4_w4a4_moe_permute_gb300 import minite as M

INVALID, SHAPE = 1, 2
FAKE = ctypes.c_void_p(1 << 12)     # never dereferenced
ODD = ctypes.c_void_p((1 << 12) + 2)


@pytest.fixture(scope="module")
def lib():
    B.build()
    return M.load()


GEMM = dict(a=FAKE, a_stride=64, w=FAKE, w_layout=0, offsets=FAKE, M=16, N=64, K=64, E=4, out=FAKE,
            out_stride=64, out_dtype=0, status=None, stream=None)


@pytest.mark.parametrize("change,rc", [
    (dict(a=None), INVALID), (dict(w=None), INVALID), (dict(offsets=None), INVALID),
    (dict(out=None), INVALID), (dict(out_dtype=2), INVALID), (dict(w_layout=2), INVALID),
    (dict(a=ODD), INVALID), (dict(w=ODD), INVALID), (dict(out=ODD), INVALID),
    (dict(M=-1), SHAPE), (dict(M=1 << 31), SHAPE), (dict(N=0), SHAPE), (dict(N=12), SHAPE),
    (dict(K=4), SHAPE), (dict(K=20, a_stride=24), SHAPE), (dict(E=0), SHAPE), (dict(E=1025), SHAPE),
    (dict(a_stride=56), SHAPE), (dict(a_stride=68), SHAPE), (dict(out_stride=32), SHAPE),
    (dict(out_stride=65), SHAPE), (dict(N=1 << 21, out_stride=1 << 21), SHAPE), (dict(M=1 << 30), SHAPE),
    (dict(N=1 << 20, K=1 << 20, a_stride=1 << 20, out_stride=1 << 20), SHAPE)])
def test_grouped_gemm(lib, change, rc):
    assert lib.minite_grouped_gemm_bf16(*{**GEMM, **change}.values()) == rc


WGRAD = dict(a=FAKE, a_stride=64, b=FAKE, b_stride=64, offsets=FAKE, M=16, Na=64, Nb=64, E=4, out=FAKE,
             out_dtype=1, accumulate=0, status=None, stream=None)


@pytest.mark.parametrize("change,rc", [
    (dict(a=None), INVALID), (dict(b=None), INVALID), (dict(offsets=None), INVALID),
    (dict(out=None), INVALID), (dict(out_dtype=3), INVALID), (dict(out_dtype=0, accumulate=1), INVALID),
    (dict(a=ODD), INVALID), (dict(b=ODD), INVALID), (dict(out=ODD), INVALID), (dict(M=-1), SHAPE),
    (dict(Na=0), SHAPE), (dict(Na=60), SHAPE), (dict(Nb=4), SHAPE), (dict(E=0), SHAPE),
    (dict(E=2000), SHAPE), (dict(a_stride=32), SHAPE), (dict(b_stride=66), SHAPE)])
def test_grouped_wgrad(lib, change, rc):
    assert lib.minite_grouped_wgrad_bf16(*{**WGRAD, **change}.values()) == rc


LOGP = dict(logits=FAKE, dtype=0, N=4, V=100, stride=100, targets=FAKE, t64=0, temperature=1.0,
            logprob=FAKE, entropy=FAKE, stats=FAKE, k=0, ids=None, lps=None, status=None, stream=None)


@pytest.mark.parametrize("change,rc", [
    (dict(logits=None), INVALID), (dict(dtype=2), INVALID), (dict(logprob=None), INVALID),
    (dict(temperature=0.0), INVALID), (dict(temperature=-1.0), INVALID),
    (dict(temperature=float("nan")), INVALID), (dict(temperature=float("inf")), INVALID),
    (dict(temperature=1e-45), INVALID), (dict(k=-1), INVALID), (dict(k=3), INVALID),
    (dict(k=3, ids=FAKE), INVALID), (dict(k=33, ids=FAKE, lps=FAKE), SHAPE),
    (dict(V=5, k=6, ids=FAKE, lps=FAKE), SHAPE), (dict(N=-1), SHAPE), (dict(V=0), SHAPE),
    (dict(V=1 << 31, stride=1 << 31), SHAPE), (dict(stride=99), SHAPE), (dict(dtype=1, logits=ODD), INVALID),
    (dict(stats=ctypes.c_void_p((1 << 12) + 4)), INVALID), (dict(targets=ODD), INVALID),
    (dict(targets=ctypes.c_void_p((1 << 12) + 4), t64=1), INVALID)])
def test_token_logprobs(lib, change, rc):
    assert lib.minite_token_logprobs(*{**LOGP, **change}.values()) == rc


BACK = dict(logits=FAKE, dtype=0, N=4, V=100, stride=100, targets=FAKE, t64=0, temperature=1.0,
            stats=FAKE, entropy=FAKE, gl=FAKE, gh=FAKE, d=ctypes.c_void_p(1 << 20), dstride=100,
            status=None, stream=None)


@pytest.mark.parametrize("change,rc", [
    (dict(logits=None), INVALID), (dict(d=None), INVALID), (dict(stats=None), INVALID),
    (dict(entropy=None), INVALID), (dict(targets=None), INVALID), (dict(dtype=5), INVALID),
    (dict(temperature=0.0), INVALID), (dict(stride=50), SHAPE), (dict(dstride=50), SHAPE),
    (dict(V=0), SHAPE), (dict(N=-2), SHAPE), (dict(d=FAKE, dstride=128), INVALID),
    (dict(dtype=1, d=ODD), INVALID)])
def test_token_logprobs_backward(lib, change, rc):
    assert lib.minite_token_logprobs_backward(*{**BACK, **change}.values()) == rc


def adamw(lib, tensor=None, **change):
    t = np.zeros(1, dtype=M.ADAMW_TENSOR)
    for k in ("param", "grad", "exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale"):
        t[k] = 1 << 12
    t["n"] = 100
    for k, v in (tensor or {}).items():
        t[k] = v
    a = dict(tensors=t.ctypes.data, n=1, pd=1, gd=1, bits=8, lr=1e-3, b1=0.9, b2=0.99, eps=1e-8, wd=0.1,
             step=1, scale=None, stream=None)
    return lib.minite_adamw_step(*{**a, **change}.values())


def test_adamw(lib):
    for k in ("param", "grad", "exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale"):
        assert adamw(lib, {k: 0}) == INVALID, k
        assert adamw(lib, {k: (1 << 12) + 1}) == INVALID, k
    assert adamw(lib, {"exp_avg": (1 << 12) + 8}, bits=32) == INVALID
    assert adamw(lib, {"param_bf16": (1 << 12) + 1}) == INVALID
    assert adamw(lib, {"n": -1}) == SHAPE
    for bad in (dict(tensors=None), dict(n=-1), dict(step=0), dict(bits=16), dict(pd=2), dict(gd=-1),
                dict(b1=1.0), dict(b1=-0.1), dict(b2=1.5), dict(eps=-1.0), dict(lr=float("nan")),
                dict(wd=float("inf")), dict(b2=float("nan"))):
        assert adamw(lib, **bad) == INVALID, bad
    assert adamw(lib, {"n": 0}) == 0            # nothing to do: nothing is enqueued
    assert adamw(lib, n=0, tensors=None) == 0


def test_calls_without_rows_enqueue_nothing(lib):
    assert lib.minite_grouped_gemm_bf16(*{**GEMM, "M": 0, "a": None}.values()) == 0
    assert lib.minite_token_logprobs(*{**LOGP, "N": 0}.values()) == 0
    assert lib.minite_token_logprobs_backward(*{**BACK, "N": 0}.values()) == 0


def test_python_calls_refuse_wrong_tensors(lib):
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    x, w, off = torch.zeros(4, 64, dtype=bf), torch.zeros(2, 32, 64, dtype=bf), torch.zeros(3, dtype=i32)
    logits, y = torch.zeros(4, 50), torch.zeros(4, dtype=i32)
    for call in (
            lambda: M.grouped_gemm_bf16(x, w, off),                                 # not on a GPU
            lambda: M.grouped_gemm_bf16(x.float(), w, off),
            lambda: M.grouped_gemm_bf16(x, w, off.long()),
            lambda: M.grouped_gemm_bf16(x, w, off[:2]),
            lambda: M.grouped_gemm_bf16(x, w, off, w_as_stored=True),               # K does not match
            lambda: M.grouped_gemm_bf16(x, w.transpose(1, 2), off, w_as_stored=True),  # not contiguous
            lambda: M.grouped_gemm_bf16(x.t(), w, off),
            lambda: M.grouped_gemm_bf16(x[:1].expand(4, 64), w, off),               # rows overlap
            lambda: M.grouped_gemm_bf16(x, w, off, out_dtype=torch.float16),
            lambda: M.grouped_gemm_bf16(x, w, off, out=torch.zeros(4, 31, dtype=bf)),
            lambda: M.grouped_wgrad_bf16(x, x[:3], off),
            lambda: M.grouped_wgrad_bf16(x, x, off, accumulate=True),
            lambda: M.token_logprobs(logits.half(), y),
            lambda: M.token_logprobs(logits, y[:3]),
            lambda: M.token_logprobs(logits, y.float()),
            lambda: M.token_logprobs(logits[:1].expand(4, 50), y),
            lambda: M.token_logprobs_backward(logits, y, dict(stats=None, entropy=None)),
            lambda: M.token_logprobs_backward(logits, y, dict(stats=torch.zeros(4, 2), entropy=torch.zeros(4)),
                                              out=torch.zeros(4, 50, dtype=bf)),
            lambda: M.AdamW([torch.zeros(4)])):
        with pytest.raises(M.MiniteError):
            call()
