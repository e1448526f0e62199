"""Refusals of the calls around the verify call (no GPU needed): the checks
read shapes, types, strides and pointers only, so CPU tensors stand in."""
import ctypes

import pytest
import torch

import speculative_decode_verify_prefix_gb300 as vsk
from speculative_decode_verify_prefix_gb300 import _native

BF16 = torch.bfloat16
ref = vsk.api._ref


@pytest.fixture(scope="module", autouse=True)
def built():
    vsk.build()


def bf(*shape):
    return torch.zeros(*shape, dtype=BF16)


def ptr(*x):
    return torch.tensor(x, dtype=torch.int32)


def call(name, args, *scalars, ws=(None, 0)):
    t = [None if a is None else ref(a) if isinstance(a, torch.Tensor) else a for a in args]
    return getattr(_native.lib(), name)(*t, *scalars, ctypes.c_void_p(ws[0]), ws[1], None)


def refused(msg, got):
    assert got == 0
    assert msg in vsk.last_error(), vsk.last_error()


PROMPT = dict(q=bf(10, 8, 64), k=bf(10, 2, 64), v=bf(10, 2, 64), o=bf(10, 8, 64), p=ptr(0, 4, 10))


@pytest.mark.parametrize("change,msg", [
    (dict(q=bf(10, 8, 64).half()), "bf16"), (dict(o=torch.zeros(10, 8, 64)), "bf16"),
    (dict(p=ptr(0, 4, 10).long()), "int32"), (dict(p=ptr(0)), "batch size"),
    (dict(q=bf(10, 7, 64), o=bf(10, 7, 64)), "multiple of h_kv"), (dict(k=bf(10, 0, 64), v=bf(10, 0, 64)), "multiple of h_kv"),
    (dict(q=bf(10, 8, 96), k=bf(10, 2, 96), v=bf(10, 2, 96), o=bf(10, 8, 96)), "head_dim 96"),
    (dict(v=bf(10, 2, 128)), "k and v must be"), (dict(v=bf(9, 2, 64)), "k and v must be"),
    (dict(k=bf(10, 4, 64)), "k and v must be"), (dict(o=bf(10, 8, 64)[:9]), "shape of q"),
    (dict(q=bf(10, 258, 64), o=bf(10, 258, 64)), "exceeds 128"),
    (dict(k=torch.zeros(10 * 128 + 4, dtype=BF16)[4:].view(10, 2, 64)), "16-byte"),
    (dict(v=bf(10, 2, 68)[:, :, :64]), "16-byte"), (dict(q=bf(10 * 8, 65)[:, :64].view(10, 8, 64)), "4-byte"),
    (dict(o=torch.zeros(10 * 512 + 1, dtype=BF16)[1:].view(10, 8, 64)), "4-byte"),
    (dict(q=bf(10, 8, 128)[:, :, ::2]), "contiguous"), (dict(k=bf(20, 64)), "3-d"), (dict(q=None), "NULL"),
])
def test_prompt_refusals(change, msg):
    a = {**PROMPT, **change}
    refused(msg, call("prompt_attn_fwd", [a["q"], a["k"], a["v"], a["o"], a["p"]], 0.0))


def test_scales_beyond_a_float_are_refused():
    refused("too large", call("prompt_attn_fwd", PROMPT.values(), 3.2e38, ws=(None, 0)))
    refused("too large", call("verify_splitkv_shared_fwd", shared_args(), 4, 100.0, 1.0, 3e38))


def test_prompt_workspace_too_small():
    refused("smaller than 256", call("prompt_attn_fwd", PROMPT.values(), 0.0, ws=(256, 255)))


def test_prompt_without_rows_launches_nothing():
    a = [bf(0, 8, 64), bf(0, 2, 64), bf(0, 2, 64), bf(0, 8, 64), ptr(0, 0)]
    assert call("prompt_attn_fwd", a, 0.0) == 1


def shared_args(**change):
    a = dict(q=bf(8, 8, 64), ke=bf(8, 2, 64), ve=bf(8, 2, 64), o=bf(8, 8, 64), kb=bf(50, 2, 64), vb=bf(50, 2, 64),
             qo=ptr(0, 4, 8), kvp=ptr(0, 10, 20), kvi=torch.arange(20), sh=torch.arange(20, 50))
    return [*{**a, **change}.values()]


@pytest.mark.parametrize("change,msg", [
    (dict(sh=torch.zeros(5)), "shared_indices must be int32 or int64"), (dict(sh=torch.zeros(5, 1).long()), "1-d"),
    (dict(sh=torch.arange(60)[::2]), "contiguous"), (dict(sh=None), "NULL"), (dict(q=bf(7, 8, 64)), "ragged"),
    (dict(ve=bf(8, 2, 128), vb=bf(50, 2, 128), o=bf(8, 8, 128)), "must be equal"),
    (dict(o=bf(8, 8, 128)), "o_extend"), (dict(kb=bf(50, 2, 64).half()), "k_buffer"),
])
def test_shared_refusals(change, msg):
    refused(msg, call("verify_splitkv_shared_fwd", shared_args(**change), 4, 1.0, 1.0, 0.0))


def test_shared_refuses_scales_that_are_not_finite():
    refused("finite", call("verify_splitkv_shared_fwd", shared_args(), 4, float("nan"), 1.0, 0.0))


def mass_args(**change):
    a = dict(q=bf(8, 8, 64), ke=bf(8, 2, 64), kb=bf(50, 2, 64), qo=ptr(0, 4, 8), kvp=ptr(0, 10, 20),
             kvi=torch.arange(20), m_in=None, m=torch.zeros(2, 20))
    return [*{**a, **change}.values()]


@pytest.mark.parametrize("change,msg", [
    (dict(m=torch.zeros(2, 20).double()), "float32"), (dict(m=torch.zeros(3, 20)), "one row per KV head"),
    (dict(m=torch.zeros(2, 19)), "one column per"), (dict(m=torch.zeros(2, 40)[:, ::2]), "contiguous"),
    (dict(m_in=torch.zeros(2, 21)), "mass_in must have one column"), (dict(m_in=bf(2, 20)), "float32"),
    (dict(m=torch.zeros(40)), "2-d"), (dict(q=bf(9, 8, 64)), "ragged"), (dict(m=None), "NULL"),
])
def test_mass_refusals(change, msg):
    refused(msg, call("verify_splitkv_mass", mass_args(**change), 4, 1.0, 0.0))


def evict_args(budget=8, recent=2, **change):
    a = dict(m=torch.zeros(2, 20), kvp=ptr(0, 10, 20), kvi=torch.arange(20), b=budget, r=recent, op=ptr(0, 0, 0),
             oi=torch.arange(16), om=torch.zeros(2, 16), f=torch.arange(20))
    return [*{**a, **change}.values()]


_KVI = torch.arange(40)


@pytest.mark.parametrize("change,msg", [
    (dict(budget=0), "budget must be"), (dict(recent=9), "recent must be"), (dict(recent=-1), "recent must be"),
    (dict(oi=torch.arange(16).int()), "type of kv_indices"), (dict(f=torch.arange(20).int()), "type of kv_indices"),
    (dict(om=torch.zeros(2, 15)), "one column per out_kv_indices"), (dict(om=torch.zeros(1, 16)), "one row per KV head"),
    (dict(op=ptr(0, 0)), "B+1"), (dict(kvp=ptr(0, 10, 20).long()), "int32"), (dict(m=torch.zeros(2, 21)), "one column per"),
    (dict(m=torch.zeros(0, 20)), "one row per KV head"), (dict(kvi=torch.zeros(20)), "int32 or int64"),
    (dict(kvi=_KVI[:20], oi=_KVI[10:26]), "overlaps"), (dict(kvi=_KVI[:20], f=_KVI[:20]), "overlaps"),
    (dict(kvp=ptr(0)), "batch size"),
])
def test_evict_refusals(change, msg):
    refused(msg, call("kv_evict", evict_args(**change)))


def test_python_calls_want_cuda_tensors():
    with pytest.raises(ValueError, match="CUDA"):
        vsk.prompt_attn_fwd(*PROMPT.values())
    a = shared_args()
    with pytest.raises(ValueError, match="CUDA"):
        vsk.verify_splitkv_shared_fwd(*a, 4)
    a = mass_args()
    with pytest.raises(ValueError, match="CUDA"):
        vsk.verify_splitkv_mass(*a[:6], a[7], 4)
    with pytest.raises(ValueError, match="CUDA"):
        vsk.kv_evict(*evict_args())
