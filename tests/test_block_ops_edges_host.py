"""Corners of the rotary, append and block-scaled cache calls that need no GPU: what
the binding does with a call's tensors before the library sees them, and which views
the library refuses (CPU tensors stand in, see test_block_ops_host.py)."""
import contextlib
import types

import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

import speculative_decode_verify_prefix_gb300 as vsk
from speculative_decode_verify_prefix_gb300 import api, block_ops

BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def built():
    vsk.build()


def bf(*shape):
    return torch.zeros(*shape, dtype=BF16)


def ints(*x):
    return torch.tensor(x, dtype=torch.int32)


# ------------------------------------------------------------------ masks that are not contiguous

@pytest.fixture
def streams(monkeypatch):
    """The streams made current, innermost last."""
    current = []

    @contextlib.contextmanager
    def stream(s):
        current.append(s)
        yield
        current.pop()

    monkeypatch.setattr(torch.cuda, "stream", stream)
    return current


class Copies(TorchDispatchMode):
    """The stream that is current at each copy."""

    def __init__(self, current):
        super().__init__()
        self.current, self.seen = current, []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        if any(n in str(func) for n in ("clone", "copy", "contiguous")):
            self.seen.append(self.current[-1] if self.current else None)
        return func(*args, **(kwargs or {}))


WIDE = (torch.arange(2 * 3 * 9) % 5 > 1).view(6, 9)


@pytest.mark.parametrize("cut", [slice(None, 7), slice(None)])
def test_block_call_copies_a_mask_on_its_own_stream(monkeypatch, streams, cut):
    got = {}
    monkeypatch.setattr(block_ops, "_run", lambda name, names, ts, *a: got.update(zip(names, ts)))
    other, mask = types.SimpleNamespace(cuda_stream=5), WIDE[:, cut]
    x = bf(6, 2, 64)
    with Copies(streams) as copies:
        vsk.verify_splitkv_block_fwd(x, x, x, x, x, x, x, x, ints(0, 3, 6), ints(0), ints(0), 16, 3, custom_mask=mask,
                                     mask_indptr=ints(0, 21, 42), stream=other)
    assert copies.seen == ([other] if cut.stop else [])
    assert torch.equal(got["custom_mask"], mask.flatten())


@pytest.mark.parametrize("cut", [slice(None, 7), slice(None)])
def test_tree_call_copies_a_mask_on_its_own_stream(monkeypatch, streams, cut):
    other, mask = types.SimpleNamespace(cuda_stream=5), WIDE[:, cut]
    kept, refs = [], api._ref
    monkeypatch.setattr(api, "_gate", lambda *a: True)
    monkeypatch.setattr(api, "_ref", lambda t: kept.append(t) or refs(t))
    monkeypatch.setattr(api._native, "lib", lambda: types.SimpleNamespace(verify_splitkv_tree_fwd=lambda *a: 1))
    x = bf(6, 2, 64)
    with Copies(streams) as copies:
        assert vsk.verify_splitkv_fwd(x, x, x, x, x, x, ints(0, 3, 6), ints(0, 0, 0), ints(0), mask, True, ints(0, 21, 42), 3, 1.0,
                                      1.0, workspace=torch.zeros(256, dtype=torch.uint8), stream=other)
    assert copies.seen == ([other] if cut.stop else [])
    assert any(t.dtype == torch.uint8 and torch.equal(t.bool(), mask.flatten()) for t in kept if t.dim() == 1)
