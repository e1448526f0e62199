"""Corners of the rotary, append and block-scaled cache calls that need no GPU: what
the binding does with a call's tensors before the library sees them, and which views
the library refuses (CPU tensors stand in, see test_block_ops_host.py)."""
import contextlib
import ctypes
import random
import types

import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

import speculative_decode_verify_prefix_gb300 as vsk
from speculative_decode_verify_prefix_gb300 import _native, api, block_ops

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
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda raw, device: types.SimpleNamespace(cuda_stream=raw))
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


# ------------------------------------------------------------------ views that share memory

def call(name, args, *scalars, ws=None):
    keep = [None if a is None else api.as_vsk(a) for a in args]
    ptrs = [None if v is None else ctypes.addressof(v) for v in keep]
    return getattr(_native.lib(), name)(*ptrs, *scalars, *([] if ws is None else [ctypes.c_void_p(ws[0]), ws[1]]), None)


def shared_bytes_refused(name, args, *scalars, ws=None):
    """The refusal for shared bytes, or none; without a GPU a call that passes ends at the device."""
    if torch.cuda.is_available():
        pytest.skip("a call that passes would run")
    assert call(name, args, *scalars, ws=ws) == 0
    return vsk.last_error() if "overlap" in vsk.last_error() else ""


ROOM = torch.zeros(1 << 14, dtype=BF16)


def rows_of(t):
    """Where a view's elements lie."""
    n, h, d = t.shape
    first = torch.arange(n)[:, None] * t.stride(0) + torch.arange(h) * t.stride(1) + t.storage_offset()
    return (first.flatten()[:, None] + torch.arange(d)).flatten()


def test_one_run_shifted_by_less_than_itself():
    k = ROOM.as_strided((1, 1, 64), (8, 8, 1), 0)
    f, pos = torch.ones(32), torch.zeros(1, dtype=torch.int64)
    for by, msg in ((8, "k_out overlaps k"), (56, "k_out overlaps k"), (64, ""), (0, "")):
        ko = ROOM.as_strided((1, 1, 64), (8, 8, 1), by)
        assert shared_bytes_refused("rope_fwd", [None, k, None, ko, pos, f], 0, 1.0) == msg


@pytest.mark.parametrize("form", ["rows", "pool"])
def test_views_of_all_strides_against_their_bytes(form):
    """Views that share a byte are refused; views of equal strides whose runs lie in order are refused only then."""
    r = random.Random(11)
    counts = [0, 0, 0]
    for _ in range(6000):
        n, h, m = r.randint(1, 3), r.randint(1, 3), r.randint(1, 4)  # (the queries' heads, or the pool's rows)
        steps = [8 * r.choice([0, 1, 3, 8, 9, 16, 17, 24, 32, 48, 64, 80]) for _ in range(4)]
        same = r.random() < 0.6
        a = ((n, m) if form == "rows" else (n, h), steps[:2])
        b = ((n, h) if form == "rows" else (m, h), steps[:2] if same else steps[2:])
        x = ROOM.as_strided((*a[0], 64), (*a[1], 1), 4096)
        y = ROOM.as_strided((*b[0], 64), (*b[1], 1), 4096 + 8 * r.randint(-60, 60))
        f, pos = torch.ones(32), torch.zeros(n, dtype=torch.int64)
        if form == "rows":  # queries against the rotated keys
            error = shared_bytes_refused("rope_fwd", [x, bf(n, h, 64), bf(n, m, 64), y, pos, f], 0, 1.0)
        else:  # values against the pool
            error = shared_bytes_refused("rope_append_fwd", [None, bf(n, h, 64), x, None, None, y, bf(m, h, 64), torch.arange(n), pos, f],
                                         0, 1.0, 1.0, 1.0, ws=(256, 256))
        bx, by = rows_of(x), rows_of(y)
        folds = by.unique().numel() < by.numel()
        shares = torch.isin(bx, by).any()
        counts[0] += bool(shares)
        if shares or folds:
            assert error, (x.shape, x.stride(), y.shape, y.stride(), x.storage_offset() - y.storage_offset())
        (s0, s1), hi = b[1], max(x.shape[1], y.shape[1])
        ordered = s1 >= 64 and s0 >= (hi - 1) * s1 + 64
        if same and ordered and not shares:
            counts[1] += 1
            assert not error, (x.shape, x.stride(), y.shape, y.stride(), x.storage_offset() - y.storage_offset())
        counts[2] += not error
    assert min(counts) > 50, counts


# ------------------------------------------------------------------ outputs over what a call reads beside q, k and v

def rope_call(**change):
    a = dict(q=bf(6, 4, 64), k=bf(6, 2, 64), q_out=bf(6, 4, 64), k_out=bf(6, 2, 64), positions=torch.arange(6), inv_freq=torch.ones(32))
    a.update(change)
    return "rope_fwd", a, (0, 1.0), None


def append_call(**change):
    a = dict(q=bf(6, 4, 64), k=bf(6, 2, 64), v=bf(6, 2, 64), q_out=bf(6, 4, 64), k_out=bf(6, 2, 64), k_buffer=bf(20, 2, 64),
             v_buffer=bf(20, 2, 64), out_cache_loc=torch.arange(6), positions=torch.arange(6), inv_freq=torch.ones(32))
    a.update(change)
    return "rope_append_fwd", a, (0, 1.0, 1.0, 1.0), (256, 256)


def cache():
    return dict(k_cache=torch.zeros(64, 2, 64, dtype=torch.uint8).view(E4M3), v_cache=torch.zeros(64, 2, 64, dtype=torch.uint8).view(E4M3),
                k_scales=torch.ones(4, 2), v_scales=torch.ones(4, 2), qo_indptr=ints(0, 3, 6),
                block_table=torch.zeros(2, 2, dtype=torch.int32))


def block_append_call(**change):
    a = dict(q=bf(6, 4, 64), k=bf(6, 2, 64), v=bf(6, 2, 64), q_out=bf(6, 4, 64), k_out=bf(6, 2, 64), **cache(), cache_lens=ints(0, 3),
             positions=torch.arange(6), inv_freq=torch.ones(32))
    a.update(change)
    return "rope_append_block_fwd", a, (16, 0, 1.0), (256, 256)


def block_call(**change):
    a = dict(q_extend=bf(6, 4, 64), k_extend=bf(6, 2, 64), v_extend=bf(6, 2, 64), o_extend=bf(6, 4, 64), **cache(), seq_lens=ints(0, 3),
             custom_mask=torch.zeros(64, dtype=torch.uint8), mask_indptr=torch.tensor([0, 9, 27]))
    a.update(change)
    return "verify_splitkv_block_fwd", a, (16, 3, 0.0), (256, 256)


READ = {rope_call: ("positions", "inv_freq"), append_call: ("positions", "inv_freq", "out_cache_loc"),
        block_append_call: ("positions", "inv_freq", "qo_indptr", "block_table", "cache_lens"),
        block_call: ("k_scales", "v_scales", "qo_indptr", "block_table", "seq_lens", "custom_mask", "mask_indptr")}
WRITTEN = {rope_call: ("q_out", "k_out"), append_call: ("q_out", "k_out", "k_buffer", "v_buffer"),
           block_append_call: ("q_out", "k_out", "k_cache", "v_cache", "k_scales", "v_scales"), block_call: ("o_extend",)}


@pytest.mark.parametrize("make", READ, ids=lambda m: m.__name__)
def test_outputs_over_indices_and_tables(make):
    def error(**change):
        name, a, scalars, ws = make(**change)
        return shared_bytes_refused(name, list(a.values()), *scalars, ws=ws)

    a = make()[1]
    assert error() == ""
    for out in WRITTEN[make]:
        for read in READ[make]:
            x, y = a[out], a[read]
            room = torch.zeros(x.nbytes + y.nbytes, dtype=torch.uint8)

            def at(t, by):
                return room[by:by + t.nbytes].view(t.dtype).view(t.shape)

            for by in (0, x.nbytes - 8):  # the first bytes of what is written, the last ones
                assert error(**{out: at(x, 0), read: at(y, by)}) == f"{out} overlaps {read}", (out, read)
            assert error(**{out: at(x, 0), read: at(y, x.nbytes)}) == "", (out, read)  # behind it
