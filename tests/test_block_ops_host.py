"""Refusals of the rotary, append and block-scaled cache calls (no GPU needed: the
checks read shapes, types, strides and pointers only, so CPU tensors stand in), and
the frequencies against their formulas in 64 bits."""
import ctypes
import math

import pytest
import torch

import speculative_decode_verify_prefix_gb300 as vsk
from speculative_decode_verify_prefix_gb300 import _native

BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn
view = vsk.api.as_vsk


@pytest.fixture(scope="module", autouse=True)
def built():
    vsk.build()


def bf(*shape):
    return torch.zeros(*shape, dtype=BF16)


def e4(*shape):
    return torch.zeros(*shape, dtype=torch.uint8).view(E4M3)


def ints(*x):
    return torch.tensor(x, dtype=torch.int32)


def call(name, args, *scalars, ws=(None, 0)):
    keep = [None if a is None else view(a) for a in args]
    ptrs = [None if v is None else ctypes.addressof(v) for v in keep]
    more = [] if ws is None else [ctypes.c_void_p(ws[0]), ws[1]]
    return getattr(_native.lib(), name)(*ptrs, *scalars, *more, None)


def refused(msg, got):
    assert got == 0
    assert msg in vsk.last_error(), vsk.last_error()


def shifted(dtype, *shape, by=1):
    """A tensor whose data begins `by` elements behind an aligned place."""
    n = math.prod(shape)
    return torch.zeros(n + by, dtype=dtype)[by:].view(*shape)


# ------------------------------------------------------------------ frequencies

def ramp(x, lo, hi):
    return min(1.0, max(0.0, (x - lo) / (hi - lo)))


@pytest.mark.parametrize("rot", [2, 16, 48, 64, 128, 256])
@pytest.mark.parametrize("base", [10000.0, 500000.0])
def test_frequencies(rot, base):
    def plain(b):
        return [b ** (-2.0 * i / rot) for i in range(rot // 2)]

    def check(got, want, size, want_size):
        assert got.dtype == torch.float32 and len(got) == rot // 2
        for g, w in zip(got.tolist(), want):
            assert abs(g - w) <= 2.0 ** -24 * 1.001 * w  # one rounding to 32 bits
        assert abs(size - want_size) <= 2.0 ** -23

    f = plain(base)
    check(*swap(vsk.rope_frequencies(rot, base, device="cpu"), f, 1.0))
    check(*swap(vsk.rope_frequencies(rot, base, "linear", 8.0, device="cpu"), [x / 8 for x in f], 1.0))
    if rot >= 4:
        check(*swap(vsk.rope_frequencies(rot, base, "base", 8.0, device="cpu"), plain(base * 8.0 ** (rot / (rot - 2.0))), 1.0))
    orig, factor = 4096.0, 16.0
    turns = [orig * x / (2 * math.pi) for x in f]
    slow = [1.0 - ramp(t, 1.0, 4.0) for t in turns]
    check(*swap(vsk.rope_frequencies(rot, base, "bands", factor, orig, device="cpu"),
                [x * (1 - s) + x / factor * s for x, s in zip(f, slow)], 1.0))
    lo, hi = (rot * math.log(orig / (r * 2 * math.pi)) / (2 * math.log(base)) for r in (32.0, 1.0))
    lo, hi = max(0.0, math.floor(lo)), min(rot - 1.0, math.ceil(hi))
    slow = [ramp(i, lo, hi if hi > lo else lo + 1e-3) for i in range(rot // 2)]
    check(*swap(vsk.rope_frequencies(rot, base, "ramp", factor, orig, device="cpu"),
                [x * (1 - s) + x / factor * s for x, s in zip(f, slow)], 1 + 0.1 * math.log(factor)))


def swap(got, want, want_size):
    return got[0], want, got[1], want_size


@pytest.mark.parametrize("args,msg", [
    ((63,), "even"), ((0,), "even"), ((64, 1.0), "base"), ((64, float("nan")), "base"), ((64, 1e4, "linear", 0.5), "factor"),
    ((64, 1e4, "ramp", 4.0), "original_len"), ((64, 1e4, "bands", 4.0, 4096, 4.0, 4.0), "low < high"),
    ((2, 1e4, "base", 4.0), "rot_dim of at least 4"), ((64, 1e4, "cubic"), "none of"),
])
def test_frequencies_refused(args, msg):
    with pytest.raises(ValueError, match=msg):
        vsk.rope_frequencies(*args, device="cpu")


# ------------------------------------------------------------------ rope_fwd

def rope_args(**change):
    a = dict(q=bf(6, 4, 64), k=bf(6, 2, 64), qo=bf(6, 4, 64), ko=bf(6, 2, 64), pos=torch.arange(6), f=torch.ones(32))
    return [*{**a, **change}.values()]


@pytest.mark.parametrize("change,msg", [
    (dict(q=None), "go together"), (dict(qo=None), "go together"), (dict(ko=None), "k_out is NULL"), (dict(k=None), "k is NULL"),
    (dict(q=bf(6, 4, 64).half()), "q must be bf16"), (dict(ko=torch.zeros(6, 2, 64)), "k_out must be bf16"),
    (dict(q=bf(5, 4, 64)), "q must be [6, 4, 64]"), (dict(qo=bf(6, 3, 64)), "q_out must be [6, 4, 64]"),
    (dict(ko=bf(6, 2, 128)), "k_out must be [6, 2, 64]"), (dict(k=bf(6, 2, 96)), "head_dim 96"),
    (dict(k=bf(6, 0, 64)), "at least one head"), (dict(q=bf(6, 0, 64), qo=bf(6, 0, 64)), "at least one head"),
    (dict(q=shifted(BF16, 6, 4, 64)), "q rows must be 16-byte aligned"),
    (dict(ko=bf(6, 2, 68)[..., :64]), "k_out rows must be 16-byte aligned"), (dict(q=bf(6, 4, 128)[..., ::2]), "contiguous"),
    (dict(pos=torch.arange(5)), "one entry per row"), (dict(pos=torch.arange(6.0)), "positions must be int32 or int64"),
    (dict(pos=torch.arange(12)[::2]), "contiguous"), (dict(pos=torch.zeros(6, 1).long()), "1-d"),
    (dict(f=torch.ones(32).double()), "inv_freq must be float32"), (dict(f=torch.ones(33)), "multiple of 16"),
    (dict(f=torch.ones(0)), "multiple of 16"), (dict(f=torch.ones(40)), "multiple of 16"), (dict(f=torch.ones(4)), "multiple of 16"),
    (dict(q=bf(6, 256)), "3-d"),
])
def test_rope_refusals(change, msg):
    refused(msg, call("rope_fwd", rope_args(**change), 0, 1.0, ws=None))


@pytest.mark.parametrize("size", [float("nan"), float("inf")])
def test_rope_refuses_a_factor_that_is_not_finite(size):
    refused("attention_factor", call("rope_fwd", rope_args(), 0, size, ws=None))


def overlap_error(args):
    """The refusal for shared bytes; without a GPU a call that passes ends at the device."""
    call("rope_fwd", args, 0, 1.0, ws=None)
    e = vsk.last_error()
    return e if "overlap" in e else ""


def test_rope_views_of_one_buffer():
    x = bf(6, 8, 64)  # 4 query, 2 key, 2 value heads a row
    q, k, v = x[:, :4], x[:, 4:6], x[:, 6:]
    y = bf(6, 6, 64)
    assert overlap_error(rope_args(q=q, k=k)) == ""
    assert overlap_error(rope_args(q=q, k=k, qo=q, ko=k)) == ""  # in place
    assert overlap_error(rope_args(q=q, k=k, qo=y[:, :4], ko=y[:, 4:])) == ""
    assert overlap_error(rope_args(q=q, k=k, qo=q, ko=v)) == ""  # over the values: no byte of q or k
    assert "k_out overlaps q" in overlap_error(rope_args(q=q, k=k, ko=x[:, 2:4]))
    assert "q_out overlaps k" in overlap_error(rope_args(q=q, k=k, qo=x[:, 4:]))
    assert "q_out overlaps q" in overlap_error(rope_args(q=q, k=k, qo=x[:, 3:7]))
    assert "k_out overlaps q_out" in overlap_error(rope_args(qo=y[:, :4], ko=y[:, 3:5]))
    z = bf(7, 8, 64)
    assert "q_out overlaps q" in overlap_error(rope_args(q=z[:6, :4], k=k, qo=z[1:, :4]))  # a row further on
    assert overlap_error(rope_args(q=z[:6, :4], k=k, qo=z[1:, 4:])) == ""
    w = bf(6, 2, 3, 64)  # two queries and a key, head after head
    assert overlap_error(rope_args(q=bf(6, 4, 64), k=w[:, :, 2], ko=w[:, :, 1])) == ""
    assert "k_out overlaps k" in overlap_error(rope_args(k=w[:, :, 2], ko=w.view(6, 6, 64)[:, 2:4]))


def test_rope_outputs_that_fold():
    assert "rows of q_out overlap" in overlap_error(rope_args(qo=bf(1, 4, 64).expand(6, 4, 64)))
    assert "rows of k_out overlap" in overlap_error(rope_args(ko=bf(6, 1, 64).expand(6, 2, 64)))
    heads_first = bf(4, 6, 64).transpose(0, 1)
    assert overlap_error(rope_args(qo=heads_first)) == ""


def test_rope_without_rows_launches_nothing():
    a = rope_args(q=bf(0, 4, 64), k=bf(0, 2, 64), qo=bf(0, 4, 64), ko=bf(0, 2, 64), pos=torch.arange(0))
    assert call("rope_fwd", a, 0, 1.0, ws=None) == 1


# ------------------------------------------------------------------ rope_append_fwd

def append_args(**change):
    a = dict(q=bf(6, 4, 64), k=bf(6, 2, 64), v=bf(6, 2, 64), qo=bf(6, 4, 64), ko=bf(6, 2, 64), kb=bf(20, 2, 64), vb=bf(20, 2, 64),
             loc=torch.arange(6), pos=torch.arange(6), f=torch.ones(32))
    return [*{**a, **change}.values()]


@pytest.mark.parametrize("change,msg", [
    (dict(v=None), "v is NULL"), (dict(v=bf(6, 3, 64)), "v must be [6, 2, 64]"), (dict(kb=e4(20, 2, 64)), "both be bf16 or both"),
    (dict(kb=torch.zeros(20, 2, 64), vb=torch.zeros(20, 2, 64)), "both be bf16 or both"), (dict(vb=bf(19, 2, 64)), "[pool, 2, 64]"),
    (dict(kb=bf(20, 1, 64)), "[pool, 2, 64]"), (dict(kb=e4(20, 2, 72)[..., :64], vb=e4(20, 2, 72)[..., :64]), "16-byte"),
    (dict(vb=shifted(BF16, 20, 2, 64)), "16-byte"), (dict(loc=torch.arange(7)), "out_cache_loc must have one entry"),
    (dict(loc=torch.arange(6.0)), "out_cache_loc must be int32 or int64"), (dict(kb=None), "NULL"),
    (dict(vb=bf(1, 2, 64).expand(20, 2, 64)), "rows of v_buffer overlap"),
])
def test_append_refusals(change, msg):
    refused(msg, call("rope_append_fwd", append_args(**change), 0, 1.0, 1.0, 1.0))


@pytest.mark.parametrize("ks,vs", [(0.0, 1.0), (1.0, -1.0), (float("nan"), 1.0), (1.0, float("inf"))])
def test_append_refuses_scales(ks, vs):
    refused("k_scale > 0", call("rope_append_fwd", append_args(), 0, 1.0, ks, vs))


def test_append_refuses_shared_bytes():
    pool = bf(40, 2, 64)
    refused("v_buffer overlaps k_buffer", call("rope_append_fwd", append_args(kb=pool[:20], vb=pool[10:30]), 0, 1.0, 1.0, 1.0))
    refused("k_buffer overlaps v", call("rope_append_fwd", append_args(v=pool[:6], kb=pool[:20]), 0, 1.0, 1.0, 1.0))
    refused("k_buffer overlaps k_out", call("rope_append_fwd", append_args(ko=pool[4:10], kb=pool[:20]), 0, 1.0, 1.0, 1.0))


def test_append_workspace_too_small():
    refused("smaller than 256", call("rope_append_fwd", append_args(), 0, 1.0, 1.0, 1.0, ws=(256, 255)))


# ------------------------------------------------------------------ rope_append_block_fwd

def block_append_args(**change):
    a = dict(q=bf(6, 4, 64), k=bf(6, 2, 64), v=bf(6, 2, 64), qo=bf(6, 4, 64), ko=bf(6, 2, 64), kc=e4(64, 2, 64), vc=e4(64, 2, 64),
             ks=torch.ones(4, 2), vs=torch.ones(4, 2), p=ints(0, 2, 6), bt=torch.zeros(2, 2, dtype=torch.int32), lens=ints(0, 3),
             pos=torch.arange(6), f=torch.ones(32))
    return [*{**a, **change}.values()]


CACHE = [
    (dict(kc=bf(64, 2, 64)), "fp8 e4m3"), (dict(kc=e4(64, 1, 64)), "[blocks * block_size, 2, 64]"),
    (dict(vc=e4(80, 2, 64)), "[blocks * block_size, 2, 64]"), (dict(kc=e4(72, 2, 64), vc=e4(72, 2, 64)), "whole number of blocks"),
    (dict(kc=e4(64, 2, 72)[..., :64]), "16-byte"), (dict(ks=torch.ones(4, 2).double()), "k_scales must be float32"),
    (dict(vs=torch.ones(5, 2)), "v_scales must be [4, 2]"), (dict(vs=torch.ones(4, 4)[:, ::2]), "contiguous"),
    (dict(ks=torch.ones(8)), "2-d"), (dict(bt=torch.zeros(2, 2).long()), "must be int32"), (dict(lens=ints(0, 3).long()), "must be int32"),
    (dict(bt=torch.zeros(3, 2, dtype=torch.int32)), "one row per sequence"), (dict(lens=ints(0)), "one entry per sequence"),
    (dict(bt=torch.zeros(2, 0, dtype=torch.int32)), "no columns"), (dict(bt=torch.zeros(2, 4, dtype=torch.int32)[:, ::2]), "contiguous"),
    (dict(bt=torch.zeros(2, dtype=torch.int32)), "2-d"), (dict(lens=None), "NULL"),
]


@pytest.mark.parametrize("change,msg", CACHE + [
    (dict(p=ints(0, 6)), "one row per sequence"), (dict(p=ints(0)), "batch size"), (dict(p=torch.tensor([0, 2, 6])), "qo_indptr must be int32"),
    (dict(v=None), "v is NULL"),
])
def test_block_append_refusals(change, msg):
    refused(msg, call("rope_append_block_fwd", block_append_args(**change), 16, 0, 1.0))


@pytest.mark.parametrize("block", [0, -16, 8, 24, 144, 256])
def test_block_sizes_refused(block):
    refused("block_size", call("rope_append_block_fwd", block_append_args(), block, 0, 1.0))
    refused("block_size", call("verify_splitkv_block_fwd", block_args(), block, 2, 0.0))


def test_block_append_refuses_shared_bytes():
    s = torch.ones(8, 2)
    refused("v_scales overlaps k_scales", call("rope_append_block_fwd", block_append_args(ks=s[:4], vs=s[2:6]), 16, 0, 1.0))
    c = e4(128, 2, 64)
    refused("v_cache overlaps k_cache", call("rope_append_block_fwd", block_append_args(kc=c[:64], vc=c[32:96]), 16, 0, 1.0))


def test_block_append_workspace_too_small():
    refused("smaller than 256", call("rope_append_block_fwd", block_append_args(), 16, 0, 1.0, ws=(256, 128)))


# ------------------------------------------------------------------ verify_splitkv_block_fwd

def block_args(**change):
    a = dict(q=bf(4, 4, 64), ke=bf(4, 2, 64), ve=bf(4, 2, 64), o=bf(4, 4, 64), kc=e4(64, 2, 64), vc=e4(64, 2, 64),
             ks=torch.ones(4, 2), vs=torch.ones(4, 2), p=ints(0, 2, 4), bt=torch.zeros(2, 2, dtype=torch.int32), lens=ints(0, 3),
             cm=None, mi=None)
    return [*{**a, **change}.values()]


MASK = torch.zeros(64, dtype=torch.uint8)


@pytest.mark.parametrize("change,msg", CACHE + [
    (dict(q=bf(5, 4, 64)), "ragged"), (dict(q=bf(4, 3, 64), o=bf(4, 3, 64)), "multiple of h_kv"),
    (dict(q=bf(4, 0, 64), o=bf(4, 0, 64)), "multiple of h_kv"),
    (dict(ke=bf(4, 2, 128)), "k_extend and v_extend must be"), (dict(ve=bf(4, 1, 64)), "k_extend and v_extend must be"),
    (dict(o=bf(4, 4, 128)), "shape of q_extend"), (dict(o=bf(4, 4, 64).half()), "must be bf16"),
    (dict(q=bf(4, 4, 96), ke=bf(4, 2, 96), ve=bf(4, 2, 96), o=bf(4, 4, 96)), "head_dim 96"),
    (dict(q=bf(4, 130, 64), o=bf(4, 130, 64)), "exceeds 128"), (dict(q=shifted(BF16, 4, 4, 64)), "4-byte"),
    (dict(ve=bf(8, 65)[:, :64].view(4, 2, 64)), "4-byte"), (dict(o=None), "NULL"),
    (dict(cm=MASK), "go together"), (dict(mi=ints(0, 10, 20)), "go together"),
    (dict(cm=MASK.int(), mi=ints(0, 10, 20)), "custom_mask must be uint8"), (dict(cm=MASK, mi=ints(0, 10)), "B+1"),
    (dict(cm=MASK, mi=torch.zeros(3)), "mask_indptr must be int32 or int64"), (dict(o=bf(4, 1, 64).expand(4, 4, 64)), "rows of o_extend"),
])
def test_block_refusals(change, msg):
    refused(msg, call("verify_splitkv_block_fwd", block_args(**change), 16, 2, 0.0))


def test_block_refuses_shared_bytes_and_scales():
    x = bf(8, 4, 64)
    refused("o_extend overlaps q_extend", call("verify_splitkv_block_fwd", block_args(q=x[:4], o=x[2:6]), 16, 2, 0.0))
    refused("sm_scale is too large", call("verify_splitkv_block_fwd", block_args(), 16, 2, 3e38))
    refused("max_len_extend", call("verify_splitkv_block_fwd", block_args(), 16, 0, 0.0))


@pytest.mark.parametrize("shape", [(0, 8, 2, 64, 4), (2, 8, 3, 64, 4), (2, 8, 2, 96, 4), (2, 8, 2, 64, 0), (2, 130, 2, 64, 2)])
def test_block_workspace_of_unsupported_shapes(shape):
    assert vsk.block_workspace_size(*shape) == 0


@pytest.mark.parametrize("name", ["rope_fwd", "rope_append_fwd", "rope_append_block_fwd", "verify_splitkv_block_fwd"])
def test_python_names_tensors_that_are_not_on_a_gpu(name):
    made = {"rope_fwd": rope_args, "rope_append_fwd": append_args, "rope_append_block_fwd": block_append_args,
            "verify_splitkv_block_fwd": block_args}[name]()
    if name == "rope_append_block_fwd":
        made = made[:12] + [16] + made[12:]
    if name == "verify_splitkv_block_fwd":
        made = made[:11] + [16, 2]
    with pytest.raises(ValueError, match="q(_extend)? must be a CUDA tensor"):
        getattr(vsk, name)(*made)
