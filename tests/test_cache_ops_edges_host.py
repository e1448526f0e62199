"""More refusals of the calls around the verify call (no GPU needed): the
checks read shapes, types, strides and pointers only, so CPU tensors stand in."""
import ctypes

import pytest
import torch

import speculative_decode_verify_prefix_gb300 as vsk
from speculative_decode_verify_prefix_gb300 import _native
from test_cache_ops_host import bf, built, call, evict_args, mass_args, ptr, ref, refused, shared_args  # noqa: F401


def test_shared_without_query_heads_is_refused():
    """The cut of the work divides by the query heads of a KV head."""
    refused("h_q must be", call("verify_splitkv_shared_fwd", shared_args(q=bf(8, 0, 64), o=bf(8, 0, 64)), 4, 1.0, 1.0, 0.0))


@pytest.mark.parametrize("name", ["verify_splitkv_mass", "kv_evict"])
def test_indices_past_32_bit_positions_are_refused(name):
    """Positions are 32-bit in the kernels, with room for a step behind the last one."""
    def sized(t, n):  # the view of a longer array (never read here)
        v = vsk.as_vsk(t)
        v.shape[t.dim() - 1] = n
        if t.dim() == 2:
            v.stride[0] = n
        return ctypes.byref(v)

    for n, msg in ((2 ** 31 - 65536 + 1, "too many"), (2 ** 31 - 1, "too many")):
        if name == "kv_evict":
            a = evict_args(m=sized(torch.zeros(2, 20), n), kvi=sized(torch.arange(20), n))
            refused(msg, call(name, a))
        else:
            a = mass_args(m=sized(torch.zeros(2, 20), n), kvi=sized(torch.arange(20), n))
            refused(msg, call(name, a, 4, 1.0, 0.0))


@pytest.mark.parametrize("k_scale,sm_scale", [(100.0, 3e38), (-100.0, 3e38), (0.1, 3e38), (1e-38, 3.2e38)])
@pytest.mark.parametrize("name", ["verify_splitkv_mass", "verify_splitkv_shared_fwd"])
def test_scales_of_keys_and_drafts_beyond_a_float_are_refused(name, k_scale, sm_scale):
    """Cached keys carry sm_scale k_scale log2 e, drafts sm_scale log2 e: with either infinite every weight is NaN, which
    kv_evict takes for the largest."""
    if name == "verify_splitkv_mass":
        got = call(name, mass_args(), 4, k_scale, sm_scale)
    else:
        got = call(name, shared_args(), 4, k_scale, 1.0, sm_scale)
    refused("too large", got)


_BIG = torch.zeros(2, 64)


@pytest.mark.parametrize("change,msg", [
    # one column off, one row off, a view that begins inside, rows of one among the other's
    (dict(m=_BIG[:, 1:21], m_in=_BIG[:, :20]), "mass overlaps mass_in"),
    (dict(m=_BIG.view(-1)[:84].as_strided((2, 20), (64, 1)), m_in=_BIG.view(-1).as_strided((2, 20), (32, 1), 64)),
     "mass overlaps mass_in"),
    (dict(m=_BIG[:, :20], m_in=_BIG[:1, :20].expand(2, 20)), "mass overlaps mass_in"),
    (dict(m=_BIG[:, :20], m_in=_BIG.view(-1).as_strided((2, 20), (44, 1))), "mass overlaps mass_in"),
    # rows of mass that share elements
    (dict(m=_BIG[:1, :20].expand(2, 20)), "rows of mass overlap"),
    (dict(m=_BIG.view(-1).as_strided((2, 20), (19, 1))), "rows of mass overlap"),
])
def test_mass_outputs_that_overlap_are_refused(change, msg):
    refused(msg, call("verify_splitkv_mass", mass_args(**change), 4, 1.0, 0.0))


_OUT = torch.arange(64)


@pytest.mark.parametrize("change,msg", [
    (dict(oi=_OUT[:16], f=_OUT[10:30]), "freed overlaps out_kv_indices"),
    (dict(om=_BIG[:1, :16].expand(2, 16)), "rows of out_mass overlap"),
    (dict(om=_BIG.view(-1).as_strided((2, 16), (15, 1))), "rows of out_mass overlap"),
    (dict(m=_BIG[:, :20], om=_BIG[:, 19:35]), "out_mass overlaps mass"),
    (dict(kvp=_OUT.int()[:3], op=_OUT.int()[3:6], kvi=_OUT[:20], f=_OUT[19:39]), "freed overlaps kv_indices"),
])
def test_evict_outputs_that_overlap_are_refused(change, msg):
    refused(msg, call("kv_evict", evict_args(**change)))


@pytest.mark.parametrize("change", [lambda: vsk.set_tuning(num_ctas=7), lambda: vsk.set_tuning(),
                                    lambda: vsk.set_tuning_shape(max_kv_heads_per_cta=1)])
def test_workspace_sizes_are_asked_again_after_tuning(change):
    """What sizes a workspace is process-wide tuning too, so a size kept from before it says nothing."""
    from speculative_decode_verify_prefix_gb300 import api, cache_ops

    kept = dict(api._WS_SIZE), dict(cache_ops._SIZES)
    try:
        api._WS_SIZE["verify"] = cache_ops._SIZES["shared"] = 1
        change()
        assert "verify" not in api._WS_SIZE and "shared" not in cache_ops._SIZES
    finally:
        vsk.set_tuning()
        vsk.set_tuning_shape()
        api._WS_SIZE.clear()
        cache_ops._SIZES.clear()
        api._WS_SIZE.update(kept[0])
        cache_ops._SIZES.update(kept[1])


def _odd(t):
    """The same values one element off the alignment that calls want."""
    flat = torch.zeros(t.numel() + 1, dtype=t.dtype)
    return flat[1:].view(t.shape)


@pytest.mark.parametrize("change,k_scale,msg", [
    (dict(kb=bf(50, 2, 64).half()), 1.0, "k_buffer must be bf16 or fp8 e4m3"), (dict(ke=bf(8, 2, 64).half()), 1.0, "q_extend and k_extend must be bf16"),
    (dict(kb=bf(50, 3, 64)), 1.0, "between k_extend and k_buffer"), (dict(ke=bf(7, 2, 64)), 1.0, "k_extend rows differ"),
    (dict(kb=_odd(bf(50, 2, 64))), 1.0, "K pool rows"), (dict(ke=_odd(bf(8, 2, 64))), 1.0, "q_extend/k_extend must be 4-byte"),
    (dict(ke=bf(8, 2, 128)), 1.0, "head_dim mismatch"), (dict(q=_odd(bf(8, 8, 64))), 1.0, "4-byte"), (dict(), float("inf"), "k_scale must be finite"),
    (dict(kb=bf(50, 2, 64, 1)), 1.0, "k_buffer must be 3-d"),
])
def test_mass_refusals_name_its_own_arguments(change, k_scale, msg):
    """The weights call has no values and no output rows."""
    assert call("verify_splitkv_mass", mass_args(**change), 4, k_scale, 0.0) == 0
    said = vsk.last_error()
    assert msg in said, said
    for other in ("v_extend", "v_buffer", "v_head_dim", "v_scale", "o_extend"):
        assert other not in said, said


def test_outputs_of_neighbouring_key_counts_are_told_apart():
    """The GPU tests that count keys take bf16 outputs within 2^-18 of count / n: with up to 64 keys of a place, one key
    more or less is outside."""
    count = torch.arange(0, 66, dtype=torch.float64)
    for n in [*range(1, 300), 4097, 20000, 40008, 65537, *torch.randint(300, 70000, (2000,), generator=torch.manual_seed(1)).tolist()]:
        x = count / n
        lo, hi = (x * (1 - 2.0 ** -18)).bfloat16(), (x * (1 + 2.0 ** -18)).bfloat16()
        assert bool((hi[:-1] < lo[1:]).all()), n
