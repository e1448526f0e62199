"""GPU tests of the rotary, append and block-scaled cache calls at corners that the
tests of their formulas do not reach."""
import ctypes
import types

import pytest
import torch

from test_block_ops_gpu import DEV, block_case, block_want, check_block, ints, vsk  # noqa: F401
from test_parity_gpu import gpu_problem, run_gpu

import workloads

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- masks that are not contiguous

def wide(mask):
    """The same mask as a slice of a wider buffer."""
    w = torch.zeros(mask.shape[0], mask.shape[1] + 5, dtype=mask.dtype, device=DEV)
    w[:, :mask.shape[1]] = mask
    return w[:, :mask.shape[1]]


@pytest.mark.parametrize("call", ["blocks", "tree"])
@pytest.mark.parametrize("given", [lambda s: s, lambda s: types.SimpleNamespace(cuda_stream=s.cuda_stream)], ids=["torch's", "another object"])
def test_mask_that_is_not_contiguous_on_another_stream(vsk, call, given):  # noqa: F811
    """The copy is made on the call's stream, so it neither waits for the current one nor is overtaken by the kernels."""
    n, l_ext = 40, 4
    g = torch.Generator(device=DEV)
    g.manual_seed(4)
    draft = torch.rand(2, l_ext, l_ext, generator=g, device=DEV) < 0.5
    mask = wide(torch.cat([torch.ones(2 * l_ext, n, dtype=torch.bool, device=DEV), draft.view(-1, l_ext)], 1))
    at = ints([0, l_ext * (n + l_ext), 2 * l_ext * (n + l_ext)])
    assert not mask.is_contiguous()
    if call == "blocks":
        c = block_case([n, n], 16, 8, 2, 64, l_ext, seed=5)

        def run(m, o=None, **kw):
            o = torch.empty_like(c["q"]) if o is None else o
            vsk.verify_splitkv_block_fwd(c["q"], c["ke"], c["ve"], o, c["kc"], c["vc"], c["ks"], c["vs"], c["qo"], c["table"],
                                         c["lens"], 16, l_ext, custom_mask=m, mask_indptr=at, **kw)
            return o

        check_block(run(mask), *block_want(c["q"], c["ke"], c["ve"], c["kc"], c["vc"], c["ks"], c["vs"], c["table"], [n, n], 16,
                                           l_ext, 64 ** -0.5, list(draft)))
    else:
        p = gpu_problem(workloads.Spec("wide_mask", (n, n), l_ext, 8, 2, 64, 64, perm=True, seed=209))

        def run(m, o=None, **kw):
            o = torch.empty_like(p["q"]) if o is None else o
            assert vsk.verify_splitkv_fwd(p["q"], p["k_ext"], p["v_ext"], o, p["k_buffer"], p["v_buffer"], p["qo_indptr"],
                                          p["kv_indptr"], p["kv_indices"], m, True, at, l_ext, p["k_scale"], p["v_scale"],
                                          sm_scale=p["sm_scale"], **kw)
            return o

        assert not torch.equal(run(mask), run_gpu(vsk, p))  # (the mask is not the causal one)
    want = run(mask.contiguous())
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run(mask.contiguous())  # the stream's workspace is there
    o = torch.zeros_like(want)
    torch.cuda.synchronize()
    late = torch.cuda.Event()
    torch.cuda._sleep(200_000_000)  # the current stream is busy for some 0.1 s
    late.record()
    run(mask, o, stream=given(side))
    over = torch.ones(mask.shape, dtype=torch.bool, device=DEV)  # the copy's memory, if it were the current stream's
    side.synchronize()
    assert not late.query()
    torch.cuda.synchronize()
    assert torch.equal(o, want) and bool(over.all())


# ---------------------------------------------------------------- mask offsets

@pytest.mark.parametrize("call", ["blocks", "tree, one launch", "tree, two launches"])
def test_mask_offsets_near_the_largest(vsk, call):  # noqa: F811
    """An offset to which the mask's size cannot be added is outside the mask like any other: causal drafts, bit 16."""
    n, l_ext = 40, 4
    flat = torch.zeros(2 * l_ext * (n + l_ext), dtype=torch.uint8, device=DEV)
    if call == "blocks":
        c = block_case([n, n], 16, 8, 2, 64, l_ext, seed=5)

        def run(m, at):
            o = torch.empty_like(c["q"])
            vsk.verify_splitkv_block_fwd(c["q"], c["ke"], c["ve"], o, c["kc"], c["vc"], c["ks"], c["vs"], c["qo"], c["table"],
                                         c["lens"], 16, l_ext, custom_mask=m, mask_indptr=at)
            return o
    else:
        p = gpu_problem(workloads.Spec("far_mask", (n, n), l_ext, 8, 2, 64, 64, perm=True, seed=210))

        def run(m, at):
            return run_gpu(vsk, p, custom_mask=m, mask_indptr=at)

        vsk.set_tuning_split_launch(2 if "two" in call else 0)
    try:
        causal = run(None, None)
        vsk.read_error_flags()
        for far in (2 ** 63 - 1, 2 ** 63 - flat.numel() // 2, -2 ** 63):
            at = torch.tensor([far, far, far], device=DEV)
            assert torch.equal(run(flat, at), causal)
            assert vsk.read_error_flags() == 16
    finally:
        vsk.set_tuning_split_launch(1)


# ---------------------------------------------------------------- the binding

def test_views_packed_in_python_are_the_modules(vsk, monkeypatch):  # noqa: F811
    from speculative_decode_verify_prefix_gb300 import _native, cache_ops

    x = torch.zeros(4, 6, 64, dtype=torch.bfloat16, device=DEV)
    tensors = (x, None, x[:, 2:4], x.transpose(0, 1), x.view(torch.uint8), x[0, 0], x[0], x[..., 0, None, None, :], x.bool(), x.double(),
               torch.zeros((), device=DEV), torch.zeros(0, 3, dtype=torch.int32, device=DEV), torch.arange(5, device=DEV))
    names = tuple(f"t{i}" for i in range(len(tensors)))
    size = ctypes.sizeof(_native.VskTensor)
    packed = [pack(names, tensors) for pack in (_native.views(), cache_ops._python_views)]
    (device, _, one), (other_device, _, other) = packed
    assert device == other_device == x.get_device()
    for a, b in zip(one, other):
        assert (a is None) == (b is None) and (a is None or ctypes.string_at(a, size) == ctypes.string_at(b, size))
    for pack in (_native.views(), cache_ops._python_views):
        with pytest.raises(ValueError, match="b must be a strided CUDA tensor"):
            pack(("a", "b"), (x, torch.ones(2, device=DEV).to_sparse()))
    # a whole call without the module
    c = block_case([40, 70], 16, 8, 2, 64, 4, seed=5)

    def run():
        o = torch.empty_like(c["q"])
        vsk.verify_splitkv_block_fwd(c["q"], c["ke"], c["ve"], o, c["kc"], c["vc"], c["ks"], c["vs"], c["qo"], c["table"], c["lens"],
                                     16, 4)
        return o

    want = run()
    assert cache_ops._views is _native.views()
    monkeypatch.setattr(cache_ops, "_views", cache_ops._python_views)
    assert torch.equal(run(), want)


# ---------------------------------------------------------------- large queries

@pytest.mark.parametrize("d,gq", [(64, 2), (128, 4), (256, 8)])
@pytest.mark.parametrize("exponent", [-40, 0, 40])
def test_block_largest_queries_against_zeros(vsk, d, gq, exponent):  # noqa: F811
    """A query's largest elements meet zeros in every key: the scores are 0, whatever the scale of query and block."""
    lens, l_ext = [70, 300], 4
    c = block_case(lens, 16, 2 * gq, 2, d, l_ext, seed=6)
    c["q"].zero_()
    c["q"][:, :, 5] = 3e38
    c["q"][1, :, 9] = -3e38
    live = c["kc"].view(torch.uint8) != 0x7F
    for col in (5, 9):
        c["kc"].view(torch.uint8)[:, :, col] = torch.where(live[:, :, col], 0x80, 0x7F).to(torch.uint8)  # -0
        c["ke"][:, :, col] = 0.0
    c["ks"][c["ks"].isfinite()] = 2.0 ** exponent
    o = torch.empty_like(c["q"])
    vsk.verify_splitkv_block_fwd(c["q"], c["ke"], c["ve"], o, c["kc"], c["vc"], c["ks"], c["vs"], c["qo"], c["table"], c["lens"], 16,
                                 l_ext)
    check_block(o, *block_want(c["q"], c["ke"], c["ve"], c["kc"], c["vc"], c["ks"], c["vs"], c["table"], lens, 16, l_ext, d ** -0.5))
