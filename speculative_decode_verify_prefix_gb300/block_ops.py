"""Python binding of the calls between the projections and the verify call:
rotary positions, the same with the keys and values stored into a pool of rows or
into a block-scaled e4m3 cache, and the verify call over that cache.

As in cache_ops.py: argument marshalling only, on the given stream (default: the
current one of the tensors' device) and without synchronising; a rejected call
raises ValueError and launches nothing; ``workspace`` as there.
"""
from __future__ import annotations

import ctypes

import torch

from . import _native
from .api import _BLOCK_SIZE as _SIZES, _flat_mask
from .cache_ops import _run

_SCALINGS = {"plain": 0, "linear": 1, "base": 2, "ramp": 3, "bands": 4}


def rope_frequencies(rot_dim, base=10000.0, scaling="plain", factor=1.0, original_len=0, low=1.0, high=None,
                     device="cuda"):
    """What every pair of rotated elements turns by per position ([rot_dim / 2]
    float32 on ``device``), and the factor the rotated elements are multiplied by.

    ``scaling`` for contexts ``factor`` times longer than the ``original_len``
    positions a model was trained on: "linear" divides every frequency by the
    factor, "base" raises the base instead, "ramp" and "bands" divide only the slow
    ones: those that turn ``low`` times or fewer over original_len, and in part
    those that turn up to ``high`` times (32 for "ramp", along a line in the pairs'
    number; 4 for "bands", along a line in the turns)."""
    if scaling not in _SCALINGS:
        raise ValueError(f"rope_frequencies: scaling {scaling!r} is none of {', '.join(_SCALINGS)}")
    if high is None:
        high = 32.0 if scaling == "ramp" else 4.0
    out = (ctypes.c_float * max(1, int(rot_dim) // 2))()
    size = _native.lib().vsk_rope_frequencies(out, int(rot_dim), float(base), _SCALINGS[scaling], float(factor),
                                              float(original_len), float(low), float(high))
    if size == 0.0:
        raise ValueError(f"rope_frequencies: {_native.last_error()}")
    return torch.tensor(list(out), dtype=torch.float32, device=device), size


def rope_fwd(q, k, q_out, k_out, positions, inv_freq, interleaved=False, attention_factor=1.0, stream=None) -> None:
    """Rotary positions of query and key rows.

    ``q`` / ``q_out``: [N, h_q, D] bf16 (both None: keys only), ``k`` / ``k_out``:
    [N, h_kv, D] bf16, D in {64, 128, 256}; an output may be its own input.
    ``positions``: [N] int32 or int64; ``inv_freq``: [R/2] float32 (see
    ``rope_frequencies``), R a multiple of 16 up to D: the first R elements of a
    head turn, in pairs (i, i + R/2) or, ``interleaved``, (2i, 2i + 1), and are
    multiplied by ``attention_factor``; the others are copied."""
    _run("rope_fwd", ("q", "k", "q_out", "k_out", "positions", "inv_freq"), (q, k, q_out, k_out, positions, inv_freq),
         (1 if interleaved else 0, float(attention_factor)), stream, None, need=0)


def rope_append_fwd(q, k, v, q_out, k_out, k_buffer, v_buffer, out_cache_loc, positions, inv_freq, k_scale=1.0,
                    v_scale=1.0, interleaved=False, attention_factor=1.0, workspace=None, stream=None) -> None:
    """``rope_fwd`` that also stores the rotated keys and ``v`` ([N, h_kv, D] bf16)
    to rows ``out_cache_loc`` ([N] int32 or int64, distinct; -1: not stored) of
    ``k_buffer`` / ``v_buffer`` ([pool, h_kv, D] bf16 or e4m3), as x / scale in the
    pool's type.  ``k_out`` None: the rotated keys go to the pool only.
    ``workspace``: 256 bytes or more (the error word)."""
    _run("rope_append_fwd",
         ("q", "k", "v", "q_out", "k_out", "k_buffer", "v_buffer", "out_cache_loc", "positions", "inv_freq"),
         (q, k, v, q_out, k_out, k_buffer, v_buffer, out_cache_loc, positions, inv_freq),
         (1 if interleaved else 0, float(attention_factor), float(k_scale), float(v_scale)), stream, workspace)


def rope_append_block_fwd(q, k, v, q_out, k_out, k_cache, v_cache, k_scales, v_scales, qo_indptr, block_table,
                          cache_lens, block_size, positions, inv_freq, interleaved=False, attention_factor=1.0,
                          workspace=None, stream=None) -> None:
    """``rope_fwd`` that also stores the rotated keys and ``v`` into an e4m3 cache
    whose blocks have a power-of-two scale for every KV head, one for K and one for
    V, that follows their rows.

    ``k_cache`` / ``v_cache``: [blocks * block_size, h_kv, D] e4m3, ``block_size`` a
    multiple of 16 up to 128; ``k_scales`` / ``v_scales``: [blocks, h_kv] float32;
    rows qo_indptr[b] .. qo_indptr[b+1] - 1 ([B+1] int32) go to cache positions
    cache_lens[b] .. ([B] int32) of sequence b, position t to row t % block_size of
    block block_table[b][t // block_size] ([B, columns] int32).  A block that holds
    earlier rows keeps its scale unless the new rows need a larger one; its earlier
    rows are then rounded again under that.  ``k_out`` may be None.
    ``workspace``: 256 bytes or more (the error word)."""
    _run("rope_append_block_fwd",
         ("q", "k", "v", "q_out", "k_out", "k_cache", "v_cache", "k_scales", "v_scales", "qo_indptr", "block_table",
          "cache_lens", "positions", "inv_freq"),
         (q, k, v, q_out, k_out, k_cache, v_cache, k_scales, v_scales, qo_indptr, block_table, cache_lens, positions,
          inv_freq),
         (int(block_size), 1 if interleaved else 0, float(attention_factor)), stream, workspace)


def block_workspace_size(max_bs, h_q, h_kv, head_dim, l_ext) -> int:
    """Workspace bytes of ``verify_splitkv_block_fwd`` for any batch of up to
    ``max_bs`` sequences of any lengths, on the current device."""
    return int(_native.lib().vsk_block_workspace_size(max_bs, h_q, h_kv, head_dim, l_ext))


def verify_splitkv_block_fwd(q_extend, k_extend, v_extend, o_extend, k_cache, v_cache, k_scales, v_scales, qo_indptr,
                             block_table, seq_lens, block_size, max_len_extend, sm_scale=None, custom_mask=None,
                             mask_indptr=None, max_bs=None, workspace=None, stream=None) -> None:
    """``verify_splitkv_fwd`` over a cache that ``rope_append_block_fwd`` filled:
    sequence b's prefix is its cache positions 0 .. seq_lens[b] - 1 ([B] int32), its
    drafts the bf16 rows ``k_extend`` / ``v_extend``, causal or, with
    ``custom_mask`` / ``mask_indptr``, in a tree (the layout of
    ``verify_splitkv_fwd``).  One draft, the new token, makes a decode step.
    (h_q / h_kv) * max_len_extend is at most 128.
    ``workspace``: ``block_workspace_size`` bytes or more."""
    mle = int(max_len_extend)
    if custom_mask is not None:
        custom_mask = _flat_mask(custom_mask, stream)

    def need():
        if q_extend.dim() != 3 or k_extend.dim() != 3 or qo_indptr.dim() != 1 or qo_indptr.shape[0] < 2:
            return 256  # the library names what is wrong
        bs = qo_indptr.shape[0] - 1
        mb = bs if (max_bs is None or max_bs < bs) else int(max_bs)
        key = (q_extend.get_device(), mb, q_extend.shape[1], k_extend.shape[1], q_extend.shape[2], mle)
        n = _SIZES.get(key)
        if n is None:
            n = _SIZES[key] = block_workspace_size(*key[1:]) or 256
        return n

    _run("verify_splitkv_block_fwd",
         ("q_extend", "k_extend", "v_extend", "o_extend", "k_cache", "v_cache", "k_scales", "v_scales", "qo_indptr",
          "block_table", "seq_lens", "custom_mask", "mask_indptr"),
         (q_extend, k_extend, v_extend, o_extend, k_cache, v_cache, k_scales, v_scales, qo_indptr, block_table, seq_lens,
          custom_mask, mask_indptr),
         (int(block_size), mle, 0.0 if sm_scale is None else float(sm_scale)), stream, workspace, need)
