"""Python binding of the calls around the verify call: attention over whole
prompts, the verify call for a batch that shares a long prefix, the attention
weight of the cached keys and the eviction that goes by it.

As in api.py: argument marshalling only, every step of the computation runs in
the library's kernels, on the given stream (default: the current one of the
tensors' device) and without synchronising.  A call that the library rejects
raises ValueError with its message and launches nothing.
"""
from __future__ import annotations

import ctypes

import torch

from . import _native
from .api import _WS, _WS_LOCK, _coerce, _ref


def _device_of(**tensors) -> torch.device:
    """The CUDA device of a call's tensors; they must all be on one."""
    dev = None
    for name, t in tensors.items():
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if dev is not None and t.device != dev:
            raise ValueError(f"{name} is on {t.device}, the call's other tensors on {dev}")
        dev = t.device
    return dev


def _workspace_of(device, stream, need):
    """The cached workspace of (device, stream), grown to ``need`` bytes.  Not
    while the stream is captured: growing it later would free the buffer that
    the graph keeps using."""
    with torch.cuda.stream(stream):
        if torch.cuda.is_current_stream_capturing():
            raise ValueError("pass workspace= to a call that is captured into a graph")
        key = (device, int(stream.cuda_stream))
        with _WS_LOCK:
            ws = _WS.get(key)
            if ws is None or ws.numel() < need:
                ws = torch.zeros(need, dtype=torch.uint8, device=device)
                _WS[key] = ws
    return ws


def _run(name, device, stream, workspace, need, *args) -> None:
    """Calls a library entry point whose last arguments are workspace, its
    bytes and the stream, with ``device`` current."""
    with torch.cuda.device(device):
        if stream is None:
            stream = torch.cuda.current_stream(device)
        if workspace is None:
            workspace = _workspace_of(device, stream, need())
        ok = getattr(_native.lib(), name)(*args, ctypes.c_void_p(workspace.data_ptr()), workspace.numel(),
                                          ctypes.c_void_p(stream.cuda_stream))
    if not ok:
        raise ValueError(f"{name}: {_native.last_error()}")


def prompt_attn_fwd(q, k, v, o, qo_indptr, sm_scale=None, workspace=None, stream=None) -> None:
    """Causal attention over whole prompts packed one after the other.

    ``q`` / ``o``: [N, h_q, D] bf16, ``k`` / ``v``: [N, h_kv, D] bf16, D in
    {64, 128, 256}; ``qo_indptr``: [B+1] int32, sequence b owns rows
    qo_indptr[b] .. qo_indptr[b+1] - 1, of any lengths.  Row i of a sequence
    attends to its rows t <= i.  Rows of ``o`` outside every sequence are left
    as they were.  ``workspace``: 256 bytes or more (the error word)."""
    dev = _device_of(q=q, k=k, v=v, o=o, qo_indptr=qo_indptr)
    _run("prompt_attn_fwd", dev, stream, workspace, lambda: 256, _ref(q), _ref(k), _ref(v), _ref(o), _ref(qo_indptr),
         0.0 if sm_scale is None else float(sm_scale))


def shared_workspace_size(max_bs, h_q, h_kv, head_dim, l_ext) -> int:
    """Workspace bytes of ``verify_splitkv_shared_fwd`` for any batch of up to
    ``max_bs`` sequences, on the current device."""
    return int(_native.lib().vsk_shared_workspace_size(max_bs, h_q, h_kv, head_dim, l_ext))


def verify_splitkv_shared_fwd(q_extend, k_extend, v_extend, o_extend, k_buffer, v_buffer, qo_indptr, kv_indptr,
                              kv_indices, shared_indices, max_len_extend, k_scale=1.0, v_scale=1.0, sm_scale=None,
                              max_bs=None, workspace=None, stream=None) -> None:
    """``verify_splitkv_fwd`` (causal drafts) for a batch whose sequences share
    a prefix: every sequence's prefix is the pool rows ``shared_indices``
    ([S] int32 or int64) followed by its own ``kv_indices`` rows.  The shared
    rows are read for the whole batch at once, not per sequence."""
    dev = _device_of(q_extend=q_extend, k_extend=k_extend, v_extend=v_extend, o_extend=o_extend, k_buffer=k_buffer,
                     v_buffer=v_buffer, qo_indptr=qo_indptr, kv_indptr=kv_indptr, kv_indices=kv_indices,
                     shared_indices=shared_indices)
    mle = int(max_len_extend)

    def need():
        if q_extend.dim() != 3 or k_extend.dim() != 3 or qo_indptr.dim() != 1 or qo_indptr.shape[0] < 2 or mle < 1:
            return 256  # the library names what is wrong
        bs = qo_indptr.shape[0] - 1
        mb = bs if (max_bs is None or max_bs < bs) else int(max_bs)
        return shared_workspace_size(mb, q_extend.shape[1], k_extend.shape[1], q_extend.shape[2], mle) or 256

    _run("verify_splitkv_shared_fwd", dev, stream, workspace, need,
         _ref(q_extend), _ref(k_extend), _ref(v_extend), _ref(o_extend), _ref(k_buffer), _ref(v_buffer),
         _ref(qo_indptr), _ref(kv_indptr), _ref(kv_indices), _ref(shared_indices), mle, _coerce(k_scale),
         _coerce(v_scale), 0.0 if sm_scale is None else float(sm_scale))


def verify_splitkv_mass(q_extend, k_extend, k_buffer, qo_indptr, kv_indptr, kv_indices, mass, max_len_extend,
                        k_scale=1.0, sm_scale=None, mass_in=None, workspace=None, stream=None) -> None:
    """Attention weight of the cached keys: writes to ``mass`` ([h_kv,
    len(kv_indices)] float32) ``mass_in`` (None: zeros; may be ``mass`` itself)
    plus, for every entry of ``kv_indices``, the sum over the draft rows and the
    query heads of the KV head of the softmax weight its key has in
    ``verify_splitkv_fwd`` (causal drafts)."""
    named = dict(q_extend=q_extend, k_extend=k_extend, k_buffer=k_buffer, qo_indptr=qo_indptr, kv_indptr=kv_indptr,
                 kv_indices=kv_indices, mass=mass)
    if mass_in is not None:
        named["mass_in"] = mass_in
    dev = _device_of(**named)
    _run("verify_splitkv_mass", dev, stream, workspace, lambda: 256, _ref(q_extend), _ref(k_extend), _ref(k_buffer),
         _ref(qo_indptr), _ref(kv_indptr), _ref(kv_indices), None if mass_in is None else _ref(mass_in), _ref(mass),
         int(max_len_extend), _coerce(k_scale), 0.0 if sm_scale is None else float(sm_scale))


def kv_evict(mass, kv_indptr, kv_indices, budget, recent, out_kv_indptr, out_kv_indices, out_mass, freed,
             workspace=None, stream=None) -> None:
    """Cuts every sequence's cache index to ``budget`` entries: its last
    ``recent`` ones and, of the others, those with the largest ``mass`` summed
    over the KV heads, in their order.

    Writes ``out_kv_indptr`` ([B+1] int32), the kept entries to
    ``out_kv_indices`` and their weights to ``out_mass`` (both packed; min(n, B *
    budget) columns always suffice) and the others, whose pool rows may be
    reused, to ``freed`` (out_kv_indptr and kv_indptr tell how many)."""
    dev = _device_of(mass=mass, kv_indptr=kv_indptr, kv_indices=kv_indices, out_kv_indptr=out_kv_indptr,
                     out_kv_indices=out_kv_indices, out_mass=out_mass, freed=freed)
    _run("kv_evict", dev, stream, workspace, lambda: 256, _ref(mass), _ref(kv_indptr), _ref(kv_indices), int(budget),
         int(recent), _ref(out_kv_indptr), _ref(out_kv_indices), _ref(out_mass), _ref(freed))
