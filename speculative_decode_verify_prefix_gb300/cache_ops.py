"""Python binding of the calls around the verify call: attention over whole
prompts, the verify call for a batch that shares a long prefix, the attention
weight of the cached keys and the eviction that goes by it.

As in api.py: argument marshalling only, every step of the computation runs in
the library's kernels, on the given stream (default: the current one of the
tensors' device) and without synchronising.  A call that the library rejects
raises ValueError with its message and launches nothing.

``workspace``: a contiguous tensor on the tensors' device, 256-byte aligned,
zero-filled once before its first use and then left to the calls, which keep
counters in it between them; calls that may overlap on the GPU (two streams, two
graphs) must each have their own.  None: the cached one of (device, stream);
a call that is captured into a graph needs its own.
"""
from __future__ import annotations

import ctypes
import functools
import struct

import torch

from . import _native
from .api import _DT, _SHARED_SIZE as _SIZES, _WS, _WS_LOCK, _coerce

# A vsk_tensor: data, dtype, ndim, shape[3], stride[3].  The views of a call are
# packed into one buffer: a fraction of the time of filling a ctypes structure
# per tensor.
_VIEW = struct.Struct("Pii6q")
assert _VIEW.size == ctypes.sizeof(_native.VskTensor)


_ARENA = {n: ctypes.c_char * (_VIEW.size * n) for n in range(1, 16)}
_pack, _SIZE, _code = _VIEW.pack_into, _VIEW.size, _DT.get


def _views(names, tensors):
    """The packed views of a call's tensors (None stays None) and their
    addresses; all tensors must be on one CUDA device, which is returned."""
    buf = _ARENA[len(tensors)]()
    at = ctypes.addressof(buf)
    device, args, off = -1, [], 0
    for t in tensors:
        if t is None:
            args.append(None)
            continue
        try:
            dev, shape, stride = t.get_device(), t.shape, t.stride()
        except AttributeError:
            dev = -1
        if dev != device or dev < 0:
            name = names[len(args)]
            if dev < 0:
                raise ValueError(f"{name} must be a CUDA tensor")
            if device >= 0:
                raise ValueError(f"{name} is on cuda:{dev}, the call's other tensors on cuda:{device}")
            device = dev
        n = len(shape)
        if n == 3:
            _pack(buf, off, t.data_ptr(), _code(t.dtype, -1), 3, *shape, *stride)
        elif n == 1:
            _pack(buf, off, t.data_ptr(), _code(t.dtype, -1), 1, shape[0], 0, 0, stride[0], 0, 0)
        else:
            _pack(buf, off, t.data_ptr(), _code(t.dtype, -1), n, *(*shape, 0, 0, 0)[:3], *(*stride, 0, 0, 0)[:3])
        args.append(at + off)
        off += _SIZE
    if device < 0:
        raise ValueError(f"{names[0]} must be a CUDA tensor")
    return device, buf, args


@functools.lru_cache(maxsize=None)
def _device(index):
    return torch.device("cuda", index)


def _workspace_of(device, stream, raw_stream, need):
    """The cached workspace of (device, stream), grown to ``need`` bytes.  Not
    while the stream is captured: growing it later would free the buffer that
    the graph keeps using."""
    if stream is None:
        capturing = torch.cuda.is_current_stream_capturing()
    else:
        with torch.cuda.stream(stream):
            capturing = torch.cuda.is_current_stream_capturing()
    if capturing:
        raise ValueError("pass workspace= to a call that is captured into a graph")
    key = (_device(device), raw_stream)
    ws = _WS.get(key)
    if ws is None or ws.numel() < need:
        with torch.cuda.stream(stream), _WS_LOCK:  # zeroed in the order of the stream that uses it
            ws = _WS.get(key)
            if ws is None or ws.numel() < need:
                ws = torch.zeros(need, dtype=torch.uint8, device=key[0])
                _WS[key] = ws
    return ws


def _run(name, names, tensors, scalars, stream, workspace, need=None, scalars_at=None) -> None:
    """Calls a library entry point: the tensors' views, the scalars (after
    ``scalars_at`` tensors; None: after all), then workspace, its bytes and the
    stream, with the tensors' device current.  ``need``: workspace bytes (None:
    the error word)."""
    device, buf, args = _views(names, tensors)
    if device != torch.cuda.current_device():
        with torch.cuda.device(device):
            return _run(name, names, tensors, scalars, stream, workspace, need, scalars_at)
    raw = torch._C._cuda_getCurrentRawStream(device) if stream is None else stream.cuda_stream
    if workspace is None:
        workspace = _workspace_of(device, stream, raw, 256 if need is None else need())
    elif not isinstance(workspace, torch.Tensor) or workspace.get_device() != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{device}")
    k = len(args) if scalars_at is None else scalars_at
    if not getattr(_native.lib(), name)(*args[:k], *scalars, *args[k:], workspace.data_ptr(), workspace.nbytes, raw):
        raise ValueError(f"{name}: {_native.last_error()}")


def prompt_attn_fwd(q, k, v, o, qo_indptr, sm_scale=None, workspace=None, stream=None) -> None:
    """Causal attention over whole prompts packed one after the other.

    ``q`` / ``o``: [N, h_q, D] bf16, ``k`` / ``v``: [N, h_kv, D] bf16, D in
    {64, 128, 256}; ``qo_indptr``: [B+1] int32, sequence b owns rows
    qo_indptr[b] .. qo_indptr[b+1] - 1, of any lengths.  Row i of a sequence
    attends to its rows t <= i.  Rows of ``o`` outside every sequence are left
    as they were.  ``workspace``: 256 bytes or more (the error word and the
    counters by which CTAs draw their work: in a buffer that was not zeroed, or
    that another call uses meanwhile, rows would be left out)."""
    _run("prompt_attn_fwd", ("q", "k", "v", "o", "qo_indptr"), (q, k, v, o, qo_indptr),
         (0.0 if sm_scale is None else float(sm_scale),), stream, workspace)


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
    rows are read for the whole batch at once, not per sequence.
    ``workspace``: ``shared_workspace_size`` bytes or more."""
    mle = int(max_len_extend)

    def need():
        if q_extend.dim() != 3 or k_extend.dim() != 3 or qo_indptr.dim() != 1 or qo_indptr.shape[0] < 2 or mle < 1:
            return 256  # the library names what is wrong
        bs = qo_indptr.shape[0] - 1
        mb = bs if (max_bs is None or max_bs < bs) else int(max_bs)
        key = (q_extend.get_device(), mb, q_extend.shape[1], k_extend.shape[1], q_extend.shape[2], mle)
        n = _SIZES.get(key)
        if n is None:
            n = _SIZES[key] = shared_workspace_size(*key[1:]) or 256
        return n

    _run("verify_splitkv_shared_fwd",
         ("q_extend", "k_extend", "v_extend", "o_extend", "k_buffer", "v_buffer", "qo_indptr", "kv_indptr",
          "kv_indices", "shared_indices"),
         (q_extend, k_extend, v_extend, o_extend, k_buffer, v_buffer, qo_indptr, kv_indptr, kv_indices,
          shared_indices),
         (mle, _coerce(k_scale), _coerce(v_scale), 0.0 if sm_scale is None else float(sm_scale)), stream, workspace,
         need)


def verify_splitkv_mass(q_extend, k_extend, k_buffer, qo_indptr, kv_indptr, kv_indices, mass, max_len_extend,
                        k_scale=1.0, sm_scale=None, mass_in=None, workspace=None, stream=None) -> None:
    """Attention weight of the cached keys: writes to ``mass`` ([h_kv,
    len(kv_indices)] float32) ``mass_in`` (None: zeros; may be ``mass`` itself)
    plus, for every entry of ``kv_indices`` that belongs to a sequence, the sum
    over the draft rows and the query heads of the KV head of the softmax weight
    its key has in ``verify_splitkv_fwd`` (causal drafts); other columns are left
    as they were.  ``workspace``: 256 bytes or more (the error word)."""
    _run("verify_splitkv_mass",
         ("q_extend", "k_extend", "k_buffer", "qo_indptr", "kv_indptr", "kv_indices", "mass_in", "mass"),
         (q_extend, k_extend, k_buffer, qo_indptr, kv_indptr, kv_indices, mass_in, mass),
         (int(max_len_extend), _coerce(k_scale), 0.0 if sm_scale is None else float(sm_scale)), stream, workspace)


def kv_evict(mass, kv_indptr, kv_indices, budget, recent, out_kv_indptr, out_kv_indices, out_mass, freed,
             workspace=None, stream=None) -> None:
    """Cuts every sequence's cache index to ``budget`` entries: its last
    ``recent`` ones and, of the others, those with the largest ``mass`` summed
    over the KV heads, in their order.

    Writes ``out_kv_indptr`` ([B+1] int32), the kept entries to
    ``out_kv_indices`` and their weights to ``out_mass`` (both packed; min(n, B *
    budget) columns always suffice) and the others, whose pool rows may be
    reused, to ``freed`` (out_kv_indptr and kv_indptr tell how many).
    ``workspace``: 256 bytes or more (the error word)."""
    _run("kv_evict",
         ("mass", "kv_indptr", "kv_indices", "out_kv_indptr", "out_kv_indices", "out_mass", "freed"),
         (mass, kv_indptr, kv_indices, out_kv_indptr, out_kv_indices, out_mass, freed), (int(budget), int(recent)),
         stream, workspace, scalars_at=3)
