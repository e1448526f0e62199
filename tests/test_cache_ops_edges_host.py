"""More refusals of the calls around the verify call (no GPU needed): the
checks read shapes, types, strides and pointers only, so CPU tensors stand in."""
import pytest
import torch

import speculative_decode_verify_prefix_gb300 as vsk
from speculative_decode_verify_prefix_gb300 import _native
from test_cache_ops_host import bf, built, call, evict_args, mass_args, ptr, ref, refused, shared_args  # noqa: F401


def test_shared_without_query_heads_is_refused():
    """The cut of the work divides by the query heads of a KV head."""
    refused("h_q must be", call("verify_splitkv_shared_fwd", shared_args(q=bf(8, 0, 64), o=bf(8, 0, 64)), 4, 1.0, 1.0, 0.0))
