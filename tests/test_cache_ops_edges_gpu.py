"""GPU tests of the calls around the verify call at their edges: host threads,
values and sizes that the tests of their formulas do not reach."""
import math
import threading

import pytest
import torch

import test_cache_ops_gpu as base
from test_cache_ops_gpu import (BF16, DEV, E4M3, F64, check_attention, gen, indptr, normal, run_mass, run_shared,  # noqa: F401
                                shared_case, shared_want, vsk)

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- host threads

@pytest.mark.parametrize("form", ["shared prefix", "stream and combine"])
def test_threads_on_one_stream_keep_their_partials(vsk, form):
    """Calls of several launches from four host threads on one stream: the threads have one workspace, in which the
    launches of a call hand partials on, so no other call's launches may come between them."""
    d, l = 128, 4
    cases = [shared_case(700, (150, 40, 333, 90), l, 8, 2, d, seed=90 + i) for i in range(4)]
    assert vsk.call_form(4, 8, 2, d, d, l, 613) == "stream_only" and vsk.launches_per_call(4, 8, 2, d, l, 613) == 2

    def run(c, o):
        if form == "shared prefix":
            vsk.verify_splitkv_shared_fwd(c["q"], c["ke"], c["ve"], o, c["kb"], c["vb"], c["qo"], c["kvp"], c["kvi"],
                                          c["sh"], l)
        else:
            assert vsk.verify_splitkv_fwd(c["q"], c["ke"], c["ve"], o, c["kb"], c["vb"], c["qo"], c["kvp"], c["kvi"], None,
                                          True, None, l, 1.0, 1.0)

    alone = []
    for c in cases:
        alone.append(torch.empty_like(c["q"]))
        run(c, alone[-1])
    if form == "shared prefix":
        for c, o in zip(cases, alone):
            check_attention(o, *shared_want(c, d ** -0.5))
    calls, outs, failed, start = 100, [[] for _ in cases], [], threading.Barrier(len(cases))
    for i, c in enumerate(cases):
        outs[i] = [torch.full_like(c["q"], float("nan")) for _ in range(calls)]
    torch.cuda.synchronize()

    def work(i):
        try:
            start.wait(30)
            for o in outs[i]:
                run(cases[i], o)
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert not failed, failed
    torch.cuda.synchronize()
    wrong = [sum(not torch.equal(o, alone[i]) for o in outs[i]) for i in range(len(cases))]
    assert wrong == [0] * len(cases), f"calls of {calls} with another call's partials: {wrong}"
    assert vsk.read_error_flags() == 0


# ---------------------------------------------------------------- sizes

def test_shared_workspace_size_of_shapes_that_no_call_takes(vsk):
    assert vsk.shared_workspace_size(2, 8, 2, 128, 4) > 0
    for shape in ((2, 0, 2, 128, 4), (2, -4, 2, 128, 4), (2, 8, 0, 128, 4), (0, 8, 2, 128, 4), (2, 8, 2, 96, 4),
                  (2, 8, 2, 128, 0), (2, 7, 2, 128, 4)):
        assert vsk.shared_workspace_size(*shape) == 0, shape
