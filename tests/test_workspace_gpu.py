"""GPU test of the workspaces that the binding keeps for a stream."""
import types

import pytest
import torch

from test_parity_gpu import gpu_problem, run_gpu, vsk  # noqa: F401

import workloads

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("launches", [1, 2])
@pytest.mark.parametrize("given", ["torch's", "another object"])
def test_first_call_on_a_stream_does_not_wait_for_the_current_one(vsk, launches, given):  # noqa: F811
    """The workspace is zeroed on the stream that uses it: in time, although the current stream is busy."""
    p = gpu_problem(workloads.Spec("first", (900, 40), 4, 8, 2, 128, 128, perm=True, seed=211))
    vsk.set_tuning_split_launch(2 if launches == 2 else 0)
    try:
        want = run_gpu(vsk, p)
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):  # memory of that stream, not zero
            dirty = torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")
            del dirty
        o = torch.zeros_like(want)
        torch.cuda.synchronize()
        late = torch.cuda.Event()
        torch.cuda._sleep(200_000_000)
        late.record()
        assert vsk.verify_splitkv_fwd(p["q"], p["k_ext"], p["v_ext"], o, p["k_buffer"], p["v_buffer"], p["qo_indptr"], p["kv_indptr"],
                                      p["kv_indices"], None, True, None, 4, p["k_scale"], p["v_scale"], sm_scale=p["sm_scale"],
                                      stream=side if given == "torch's" else types.SimpleNamespace(cuda_stream=side.cuda_stream))
        side.synchronize()
        assert not late.query()
        torch.cuda.synchronize()
        assert torch.equal(o, want) and vsk.read_error_flags(stream=side) == 0
    finally:
        vsk.set_tuning_split_launch(1)
