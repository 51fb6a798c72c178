"""Where the Muon step's buffers come from when a step runs on a stream of its own."""
import pytest
import torch

from zero_sharded_optimizer_reduce_amd.drivers import MuonStep

pytestmark = pytest.mark.gpu


def _stream_of(tensor):
    """The stream that the caching allocator's segment of a tensor belongs to."""
    at = tensor.data_ptr()
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= at < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not in the allocator's memory")


@pytest.mark.parametrize("as_handle", [False, True])
def test_the_first_clipped_steps_buffers_belong_to_its_stream(as_handle):
    # Memory that the allocator took back on another stream may still be in use
    # there: buffers made inside a step have to be that step's stream's.
    st = MuonStep([(64, 96)], 2)
    grads = [torch.zeros(st.psi_pad, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    st.load_master(torch.zeros(st.psi_pad, device="cuda"))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    st.step(grads, [0.5, 0.5], dict(lr=1e-2, momentum=0.9), max_norm=1.0,
            stream=side.cuda_stream if as_handle else side)
    side.synchronize()
    for t in (*st.grad, st.norm_parts, st.norm_sq, st.clip):
        assert _stream_of(t) == side.cuda_stream
    assert float(st.clip) == 1.0
