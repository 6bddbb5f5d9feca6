"""Where the outputs and workspaces that the products allocate belong."""
import pytest
import torch

import gpu_util as G
from nvfp4_block_numerics_b200 import binding as nv4

pytestmark = pytest.mark.gpu


def owner(t):
    """The stream, as a handle, to whose pool the caching allocator counts t's memory."""
    at = [s["stream"] for s in torch.cuda.memory_snapshot() if s["address"] <= t.data_ptr() < s["address"] + s["total_size"]]
    assert len(at) == 1
    return at[0]


@pytest.mark.parametrize("kind", ["none", "default", "handle 0", "stream", "handle"])
def test_outputs_belong_to_the_stream_of_the_call(kind):
    """Memory of another stream could be handed to that stream's next tensor while the call still writes it.
    Handle 0 is the default stream, whatever stream is current."""
    q, sc = torch.zeros((40, 64), dtype=torch.uint8, device=G.DEV), torch.full((40, 8), 0x38, dtype=torch.uint8, device=G.DEV)
    x, s2 = torch.ones((3, 128), dtype=torch.bfloat16, device=G.DEV), torch.ones(1, device=G.DEV)
    torch.cuda.synchronize()
    side, current = torch.cuda.Stream(), torch.cuda.Stream()
    stream, want = {"none": (None, current.cuda_stream), "default": (torch.cuda.default_stream(), 0), "handle 0": (0, 0),
                    "stream": (side, side.cuda_stream), "handle": (side.cuda_stream, side.cuda_stream)}[kind]
    with torch.cuda.stream(current):
        y = nv4.linear_w4a16(x, q, sc, s2, stream=stream)
        sm = nv4.mxfp4_quant_mma(x, stream=stream)[1]
    torch.cuda.synchronize()
    assert owner(y) == want and owner(sm) == want
    assert torch.all(y == 0)
