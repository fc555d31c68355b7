"""The paged cache on the GPU at the borders of its arguments: calls side by side on several streams,
the largest groups of heads, and values and scales at the ends of their types.  Setup, oracle and
tolerances are those of test_cache_gpu."""
import pytest
import torch

from test_cache_gpu import BF, Setup

pytestmark = pytest.mark.gpu


# ----------------------------------------------------------------------------- streams
def test_default_workspaces_on_two_unordered_streams(lib, cuda_dev):
    """Calls on the current stream and on a side stream in turn, nothing between them, each with the
    workspace and the output that the binding allocates: every result is the one of its own call."""
    s = Setup(lib, cuda_dev, "e2m1", B=2, ctx=3000, page=64, HKV=4, DQK=64, DV=64, fill=False)
    pos = torch.arange(3000, dtype=torch.int32, device=cuda_dev).expand(2, -1).contiguous()
    g = torch.Generator(device=cuda_dev).manual_seed(3)
    rand = lambda *sh: torch.randn(*sh, generator=g, device=cuda_dev).to(BF)  # noqa: E731
    lib.dsa_cache_append(s.cache, pos, rand(2, 3000, 4, 64), rand(2, 3000, 4, 64))
    last = torch.tensor([[2999], [1500]], dtype=torch.int32, device=cuda_dev)
    q = [rand(2, 1, 8, 64) for _ in range(2)]
    want = [lib.dsa_cache_attn(x, s.cache, last) for x in q]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(200):
        got[0].append(lib.dsa_cache_attn(q[0], s.cache, last))
        got[1].append(lib.dsa_cache_attn(q[1], s.cache, last, stream=side))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, want[i]) for x in got[i])


def test_a_side_stream_takes_no_block_of_the_current_one(lib, cuda_dev):
    """Blocks that the current stream has just given back are not what a call on another stream
    writes its output to."""
    s = Setup(lib, cuda_dev, "e2m1", B=2, ctx=900, page=64, HKV=4, DQK=64, DV=64)
    pos = torch.tensor([[899], [500]], dtype=torch.int32, device=cuda_dev)
    q = s.cuda(s.normal(2, 1, 8, 64))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    freed = [torch.empty_like(q) for _ in range(8)]
    at = {t.data_ptr() for t in freed}
    del freed
    outs = [lib.dsa_cache_attn(q, s.cache, pos, stream=side) for _ in range(8)]
    outs += [t for _ in range(4) for t in lib.dsa_cache_read(s.cache, pos, stream=side)]
    outs += [lib.dsa_window_attn(q, q, q, 1, stream=side)]
    assert not at & {t.data_ptr() for t in outs}
    torch.cuda.synchronize()
