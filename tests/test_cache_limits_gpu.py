"""The paged cache on the GPU at the borders of its arguments: calls side by side on several streams,
the largest groups of heads, and values and scales at the ends of their types.  Setup, oracle and
tolerances are those of test_cache_gpu."""
import numpy as np
import pytest
import torch

from oracle import cache_oracle as O
from test_cache_gpu import BF, Setup, check, run_attn

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


# ----------------------------------------------------------------------------- sizes past an int
@pytest.mark.parametrize("dtype,D,S", [(BF, 128, 70), (BF, 64, 70), (torch.float32, 64, 9)])
def test_contiguous_windows_past_an_int(lib, cuda_dev, dtype, D, S):
    """A window of any size past the context is the window of the whole context; one below the range
    of an int is as negative as any other."""
    g = torch.Generator(device=cuda_dev).manual_seed(D + S)
    rand = lambda *sh: torch.randn(*sh, generator=g, device=cuda_dev).to(dtype)  # noqa: E731
    q, k, v = rand(2, S, 4, D), rand(2, 90, 2, D), rand(2, 90, 2, D)
    sink_k, sink_v = rand(3, 2, D), rand(3, 2, D)
    for kw in (dict(), dict(n_first=5), dict(sink_k=sink_k, sink_v=sink_v)):
        every = lib.dsa_window_attn(q, k, v, 90, **kw)
        for window in (2**31 - 1, 2**32, 2**32 + 8, 2**40):
            assert torch.equal(lib.dsa_window_attn(q, k, v, window, **kw), every)
        for window in (-2**32, -2**32 + 8):
            with pytest.raises(lib.DSAError):
                lib.dsa_window_attn(q, k, v, window, **kw)
    for n_first in (-2**32, -2**32 + 8):
        with pytest.raises(lib.DSAError):
            lib.dsa_window_attn(q, k, v, 8, n_first=n_first)


def test_cache_windows_below_an_int_are_refused(lib, cuda_dev):
    s = Setup(lib, cuda_dev, "e2m1", B=1, ctx=40, page=16, HKV=2, DQK=64, DV=64)
    q, pos = s.cuda(s.normal(1, 1, 4, 64)), torch.tensor([[39]], dtype=torch.int32, device=cuda_dev)
    for window, n_first in ((-2**32, 0), (-2**32 + 5, 0), (8, -2**32), (8, -2**32 + 4)):
        with pytest.raises(lib.DSAError):
            lib.dsa_cache_attn(q, s.cache, pos, window=window, n_first=n_first)


# ----------------------------------------------------------------------------- refused calls
def test_a_refused_call_leaves_the_next_one_alone(lib, cuda_dev):
    """No selected keys at all are refused; the whole context of the same rows is then as before."""
    s = Setup(lib, cuda_dev, "e2m1", B=2, ctx=900, page=64, HKV=4, DQK=64, DV=64)
    q = s.cuda(s.normal(2, 1, 8, 64))
    pos = torch.tensor([[899], [500]], dtype=torch.int32, device=cuda_dev)
    want = lib.dsa_cache_attn(q, lib.Cache(s.pages, s.table, 4, 64, 64), pos)
    with pytest.raises(lib.DSAError):
        lib.dsa_cache_sparse_attn(q, s.cache, pos, pos.new_empty(2, 1, 0))
    assert torch.equal(lib.dsa_cache_attn(q, s.cache, pos), want)


# ----------------------------------------------------------------------------- values and scales
@pytest.mark.parametrize("k_scale,v_scale", [(0.25, 0.3), (0.3, 2.0**-20), (2.0**-90, 1e-30)])
def test_values_past_the_range_of_a_quotient_saturate(lib, cuda_dev, k_scale, v_scale):
    """Finite values whose quotient by the tensor's scale float32 does not hold: codes of 6 and scales
    of 448, as where the quotient is merely large; NaN is for infinities and NaN alone."""
    s = Setup(lib, cuda_dev, "e2m1", B=1, ctx=4, page=4, HKV=2, DQK=64, DV=64, k_scale=k_scale,
              v_scale=v_scale, fill=False)
    k, v = s.normal(1, 4, 2, 64), s.normal(1, 4, 2, 64)
    for x in (k, v):
        x[0, 0, 0, 3], x[0, 0, 0, 20] = 3.3e38, -3.3e38
        x[0, 0, 1, :16] = np.linspace(-3.3e38, 3.3e38, 16)
        x[0, 1, 0] = np.ldexp(1.5, np.arange(64) * 4 - 126)
        x[0, 1, 1, 5], x[0, 1, 1, 6] = np.inf, 3e38
        x[0, 2, 0, 40], x[0, 2, 0, 41], x[0, 2, 1, 0] = np.nan, 1e38, -np.inf
    k, v = O.to_bf16(k), O.to_bf16(v)
    pos = torch.arange(4, dtype=torch.int32, device=cuda_dev)[None]
    lib.dsa_cache_append(s.cache, pos, s.cuda(k), s.cuda(v))
    rows = s.pages[s.table[0, 0].item()].cpu().numpy()
    for t in range(4):
        want, kd, vd = O.row_of(k[0, t], v[0, t], "e2m1", k_scale, v_scale)
        assert np.array_equal(rows[t][:144], want[:144])
        assert np.isfinite(kd).all() == np.isfinite(k[0, t]).all()
    # read back: 6 * 448 * scale of a saturated group's largest, in bf16
    k2, _ = lib.dsa_cache_read(s.cache, pos)
    top = float(torch.tensor(6 * 448 * float(np.float32(k_scale)), dtype=torch.float32).to(BF))
    assert k2[0, 0, 0, 3].item() == top and k2[0, 0, 0, 20].item() == -top
    assert k2[0, 1, 1, :16].isnan().all() and not k2[0, 1, 1, 16:].isnan().any()


@pytest.mark.parametrize("v_scale", [2.0**-120, 2.0**-126, 2.0**100])
@pytest.mark.parametrize("S,ctx,low", [(1, 2500, 1), (1200, 40, 1), (1200, 2000, 64)])
def test_a_small_tensor_scale_keeps_the_output(lib, cuda_dev, v_scale, S, ctx, low):
    """Large sums of probabilities (the most where the first steps' scores are 8 lower in log2 units
    than the others) beside a scale at the end of float32's range: neither 1 / L times the scale nor the
    scale times the gate is what the output is.  Rows in pieces, and rows taken whole."""
    s = Setup(lib, cuda_dev, "e2m1", B=1, ctx=ctx, page=64, HKV=1, DQK=64, DV=64, v_scale=v_scale,
              fill=False)
    k = np.zeros((1, ctx, 1, 64))
    k[0, low:] = 6.0  # exact in 4 bits; the first keys' scores are 0, the others' 8 in log2 units
    v = O.to_bf16(s.normal(1, ctx, 1, 64) * v_scale)  # (what the call gets, below 2^-126 too)
    every = torch.arange(ctx, dtype=torch.int32, device=cuda_dev)[None]
    lib.dsa_cache_append(s.cache, every, s.cuda(k), s.cuda(v))
    for t in range(ctx):
        _, s.k[0, t], s.v[0, t] = O.row_of(k[0, t], v[0, t], "e2m1", 1.0, v_scale)
    q = np.full((4, 64), 1.0)
    gate = np.array([-20.0, 0.0, 1.0, 5.0])
    sm = 8 * np.log(2) / (6.0 * 64)
    pos = torch.full((1, S), ctx - 1, dtype=torch.int32, device=cuda_dev)
    rows = lambda x: s.cuda(np.broadcast_to(x, (1, S, *x.shape)).copy())  # noqa: E731
    out = lib.dsa_cache_attn(rows(q), s.cache, pos, gate=rows(gate), sm_scale=sm)
    want, mag = O.attend(q, s.k[0], s.v[0], list(range(ctx)), float(np.float32(sm)), gate)
    # below bf16's and float32's normal range a result is off by half a step of it
    for i in {0, S // 2, S - 1}:
        check(out[0, i], want, mag, floor=2.0**-134 + 3 * 2.0**-150)


# ----------------------------------------------------------------------------- groups of heads
@pytest.mark.parametrize("fmt", ["bf16", "e2m1"])
@pytest.mark.parametrize("G,DQK,DV", [(33, 192, 128), (40, 192, 128), (41, 64, 64), (48, 128, 64),
                                      (56, 64, 128), (57, 192, 64), (64, 192, 128), (64, 128, 128)])
def test_more_than_32_heads_of_one_key_head(lib, cuda_dev, fmt, G, DQK, DV):
    """Groups of five to eight times 8 heads, with more warps than the formats' usual CTA: whole
    contexts in many pieces and in one, a window, selected keys, rows in plenty."""
    s = Setup(lib, cuda_dev, fmt, B=2, ctx=700, page=48, HKV=1, DQK=DQK, DV=DV,
              k_scale=1.0 if fmt == "bf16" else 0.5, v_scale=1.0 if fmt == "bf16" else 2.0)
    run_attn(s, np.array([[699], [17]]), G, gate=True)
    run_attn(s, np.array([[699], [-1]]), G, window=100, n_first=9)
    idx = np.full((2, 1, 333), -1)
    for b in range(2):
        idx[b, 0, :200] = np.sort(s.r.permutation(700)[:200])
    run_attn(s, np.array([[650], [300]]), G, idx=idx)
    run_attn(s, s.r.integers(-1, 700, (2, 620)), G, window=3)


def test_two_key_heads_of_32_heads(lib, cuda_dev):
    for fmt in ("bf16", "e2m1"):
        s = Setup(lib, cuda_dev, fmt, B=1, ctx=900, page=100, HKV=2, DQK=192, DV=128)
        run_attn(s, np.array([[899]]), 64, gate=True, gate_mode="silu")


# ----------------------------------------------------------------------------- probabilities
@pytest.mark.parametrize("fmt", ["bf16", "e2m1"])
@pytest.mark.parametrize("HKV,G", [(8, 1), (2, 3), (8, 4), (2, 5), (4, 8), (2, 12)])
def test_values_that_cancel(lib, cuda_dev, fmt, HKV, G):
    """Two keys of nearly equal scores whose values are c and -c: the output is c times the difference
    of the probabilities, tanh of half the scores' difference (keys and c as the cache holds them).  One dim of q alone is not zero, so scores are
    one product, below 2^3 in log2 units: float32 roundings (2^3 * 2^-24 * 3) and an exponential within
    2^-22 give p within 2^-19, and a pair of bf16 holds it within 2^-17 (of f16 within 2^-21)."""
    s = Setup(lib, cuda_dev, fmt, B=1, ctx=2, page=16, HKV=HKV, DQK=64, DV=64, fill=False)
    k, v = np.zeros((1, 2, HKV, 64)), np.ones((1, 2, HKV, 64))
    k[0, 0, :, 0], k[0, 1, :, 0], v[0, 1] = 6.0, 4.0, -1.0
    every = torch.tensor([[0, 1]], dtype=torch.int32, device=cuda_dev)
    lib.dsa_cache_append(s.cache, every, s.cuda(k), s.cuda(v))
    H, n = HKV * G, 40
    q = np.zeros((n, H, 64))
    q[..., 0] = O.to_bf16(2.0 ** s.r.uniform(-7, -3, (n, H)))
    pos = torch.ones(1, n, dtype=torch.int32, device=cuda_dev)
    out = lib.dsa_cache_attn(s.cuda(q[None]), s.cache, pos, sm_scale=1.0)[0].double().cpu().numpy()
    (_, k0, v0), (_, k1, v1) = (O.row_of(k[0, t], v[0, t], fmt, 1.0, 1.0) for t in range(2))
    c = v0[0, 0]
    assert (v0 == c).all() and (v1 == -c).all() and c < 1.04
    want = c * np.tanh(q[..., :1] * (k0 - k1)[0, 0] / 2)
    assert (np.abs(out - want) <= want * 2.0**-8 + 2.0**-16).all()


# ----------------------------------------------------------------------------- graphs
def test_graphs_with_side_streams_and_at_the_same_time(lib, cuda_dev):
    """A step whose layers run on two streams, captured twice with the workspaces that the binding
    allocates, and both graphs replayed at the same time: each gives its own queries' results."""
    s = Setup(lib, cuda_dev, "e2m1", B=2, ctx=900, page=64, HKV=4, DQK=64, DV=64)
    pos = torch.tensor([[899], [500]], dtype=torch.int32, device=cuda_dev)
    idx = torch.arange(0, 900, 3, dtype=torch.int32, device=cuda_dev).expand(2, 1, -1).contiguous()
    side = torch.cuda.Stream()

    def step(q):
        side.wait_stream(torch.cuda.current_stream())
        a = lib.dsa_cache_attn(q, s.cache, pos)
        b = lib.dsa_cache_sparse_attn(q, s.cache, pos, idx, stream=side)
        c, _ = lib.dsa_cache_read(s.cache, pos, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        return a, b, c

    qs = [s.cuda(s.normal(2, 1, 8, 64)) for _ in range(2)]
    want = [step(q) for q in qs]
    torch.cuda.synchronize()
    graphs, held = [], []
    for q in qs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            held.append(step(q))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for got, right in zip(held, want):
        for x, y in zip(got, right):
            assert torch.equal(x, y)


def test_a_small_key_scale_beside_large_queries(lib, cuda_dev):
    """Scores of ordinary size from q near 2^128, a key scale of 2^-100 and sm_scale 2^-46, whose product
    with the key scale alone has 4 bits left in float32: keys of one value each, scores up to 2.
    (float32: sums of 192 equal products and three scalings, 2^-20 of scores below 2^2 in log2 units.)"""
    s = Setup(lib, cuda_dev, "e2m1", B=1, ctx=64, page=16, HKV=1, DQK=192, DV=64, k_scale=2.0**-100,
              fill=False)
    codes = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -6, -4, -3, -2, -1.5, -1, -.5, 5.0])
    k = np.broadcast_to((np.tile(codes, 4) * 448 * 2.0**-100)[None, :, None, None], (1, 64, 1, 192))
    v = s.normal(1, 64, 1, 64)
    every = torch.arange(64, dtype=torch.int32, device=cuda_dev)[None]
    lib.dsa_cache_append(s.cache, every, s.cuda(k.copy()), s.cuda(v))
    for t in range(64):
        _, s.k[0, t], s.v[0, t] = O.row_of(O.to_bf16(k[0, t]), v[0, t], "e2m1", 2.0**-100, 1.0)
    q, sm = np.full((4, 192), 1.75 * 2.0**127), 2.0**-46
    out = lib.dsa_cache_attn(s.cuda(q[None, None]), s.cache, every[:, -1:].contiguous(), sm_scale=sm)
    check(out[0, 0], *O.attend(q, s.k[0], s.v[0], list(range(64)), sm))
