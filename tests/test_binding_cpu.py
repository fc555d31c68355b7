"""The Python binding without a GPU: a library that only answers, CPU tensors in the place of device
memory, and what the binding allocates and passes looked at."""
import contextlib

import pytest
import torch

import sparse_attention_15_b200 as dsa

BF = torch.bfloat16


class Answers:
    """Every entry point succeeds and is recorded; workspaces have 4096 bytes, cache rows their size."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            if name == "dsa_cache_row_bytes":
                fmt, kv, dqk, dv = args
                n = kv * (dqk + dv)
                return 2 * n if fmt == 0 else (n // 2 + n // 16 + 15) // 16 * 16
            return 4096 if name.endswith("workspace_bytes") else 0

        return call

    def last(self, name):
        return next(args for n, args in reversed(self.calls) if n == name)


class Stream:
    """Stands for a CUDA stream of the caller."""
    cuda_stream = 0x5000


class Current:
    cuda_stream = 0


@pytest.fixture
def answers(monkeypatch):
    """The binding on CPU tensors; `.made` lists (shape, dtype, inside the side stream's context) of
    each tensor that it makes, `.recorded` those kept for the current stream."""
    a = Answers()
    a.made, a.recorded, a.inside = [], [], False
    empty = torch.empty

    def made(*args, **kw):
        t = empty(*args, **kw)
        a.made.append((t, a.inside))
        return t

    @contextlib.contextmanager
    def on(stream):
        assert stream is Stream
        a.inside = True
        yield
        a.inside = False

    monkeypatch.setattr(dsa, "_LIB", a)
    monkeypatch.setattr(dsa, "_dev", lambda *ts: None)
    monkeypatch.setattr(dsa, "_cuda", lambda *ts: None)
    monkeypatch.setattr(torch, "empty", made)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: Stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Current)
    monkeypatch.setattr(dsa, "_raw_stream", lambda stream, device: (stream or Current).cuda_stream)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: None)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: a.recorded.append((t, s)))
    return a


def some_cache(fmt="e2m1", B=2, kv=2, D=64):
    return dsa.Cache(dsa.dsa_cache_pages(fmt, 8, 16, kv, D, D, device="cpu"),
                     torch.zeros(B, 4, dtype=torch.int32), kv, D, D)


def calls():
    """Each call that allocates, all of its outputs and workspace left to it."""
    z = lambda *s, dtype=BF: torch.zeros(*s, dtype=dtype)  # noqa: E731
    i32 = torch.int32
    qi, ki, w = z(2, 1, 4, 64), z(2, 32, 64), z(2, 1, 4, dtype=torch.float32)
    q, k = z(2, 1, 4, 64), z(2, 32, 4, 64)
    idx, pos = z(2, 1, 8, dtype=i32), z(2, 1, dtype=i32)
    kv, new = z(2, 32, 576), z(2, 1, 2, 64)
    c = some_cache()
    inv = torch.ones(16)
    return [
        (dsa.dsa_index_scores, (qi, ki, w, 1.0), {}),
        (dsa.dsa_index_scores_collapsed, (qi, ki, w, 1.0), {}),
        (dsa.dsa_hadamard_rotate, (qi,), {}),
        (dsa.dsa_topk, (z(2, 1, 32, dtype=torch.float32), 8), {}),
        (dsa.dsa_index_topk, (qi, ki, w, 1.0, 8), {}),
        (dsa.dsa_sparse_attn, (q, k, k, idx), {}),
        (dsa.dsa_sparse_attn_sinks, (q, k, k, idx, z(3, 4, 64), z(3, 4, 64)), {}),
        (dsa.dsa_sparse_attn_noalloc, (q, k, k, idx), {}),
        (dsa.dsa_sparse_attn_latent, (z(2, 1, 4, 576), kv, idx), {}),
        (dsa.dsa_forward, (qi, ki, w, 1.0, 8, q, k, k), {}),
        (dsa.dsa_window_attn, (q, k, k, 8), {}),
        (dsa.dsa_window_attn, (q, k, k, 8), dict(n_first=4)),
        (dsa.dsa_cache_append, (c, pos, new, new), dict(rope="half", inv_freq=inv, q=q)),
        (dsa.dsa_cache_read, (c, pos), {}),
        (dsa.dsa_cache_attn, (q, c, pos), {}),
        (dsa.dsa_cache_sparse_attn, (q, c, pos, idx), {}),
    ]


@pytest.mark.parametrize("n", range(16))
def test_a_call_on_another_stream_allocates_there(answers, n):
    """A block of the current stream's pool may still be in use there, so outputs and workspaces of a
    call on another stream come from that stream's own; outputs are kept for the current one."""
    fn, args, kw = calls()[n]
    answers.made.clear()
    out = fn(*args, stream=Stream(), **kw)
    assert answers.made and all(inside for _, inside in answers.made), fn.__name__
    out = [t for t in (out if isinstance(out, tuple) else (out,)) if t is not None]
    assert [t.data_ptr() for t, s in answers.recorded if s is Current] == \
        [t.data_ptr() for t, _ in answers.made if any(t is o for o in out)]
    assert len(answers.recorded) == len(out)


def test_calls_on_the_current_stream_allocate_plainly(answers):
    for fn, args, kw in calls():
        fn(*args, **kw)
    assert not answers.recorded and not any(inside for _, inside in answers.made)


# ----------------------------------------------------------------------------- sizes past an int
TOP = 2**31 - 1


@pytest.mark.parametrize("given,passed", [(8, 8), (TOP, TOP), (2**31, TOP), (2**32, TOP),
                                          (2**32 + 8, TOP), (2**40, TOP), (-1, -1),
                                          (-2**32, -TOP - 1), (-2**32 + 8, -TOP - 1)])
def test_sizes_past_an_int_do_not_wrap(answers, given, passed):
    """What a C int does not hold arrives as its last value on that side."""
    q, k, sink = torch.zeros(2, 1, 4, 64, dtype=BF), torch.zeros(2, 32, 4, 64, dtype=BF), \
        torch.zeros(3, 4, 64, dtype=BF)
    c, pos = some_cache(), torch.zeros(2, 1, dtype=torch.int32)
    qi, ki, w = q[:, :, :, :64], torch.zeros(2, 32, 64, dtype=BF), torch.zeros(2, 1, 4)
    dsa.dsa_window_attn(q, k, k, given)
    assert answers.last("dsa_window_attn")[7] == passed
    dsa.dsa_window_attn(q, k, k, given, sink_k=sink, sink_v=sink)
    assert answers.last("dsa_window_attn_sinks")[10] == passed
    dsa.dsa_window_attn(q, k, k, given, n_first=given)
    args = answers.last("dsa_window_attn_first")
    assert (args[4], args[8]) == (passed, passed)
    dsa.dsa_cache_attn(q, c, pos, window=given, n_first=given)
    assert answers.last("dsa_cache_attn_workspace_bytes")[4:] == (passed, passed)
    assert answers.last("dsa_cache_attn")[3:5] == (passed, passed)
    if given > 0:
        idx = torch.zeros(2, 1, 32, dtype=torch.int32)
        dsa.dsa_index_topk(qi, ki, w, 1.0, given, idx=idx)
        assert answers.last("dsa_index_topk")[11] == passed
        assert answers.last("dsa_index_topk_workspace_bytes")[3] == passed
        dsa.dsa_forward(qi, ki, w, 1.0, given, q, k, k, idx_out=idx)
        assert answers.last("dsa_forward")[0]._obj.K == passed


def test_a_window_past_an_int_is_refused_or_sees_every_key(lib):
    """The library's part: a window of any positive size is taken, a negative one is not."""
    L, FAKE = lib.lib(), 0x10000
    for window in (-TOP - 1, -1, 0):
        assert L.dsa_window_attn_first(1, FAKE, FAKE, FAKE, 4, None, 0, 0.0, window, 1, 64, 64, 4, 2,
                                       128, 128, 0, FAKE, None) == 1
    assert L.dsa_window_attn_first(1, FAKE, FAKE, FAKE, -TOP - 1, None, 0, 0.0, 8, 1, 64, 64, 4, 2,
                                   128, 128, 0, FAKE, None) == 1


# ----------------------------------------------------------------------------- workspaces
def test_the_two_forms_share_no_workspace_size(answers):
    """A call over no selected keys, which the library refuses, leaves the size of the whole-context
    workspace alone, and the other way round."""
    q, pos = torch.zeros(2, 1, 4, 64, dtype=BF), torch.zeros(2, 1, dtype=torch.int32)
    none = torch.zeros(2, 1, 0, dtype=torch.int32)
    sizes = {"dsa_cache_attn_workspace_bytes": 4096, "dsa_cache_sparse_attn_workspace_bytes": 0}

    class Sizes(Answers):
        def __getattr__(self, name):
            got = super().__getattr__(name)
            return (lambda *args: (got(*args), sizes[name])[1]) if name in sizes else got

    for first in (0, 1):
        dsa._LIB, c = Sizes(), some_cache()
        forms = [lambda: dsa.dsa_cache_sparse_attn(q, c, pos, none), lambda: dsa.dsa_cache_attn(q, c, pos)]
        forms[first]()
        forms[1 - first]()
        assert dsa._LIB.last("dsa_cache_attn")[13] == 4096
        assert dsa._LIB.last("dsa_cache_sparse_attn")[13] == 0


# ----------------------------------------------------------------------------- a cache's tensors
def test_a_cache_is_not_changed(answers):
    """Another page table, or other sizes, would not reach the library: they take a new Cache."""
    c, pos = some_cache(), torch.zeros(2, 1, dtype=torch.int32)
    for name, value in (("table", torch.zeros(2, 9, dtype=torch.int32)), ("pages", c.pages.clone()),
                        ("kv_heads", 1), ("dqk", 128), ("device", "cpu"), ("args", None)):
        with pytest.raises(AttributeError):
            setattr(c, name, value)
    c.lengths = [3]  # what a program keeps with it is its own
    c.lengths = [4]
    dsa.dsa_cache_read(c, pos)
    c.table[:] = 3  # the entries may change
    dsa.dsa_cache_read(c, pos)


@pytest.mark.parametrize("which,shape", [("table", (2, 3)), ("table", (2, 4000)),
                                         ("pages", (800, 16, 144))])
def test_a_cache_whose_tensors_were_resized_is_refused(answers, which, shape):
    c, pos = some_cache(), torch.zeros(2, 1, dtype=torch.int32)
    q, new = torch.zeros(2, 1, 4, 64, dtype=BF), torch.zeros(2, 1, 2, 64, dtype=BF)
    getattr(c, which).resize_(shape)
    n = len(answers.calls)
    for call in (lambda: dsa.dsa_cache_append(c, pos, new, new), lambda: dsa.dsa_cache_read(c, pos),
                 lambda: dsa.dsa_cache_attn(q, c, pos),
                 lambda: dsa.dsa_cache_sparse_attn(q, c, pos, pos[..., None])):
        with pytest.raises(ValueError):
            call()
    assert len(answers.calls) == n


# ----------------------------------------------------------------------------- devices
class On:
    """As much of a CUDA tensor as the binding's check looks at."""
    is_cuda = True

    def __init__(self, index):
        self.index, self.device = index, f"cuda:{index}"

    def is_contiguous(self):
        return True

    def get_device(self):
        return self.index


def test_tensors_of_another_device_are_refused(monkeypatch):
    """Kernels run on the current device, which may not reach another one's memory."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    dsa._dev(On(1), None, On(1))
    for ts in ((On(0),), (On(1), On(0)), (None, On(1), On(2))):
        with pytest.raises(ValueError, match="not the current device"):
            dsa._dev(*ts)
    for call in (lambda: dsa.dsa_window_attn(On(1), On(0), On(0), 8, n_first=4),
                 lambda: dsa.dsa_topk(On(0), 4)):
        with pytest.raises(ValueError, match="not the current device"):
            call()


# ----------------------------------------------------------------------------- shapes and types
def test_window_attn_refuses_tensors_that_do_not_go_together(answers):
    """What the library would read or write past the end, or as another type."""
    z = lambda *s, dtype=BF: torch.zeros(*s, dtype=dtype)  # noqa: E731
    q, k, v = z(2, 3, 4, 64), z(2, 32, 2, 64), z(2, 32, 2, 128)
    good = dict(gate=z(2, 3, 4), out=z(2, 3, 4, 128))
    for more in (dict(n_first=4), dict(), dict(sink_k=z(5, 2, 64), sink_v=z(5, 2, 128))):
        dsa.dsa_window_attn(q, k, v, 8, **good, **more)
    dsa.dsa_window_attn(q, z(3, 32, 2, 64), z(3, 32, 2, 128), 8, out=z(9, 3, 4, 128))  # room to spare
    n = len(answers.calls)
    f32 = torch.float32
    bad = [dict(k=z(1, 32, 2, 64)), dict(k=z(2, 31, 2, 64)), dict(k=z(2, 32, 2, 128)),
           dict(k=z(2, 32, 2, 64, dtype=f32)), dict(q=z(2, 3, 4, 64, dtype=f32)),
           dict(v=z(2, 32, 1, 128)), dict(v=z(1, 32, 2, 128)), dict(v=z(2, 32, 2, 128, dtype=f32)),
           dict(gate=z(2, 3, 3)), dict(gate=z(2, 3, 4, dtype=f32)), dict(out=z(2, 3, 4, 64)),
           dict(out=z(2, 3, 4, 128, dtype=f32)), dict(sink_k=z(5, 2, 64)),
           dict(sink_k=z(5, 2, 64), sink_v=z(4, 2, 128)), dict(sink_k=z(5, 1, 64), sink_v=z(5, 2, 128))]
    for change in bad:
        for n_first in (0, 4):
            args = dict(dict(q=q, k=k, v=v), **change)
            with pytest.raises(ValueError):
                dsa.dsa_window_attn(window=8, n_first=n_first, **args)
    assert len(answers.calls) == n
