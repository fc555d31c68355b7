"""The paged key/value cache on the GPU: appending with rotation (whole pages compared to the bit),
reading back, attention over windows, whole contexts and selected keys, against the float64 oracle.

Tolerance of an attention output, element by element: half a step of its bf16 rounding, 2^-8 |o|,
and for the probabilities 2^-10 sum_t p_t |v_t|: each is f16 (half a step 2^-11; bf16 rows: a pair,
2^-16), and the other 2^-11 covers float32 scores of up to 2^6 in log2 units (2^6 * 2^-23 * a few
roundings), the exponential and the sums.

f16 has a smallest step as well, 2^-24.  The largest probability of a row is held at 2^6 or above, so
a term is off by at most half that step over 2^6, 2^-31 of the largest, whose value the sum of n terms
cannot fall below: n 2^-31 max|v| in all, which counts where the weighted values are zero but for
terms that small (4-bit values often are exactly zero)."""
import numpy as np
import pytest
import torch

from oracle import cache_oracle as O

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


class Setup:
    """A cache with shuffled pages and every row filled by its own token, and the oracle's view."""

    def __init__(self, lib, dev, fmt="e2m1", B=2, ctx=70, page=16, HKV=2, DQK=64, DV=64, k_scale=1.0,
                 v_scale=1.0, seed=0, fill=True):
        self.lib, self.dev, self.fmt, self.page = lib, dev, fmt, page
        self.B, self.ctx, self.HKV, self.DQK, self.DV = B, ctx, HKV, DQK, DV
        self.r = np.random.default_rng(seed)
        self.each = -(-ctx // page)
        self.n_pages = B * self.each + 2
        table = self.r.permutation(self.n_pages)[: B * self.each].reshape(B, self.each)
        self.table = torch.tensor(table, dtype=torch.int32, device=dev)
        self.pages = lib.dsa_cache_pages(fmt, self.n_pages, page, HKV, DQK, DV, device=dev)
        # what no token was appended to holds garbage: NaN in either format
        self.pages.view(torch.uint8).fill_(0xFF)
        self.scales = (k_scale, v_scale)
        self.cache = lib.Cache(self.pages, self.table, HKV, DQK, DV, k_scale=k_scale,
                               v_scale=v_scale)
        self.k = np.full((B, ctx, HKV, DQK), np.nan)  # as held
        self.v = np.full((B, ctx, HKV, DV), np.nan)
        if fill:
            self.fill()

    def normal(self, *shape):
        return O.to_bf16(self.r.standard_normal(shape))

    def cuda(self, x):
        return torch.tensor(np.asarray(x), dtype=torch.float32).to(BF).to(self.dev)

    def fill(self):
        k, v = self.normal(*self.k.shape), self.normal(*self.v.shape)
        pos = torch.arange(self.ctx, dtype=torch.int32, device=self.dev).expand(self.B, -1)
        self.lib.dsa_cache_append(self.cache, pos.contiguous(), self.cuda(k), self.cuda(v))
        for b in range(self.B):
            for t in range(self.ctx):
                _, self.k[b, t], self.v[b, t] = O.row_of(k[b, t], v[b, t], self.fmt, *self.scales)


def check(got, want, mag, floor=0.0):
    got = got.float().cpu().numpy().astype(np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    ok = ~np.isnan(want)
    err = np.abs(got - want)[ok]
    bound = (np.abs(want) * 2.0**-8 + mag * 2.0**-10 + floor)[ok]
    assert (err <= bound).all(), f"worst {np.max(err / np.maximum(bound, 1e-30))} of the bound"


def run_attn(s, pos, H, window=0, n_first=0, idx=None, gate=False, gate_mode=None, sm_scale=0.0,
             skip=lambda b, t: False):
    """The call and the oracle's rows for queries at pos [B, S] (numpy)."""
    B, S = pos.shape
    q = s.normal(B, S, H, s.DQK)
    g = s.normal(B, S, H) if gate else None
    pt = torch.tensor(pos, dtype=torch.int32, device=s.dev)
    gt = s.cuda(g) if gate else None
    if idx is None:
        got = s.lib.dsa_cache_attn(s.cuda(q), s.cache, pt, window=window, n_first=n_first, gate=gt,
                                   gate_mode=gate_mode, sm_scale=sm_scale)
    else:
        it = torch.tensor(idx, dtype=torch.int32, device=s.dev)
        got = s.lib.dsa_cache_sparse_attn(s.cuda(q), s.cache, pt, it, gate=gt, gate_mode=gate_mode,
                                          sm_scale=sm_scale)
    want, mag = np.zeros((B, S, H, s.DV)), np.zeros((B, S, H, s.DV))
    for b in range(B):
        for i in range(S):
            p = int(pos[b, i])
            keys = O.window_keys(p, window, n_first) if idx is None else [
                t for t in idx[b, i] if 0 <= t <= p]
            keys = [t for t in keys if t < s.ctx and not skip(b, t)]
            want[b, i], mag[b, i] = O.attend(q[b, i], s.k[b], s.v[b], keys,
                                             sm_scale if sm_scale > 0 else s.DQK**-0.5,
                                             None if g is None else g[b, i],
                                             gate_mode or "sigmoid")
    check(got, want, mag)
    assert s.lib.dsa_device_status() == 0
    return got


# ----------------------------------------------------------------------------- append
@pytest.mark.parametrize("fmt", ["bf16", "e2m1"])
@pytest.mark.parametrize("rope", ["off", "interleaved", "half"])
@pytest.mark.parametrize("HKV,G,DQK,DV,rd", [(1, 3, 64, 64, 32), (3, 1, 128, 64, 64),
                                             (8, 4, 192, 128, 64), (2, 2, 128, 128, 128),
                                             (5, 2, 64, 128, 64), (4, 1, 192, 64, 192)])
def test_append_writes_the_pages_to_the_bit(lib, cuda_dev, fmt, rope, HKV, G, DQK, DV, rd):
    ks, vs = (1.0, 1.0) if fmt == "bf16" else (0.37, 4.0)
    s = Setup(lib, cuda_dev, fmt, B=3, ctx=50, page=7, HKV=HKV, DQK=DQK, DV=DV, k_scale=ks,
              v_scale=vs, fill=False)
    S, H = 5, HKV * G
    # far positions in a wide table would need a huge cache: the pages repeat instead
    pos = np.array([[0, 1, 2, 3, 4], [49, 48, 7, 13, 14], [-1, 20, -7, 21, 60]])
    s.table[1, 2] = -1           # positions 14..20 of sequence 1 have no page
    s.table[2, 2] = s.n_pages    # the same for sequence 2
    inv = (100.0 ** (-np.arange(rd // 2) / (rd // 2))).astype(np.float32)
    q, k, v = s.normal(3, S, H, DQK), s.normal(3, S, HKV, DQK), s.normal(3, S, HKV, DV)
    before = s.pages.clone()
    kt = s.cuda(k)
    q_out, k_out = lib.dsa_cache_append(
        s.cache, torch.tensor(pos, dtype=torch.int32, device=cuda_dev), kt, s.cuda(v),
        rope=rope, inv_freq=torch.tensor(inv, device=cuda_dev), q=s.cuda(q),
        k_out=torch.empty_like(kt))
    want = before.view(torch.uint8).cpu().numpy().reshape(s.n_pages, 7, -1).copy()
    tab = s.table.cpu().numpy()
    for b in range(3):
        for i in range(S):
            p = int(pos[b, i])
            kr = O.rotate(k[b, i], p, inv, rope) if p >= 0 else k[b, i] * 0
            qr = O.rotate(q[b, i], p, inv, rope) if p >= 0 else q[b, i] * 0
            assert np.array_equal(k_out[b, i].float().cpu().numpy(), kr)
            if rope != "off":
                assert np.array_equal(q_out[b, i].float().cpu().numpy(), qr)
            if p < 0 or p // 7 >= s.each or not 0 <= tab[b, p // 7] < s.n_pages:
                continue
            want[tab[b, p // 7], p % 7] = O.row_of(kr, v[b, i], fmt, ks, vs)[0]
    got = s.pages.view(torch.uint8).cpu().numpy().reshape(want.shape)
    if fmt == "e2m1":  # the pad bytes of a row are not part of the contract
        n = HKV * (DQK + DV) * 9 // 16
        got, want = got[..., :n], want[..., :n]
    assert np.array_equal(got, want)


@pytest.mark.parametrize("rope", ["interleaved", "half"])
def test_append_far_positions_and_in_place(lib, cuda_dev, rope):
    """Angles of far positions keep their value (float64), and q and k may be rotated in place."""
    s = Setup(lib, cuda_dev, "bf16", B=1, ctx=16, page=4, HKV=2, DQK=128, DV=64, fill=False)
    far = 987_654_321
    wide = s.table.new_full((1, far // 4 + 1), -1)
    wide[0, far // 4] = s.table[0, 0]
    cache = lib.Cache(s.pages, wide, 2, 128, 64)
    inv = (10000.0 ** (-np.arange(32) / 32)).astype(np.float32)
    q, k, v = s.normal(1, 1, 4, 128), s.normal(1, 1, 2, 128), s.normal(1, 1, 2, 64)
    qt, kt = s.cuda(q), s.cuda(k)
    pos = torch.tensor([[far]], dtype=torch.int32, device=cuda_dev)
    lib.dsa_cache_append(cache, pos, kt, s.cuda(v), rope=rope,
                         inv_freq=torch.tensor(inv, device=cuda_dev), q=qt, q_out=qt, k_out=kt)
    assert np.array_equal(qt[0, 0].float().cpu().numpy(), O.rotate(q[0, 0], far, inv, rope))
    assert np.array_equal(kt[0, 0].float().cpu().numpy(), O.rotate(k[0, 0], far, inv, rope))
    k2, v2 = lib.dsa_cache_read(cache, pos)
    assert torch.equal(k2, kt) and np.array_equal(v2.float().cpu().numpy(), v)


def test_encoding_of_edge_values(lib, cuda_dev):
    """Ties, saturation, subnormal scales, zeros, infinities and NaN, group by group."""
    s = Setup(lib, cuda_dev, "e2m1", B=1, ctx=4, page=4, HKV=1, DQK=192, DV=128, fill=False)
    k = np.zeros((1, 4, 1, 192))
    k[0, 0, 0, :16] = np.array([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -1.75,
                                -2.5, -3.5, -5, 4.5])
    k[0, 0, 0, 16:32] = 3.0e38
    k[0, 0, 0, 32:48] = np.linspace(-1, 1, 16) * 2.0**-11   # the scale rounds to 0
    k[0, 0, 0, 48:64] = np.linspace(-1, 1, 16) * 2.0**-7    # a subnormal scale
    k[0, 0, 0, 64] = np.inf
    k[0, 0, 0, 80:96] = np.nan
    k[0, 0, 0, 96] = -0.0
    k[0, 1, 0] = self_k = np.linspace(-3000, 3000, 192)
    k[0, 1, 0] = O.to_bf16(self_k)
    k[0, 2, 0] = O.to_bf16(np.sign(self_k) * 2.0 ** np.linspace(-30, 30, 192))
    k = O.to_bf16(k)
    v = s.normal(1, 4, 1, 128)
    pos = torch.arange(4, dtype=torch.int32, device=cuda_dev)[None]
    lib.dsa_cache_append(s.cache, pos, s.cuda(k), s.cuda(v))
    rows = s.pages[s.table[0, 0].item()].cpu().numpy()
    for t in range(4):
        want, kd, vd = O.row_of(k[0, t], v[0, t], "e2m1", 1.0, 1.0)
        assert np.array_equal(rows[t], want) or np.array_equal(rows[t][:180], want[:180])
    k2, v2 = lib.dsa_cache_read(s.cache, pos)
    for t in range(4):
        _, kd, vd = O.row_of(k[0, t], v[0, t], "e2m1", 1.0, 1.0)
        assert np.array_equal(k2[0, t].float().cpu().numpy(), kd, equal_nan=True)
        assert np.array_equal(v2[0, t].float().cpu().numpy(), vd)


def test_read_back_without_a_row_is_zero(lib, cuda_dev):
    s = Setup(lib, cuda_dev, "e2m1", B=2, ctx=20, page=8, HKV=3, DQK=128, DV=128)
    s.table[1, 1] = -5
    pos = torch.tensor([[0, -1, 19], [8, 24, 7]], dtype=torch.int32, device=cuda_dev)
    k, v = lib.dsa_cache_read(s.cache, pos)
    for b, i in ((0, 1), (1, 0), (1, 1)):
        assert not k[b, i].any() and not v[b, i].any()
    for b, i, t in ((0, 0, 0), (0, 2, 19), (1, 2, 7)):
        assert np.array_equal(k[b, i].float().cpu().numpy(), s.k[b, t])
        assert np.array_equal(v[b, i].float().cpu().numpy(), s.v[b, t])


# ----------------------------------------------------------------------------- attention
SHAPES = [  # HKV, G, DQK, DV: one to many KV heads, groups below, at and past 8 columns
    (1, 1, 64, 64), (1, 32, 192, 128), (2, 12, 128, 64), (3, 20, 64, 128), (4, 1, 128, 128),
    (8, 4, 192, 128), (20, 1, 128, 128), (10, 2, 192, 64), (16, 4, 64, 64), (7, 9, 128, 128),
    (64, 1, 192, 128), (9, 1, 192, 128)]


@pytest.mark.parametrize("fmt", ["bf16", "e2m1"])
@pytest.mark.parametrize("HKV,G,DQK,DV", SHAPES)
def test_whole_context(lib, cuda_dev, fmt, HKV, G, DQK, DV):
    s = Setup(lib, cuda_dev, fmt, B=2, ctx=300, page=48, HKV=HKV, DQK=DQK, DV=DV,
              k_scale=1.0 if fmt == "bf16" else 0.5, v_scale=1.0 if fmt == "bf16" else 2.0)
    run_attn(s, np.array([[299], [17]]), HKV * G, gate=True)


@pytest.mark.parametrize("fmt", ["bf16", "e2m1"])
@pytest.mark.parametrize("window,n_first", [(1, 0), (1, 3), (16, 4), (100, 1), (129, 130), (1000, 5),
                                            (64, 1000)])
def test_window_with_first_tokens(lib, cuda_dev, fmt, window, n_first):
    s = Setup(lib, cuda_dev, fmt, B=3, ctx=260, page=100, HKV=2, DQK=128, DV=128)
    pos = np.array([[0, 259, 3], [-1, 16, 100], [128, 129, 255]])
    out = run_attn(s, pos, 6, window=window, n_first=n_first)
    assert not out[1, 0].any()  # padding


@pytest.mark.parametrize("fmt", ["bf16", "e2m1"])
@pytest.mark.parametrize("K", [1, 15, 16, 17, 200])
def test_selected_keys(lib, cuda_dev, fmt, K):
    s = Setup(lib, cuda_dev, fmt, B=2, ctx=200, page=1, HKV=4, DQK=192, DV=128)
    pos = np.array([[199, 5, -1], [100, 0, 198]])
    idx = np.full((2, 3, K), -1)
    for b in range(2):
        for i in range(3):
            n = min(K, s.ctx)
            idx[b, i, :n] = np.sort(s.r.permutation(s.ctx)[:n])  # past pos too: skipped
    idx[0, 0, K // 2] = 5000
    idx[1, 0, 0] = -9
    run_attn(s, pos, 8, idx=idx, gate=True, gate_mode="silu")


@pytest.mark.parametrize("fmt", ["bf16", "e2m1"])
def test_unsorted_and_sparse_lists(lib, cuda_dev, fmt):
    """Entries in any order, with skipped ones anywhere: whole stages of them, single ones."""
    s = Setup(lib, cuda_dev, fmt, B=1, ctx=150, page=16, HKV=1, DQK=64, DV=64)
    idx = np.full((1, 1, 900), -1)
    at = s.r.permutation(900)[:150]
    idx[0, 0, at] = s.r.permutation(150)
    run_attn(s, np.array([[149]]), 5, idx=idx)
    idx[:] = -1
    run_attn(s, np.array([[149]]), 5, idx=idx)  # nothing left: zeros
    idx[0, 0, 899] = 149
    run_attn(s, np.array([[149]]), 5, idx=idx)


@pytest.mark.parametrize("fmt", ["bf16", "e2m1"])
@pytest.mark.parametrize("HKV,G", [(2, 2), (8, 1)])
def test_missing_pages_are_not_seen(lib, cuda_dev, fmt, HKV, G):
    s = Setup(lib, cuda_dev, fmt, B=2, ctx=96, page=8, HKV=HKV, DQK=64, DV=64)
    s.table[0, 3] = -1
    s.table[1, :] = s.n_pages + 7
    s.table[0, 11] = -2**31
    skip = lambda b, t: b == 1 or t // 8 in (3, 11)  # noqa: E731
    pos = np.array([[95, 24], [95, 3]])
    out = run_attn(s, pos, HKV * G, skip=skip)
    assert not out[1].any()
    run_attn(s, pos, HKV * G, window=9, n_first=30, skip=skip)


def test_positions_past_the_table(lib, cuda_dev):
    s = Setup(lib, cuda_dev, "e2m1", B=1, ctx=64, page=16, HKV=2, DQK=64, DV=64)
    pos = np.array([[64, 2**31 - 1, 80]])
    q = s.normal(1, 3, 2, 64)
    out = s.lib.dsa_cache_attn(s.cuda(q), s.cache, torch.tensor(pos, dtype=torch.int32,
                                                               device=cuda_dev), window=10, n_first=4)
    for i, keys in enumerate(([0, 1, 2, 3] + list(range(55, 64)), [0, 1, 2, 3], [0, 1, 2, 3])):
        want, mag = O.attend(q[0, i], s.k[0], s.v[0], keys, 0.125)
        check(out[0, i], want, mag)


@pytest.mark.parametrize("fmt", ["bf16", "e2m1"])
def test_unseen_keys_may_hold_anything(lib, cuda_dev, fmt):
    """NaN and infinities in rows that a query does not see, in pages shared with rows it sees."""
    s = Setup(lib, cuda_dev, fmt, B=1, ctx=64, page=16, HKV=2, DQK=64, DV=64)
    bad = torch.full((1, 2, 2, 64), float("nan"), dtype=BF, device=cuda_dev)
    bad[:, 1] = float("inf")
    s.lib.dsa_cache_append(s.cache, torch.tensor([[21, 41]], dtype=torch.int32, device=cuda_dev),
                           bad, bad)
    run_attn(s, np.array([[20, 40]]), 4, window=19)
    idx = np.array([[[3, 20, 22, 40, 42, 63]]])
    run_attn(s, np.array([[63]]), 4, idx=idx)
    # a query that sees one gets NaN, and its neighbours do not
    q = torch.ones(1, 2, 4, 64, dtype=BF, device=cuda_dev)
    out = s.lib.dsa_cache_attn(q, s.cache, torch.tensor([[21, 20]], dtype=torch.int32,
                                                        device=cuda_dev))
    assert out[0, 0].isnan().all() and not out[0, 1].isnan().any()


@pytest.mark.parametrize("fmt", ["bf16", "e2m1"])
def test_large_and_small_queries(lib, cuda_dev, fmt):
    """Query magnitudes past f16's range on both sides, scores that spread over 2^10."""
    s = Setup(lib, cuda_dev, fmt, B=1, ctx=120, page=16, HKV=1, DQK=64, DV=64)
    for scale, sm in ((2.0**60, 2.0**-60), (2.0**-60, 2.0**57), (1.0, 4.0), (2.0**-126, 1.0)):
        q = s.normal(1, 1, 8, 64) * scale
        out = s.lib.dsa_cache_attn(s.cuda(q), s.cache, torch.tensor([[119]], dtype=torch.int32,
                                                                   device=cuda_dev), sm_scale=sm)
        # scores of size x carry a float32 error of about x * 2^-22, p the same relative error
        want, mag = O.attend(q[0, 0], s.k[0], s.v[0], list(range(120)), sm)
        top = np.abs(s.k[0, :120, 0] @ q[0, 0].T * sm).max()
        floor = 120 * 2.0**-31 * np.abs(s.v[0, :120]).max() if fmt == "e2m1" else 0.0
        check(out[0, 0], want, mag * (1 + top * 2.0**-10), floor)


def test_long_context_in_slices(lib, cuda_dev):
    """Many slices per row, pages that end inside stages, rows of very different lengths."""
    s = Setup(lib, cuda_dev, "e2m1", B=3, ctx=2500, page=37, HKV=2, DQK=64, DV=64)
    run_attn(s, np.array([[2499], [0], [1203]]), 4)
    run_attn(s, np.array([[2499], [700], [64]]), 4, window=640, n_first=33)


@pytest.mark.parametrize("fmt,HKV", [("e2m1", 8), ("e2m1", 24), ("bf16", 16)])
def test_groups_of_heads_side_by_side(lib, cuda_dev, fmt, HKV):
    """Rows whose heads several CTAs share: every share of the grid at work, and a part of them."""
    s = Setup(lib, cuda_dev, fmt, B=2, ctx=4807, page=64, HKV=HKV, DQK=64, DV=64)
    for pos in ([[4806], [4790]], [[4000], [-1]], [[-1], [40]]):
        run_attn(s, np.array(pos), HKV, gate=True)


@pytest.mark.parametrize("fmt", ["bf16", "e2m1"])
def test_windows_past_an_int(lib, cuda_dev, fmt):
    """A window, or first tokens, of any size: past the context, every key."""
    s = Setup(lib, cuda_dev, fmt, B=2, ctx=90, page=16, HKV=2, DQK=64, DV=64)
    q = s.cuda(s.normal(2, 1, 4, 64))
    pos = torch.tensor([[89], [30]], dtype=torch.int32, device=cuda_dev)
    every = lib.dsa_cache_attn(q, s.cache, pos).float()
    for window, n_first in ((90, 0), (2**31 - 1, 0), (2**32, 0), (2**40, 2**32), (1, 2**32), (3, 90)):
        out = lib.dsa_cache_attn(q, s.cache, pos, window=window, n_first=n_first).float()
        # two results for the same sums, each within the bound of it (sum p |v| <= max |v|)
        bound = 2.0**-8 * torch.maximum(out.abs(), every.abs()) + 2.0**-10 * np.abs(s.v).max()
        assert ((out - every).abs() <= 2 * bound).all()
    kv = s.cuda(s.normal(1, 40, 2, 64))
    with pytest.raises(lib.DSAError):
        lib.dsa_window_attn(kv, kv, kv, 8, n_first=2**32)


def test_same_result_every_time_and_out_given(lib, cuda_dev):
    s = Setup(lib, cuda_dev, "e2m1", B=4, ctx=700, page=64, HKV=4, DQK=64, DV=64)
    q = s.cuda(s.normal(4, 2, 8, 64))
    pos = torch.tensor([[699, 698], [5, 6], [300, 301], [64, 63]], dtype=torch.int32,
                       device=cuda_dev)
    ref = lib.dsa_cache_attn(q, s.cache, pos)
    for _ in range(5):
        out = torch.full_like(ref, float("nan"))
        assert lib.dsa_cache_attn(q, s.cache, pos, out=out) is out
        assert torch.equal(out, ref)


def test_captured_and_replayed_on_another_stream(lib, cuda_dev):
    """A decode step (append, read, window and selected attention) captured once and replayed with
    new tokens at new positions, and the same calls on a side stream, against eager calls."""
    s = Setup(lib, cuda_dev, "e2m1", B=2, ctx=200, page=16, HKV=2, DQK=64, DV=64)
    q, k, v = (torch.empty(2, 1, n, 64, dtype=BF, device=cuda_dev) for n in (4, 2, 2))
    pos = torch.zeros(2, 1, dtype=torch.int32, device=cuda_dev)
    idx = torch.zeros(2, 1, 40, dtype=torch.int32, device=cuda_dev)
    inv = torch.tensor([1.0, 0.1, 0.01] + [0.001] * 13, device=cuda_dev)

    def step(stream=None):
        qr, _ = lib.dsa_cache_append(s.cache, pos, k, v, rope="half", inv_freq=inv, q=q,
                                     stream=stream)
        a = lib.dsa_cache_attn(qr, s.cache, pos, window=150, n_first=4, stream=stream)
        b = lib.dsa_cache_sparse_attn(qr, s.cache, pos, idx, stream=stream)
        return a, b

    def inputs(seed):
        g = torch.Generator(device=cuda_dev).manual_seed(seed)
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, generator=g, device=cuda_dev))
        pos.copy_(torch.randint(100, 199, (2, 1), generator=g, device=cuda_dev))
        for b in range(2):
            idx[b, 0] = torch.randperm(100, generator=g, device=cuda_dev)[:40].sort().values

    inputs(1)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for seed in (2, 3):
        inputs(seed)
        graph.replay()
        got = [x.clone() for x in held]
        eager = step()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        other = step(stream=side)
        torch.cuda.current_stream().wait_stream(side)
        for x, y, z in zip(got, eager, other):
            assert torch.equal(x, y) and torch.equal(x, z)


@pytest.mark.parametrize("fmt", ["bf16", "e2m1"])
def test_decode_step_against_the_contiguous_layers(lib, cuda_dev, fmt):
    """The path as it is used: a prompt appended and run through the contiguous window layer, then
    tokens one by one over the cache: the same rows as the contiguous layers over everything, a DSA
    layer on the indexer's own top-k among them."""
    B, S, new, H, HKV, D = 2, 130, 4, 4, 4, 128
    s = Setup(lib, cuda_dev, fmt, B=B, ctx=S + new, page=16, HKV=HKV, DQK=D, DV=D, fill=False)
    T = S + new
    q, k, v = s.cuda(s.normal(B, T, H, D)), s.cuda(s.normal(B, T, HKV, D)), s.cuda(s.normal(B, T, HKV, D))
    qi = torch.randint(-2, 3, (B, T, 16, 64), device=cuda_dev).to(BF)
    ki = torch.randint(-2, 3, (B, T, 64), device=cuda_dev).to(BF)
    w = torch.randint(1, 5, (B, T, 16), device=cuda_dev).float()
    inv = torch.tensor(10000.0 ** (-np.arange(32) / 32), dtype=torch.float32, device=cuda_dev)
    pos = torch.arange(T, dtype=torch.int32, device=cuda_dev).expand(B, -1).contiguous()
    qr, kr = torch.empty_like(q), torch.empty_like(k)

    def append(a, b):
        part = [x[:, a:b].contiguous() for x in (pos, k, v, q)]
        out = lib.dsa_cache_append(s.cache, part[0], part[1], part[2], rope="interleaved",
                                   inv_freq=inv, q=part[3], k_out=torch.empty_like(part[1]))
        qr[:, a:b], kr[:, a:b] = out
        return part[0]

    append(0, S)
    for t in range(S, T):
        append(t, t + 1)
    kc, vc = lib.dsa_cache_read(s.cache, pos)
    if fmt == "bf16":
        assert torch.equal(kc, kr) and torch.equal(vc, v)
    whole = lib.dsa_window_attn(qr, kc, vc, 64, n_first=4)
    idx = lib.dsa_topk(lib.dsa_index_scores(qi, ki, w, 0.0625), 32)
    dsa_all = lib.dsa_sparse_attn(qr, kc, vc, idx)
    for t in range(S, T):
        p, qt = pos[:, t : t + 1].contiguous(), qr[:, t : t + 1].contiguous()
        a = lib.dsa_cache_attn(qt, s.cache, p, window=64, n_first=4)
        b = lib.dsa_cache_sparse_attn(qt, s.cache, p, idx[:, t : t + 1].contiguous())
        # both sides are within 2^-8 |o| + 2^-10 sum p|v| <= 2^-8 |o| + 2^-10 max|v| of the truth
        for x, y in ((a, whole[:, t : t + 1]), (b, dsa_all[:, t : t + 1])):
            x, y = x.float(), y.float()
            assert ((x - y).abs() <= y.abs() * 2.0**-6 + 2.0**-9 * vc.abs().max().float()).all()


# ----------------------------------------------------------------------------- window_attn, n_first
def window_oracle(q, k, v, window, n_first, gate):
    B, S, H, D = q.shape
    T = k.shape[1]
    want, mag = np.zeros((B, S, H, v.shape[3])), np.zeros((B, S, H, v.shape[3]))
    for b in range(B):
        for i in range(S):
            keys = O.window_keys(T - S + i, window, n_first)
            want[b, i], mag[b, i] = O.attend(q[b, i], k[b], v[b], keys, D**-0.5,
                                             None if gate is None else gate[b, i])
    return want, mag


@pytest.mark.parametrize("algo", ["gather", "masked_tile"])
@pytest.mark.parametrize("B,S,T,window,n_first", [
    (1, 70, 70, 8, 4), (2, 130, 300, 64, 1), (1, 5, 261, 3, 128), (1, 200, 400, 128, 127),
    (1, 300, 300, 1, 2), (1, 129, 129, 1000, 64), (1, 150, 600, 40, 65), (1, 64, 512, 256, 33)])
def test_window_attn_first_tokens(lib, cuda_dev, algo, B, S, T, window, n_first):
    r = np.random.default_rng(S)
    H, HKV, D = 4, 2, 128
    q, k, v = (O.to_bf16(r.standard_normal(sh)) for sh in ((B, S, H, D), (B, T, HKV, D),
                                                           (B, T, HKV, D)))
    gate = O.to_bf16(r.standard_normal((B, S, H))) if S % 2 else None
    c = lambda x: None if x is None else torch.tensor(x, dtype=torch.float32).to(BF).to(cuda_dev)  # noqa: E731
    out = lib.dsa_window_attn(c(q), c(k), c(v), window, gate=c(gate), n_first=n_first, algo=algo)
    check(out, *window_oracle(q, k, v, window, n_first, gate))
    assert lib.dsa_device_status() == 0


@pytest.mark.parametrize("D,DV", [(64, 32), (192, 128)])
def test_window_attn_first_tokens_float32(lib, cuda_dev, D, DV):
    r = np.random.default_rng(3)
    q, k, v = (r.standard_normal(sh).astype(np.float32) for sh in ((1, 40, 4, D), (1, 90, 2, D),
                                                                   (1, 90, 2, DV)))
    t = lambda x: torch.tensor(x, device=cuda_dev)  # noqa: E731
    out = lib.dsa_window_attn(t(q), t(k), t(v), 7, n_first=5).cpu().numpy()
    want, mag = window_oracle(q.astype(np.float64), k.astype(np.float64), v.astype(np.float64), 7,
                              5, None)
    # float32 scores below 2^4 in log2 units and ex2 within 2^-22: p within 2^-18
    assert (np.abs(out - want) <= np.abs(want) * 2.0**-24 + mag * 2.0**-17).all()


def test_window_attn_192_wide_and_no_first(lib, cuda_dev):
    """The hybrid block's dims through the tensor-core tiles; n_first = 0 is the plain window, and
    first tokens inside every window change nothing."""
    g = torch.Generator(device=cuda_dev).manual_seed(5)
    rand = lambda *s: torch.randn(*s, generator=g, device=cuda_dev).to(BF)  # noqa: E731
    q, k, v = rand(1, 300, 8, 192), rand(1, 420, 2, 192), rand(1, 420, 2, 128)
    plain = lib.dsa_window_attn(q, k, v, 100)
    assert torch.equal(plain, lib.dsa_window_attn(q, k, v, 100, n_first=0))
    wide = lib.dsa_window_attn(q, k, v, 420)
    assert torch.equal(wide, lib.dsa_window_attn(q, k, v, 420, n_first=128))
    f64 = lambda x: x.float().cpu().numpy().astype(np.float64)  # noqa: E731
    out = lib.dsa_window_attn(q, k, v, 100, n_first=20)
    check(out, *window_oracle(f64(q), f64(k), f64(v), 100, 20, None))


# ----------------------------------------------------------------------------- further calls
@pytest.mark.parametrize("fmt", ["bf16", "e2m1"])
def test_more_rows_than_the_gpu_holds(lib, cuda_dev, fmt):
    """Rows in plenty are taken whole, one CTA each; those without keys get zeros there too."""
    s = Setup(lib, cuda_dev, fmt, B=3, ctx=90, page=16, HKV=2, DQK=64, DV=64)
    pos = s.r.integers(-2, 90, (3, 250))
    out = run_attn(s, pos, 2, window=20, n_first=2)
    assert not out[torch.tensor(pos < 0, device=cuda_dev)].any()
    idx = np.sort(s.r.integers(0, 90, (3, 250, 1)), -1)
    run_attn(s, pos, 2, idx=idx)


@pytest.mark.parametrize("fmt", ["bf16", "e2m1"])
def test_a_query_that_is_not_finite_stays_alone(lib, cuda_dev, fmt):
    """An infinite or NaN query head gives NaN for itself, and nothing to the other heads and rows."""
    s = Setup(lib, cuda_dev, fmt, B=2, ctx=70, page=16, HKV=2, DQK=64, DV=64)
    q = s.cuda(s.normal(2, 2, 8, 64))
    pos = torch.tensor([[69, 68], [30, 3]], dtype=torch.int32, device=cuda_dev)
    clean = lib.dsa_cache_attn(q, s.cache, pos)
    q[0, 1, 2, 5] = float("inf")
    q[1, 0, 7, 0] = float("nan")
    got = lib.dsa_cache_attn(q, s.cache, pos)
    bad = torch.zeros(2, 2, 8, dtype=torch.bool, device=cuda_dev)
    bad[0, 1, 2] = bad[1, 0, 7] = True
    assert got[bad].isnan().all() and torch.equal(got[~bad], clean[~bad])


def test_two_streams_at_once(lib, cuda_dev):
    """Calls on two streams, each with its own workspace or outputs, at the same time."""
    s = Setup(lib, cuda_dev, "e2m1", B=2, ctx=900, page=64, HKV=4, DQK=64, DV=64)
    q = [s.cuda(s.normal(2, 1, 8, 64)) for _ in range(2)]
    pos = torch.tensor([[899], [500]], dtype=torch.int32, device=cuda_dev)
    want = [lib.dsa_cache_attn(x, s.cache, pos) for x in q]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    need = int(lib.lib().dsa_cache_attn_workspace_bytes(s.cache.ref, 2, 1, 8, 0, 0))
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device=cuda_dev)
    got = [[], []]
    for _ in range(20):
        got[0].append(lib.dsa_cache_attn(q[0], s.cache, pos, stream=streams[0], ws=ws))
        got[1].append(lib.dsa_cache_attn(q[1], s.cache, pos, stream=streams[1]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, want[i]) for x in got[i])
    with pytest.raises(ValueError):
        lib.dsa_cache_attn(q[0], s.cache, pos, ws=ws[: need - 1])


def test_rows_past_four_gigabytes(lib, cuda_dev):
    """Offsets in a large pool do not fit 32 bits: the last pages of 5.5 GB."""
    HKV, DQK, DV, page, n_pages = 8, 192, 128, 64, 60000
    pages = lib.dsa_cache_pages("e2m1", n_pages, page, HKV, DQK, DV, device=cuda_dev)
    assert pages.numel() > 1 << 32
    table = torch.tensor([[n_pages - 1, 3, n_pages - 2]], dtype=torch.int32, device=cuda_dev)
    cache = lib.Cache(pages, table, HKV, DQK, DV)
    small = Setup(lib, cuda_dev, "e2m1", B=1, ctx=192, page=page, HKV=HKV, DQK=DQK, DV=DV, fill=False)
    g = torch.Generator(device=cuda_dev).manual_seed(1)
    rand = lambda *s: torch.randn(*s, generator=g, device=cuda_dev).to(BF)  # noqa: E731
    pos = torch.arange(192, dtype=torch.int32, device=cuda_dev)[None]
    k, v, q = rand(1, 192, HKV, DQK), rand(1, 192, HKV, DV), rand(1, 192, 32, DQK)
    for c in (cache, small.cache):
        lib.dsa_cache_append(c, pos, k, v)
    for x, y in zip(lib.dsa_cache_read(cache, pos), lib.dsa_cache_read(small.cache, pos)):
        assert torch.equal(x, y)
    last = pos[:, -3:].contiguous()
    assert torch.equal(lib.dsa_cache_attn(q[:, -3:].contiguous(), cache, last),
                       lib.dsa_cache_attn(q[:, -3:].contiguous(), small.cache, last))


def test_rows_around_the_appended_ones_keep_their_bytes(lib, cuda_dev):
    """Appending to one row of a page leaves the others, the pad bytes of its own among them."""
    for fmt in ("bf16", "e2m1"):
        s = Setup(lib, cuda_dev, fmt, B=1, ctx=32, page=8, HKV=1, DQK=64, DV=64, fill=False)
        before = s.pages.view(torch.uint8).clone()
        pos = torch.tensor([[9]], dtype=torch.int32, device=cuda_dev)
        s.lib.dsa_cache_append(s.cache, pos, s.cuda(s.normal(1, 1, 1, 64)),
                               s.cuda(s.normal(1, 1, 1, 64)))
        changed = (s.pages.view(torch.uint8) != before).any(-1)
        row = torch.zeros_like(changed)
        row[s.table[0, 1], 1] = True
        assert torch.equal(changed, row)
        if fmt == "e2m1":
            assert torch.equal(s.pages[..., 72:], before[..., 72:])


def test_binding_refuses_what_does_not_fit(lib, cuda_dev):
    s = Setup(lib, cuda_dev, "e2m1", B=2, ctx=32, page=8, HKV=2, DQK=64, DV=64)
    pos = torch.zeros(2, 1, dtype=torch.int32, device=cuda_dev)
    q, k = s.cuda(s.normal(2, 1, 4, 64)), s.cuda(s.normal(2, 1, 2, 64))
    inv = torch.ones(16, device=cuda_dev)
    bad = [
        lambda: lib.dsa_cache_attn(q.float(), s.cache, pos),
        lambda: lib.dsa_cache_attn(q[:1], s.cache, pos),
        lambda: lib.dsa_cache_attn(q.cpu(), s.cache, pos),
        lambda: lib.dsa_cache_attn(q.transpose(1, 2), s.cache, pos),
        lambda: lib.dsa_cache_attn(q, s.cache, pos.long()),
        lambda: lib.dsa_cache_attn(q, s.cache, pos[:1]),
        lambda: lib.dsa_cache_attn(q, s.cache, pos, gate=q[..., 0, 0]),
        lambda: lib.dsa_cache_attn(q, s.cache, pos, out=q.float()),
        lambda: lib.dsa_cache_sparse_attn(q, s.cache, pos, pos.long()[..., None]),
        lambda: lib.dsa_cache_append(s.cache, pos, k, q),
        lambda: lib.dsa_cache_append(s.cache, pos, k, k, rope="half"),
        lambda: lib.dsa_cache_append(s.cache, pos, k, k, q_out=q),
        lambda: lib.dsa_cache_append(s.cache, pos, k, k, rope="half", inv_freq=inv, q_out=q),
        lambda: lib.dsa_cache_append(s.cache, pos, k, k, rope="half", inv_freq=inv.double()),
        lambda: lib.dsa_cache_read(s.cache, pos, k=q),
        lambda: lib.Cache(s.pages, s.table.long(), 2, 64, 64),
        lambda: lib.Cache(s.pages, s.table, 4, 64, 64),
        lambda: lib.Cache(s.pages.float(), s.table, 2, 64, 64)]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    for call in (lambda: lib.dsa_cache_attn(q, s.cache, pos, n_first=3),
                 lambda: lib.dsa_cache_attn(q, s.cache, pos, window=-1),
                 lambda: lib.dsa_cache_append(s.cache, pos, k, k, rope="half", inv_freq=inv[:8])):
        with pytest.raises(lib.DSAError):
            call()
