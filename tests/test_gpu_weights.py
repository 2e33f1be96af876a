"""Decode with page weights, and the choice of the pages that stay, on the GPU
against the 64-bit oracle.

Tolerances. A score is a sum of 128 products in fp32, off by at most 128 2^-24
sum |q k| scale: below 1e-4 for N(0, 1) inputs (sum |q k| about 82, scale
1/sqrt(128)); a weight is the exponential of the difference of two of them
and of sums no less exact: 2.5e-4 of its value. fp32 pools of d = 64: the
same with 64 products. On top, 1e-6 for what decay adds. The output is
hswa_decode's: equal bits where the same kernel runs, else the usual 2e-2 for
bf16 and 1e-5 for fp32. The choice of pages is exact."""
import math

import numpy as np
import pytest
import torch

import hswa_workloads as wl
import oracle
from oracle import serving
from oracle.fp8 import e4m3_decode
import hybrid_sliding_window_dual_gb300 as H
from hybrid_sliding_window_dual_gb300.session import DualPoolSession
from scenario import fill_normal_

F32, BF16, FP8 = wl.DTYPE_F32, wl.DTYPE_BF16, H.HSWA_DTYPE_FP8_E4M3


class Case:
    def __init__(self, lens, hq, hkv, d, P, dtype, seed=0, spare=2):
        S = len(lens)
        self.lens, self.P, self.dtype, self.hq, self.hkv, self.d = np.array(lens), P, dtype, hq, hkv, d
        pages = sum(-(-L // P) for L in lens) + 1
        mp = max(-(-L // P) for L in lens) + spare
        cfg = H.Config(window=128, page_size=P, n_q_heads=hq, n_kv_heads=hkv, head_dim=d, dtype=dtype, full_pages=pages,
                       swa_pages=pages, max_seqs=S, max_pages_per_seq=mp)
        self.sess = DualPoolSession(cfg, [wl.KIND_FULL], wl.permutation(pages, seed))
        self.sess.reserve(range(S), lens)
        self.sess.sync()
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        k, v = self.sess.k[0], self.sess.v[0]
        if dtype == FP8:
            for x in (k, v):
                x.copy_((torch.randn(x.shape, generator=g, device="cuda") * 120).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
            for x in (self.sess.ks[0], self.sess.vs[0]):
                x.copy_(0.004 + 0.008 * torch.rand(x.shape, generator=g, device="cuda"))
        else:
            fill_normal_(k, seed + 1)
            fill_normal_(v, seed + 2)
        self.q = wl.normal((S, hq, d), seed + 3, F32 if dtype == F32 else BF16, "cuda")
        self.w_in = torch.rand(S, mp, generator=g, device="cuda") * 3
        self.scale = 1 / math.sqrt(d)
        self.S, self.mp = S, mp

    def values(self, which):
        x = (self.sess.k if which == "k" else self.sess.v)[0]
        if self.dtype != FP8:
            return x.double().cpu().numpy()
        s = (self.sess.ks if which == "k" else self.sess.vs)[0].double().cpu().numpy()  # [pages][Hkv][P][1]
        x = e4m3_decode(x.cpu().numpy())
        return (x if which == "k" else x.transpose(0, 1, 3, 2)) * s

    def exact(self):
        full = self.sess.d_full_bt.cpu().numpy()
        return serving.decode_weights(self.q.double().cpu().numpy(), self.values("k"), self.values("v"), full, self.sess.d_seq_len.cpu().numpy(), self.scale)

    def run(self, w_in, decay, w_out=None):
        o = torch.full_like(self.q, 9)
        w = torch.full((self.S, self.mp), 9.0, device="cuda") if w_out is None else w_out
        self.sess.decode_weights(0, self.q, o, self.S, self.scale, w_in, decay, w)
        return o, w

    def check(self, decay=0.75, expect_kernel=None):
        o, w = self.run(self.w_in, decay)
        name = H.hswa_last_kernel()
        assert self.sess.check() == 0
        assert expect_kernel is None or name == expect_kernel, name
        exact_o, exact_w = self.exact()
        tol = 1e-5 if self.dtype == F32 else 2e-2
        assert np.abs(o.double().cpu().numpy() - exact_o).max() <= tol
        used = np.arange(self.mp)[None] * self.P < self.sess.d_seq_len.cpu().numpy()[:, None]
        carried = np.where(used, decay * self.w_in.double().cpu().numpy(), 0)
        got = w.double().cpu().numpy()
        assert (np.abs(got - (exact_w + carried)) <= 2.5e-4 * exact_w + 1e-6).all()
        assert (got[~used] == 0).all()
        if "weights_any" not in name:
            ref = torch.empty_like(o)
            self.sess.decode(0, self.q, ref, self.S, self.scale)
            assert torch.equal(o, ref)
        again = self.run(self.w_in, decay)
        assert torch.equal(again[0], o) and torch.equal(again[1], w)  # equal inputs, equal bits
        return o, w


LENS = [1, 63, 64, 65, 128, 700, 0, 3001, 64 * 33, 9000]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, FP8])
@pytest.mark.parametrize("hkv", [1, 3, 8])
def test_decode_weights_match_oracle(dtype, hkv):
    c = Case(LENS, 8 * hkv, hkv, 128, 64, dtype, seed=hkv)
    c.check(expect_kernel="decode_mma_%s_d128+weights" % ("bf16" if dtype == BF16 else "fp8"))


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv,d,P,dtype", [(4, 1, 64, 16, F32), (6, 2, 64, 16, BF16), (8, 8, 96, 5, BF16), (3, 1, 256, 64, F32), (12, 2, 128, 64, F32),
                                              (5, 5, 7, 1, F32), (16, 2, 128, 32, BF16)])
def test_decode_weights_any_shape(hq, hkv, d, P, dtype):
    c = Case([1, 15, 16, 17, 0, 300, 777], hq, hkv, d, P, dtype, seed=d)
    c.check(expect_kernel="decode_weights_any_%s" % ("f32" if dtype == F32 else "bf16"))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, FP8, F32])
def test_decode_weights_one_long_sequence(dtype):
    """One sequence split over every CTA; for fp32 a shorter one."""
    c = Case([70001] if dtype != F32 else [4001], *((8, 1, 128, 64) if dtype != F32 else (4, 1, 64, 16)), dtype, seed=4)
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, FP8])
def test_decode_weights_many_short_sequences(dtype):
    c = Case([(i * 37) % 200 for i in range(600)], 16, 2, 128, 64, dtype, seed=5)
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, FP8, F32])
def test_decode_weights_accumulate(dtype):
    """In place, over layers and steps; starting anew whatever was there."""
    c = Case([5, 200, 0, 1000], *((16, 2, 128, 64) if dtype != F32 else (4, 2, 64, 16)), dtype, seed=6)
    _, once = c.run(None, 0.5)
    nan = torch.full_like(once, float("nan"))
    _, anew = c.run(nan, 0.0, nan)
    assert anew is nan and torch.equal(anew, once)
    total = once.clone()
    c.run(total, 1.0, total)
    c.run(total, 1.0, total)
    assert torch.allclose(total, 3 * once, rtol=2.0 ** -22, atol=0)
    rows = once.double().sum(1).cpu().numpy()
    assert np.allclose(rows[c.lens > 0], c.hq, rtol=1e-4) and (rows[c.lens == 0] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, FP8, F32])
def test_decode_weights_one_key_with_everything(dtype):
    """Scores far apart: the page of the largest gets the whole weight, the
    others underflow to 0, never to NaN."""
    c = Case([64 * 9 + 3, 130], *((8, 1, 128, 64) if dtype != F32 else (4, 1, 64, 16)), dtype, seed=7)
    c.scale = 60.0 if dtype != F32 else 200.0
    _, w = c.run(None, 0)
    assert c.sess.check() == 0
    _, exact = c.exact()
    assert torch.isfinite(w).all()
    # an absolute error of a score of size |s| is at most 2^-17 |s| (as above), here |s| up to 60 * 45: 2e-2
    assert np.abs(w.double().cpu().numpy() - exact).max() <= 0.05 * c.hq
    c.scale = 0.0  # all keys alike
    _, w = c.run(None, 0)
    _, exact = c.exact()
    assert np.allclose(w.double().cpu().numpy(), exact, rtol=1e-5)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, FP8, F32])
def test_decode_weights_skip_pages_with_a_bad_entry(dtype):
    c = Case([300, 64, 1000], *((16, 2, 128, 64) if dtype != F32 else (4, 2, 64, 16)), dtype, seed=8)
    good = c.run(None, 0)[1].clone()
    c.sess.d_full_bt[0, 1] = -1
    c.sess.d_full_bt[1, 0] = c.sess.cfg.full_pages  # P = 64: its only page
    o, w = c.run(None, 0)
    assert c.sess.check() == H.HSWA_ERR_BOUNDS
    c.sess.d_full_bt[1, 0] = -1
    exact_o, exact_w = c.exact()
    assert np.abs(w.double().cpu().numpy() - exact_w).max() <= 2.5e-4 * c.hq
    assert np.abs(o.double().cpu().numpy() - exact_o).max() <= (1e-5 if dtype == F32 else 2e-2)
    assert w[0, 1] == 0 and torch.equal(w[2], good[2])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, FP8, F32])
@pytest.mark.parametrize("excess", [1, 200])
def test_decode_weights_of_lengths_past_the_table(dtype, excess):
    # the keys past the last entry of a table row are left out and reported; no
    # other row's weights are touched
    P = 64 if dtype != F32 else 16
    c = Case([3 * P, 10 * P, 5], *((16, 2, 128, P) if dtype != F32 else (4, 2, 64, P)), dtype, seed=11, spare=0)
    good_o, good_w = c.run(c.w_in, 0.5)
    c.sess.d_seq_len[1] += excess
    w = torch.full((c.S + 2, c.mp), 9.0, device="cuda")
    o, _ = c.run(c.w_in, 0.5, w[1:-1])
    assert c.sess.check() == H.HSWA_ERR_BOUNDS
    assert torch.equal(w[1:-1], good_w) and torch.equal(o, good_o)
    assert (w[0] == 9).all() and (w[-1] == 9).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, FP8, F32])
def test_decode_weights_of_the_first_sequences(dtype):
    # fewer sequences than the tables have rows: the others' rows are left alone
    P = 64 if dtype != F32 else 16
    c = Case([300, 70, 1000, 5], *((16, 2, 128, P) if dtype != F32 else (4, 2, 64, P)), dtype, seed=14)
    exact_o, exact_w = c.exact()
    for n in (0, 1, 3):
        o, w = torch.full_like(c.q, 9), torch.full((c.S, c.mp), 9.0, device="cuda")
        c.sess.decode_weights(0, c.q, o, n, c.scale, None, 0, w)
        assert c.sess.check() == 0
        assert (np.abs(w[:n].double().cpu().numpy() - exact_w[:n]) <= 2.5e-4 * exact_w[:n] + 1e-6).all()
        assert n == 0 or np.abs(o[:n].double().cpu().numpy() - exact_o[:n]).max() <= (1e-5 if dtype == F32 else 2e-2)
        assert (w[n:] == 9).all() and (o[n:] == 9).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, FP8])
@pytest.mark.parametrize("hkv", [1, 2, 4, 8])
@pytest.mark.parametrize("lens", [[1566, 14213], [64, 65, 3000, 1, 0], [30000], [20000, 700]], ids=str)
def test_decode_weights_of_few_segments(lens, hkv, dtype):
    Case(lens, 8 * hkv, hkv, 128, 64, dtype, seed=20 + hkv).check()


@pytest.mark.gpu
def test_decode_weights_two_calls_at_once():
    # two streams, a workspace each; then two captured calls that share one, in turn
    a, b = Case([3000, 70, 900], 64, 8, 128, 64, BF16, seed=12), Case([12000], 64, 8, 128, 64, BF16, seed=13)
    want = [c.run(c.w_in, 0.5) for c in (a, b)]
    for c in (a, b):
        c.sess.stream = torch.cuda.Stream()
        c.sess.stream.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        got = [c.run(c.w_in, 0.5) for c in (a, b)]
        torch.cuda.synchronize()
        for (o, w), (o1, w1) in zip(want, got):
            assert torch.equal(o, o1) and torch.equal(w, w1)
    ws = torch.empty(max(H.hswa_decode_weights_workspace_size(c.sess.pool, c.S) for c in (a, b)), dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    for c in (a, b):
        o, w, g = torch.zeros_like(c.q), torch.zeros_like(c.w_in), torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            H.hswa_decode_weights(c.sess.pool, c.sess.layers[0], c.q, o, c.sess.d_full_bt, c.sess.d_seq_len, c.S, c.scale, c.w_in, 0.5, w, ws, ws.numel(),
                                  torch.cuda.current_stream())
        graphs.append(g)
        outs.append((o, w))
    for _ in range(3):
        for g in graphs:
            g.replay()
    assert H.hswa_check() == 0
    for (o, w), (o1, w1) in zip(want, outs):
        assert torch.equal(o, o1) and torch.equal(w, w1)


@pytest.mark.gpu
def test_decode_weights_on_a_stream_and_in_a_graph():
    c = Case([100, 5000, 3], 64, 8, 128, 64, BF16, seed=9)
    o, w = c.check()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c.sess.stream = side
    o2, w2 = c.run(c.w_in, 0.75)
    assert c.sess.check() == 0 and torch.equal(o2, o) and torch.equal(w2, w)
    c.sess.stream = None
    ws = torch.empty(H.hswa_decode_weights_workspace_size(c.sess.pool, 3), dtype=torch.uint8, device="cuda")
    o3, w3 = torch.zeros_like(o), torch.zeros_like(w)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        H.hswa_decode_weights(c.sess.pool, c.sess.layers[0], c.q, o3, c.sess.d_full_bt, c.sess.d_seq_len, 3, c.scale, c.w_in, 0.75, w3, ws, ws.numel(),
                              torch.cuda.current_stream())
    ws.fill_(255)  # nothing of the workspace is read before it is written
    for _ in range(2):
        o3.zero_(), w3.zero_()
        g.replay()
        assert H.hswa_check() == 0 and torch.equal(o3, o) and torch.equal(w3, w)


# ---------------------------------------------------------------- selection
def select(lens, w, budget, P, sink, recent, window=128, in_place=False):
    S, mp = w.shape
    pool = H.hswa_pool_create(H.Config(window=window, page_size=P, n_q_heads=8, n_kv_heads=1, head_dim=128, dtype=BF16, full_pages=1, swa_pages=1,
                                       max_seqs=S, max_pages_per_seq=mp))
    d_w = torch.as_tensor(w, device="cuda")
    keep = torch.full((S, mp), -7, dtype=torch.int32, device="cuda")
    n_keep = torch.full((S,), -7, dtype=torch.int32, device="cuda")
    w_out = d_w.clone() if in_place else torch.full_like(d_w, 9)
    H.hswa_evict_select(pool, torch.as_tensor(np.asarray(lens, np.int32), device="cuda"), w_out if in_place else d_w,
                        torch.as_tensor(np.asarray(budget, np.int32), device="cuda"), S, sink, recent, keep, n_keep, w_out)
    assert H.hswa_check() == 0
    H.hswa_pool_destroy(pool)
    keep, n_keep, got = keep.cpu().numpy(), n_keep.cpu().numpy(), w_out.cpu().numpy()
    for i, stay in enumerate(serving.evict_select(lens, w, budget, P, sink, recent)):
        assert n_keep[i] == len(stay)
        assert keep[i].tolist() == stay + [-1] * (mp - len(stay))
        assert np.array_equal(got[i].view(np.int32), np.concatenate([w[i, stay], np.zeros(mp - len(stay), np.float32)]).view(np.int32))


def weights(rng, S, mp, kind):
    w = np.exp(2.5 * rng.standard_normal((S, mp))).astype(np.float32)
    if kind == "ties":
        w = np.floor(w).clip(0, 3)
    elif kind == "equal":
        w[:] = 1.25
    elif kind == "close":
        w = np.float32(1) + np.arange(S * mp).reshape(S, mp)[:, ::-1] % 5 * np.float32(2 ** -23)
    elif kind == "odd":
        w *= rng.choice([-1, 1], w.shape).astype(np.float32)
        at = rng.random(w.shape)
        for i, x in enumerate((np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-45, -1e-45)):
            w[(at >= i * 0.08) & (at < (i + 1) * 0.08)] = x
    return np.ascontiguousarray(w, np.float32)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["plain", "ties", "equal", "close", "odd"])
@pytest.mark.parametrize("mp", [1, 7, 33, 1024, 1025, 5000])
def test_select_matches_oracle(kind, mp):
    rng = np.random.default_rng(mp)
    P, S = 16, 12
    pages = rng.integers(0, mp + 1, S)
    pages[0] = mp
    lens = np.maximum(pages * P - rng.integers(0, P, S), 0)
    lens[1] = 0
    w = weights(rng, S, mp, kind)
    budget = rng.integers(-2, mp + 3, S)
    budget[2:4] = 0, mp
    select(lens, w, budget, P, 2, 130)
    select(lens, w, budget, P, 0, 128, in_place=True)


@pytest.mark.gpu
@pytest.mark.parametrize("mp", [16384, 16385, 40000])
def test_select_long_rows(mp):
    rng = np.random.default_rng(mp)
    for kind in ("plain", "ties", "odd"):
        select([mp * 16, mp * 16 - 5, 16 * 9000], weights(rng, 3, mp, kind), [mp // 7, mp - 9, 400], 16, 3, 1000, in_place=kind == "ties")


@pytest.mark.gpu
def test_select_window_edges():
    """Which pages may go at every length around a page's end, with windows
    that do and do not end on a page."""
    rng = np.random.default_rng(3)
    for P, window, recent in ((16, 128, 128), (16, 100, 117), (5, 128, 131), (1, 128, 128), (64, 128, 2 ** 31 - 1)):
        lens = np.arange(recent, recent + 40) if recent < 2 ** 30 else np.arange(500, 540)
        mp = int(-(-lens.max() // P))
        select(lens, weights(rng, 40, mp, "plain"), np.zeros(40, int), P, 1, recent, window)
        select(lens, weights(rng, 40, mp, "plain"), np.zeros(40, int), P, mp + 5, recent, window)  # every page a sink


@pytest.mark.gpu
def test_select_many_sequences():
    rng = np.random.default_rng(4)
    lens = rng.integers(0, 64 * 90, 3000)
    select(lens, weights(rng, 3000, 90, "ties"), rng.integers(0, 90, 3000), 64, 1, 128)


@pytest.mark.gpu
@pytest.mark.parametrize("mp", [300, 700, 1500, 5000, 12000, 30000])
def test_select_needs_every_bit(mp):
    # two far outliers and the rest within 1000 units in the last place, or in
    # clusters of that kind at several magnitudes: the range narrows by steps
    rng = np.random.default_rng(mp)
    w = np.empty((6, mp), np.float32)
    for i in range(6):
        base = np.float32(1) if i < 3 else rng.choice(np.float32([1e-30, 1, 1e30, -1, -1e30]), mp)
        w[i] = (np.broadcast_to(base, mp).astype(np.float32).view(np.int32) + rng.integers(0, 1000 if i % 3 else 40, mp).astype(np.int32)).view(np.float32)
    w[:3, 17], w[:3, mp // 2] = np.inf, -np.inf
    lens = [mp * 16, mp * 16 - 7, mp * 11, mp * 16, mp * 16 - 3, mp * 9]
    for budget in (mp // 2, mp // 10, mp - 20):
        select(lens, w, [budget] * 6, 16, 3, 200)
        select(lens, w, [budget] * 6, 16, 0, 128, in_place=True)


@pytest.mark.gpu
@pytest.mark.parametrize("S,mp", [(1, 2049), (76, 4096), (77, 4096), (1, 8193), (19, 16384), (20, 16384), (40, 5000)])
@pytest.mark.parametrize("kind", ["plain", "ties"])
def test_select_split_rows(S, mp, kind):
    # rows over several CTAs, and the same sizes with too many rows for that;
    # lengths from nothing to the whole row, ends inside each CTA's part
    rng = np.random.default_rng(mp + S)
    w = weights(rng, S, mp, kind)
    lens = np.linspace(0, mp * 16, S).astype(np.int64) if S > 1 else np.array([mp * 16])
    budget = rng.integers(0, mp, S)
    select(lens, w, budget, 16, 5, 200)
    select(lens[::-1], w, budget // 4, 16, 0, 128, in_place=True)


# ------------------------------------------------- scores far below zero
@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, FP8, F32])
def test_decode_weights_of_scores_far_below_zero(dtype):
    """A softmax does not change when every score moves by the same amount:
    with K near -c q all of them are about -150, whatever part of a page is
    used. A score is off by at most d 2^-24 sum |q k| scale, here 128 2^-24 200
    = 1.6e-3, a weight by the exponential of the difference of two: 3.2e-3;
    their logarithms, about 216 in powers of two, by 2^-17 each: 4e-3."""
    c = Case([1, 17, 48, 64 * 3 + 3, 0, 16, 33, 64, 1000], *((16, 2, 128, 64) if dtype != F32 else (4, 2, 64, 16)), dtype, seed=31)
    base = wl.normal((1, c.hkv, 1, c.d), 32, F32, "cuda")  # the queries of a kv head are nearly alike
    c.q.copy_((base + 0.1 * wl.normal((c.S, c.hkv, c.hq // c.hkv, c.d), 33, F32, "cuda")).view(c.S, c.hq, c.d))
    far = 150 / (c.scale * (base * base).sum(-1, keepdim=True))
    k = wl.normal(tuple(c.sess.k[0].shape), 34, F32, "cuda") - far * base
    if dtype == FP8:
        c.sess.ks[0].fill_(0.125)
        c.sess.k[0].copy_((k * 8).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
    else:
        c.sess.k[0].copy_(k)
    o, w = c.run(None, 0)
    assert c.sess.check() == 0
    exact_o, exact_w = c.exact()
    got = w.double().cpu().numpy()
    assert (np.abs(got - exact_w) <= 4e-3 * exact_w + 1e-6).all()
    assert np.allclose(got.sum(1)[c.lens > 0], c.hq, rtol=4e-3)  # a row gains every head's weight
    assert np.abs(o.double().cpu().numpy() - exact_o).max() <= (4e-3 * np.abs(c.values("v")).max() if dtype == F32 else 3e-2)


# ------------------------------------------------------ NaN and infinities
def same_with_nan(got, exact, tol_rel, tol_abs):
    got = got.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(exact))
    fine = ~np.isnan(exact)
    assert (np.abs(got - exact)[fine] <= (tol_rel * np.abs(exact) + tol_abs)[fine]).all()


def check_nan(c, places):
    """Break q ("q", sequence, head), one key ("k", sequence, position, kv
    head), or a page's ("page", sequence, page, kv head): outputs and weights are
    the oracle's, NaN where it has NaN, and a sequence that is not broken keeps
    its bits."""
    whole_o, whole_w = c.run(None, 0)
    table = c.sess.d_full_bt.cpu().numpy()
    k, broken = c.sess.k[0], set()
    for (what, s, at, *rest), value in places:
        broken.add(s)
        if what == "q":
            c.q[s, at, 3] = value
        elif what == "page":
            k[table[s, at], rest[0], :, 3] = value
        elif c.dtype == FP8:
            assert math.isnan(value)
            k[table[s, at // c.P], rest[0], at % c.P, 3] = 0x7F
        else:
            k[table[s, at // c.P], rest[0], at % c.P, 3] = value
    o, w = c.run(None, 0)
    assert c.sess.check() == 0
    with np.errstate(invalid="ignore"):
        exact_o, exact_w = c.exact()
    same_with_nan(o, exact_o, 0, 1e-5 if c.dtype == F32 else 2e-2)
    same_with_nan(w, exact_w, 2.5e-4, 1e-6)
    sound = [s for s in range(c.S) if s not in broken]
    assert torch.equal(o[sound], whole_o[sound]) and torch.equal(w[sound], whole_w[sound])
    plain = torch.empty_like(o)
    c.sess.decode(0, c.q, plain, c.S, c.scale)
    return o, w, plain


NAN, INF = float("nan"), float("inf")


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv,d,P,dtype", [(4, 2, 64, 16, F32), (6, 2, 64, 16, BF16), (12, 2, 128, 64, F32), (3, 1, 256, 16, BF16)])
def test_decode_weights_any_shape_keeps_nan(hq, hkv, d, P, dtype):
    """A head with a NaN, or a score of +inf, has NaN for its output as
    hswa_decode has, and for its weight on every page; a score of -inf weighs
    nothing; all of them -inf leave NaN."""
    lens = [300, 1, 700, 0, 40, 500, 333, 20]
    c = Case(lens, hq, hkv, d, P, dtype, seed=41)
    o, _, plain = check_nan(c, [(("q", 0, 1), NAN), (("q", 1, 0), NAN), (("k", 2, 650, 0), NAN), (("k", 4, 0, 0), NAN), (("k", 5, 499, 0), INF)])
    assert torch.equal(torch.isnan(o), torch.isnan(plain)) and torch.isnan(o).any()
    c = Case(lens, hq, hkv, d, P, dtype, seed=42)
    c.q[..., 3] = c.q[..., 3].abs() + 0.5
    check_nan(c, [(("k", 0, 17, 0), -INF), (("page", 2, 0, 0), -INF), (("page", 6, 1, 0), -INF)]
              + [(("page", 7, p, 0), -INF) for p in range(-(-20 // P))])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, FP8])
@pytest.mark.parametrize("lens,hkv", [([300, 1, 9000, 0, 700, 40], 1), ([300, 1, 9000, 0, 700, 40], 8), ([30000, 5], 1), ([(i * 37) % 900 for i in range(300)], 2)],
                         ids=["few", "some", "long", "many"])
def test_decode_weights_keep_nan(lens, hkv, dtype):
    """The weights of a head with a NaN are NaN on every page of the sequence,
    whether one CTA or many went over it."""
    c = Case(lens, 8 * hkv, hkv, 128, 64, dtype, seed=43)
    places = [(("q", 0, 1), NAN)]
    if len(lens) == 2:
        places = [(("k", 0, 29999, 0), NAN)]
    else:
        places += [(("q", 1, 7), NAN), (("k", 2, lens[2] - 1, hkv - 1), NAN), (("k", 4, 0, 0), NAN)]
        if dtype == BF16:
            places.append((("k", 5, 39, 0), INF))
    o, w, plain = check_nan(c, places)
    assert torch.equal(torch.isnan(o), torch.isnan(plain)) and torch.equal(o.nan_to_num(7), plain.nan_to_num(7))
    assert torch.isnan(w).any()


@pytest.mark.gpu
@pytest.mark.parametrize("mp", [10, 600, 1500, 5000, 20000])
@pytest.mark.parametrize("excess", [1, 16, 100000])
def test_select_of_lengths_past_the_table(mp, excess):
    """A length past a table row is reported and ends where the row does."""
    rng = np.random.default_rng(mp)
    P, S = 16, 5
    w = torch.as_tensor(weights(rng, S, mp, "plain"), device="cuda")
    lens = torch.tensor([mp * P, mp * P + excess, 77, mp * P, 0], dtype=torch.int32, device="cuda")
    budget = torch.tensor([mp // 3] * S, dtype=torch.int32, device="cuda")
    pool = H.hswa_pool_create(H.Config(window=128, page_size=P, n_q_heads=8, n_kv_heads=1, head_dim=128, dtype=BF16, full_pages=1, swa_pages=1,
                                       max_seqs=S, max_pages_per_seq=mp))
    keep = torch.full((S + 2, mp), -7, dtype=torch.int32, device="cuda")
    n_keep, out = torch.full((S,), -7, dtype=torch.int32, device="cuda"), torch.full((S + 2, mp), 9.0, device="cuda")
    H.hswa_evict_select(pool, lens, w, budget, S, 2, 130, keep[1:-1], n_keep, out[1:-1])
    assert H.hswa_check() == H.HSWA_ERR_BOUNDS
    H.hswa_pool_destroy(pool)
    exp = serving.evict_select(lens.clamp(max=mp * P).tolist(), w.cpu().numpy(), budget.tolist(), P, 2, 130)
    assert [k[:n].tolist() for k, n in zip(keep[1:-1].cpu().numpy(), n_keep.tolist())] == exp
    assert (keep[[0, -1]] == -7).all() and (out[[0, -1]] == 9).all()


@pytest.mark.gpu
def test_session_weights_first_called_inside_a_capture():
    """The session's workspace is made by its first call; when that is being
    captured, eager calls after the graph is gone still have it."""
    c = Case([100, 5000, 3], 64, 8, 128, 64, BF16, seed=15)
    ref = Case([100, 5000, 3], 64, 8, 128, 64, BF16, seed=15)
    want_o, want_w = ref.run(ref.w_in, 0.75)  # sets the kernels up
    o, w, g = torch.zeros_like(c.q), torch.zeros_like(c.w_in), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        c.sess.stream = torch.cuda.current_stream()
        c.sess.decode_weights(0, c.q, o, c.S, c.scale, c.w_in, 0.75, w)
    c.sess.stream = None
    kept = c.sess.weights_ws
    for _ in range(2):
        o.zero_(), w.zero_()
        g.replay()
        assert H.hswa_check() == 0 and torch.equal(o, want_o) and torch.equal(w, want_w)
    del g
    torch.cuda.empty_cache()
    other = [torch.full((kept.numel(),), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
    assert all(x.data_ptr() != kept.data_ptr() for x in other)
    got_o, got_w = c.run(c.w_in, 0.75)
    assert c.sess.weights_ws is kept and all((x == 255).all() for x in other)
    assert torch.equal(got_o, want_o) and torch.equal(got_w, want_w)
