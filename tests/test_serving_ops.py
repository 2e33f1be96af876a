"""The operators around an attention step without a GPU: the pool's truncate
and evict against the oracle on random call traces, the oracle itself against
closed forms, and what every entry point refuses before it launches anything."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from oracle import serving
import hybrid_sliding_window_dual_gb300 as H
from hybrid_sliding_window_dual_gb300.session import DualPoolSession
from test_abi import assert_same_state, make_pair

INVALID, UNSUPPORTED = H.HSWA_ERR_INVALID_ARG, H.HSWA_ERR_UNSUPPORTED


def refused(status, call, *args):
    with pytest.raises(H.HswaError) as e:
        call(*args)
    assert e.value.status == status, e.value


# ------------------------------------------------------------ bookkeeping
@pytest.mark.parametrize("seed", range(6))
def test_truncate_and_evict_match_oracle_on_random_trace(seed):
    rng = np.random.default_rng(seed)
    cfg, lp, ora = make_pair(W=24, P=8, full=260, swa=120, S=6, MP=64, seed=seed)
    for step in range(500):
        op = rng.choice(["reserve", "reserve", "release", "free", "truncate", "truncate", "evict", "drop_restore"])
        ids = rng.permutation(np.sort(rng.choice(cfg.max_seqs, size=int(rng.integers(1, 5)), replace=False)))
        if op == "reserve":
            ids, n_new = np.sort(ids), rng.choice([0, 1, 4, 9, 60], size=len(ids))
            try:
                exp = ora.reserve(ids, n_new)
            except (oracle.NoSpace, ValueError):
                with pytest.raises(H.HswaError):
                    H.hswa_reserve(lp, ids, n_new)
            else:
                got = H.hswa_reserve(lp, ids, n_new)
                assert np.array_equal(got[0], exp[0]) and np.array_equal(got[1], exp[1])
        elif op == "release":
            assert H.hswa_swa_release(lp, ids) == ora.swa_release(ids)
        elif op == "free":
            H.hswa_seq_free(lp, ids[:1])
            ora.seq_free(ids[:1])
        elif op == "truncate":
            back = rng.choice([0, 1, 3, 8, 30, 1000], size=len(ids))
            new = np.maximum(ora.seq_len[ids] - back, 0)
            try:
                exp = ora.truncate(ids, new)
            except ValueError:
                refused(INVALID, H.hswa_seq_truncate, lp, ids, new)
            else:
                assert H.hswa_seq_truncate(lp, ids, new) == exp
        elif op == "evict":
            keep = []
            for s in ids:
                pages = -(-int(ora.seq_len[s]) // cfg.page_size)
                old = max(0, int(ora.seq_len[s]) - cfg.window) // cfg.page_size
                old += rng.random() < 0.1  # now and then a page of the window
                keep.append([p for p in range(pages) if p >= old or rng.random() < 0.6])
            lists = np.full((len(ids), cfg.max_pages_per_seq), -1, np.int32)
            for i, k in enumerate(keep):
                lists[i, :len(k)] = k
            n_keep = [len(k) for k in keep]
            try:
                exp = ora.evict(ids, keep)
            except ValueError:
                refused(INVALID, H.hswa_evict, lp, ids, n_keep, lists)
            else:
                assert H.hswa_evict(lp, ids, n_keep, lists) == exp
        else:
            assert H.hswa_swa_drop(lp, ids) == ora.swa_drop(ids)
            try:
                n = ora.swa_restore(ids)
            except oracle.NoSpace:
                with pytest.raises(H.NoSpace):
                    H.hswa_swa_restore(lp, ids)
            else:
                assert H.hswa_swa_restore(lp, ids) == n
        assert_same_state(cfg, lp, ora)
    for kind, ref in ((H.HSWA_KIND_FULL, ora.full_ref), (H.HSWA_KIND_SWA, ora.swa_ref)):
        assert np.array_equal(H.hswa_get_page_refs(lp, kind, len(ref)), ref)
    H.hswa_pool_destroy(lp)


def test_truncate_refusals_change_nothing():
    cfg, lp, ora = make_pair(W=16, P=8, full=40, swa=40, S=3, MP=16, seed=3)
    for pool in (lp,):
        H.hswa_reserve(pool, [0, 1], [60, 20])
        ora.reserve([0, 1], [60, 20])
    refused(INVALID, H.hswa_seq_truncate, lp, [0], [61])
    refused(INVALID, H.hswa_seq_truncate, lp, [0], [-1])
    refused(INVALID, H.hswa_seq_truncate, lp, [0, 0], [5, 5])
    refused(INVALID, H.hswa_seq_truncate, lp, [1, 3], [5, 0])
    H.hswa_swa_release(lp, [0])
    ora.swa_release([0])  # keeps positions 40..59: pages 5, 6, 7
    refused(INVALID, H.hswa_seq_truncate, lp, [1, 0], [5, 55])  # 55 - 16 = 39 lies on released page 4; nothing of 1 goes
    assert_same_state(cfg, lp, ora)
    assert H.hswa_seq_truncate(lp, [0], [56]) == ora.truncate([0], [56])
    assert_same_state(cfg, lp, ora)
    H.hswa_pool_destroy(lp)


def test_truncate_does_not_cut_into_a_cached_prefix():
    cfg, lp, _ = make_pair(W=16, P=8, full=40, swa=40, S=3, MP=16, seed=4)
    tree = H.hswa_tree_create(lp)
    tokens = np.arange(64)
    H.hswa_reserve(lp, [0], [40])
    assert H.hswa_tree_insert(tree, 0, tokens[:40]) == 5
    refused(INVALID, H.hswa_seq_truncate, lp, [0], [37])
    assert H.hswa_seq_truncate(lp, [0], [32]) == 0  # the tree keeps the page
    full, _ = H.hswa_reserve(lp, [0], [1])
    assert full[0] // 8 not in H.hswa_tree_nodes(tree)[:, 3]
    assert H.hswa_seq_truncate(lp, [0], [32]) == 1
    H.hswa_tree_destroy(tree)
    H.hswa_pool_destroy(lp)


def test_evicted_sequences_are_not_cached_past_the_gap():
    cfg, lp, _ = make_pair(W=16, P=8, full=40, swa=40, S=3, MP=16, seed=5)
    tree = H.hswa_tree_create(lp)
    tokens = np.arange(80)
    H.hswa_reserve(lp, [0], [80])
    keep = np.array([[0, 1, 4, 6, 7, 8, 9]], np.int32)
    assert H.hswa_evict(lp, [0], [7], keep) == 3
    refused(INVALID, H.hswa_tree_insert, tree, 0, tokens[:24])
    assert H.hswa_tree_insert(tree, 0, tokens[:23]) == 2
    # taken back to the gap, the text goes on from there
    refused(INVALID, H.hswa_seq_truncate, lp, [0], [15])  # shared with the tree now
    assert H.hswa_seq_truncate(lp, [0], [16]) == 5
    H.hswa_reserve(lp, [0], [16])
    assert H.hswa_tree_insert(tree, 0, tokens[:32]) == 2
    H.hswa_seq_free(lp, [0])
    H.hswa_tree_destroy(tree)
    H.hswa_pool_destroy(lp)


def test_evict_refusals_change_nothing():
    cfg, lp, ora = make_pair(W=16, P=8, full=40, swa=40, S=3, MP=16, seed=6)
    H.hswa_reserve(lp, [0, 1], [60, 20])
    ora.reserve([0, 1], [60, 20])
    ok = list(range(8))
    for n, lists in ((7, ok[:7]), (7, ok[1:6] + [7, 7]), (8, ok[:7] + [8]), (8, [1, 0] + ok[2:]), (7, ok[:5] + [6, 7]),
                     (9, ok + [8]), (-1, ok), (0, ok)):
        k = np.full((2, 10), -1, np.int32)
        k[0, :3], k[1, :len(lists)] = [0, 1, 2], lists
        refused(INVALID, H.hswa_evict, lp, [1, 0], [3, n], k)
    refused(INVALID, H.hswa_evict, lp, [0], [8], np.zeros((1, 7), np.int32))  # longer than its row
    refused(INVALID, H.hswa_evict, lp, [3], [0], np.zeros((1, 7), np.int32))
    refused(INVALID, H.hswa_evict, lp, [0, 0], [8, 8], np.array([ok, ok], np.int32))
    assert_same_state(cfg, lp, ora)
    assert H.hswa_evict(lp, [0], [4], np.array([[0, 5, 6, 7]], np.int32)) == ora.evict([0], [[0, 5, 6, 7]]) == 4
    assert_same_state(cfg, lp, ora)
    assert H.hswa_evict(lp, [2], [0], np.zeros((1, 0), np.int32)) == 0  # nothing there
    H.hswa_pool_destroy(lp)


# ----------------------------------------------------------------- oracle
def test_oracle_rope_closed_forms():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 2, 8))
    same = serving.rope(x, np.zeros((2, 5)), 8, [3, 1])
    assert np.array_equal(same, x)
    # one axis, both pairings: the same numbers, the pairs elsewhere
    pos = np.array([[0, 1, 7, 1000, -3]])
    a = serving.rope(x, pos, 8, [4])
    order = [0, 2, 4, 6, 1, 3, 5, 7]  # adjacent pairs laid out as halves
    b = serving.rope(x[:, :, np.argsort(order)], pos, 8, [4], adjacent=True)
    assert np.allclose(b[:, :, order], a, atol=1e-12)
    # scores depend on the distance alone, on every axis
    for shift in ([5, 5], [11, -2]):
        p = np.array([[3], [9]])
        q1, k1 = serving.rope(x[:1], p, 8, [2, 2]), serving.rope(x[1:2], p * 0, 8, [2, 2])
        s = np.array(shift)[:, None]
        q2, k2 = serving.rope(x[:1], p + s, 8, [2, 2]), serving.rope(x[1:2], p * 0 + s, 8, [2, 2])
        assert np.allclose((q1 * k1).sum(-1), (q2 * k2).sum(-1), atol=1e-12)
    assert serving.pair_axes(8, [4, 2, 2], True) == [0, 1, 2, 0, 1, 2, 0, 0]
    assert serving.pair_axes(8, [4, 2, 2], False) == [0, 0, 0, 0, 1, 1, 2, 2]


def test_oracle_weights_and_selection_closed_forms():
    q = np.zeros((1, 4, 8))
    k = np.random.default_rng(1).standard_normal((3, 2, 4, 8))
    o, w = serving.decode_weights(q, k, k, np.array([[2, 0, 1, -1]]), [10], 1.0)
    assert np.allclose(w, [[1.6, 1.6, 0.8, 0]])  # equal weights: keys a page over 10, 4 heads
    nan = float("nan")
    w = np.array([[9, 1, 5, 5, nan, 0, 7, 8]])
    assert serving.evict_select([61], w, [4], 8, 1, 16) == [[0, 5, 6, 7]]  # pages 5..7 meet the last 16 tokens
    assert serving.evict_select([61], w, [5], 8, 1, 16) == [[0, 2, 5, 6, 7]]  # of equals the lower
    assert serving.evict_select([61], w, [7], 8, 1, 16) == [[0, 1, 2, 3, 5, 6, 7]]
    assert serving.evict_select([61], w, [99], 8, 1, 16) == [list(range(8))]
    assert serving.evict_select([0], w, [3], 8, 1, 16) == [[]]


def test_oracle_verify_keeps_the_targets_distribution():
    """Over drafts from q and uniform numbers on a grid, the first token is
    distributed as p."""
    p, q = np.array([0.5, 0.25, 0.125, 0.125]), np.array([0.125, 0.125, 0.5, 0.25])
    grid = (np.arange(64) + 0.5) / 64
    hist = np.zeros(4)
    for x in range(4):
        for u0 in grid:
            for u1 in grid:
                a, t = serving.verify(np.stack([p, p])[None], q[None, None], np.array([[x]]), None, np.array([[u0, u1]]))
                hist[t[0, 0]] += q[x] / 64 ** 2
    assert np.allclose(hist, p, atol=1e-9)
    # greedy drafts: q is 1 at the draft
    a, t = serving.verify(np.stack([p, p])[None], None, np.array([[1]]), None, np.array([[0.2499, 0.9]]))
    assert a[0] == 1 and t.tolist() == [[1, 3]]
    a, t = serving.verify(np.stack([p, p])[None], None, np.array([[1]]), None, np.array([[0.25, 0.7]]))
    assert a[0] == 0 and t.tolist() == [[2, -1]]  # 0.5, 0.125, 0.125 left; 0.7 * 0.75 = 0.525 lies in the second


# --------------------------------------------------------------- refusals
X = 1 << 20  # an address that is never followed: each call below returns before a launch


def layer(kind=None, **over):
    f = dict(kind=H.HSWA_KIND_FULL if kind is None else kind, window=128, k_pool=X, v_pool=X, k_scale=X, v_scale=X)
    f.update(over)
    return H.Layer(**f)


def pool(dtype=None, d=128, hq=16, hkv=2, P=64, S=4, MP=8):
    return H.hswa_pool_create(H.Config(window=128, page_size=P, n_q_heads=hq, n_kv_heads=hkv, head_dim=d,
                                       dtype=H.HSWA_DTYPE_BF16 if dtype is None else dtype, full_pages=16, swa_pages=16,
                                       max_seqs=S, max_pages_per_seq=MP))


def test_rope_create_refusals():
    make = H.hswa_rope_create
    for args in ((0, [0]), (3, [1]), (258, [129]), (128, [63]), (128, [65, -1]), (128, []), (128, [16] * 5)):
        refused(INVALID, make, *args)
    for theta in (0.0, -1.0, float("inf"), float("nan")):
        refused(INVALID, make, 4, [2], theta)
    refused(INVALID, make, 4, [2], 10000.0, [1.0, float("nan")])
    refused(INVALID, make, 16, [2, 3, 3], 10000.0, None, True)  # axis 2 has turns for 2 pairs only
    H.hswa_rope_destroy(make(16, [3, 3, 2], interleaved=True))
    refused(INVALID, H.hswa_rope_destroy, None)
    cfg = H.RopeConfig(rotary_dim=4, n_axes=1, theta=1e4)
    cfg.section[0] = 2
    out = ctypes.c_void_p()
    for name in ("pairing", "order"):
        for v in (-1, 2):
            setattr(cfg, name, v)
            assert H.lib.hswa_rope_create(ctypes.byref(cfg), ctypes.byref(out)) == INVALID
        setattr(cfg, name, 0)
    assert H.lib.hswa_rope_create(None, ctypes.byref(out)) == INVALID
    assert H.lib.hswa_rope_create(ctypes.byref(cfg), None) == INVALID


def test_rope_append_refusals():
    p, r = pool(), H.hswa_rope_create(128, [64])
    q, k, v, o = X, X << 4, X << 5, X << 6
    ok = dict(pool=p, layer=layer(), rope=r, q=q, q_stride=2048, k=k, k_stride=256, v=v, v_stride=256, d_pos=X, d_slots=X,
              q_out=o, n_tokens=5)

    def bad(status, **over):
        refused(status, H.hswa_rope_append, *{**ok, **over}.values())

    for name in ("pool", "rope", "q", "k", "v", "d_pos", "d_slots", "q_out"):
        bad(INVALID, **{name: None})
    bad(INVALID, n_tokens=-1)
    bad(INVALID, layer=layer(kind=2))
    bad(INVALID, layer=layer(k_pool=None))
    bad(INVALID, q_stride=2047)
    bad(INVALID, k_stride=255)
    bad(INVALID, v_stride=-256)
    bad(INVALID, q=q + 1)
    bad(INVALID, q_out=q, q_stride=2304)  # in place, but not packed
    bad(INVALID, q_out=q + 2)             # partly over q
    bad(INVALID, q_out=k)
    bad(INVALID, q_out=v - 2)
    small = pool(d=64)
    bad(INVALID, pool=small)  # rotary_dim 128 on heads of 64
    big = pool(d=512)
    bad(UNSUPPORTED, pool=big)
    f8, f8_64 = pool(dtype=H.HSWA_DTYPE_FP8_E4M3), pool(dtype=H.HSWA_DTYPE_FP8_E4M3, d=64)
    bad(INVALID, pool=f8, layer=layer(k_scale=None))
    r64 = H.hswa_rope_create(64, [32])
    bad(UNSUPPORTED, pool=f8_64, rope=r64)
    H.hswa_rope_append(*{**ok, "n_tokens": 0, "q": None, "k": None, "v": None}.values())  # nothing to do
    for x in (p, small, big, f8, f8_64):
        H.hswa_pool_destroy(x)
    H.hswa_rope_destroy(r)
    H.hswa_rope_destroy(r64)


def test_decode_weights_and_select_refusals():
    p = pool()
    need = H.hswa_decode_weights_workspace_size(p, 4)
    assert need >= H.hswa_decode_workspace_size(p, 4) + 4 * 16 * 8 * 4
    assert H.hswa_decode_weights_workspace_size(p, -1) == 0
    ok = dict(pool=p, layer=layer(), q=X, o=X, bt=X, lens=X, n=4, scale=1.0, w_in=None, decay=0.0, w_out=X, ws=X, ws_bytes=need)

    def bad(status, **over):
        refused(status, H.hswa_decode_weights, *{**ok, **over}.values())

    for name in ("pool", "q", "o", "bt", "lens", "w_out", "ws"):
        bad(INVALID, **{name: None})
    bad(INVALID, n=-1)
    bad(INVALID, n=5)
    bad(INVALID, layer=layer(kind=H.HSWA_KIND_SWA))
    bad(INVALID, layer=layer(v_pool=None))
    bad(INVALID, ws=X + 128)
    bad(INVALID, ws_bytes=need - 1)
    H.hswa_decode_weights(*{**ok, "n": 0, "ws": None}.values())
    wide = pool(d=264, hq=2)
    bad(UNSUPPORTED, pool=wide, ws_bytes=1 << 30)
    f8 = pool(dtype=H.HSWA_DTYPE_FP8_E4M3, hq=8)  # 4 query heads a kv head
    bad(UNSUPPORTED, pool=f8, ws_bytes=1 << 30)

    ok = dict(pool=p, lens=X, w_in=X, budget=X, n=4, sink=1, recent=128, keep=X, n_keep=X, w_out=X)

    def bad(status, **over):  # noqa: F811
        refused(status, H.hswa_evict_select, *{**ok, **over}.values())

    for name in ("pool", "lens", "w_in", "budget", "keep", "n_keep", "w_out"):
        bad(INVALID, **{name: None})
    bad(INVALID, n=5)
    bad(INVALID, n=-1)
    bad(INVALID, sink=-1)
    bad(INVALID, recent=127)  # less than the window
    for x in (p, wide, f8):
        H.hswa_pool_destroy(x)


def test_verify_refusals():
    ok = dict(dtype=H.HSWA_DTYPE_F32, p=X, p_stride=100, q=X, q_stride=100, draft=X, n_draft=None, u=X, n=2, n_tok=4, vocab=100,
              n_accept=X, tokens=X)

    def bad(status, **over):
        refused(status, H.hswa_verify_draft, *{**ok, **over}.values())

    for name in ("p", "draft", "u", "n_accept", "tokens"):
        bad(INVALID, **{name: None})
    bad(INVALID, n=-1)
    bad(INVALID, n_tok=0)
    bad(INVALID, n_tok=17)
    bad(INVALID, vocab=0)
    bad(INVALID, p_stride=99)
    bad(INVALID, q_stride=99)
    bad(INVALID, p=X + 2)
    bad(INVALID, q=X + 1)
    bad(UNSUPPORTED, dtype=H.HSWA_DTYPE_FP8_E4M3)
    bad(UNSUPPORTED, vocab=(1 << 20) + 1, p_stride=1 << 21, q_stride=1 << 21)
    H.hswa_verify_draft(*{**ok, "n": 0, "p": None}.values())


def test_outputs_across_their_inputs_are_refused():
    p = pool()
    need = H.hswa_decode_weights_workspace_size(p, 4)
    row = 8 * 4  # bytes of a row of weights
    for at in (X - 4 * row + 4, X - 4, X + 4, X + 4 * row - 4):
        refused(INVALID, H.hswa_decode_weights, p, layer(), X, X, X, X, 4, 1.0, X, 0.5, at, X, need)
        refused(INVALID, H.hswa_evict_select, p, X, X, X, 4, 1, 128, X, X, at)
    H.hswa_pool_destroy(p)


def test_session_refuses_shapes_that_do_not_fit():
    cfg = H.Config(window=128, page_size=64, n_q_heads=4, n_kv_heads=2, head_dim=16, dtype=H.HSWA_DTYPE_F32, full_pages=4, swa_pages=4, max_seqs=2,
                   max_pages_per_seq=4)
    s = DualPoolSession(cfg, [H.HSWA_KIND_FULL], device="cpu")
    rope = H.hswa_rope_create(16, [8])
    f = torch.zeros  # shapes only
    i32 = dict(dtype=torch.int32)
    for q, k, v in ((f(3, 64), f(2, 32), f(3, 32)), (f(3, 64), f(3, 32), f(4, 32)), (f(3, 63), f(3, 32), f(3, 32)), (f(3, 4, 16), f(3, 1, 16), f(3, 32)),
                    (f(64), f(32), f(32)), (f(3, 128)[:, ::2], f(3, 32), f(3, 32)), (f(3, 16, 4).transpose(1, 2), f(3, 32), f(3, 32))):
        with pytest.raises(ValueError):
            s.rope_append(0, rope, q, k, v, f(1, 3, **i32), f(3, **i32), f(3, 64))
    out = f(2, **i32), f(2, 3, **i32)
    draft, u = f(2, 2, **i32), f(2, 3)
    p = f(2, 3, 50)
    for p, q in ((p, f(2, 2, 49)), (p, f(2, 3, 50)), (p, f(1, 2, 50)), (p, f(2, 2, 50).bfloat16()), (p.double(), None), (f(3, 2, 50).transpose(0, 1), None),
                 (f(2, 3, 100)[:, :, ::2], None), (f(2, 4, 50)[:, :3], None), (p, f(2, 5, 50)[:, :2])):
        with pytest.raises(ValueError):
            s.verify(p, q, draft, None, u, *out)
    assert s._row_stride(f(5, 3, 50)[:, :1]) == 150 and s._row_stride(f(1, 3, 60)[:, :, :50]) == 60
    assert s._row_stride(f(50)[None, None]) == 50 and s._row_stride(f(3, 2, 1)) == 1
    H.hswa_rope_destroy(rope)
    s.close()


def test_binding_takes_subclasses_of_arrays_and_integers(tmp_path):
    """What stands for an address or an array may be a subclass of one: a
    mapped file for gathered windows, a masked array, an IntEnum, a bool."""
    import enum
    from hybrid_sliding_window_dual_gb300 import _binding as B

    a = np.arange(6, dtype=np.int32)
    mapped = np.memmap(tmp_path / "window", np.uint8, "w+", shape=(4096,))
    masked = np.ma.masked_array(a, a > 3)
    place = enum.IntEnum("place", {"X": X})
    assert B._ptr(mapped) == mapped.ctypes.data and B._ptr(masked) == masked.ctypes.data and B._ptr(a.view(np.matrix)) == a.ctypes.data
    assert B._ptr(place.X) == X and B._ptr(False) == 0 and B._ptr(None) is None and B._ptr(X) == X
    t = torch.arange(3)
    assert B._ptr(t) == t.data_ptr() and B._ptr(torch.nn.Parameter(torch.ones(2))) != 0
    p = pool()
    H.hswa_append_kv(p, layer(), mapped, mapped, place.X, 0)  # no tokens: nothing is followed
    H.hswa_pool_destroy(p)


def test_oracle_verify_infinities():
    """u q < p as it stands: an infinite p keeps any draft that u q is below,
    NaN (0 times infinity among them) refuses; the draw clamps to [0, 1]."""
    inf, nan = float("inf"), float("nan")
    for u, q, p, stays in ((0.5, 0.5, inf, True), (0.5, 0.5, -inf, False), (inf, 0.5, 1.0, False), (-inf, 0.5, 0.0, True), (-inf, 0.5, -inf, False),
                           (inf, 0.5, inf, False), (0.0, inf, 1.0, False), (0.5, inf, 1.0, False), (-0.5, inf, -1.0, True), (inf, 0.0, 1.0, False),
                           (nan, 0.5, inf, False), (0.5, nan, inf, False), (0.5, 0.5, nan, False)):
        row = np.array([0.5, p, 0.25, 0.0])
        a, t = serving.verify(np.stack([row, row])[None], np.array([[[0.0, q, 0.0, 0.0]]]), np.array([[1]]), None, np.array([[u, 0.0]]))
        assert bool(a[0]) == stays, (u, q, p)
        assert t[0, a[0]] == 0  # the first of what is left, 0.5 at token 0
    row = np.array([-inf, 0.5, inf, 0.0])
    assert [serving.verify(row[None, None], None, np.zeros((1, 0), int), None, np.array([[u]]))[1][0, 0] for u in (-inf, 0.0, 0.33, 0.34, inf)] == [1, 1, 1, 2, 2]
