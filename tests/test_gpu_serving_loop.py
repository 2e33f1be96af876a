"""The operators of a serving step as they are used together: drafts are
rotated and appended, attended to in one multi-token decode, verified against
the target's probabilities, the refused ones taken back; now and then the
attention weight is added up and the Full cache cut to a budget. Every
attention output is checked against a dense softmax over plain lists of the
rows that each sequence should still hold, so that slots, tables, lengths and
text positions have to agree after any number of steps."""
import math

import numpy as np
import pytest
import torch

import hswa_workloads as wl
from oracle import serving
from oracle.fp8 import e4m3_decode
import hybrid_sliding_window_dual_gb300 as H
from hybrid_sliding_window_dual_gb300.session import DualPoolSession

BF16, FP8 = wl.DTYPE_BF16, H.HSWA_DTYPE_FP8_E4M3
HQ, HKV, D, P, W = 16, 2, 128, 64, 128
SECTIONS = [32, 16, 16]
VOCAB = 501
SCALE = 1 / math.sqrt(D)


def dense(q, rows, first):
    """q [Hq][d] over rows[first:], a list of (k, v) [Hkv][d]."""
    k = np.stack([r[0] for r in rows[first:]])
    v = np.stack([r[1] for r in rows[first:]])
    g = np.arange(HQ) * HKV // HQ
    s = np.einsum("hd,khd->hk", q, k[:, g]) * SCALE
    e = np.exp(s - s.max(1, keepdims=True))
    e /= e.sum(1, keepdims=True)
    return np.einsum("hk,khd->hd", e, v[:, g]), e


class Loop:
    def __init__(self, dtype, S, seed):
        self.rng, self.S, self.dtype = np.random.default_rng(seed), S, dtype
        cfg = H.Config(window=W, page_size=P, n_q_heads=HQ, n_kv_heads=HKV, head_dim=D, dtype=dtype, full_pages=80, swa_pages=60, max_seqs=S,
                       max_pages_per_seq=20)
        self.sess = DualPoolSession(cfg, [wl.KIND_FULL, wl.KIND_SWA], wl.permutation(80, seed), wl.permutation(60, seed + 1))
        self.rope = H.hswa_rope_create(D, SECTIONS, interleaved=True)
        self.held = [[[] for _ in range(S)] for _ in range(2)]  # rows each layer's cache should hold
        self.text = np.zeros(S, np.int64)                       # tokens of the text so far
        self.weights = torch.zeros(S, 20, device="cuda")
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.head = torch.randn(HQ * D, VOCAB, generator=g, device="cuda") * 0.05
        self.g = g

    def read_back(self, layer, slots):
        """Rows of the layer's pool as values, [T][Hkv][d] each."""
        s = torch.as_tensor(slots, device="cuda").long()
        page, row = s // P, s % P
        out = []
        for pool, scale in ((self.sess.k[layer], self.sess.ks[layer]), (self.sess.v[layer], self.sess.vs[layer])):
            if self.dtype == FP8:
                x = (pool[page, :, row] if pool is self.sess.k[layer] else pool[page, :, :, row]).cpu().numpy()
                out.append(e4m3_decode(x) * scale[page, :, row].double().cpu().numpy())
            else:
                out.append(pool[page, :, row].double().cpu().numpy())
        return out

    def project(self, T):
        """A projection's output and where its tokens stand: [T][(Hq + 2 Hkv) d]."""
        x = torch.randn(T, (HQ + 2 * HKV) * D, generator=self.g, device="cuda").bfloat16()
        return x, x.split([HQ * D, HKV * D, HKV * D], 1)

    def append(self, n_new):
        """n_new tokens of every sequence through both layers: q of each."""
        ids = np.flatnonzero(n_new)
        slots = self.sess.reserve(ids, n_new[ids])
        self.sess.sync()
        T = int(n_new.sum())
        pos = np.concatenate([self.text[s] + np.arange(n_new[s]) for s in ids])
        pos = np.stack([pos, pos // 3, pos % 7])  # an image's rows and columns
        d_pos = torch.as_tensor(pos.astype(np.int32), device="cuda")
        qs = []
        for layer in range(2):
            x, (q, k, v) = self.project(T)
            q_out = torch.empty(T, HQ, D, dtype=torch.bfloat16, device="cuda")
            self.sess.rope_append(layer, self.rope, q, k, v, d_pos, torch.as_tensor(slots[layer], device="cuda"), q_out)
            kk, vv = self.read_back(layer, slots[layer])
            turned = [serving.rope(a.double().cpu().numpy().reshape(T, -1, D), pos, D, SECTIONS, interleaved=True) for a in (q, k)]
            assert np.abs(q_out.double().cpu().numpy() - turned[0]).max() <= 2.0 ** -8 * np.abs(turned[0]).max() + 1e-5
            step = 2.0 ** -8 if self.dtype == BF16 else 2.0 ** -4
            assert np.abs(kk - turned[1]).max() <= step * np.abs(turned[1]).max() + 1e-5
            assert np.abs(vv - v.double().cpu().numpy().reshape(T, HKV, D)).max() <= (0 if self.dtype == BF16 else step * 6)
            at = 0
            for s in ids:
                self.held[layer][s] += [(kk[at + i], vv[at + i]) for i in range(n_new[s])]
                at += n_new[s]
            qs.append(q_out)
        self.text += n_new
        return qs

    def check_attention(self, layer, q, o, n_tok):
        q, o = q.double().cpu().numpy(), o.double().cpu().numpy()
        for s in range(self.S):
            rows = self.held[layer][s]
            for w in range(n_tok):
                end = len(rows) - n_tok + 1 + w
                exp, _ = dense(q[s * n_tok + w], rows[:end], max(0, end - W) if layer else 0)
                assert np.abs(o[s * n_tok + w] - exp).max() <= 2e-2

    def lengths(self):
        _, _, lens = self.sess.tables()
        assert lens.tolist() == [len(x) for x in self.held[0]] == [len(x) for x in self.held[1]]
        return lens

    def prompt(self, n):
        ids = np.arange(self.S)
        qs = self.append(n)
        start = torch.as_tensor(np.concatenate([[0], np.cumsum(n)]).astype(np.int32), device="cuda")
        zero = torch.zeros(self.S, dtype=torch.int32, device="cuda")
        for layer, q in enumerate(qs):
            o = torch.empty_like(q)
            self.sess.prefill(layer, q, o, zero, start, self.S, int(n.max()), SCALE)
            last = np.cumsum(n) - 1
            self.check_attention(layer, q[last], o[last], 1)
        self.sess.release(ids)

    def draft_step(self, n_tok):
        self.sess.release(range(self.S))
        n = np.full(self.S, n_tok)
        qs = self.append(n)
        for layer, q in enumerate(qs):
            o = torch.empty_like(q)
            self.sess.decode_multi(layer, q, o, self.S, n_tok, SCALE)
            self.check_attention(layer, q, o, n_tok)
        p = torch.softmax(o.float().view(self.S, n_tok, -1) @ self.head, -1)
        d = torch.softmax(torch.log(p[:, :n_tok - 1]) + 0.7 * torch.randn(self.S, n_tok - 1, VOCAB, generator=self.g, device="cuda"), -1)
        draft = torch.multinomial(d.view(-1, VOCAB), 1, generator=self.g).view(self.S, n_tok - 1).int()
        u = torch.rand(self.S, n_tok, generator=self.g, device="cuda")
        acc = torch.empty(self.S, dtype=torch.int32, device="cuda")
        tok = torch.empty(self.S, n_tok, dtype=torch.int32, device="cuda")
        self.sess.verify(p, d, draft, None, u, acc, tok)
        assert self.sess.check() == 0
        acc, tok = acc.cpu().numpy(), tok.cpu().numpy()
        exp = serving.verify(p.double().cpu().numpy(), d.double().cpu().numpy(), draft.cpu().numpy(), None, u.double().cpu().numpy())
        assert np.array_equal(acc, exp[0]) and np.array_equal(tok, exp[1])
        back = n_tok - 1 - acc
        self.sess.truncate(range(self.S), self.lengths() - back)
        for layer in range(2):
            for s in range(self.S):
                del self.held[layer][s][len(self.held[layer][s]) - back[s]:]
        self.text -= back
        self.sess.sync()
        return acc

    def weigh_step(self):
        self.sess.release(range(self.S))
        qs = self.append(np.ones(self.S, int))
        o = torch.empty_like(qs[0])
        before = self.weights.double().cpu().numpy()
        self.sess.decode_weights(0, qs[0], o, self.S, SCALE, self.weights, 0.5, self.weights)
        self.check_attention(0, qs[0], o, 1)
        got = self.weights.double().cpu().numpy()
        for s in range(self.S):
            rows = self.held[0][s]
            n = -(-len(rows) // P)
            _, e = dense(qs[0][s].double().cpu().numpy(), rows, 0)
            exp = np.pad(e.sum(0), (0, n * P - len(rows))).reshape(n, P).sum(1)
            assert (np.abs(got[s, :n] - exp - 0.5 * before[s, :n]) <= 2.5e-4 * exp + 1e-5).all()
            assert (got[s, n:] == 0).all()
        o = torch.empty_like(qs[1])
        self.sess.decode(1, qs[1], o, self.S, SCALE)
        self.check_attention(1, qs[1], o, 1)

    def evict_step(self, budget):
        lens = self.lengths()
        keep = torch.empty(self.S, 20, dtype=torch.int32, device="cuda")
        n_keep = torch.empty(self.S, dtype=torch.int32, device="cuda")
        w = self.weights.cpu().numpy()
        self.sess.evict_select(self.weights, torch.full((self.S,), budget, dtype=torch.int32, device="cuda"), self.S, 1, W, keep, n_keep, self.weights)
        assert self.sess.check() == 0
        keep, n_keep = keep.cpu().numpy(), n_keep.cpu().numpy()
        exp = serving.evict_select(lens, w, [budget] * self.S, P, 1, W)
        assert [k[:n].tolist() for k, n in zip(keep, n_keep)] == exp
        gone = sum(-(-int(x) // P) for x in lens) - int(n_keep.sum())
        assert self.sess.evict_pages(range(self.S), n_keep, keep) == gone
        for layer in range(2):
            for s in range(self.S):
                rows = self.held[layer][s]
                self.held[layer][s] = [r for p in exp[s] for r in rows[p * P:(p + 1) * P]]
        self.sess.sync()
        self.lengths()
        return gone


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, FP8])
def test_draft_verify_take_back_and_evict(dtype):
    loop = Loop(dtype, 5, seed=40 + dtype)
    loop.prompt(np.array([3, 64, 200, 450, 700]))
    accepted, gone = 0, 0
    for step in range(8):
        accepted += int(loop.draft_step(2 + step % 5).sum())
        loop.weigh_step()
        if step % 3 == 2:
            gone += loop.evict_step(5 - step // 3)
    assert accepted > 0 and gone > 0
    assert loop.text[4] > loop.lengths()[4]  # the text went on, the cache did not
    H.hswa_rope_destroy(loop.rope)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, FP8])
def test_step_captured_once_and_replayed(dtype):
    """One graph holds the device side of a step; it is replayed as the
    sequences grow, on new projections, beside an eager run of the same."""
    S, n_tok, steps = 3, 4, 3
    sess = []
    for _ in range(2):
        cfg = H.Config(window=W, page_size=P, n_q_heads=HQ, n_kv_heads=HKV, head_dim=D, dtype=dtype, full_pages=40, swa_pages=40, max_seqs=S,
                       max_pages_per_seq=10)
        sess.append(DualPoolSession(cfg, [wl.KIND_FULL], wl.permutation(40, 1), wl.permutation(40, 2)))
    rope = H.hswa_rope_create(D, SECTIONS)
    T = S * n_tok
    g = torch.Generator(device="cuda")
    g.manual_seed(50)
    x = torch.empty(T, (HQ + 2 * HKV) * D, dtype=torch.bfloat16, device="cuda")
    q, k, v = x.split([HQ * D, HKV * D, HKV * D], 1)
    pos, slots = torch.zeros(3, T, dtype=torch.int32, device="cuda"), torch.zeros(T, dtype=torch.int32, device="cuda")
    head = torch.randn(HQ * D, VOCAB, generator=g, device="cuda") * 0.05
    draft, u = torch.zeros(S, n_tok - 1, dtype=torch.int32, device="cuda"), torch.zeros(S, n_tok, device="cuda")
    outs = []
    for s in sess:
        s.workspace(S, n_tok)
        s.weights_ws = torch.empty(H.hswa_decode_weights_workspace_size(s.pool, S), dtype=torch.uint8, device="cuda")
        outs.append(dict(q=torch.zeros(T, HQ, D, dtype=torch.bfloat16, device="cuda"), o=torch.zeros(T, HQ, D, dtype=torch.bfloat16, device="cuda"),
                         o1=torch.zeros(S, HQ, D, dtype=torch.bfloat16, device="cuda"), w=torch.zeros(S, 10, device="cuda"),
                         keep=torch.zeros(S, 10, dtype=torch.int32, device="cuda"), n_keep=torch.zeros(S, dtype=torch.int32, device="cuda"), w2=torch.zeros(S, 10, device="cuda"),
                         acc=torch.zeros(S, dtype=torch.int32, device="cuda"), tok=torch.zeros(S, n_tok, dtype=torch.int32, device="cuda")))
    budget = torch.full((S,), 2, dtype=torch.int32, device="cuda")

    def step(s, o):
        s.rope_append(0, rope, q, k, v, pos, slots, o["q"])
        s.decode_multi(0, o["q"], o["o"], S, n_tok, SCALE)
        p = torch.softmax(o["o"].float().view(S, n_tok, -1) @ head, -1)
        s.verify(p, None, draft, None, u, o["acc"], o["tok"])
        s.decode_weights(0, o["q"].view(S, n_tok, HQ, D)[:, -1].contiguous(), o["o1"], S, SCALE, o["w"], 0.9, o["w"])
        s.evict_select(o["w"], budget, S, 1, W, o["keep"], o["n_keep"], o["w2"])

    for s in sess:  # the lengths before capture, and the first set-up of every kernel
        s.reserve(range(S), [1, 100, 200])
        s.sync()
    x.normal_(generator=g)
    slots.fill_(-1)
    step(sess[0], {k_: t.clone() for k_, t in outs[0].items()})
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        sess[1].stream = torch.cuda.current_stream()
        step(sess[1], outs[1])
    sess[1].stream = None
    outs[0]["w"].zero_(), outs[1]["w"].zero_()
    for i in range(steps):
        x.normal_(generator=g)
        draft.random_(0, VOCAB, generator=g)
        u.uniform_(generator=g)
        u[:, :n_tok - 1] *= 0.004
        pos.random_(0, 100000, generator=g)
        for s in sess:
            full, _ = s.reserve(range(S), [n_tok] * S)
            s.sync()
        slots.copy_(torch.as_tensor(full))
        step(sess[0], outs[0])
        graph.replay()
        torch.cuda.synchronize()
        assert sess[0].check() == 0
        for name in outs[0]:
            assert torch.equal(outs[0][name], outs[1][name]), (i, name)
        assert torch.equal(sess[0].k[0], sess[1].k[0]) and torch.equal(sess[0].v[0], sess[1].v[0])
    H.hswa_rope_destroy(rope)
