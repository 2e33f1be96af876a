"""A serving step on FP4 pools as its operators are used together: tokens are
rotated and appended, attended to in one multi-token decode, the output layer's
logits become probabilities under penalties, biases and a grammar, drafts are
verified against them, the tokens that stay are counted for the next step and the
refused ones taken back. Attention is checked against plain lists of the rows
(as hswa_read_kv gives them) that each sequence should still hold."""
import math

import numpy as np
import pytest
import torch

import hswa_workloads as wl
from oracle import serving
from test_gpu_fp4 import tolerance
from test_gpu_logits import bits, check
import hybrid_sliding_window_dual_gb300 as H
from hybrid_sliding_window_dual_gb300.session import DualPoolSession

HQ, HKV, D, P, W = 16, 2, 128, 64, 128
SECTIONS = [32, 16, 16]
VOCAB = 501
SCALE = 1 / math.sqrt(D)


def session(S, seed, kinds=(wl.KIND_FULL, wl.KIND_SWA), pages=80):
    cfg = H.Config(window=W, page_size=P, n_q_heads=HQ, n_kv_heads=HKV, head_dim=D, dtype=H.HSWA_DTYPE_FP4, full_pages=pages, swa_pages=60, max_seqs=S,
                   max_pages_per_seq=20)
    return DualPoolSession(cfg, list(kinds), wl.permutation(pages, seed), wl.permutation(60, seed + 1))


class Loop:
    def __init__(self, S, seed):
        self.rng, self.S = np.random.default_rng(seed), S
        self.sess = session(S, seed)
        self.rope = H.hswa_rope_create(D, SECTIONS, interleaved=True)
        self.held = [[[] for _ in range(S)] for _ in range(2)]
        self.text = [[] for _ in range(S)]  # tokens so far
        self.prompts = np.zeros(S, int)
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)
        self.head = torch.randn(HQ * D, VOCAB, generator=self.g, device="cuda") * 0.05
        self.counts = torch.zeros(S, VOCAB, dtype=torch.int16, device="cuda")
        # greedy, without penalties, and with all of them
        params = np.stack((self.rng.uniform(0.5, 1.5, S), self.rng.uniform(0.8, 1.3, S), self.rng.uniform(-0.5, 0.5, S), self.rng.uniform(-0.5, 0.5, S)), 1)
        params[0, 0], params[1, 1:] = 0, (1, 0, 0)
        self.params = torch.as_tensor(params.astype(np.float32), device="cuda")
        self.bias_token = torch.as_tensor(self.rng.integers(0, VOCAB, (S, 4)).astype(np.int32), device="cuda")
        self.bias = torch.randn(S, 4, generator=self.g, device="cuda")

    def append(self, n_new):
        """n_new tokens of every sequence through both layers: q of each."""
        ids = np.arange(self.S)
        start = np.array([len(h) for h in self.held[0]])
        slots = self.sess.reserve(ids, n_new)
        self.sess.sync()
        T = int(n_new.sum())
        pos = np.concatenate([start[s] + np.arange(n_new[s]) for s in ids])
        pos = np.stack([pos, pos // 3, pos % 7])
        d_pos = torch.as_tensor(pos.astype(np.int32), device="cuda")
        qs = []
        for layer in range(2):
            x = torch.randn(T, (HQ + 2 * HKV) * D, generator=self.g, device="cuda").bfloat16()
            q, k, v = x.split([HQ * D, HKV * D, HKV * D], 1)
            q_out = torch.empty(T, HQ, D, dtype=torch.bfloat16, device="cuda")
            d_slots = torch.as_tensor(slots[layer], device="cuda")
            self.sess.rope_append(layer, self.rope, q, k, v, d_pos, d_slots, q_out)
            kk, vv = (torch.empty(T, HKV, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
            self.sess.read(layer, d_slots, kk, vv)
            kk, vv = kk.double().cpu().numpy(), vv.double().cpu().numpy()
            # A step between codes is at most 2 scales, a scale at most amax / 6 (1 + 2^-4)
            # (rounded down by as much, amax is cut by less): half a step, and
            # the rotation's roundings in fp32.
            for got, want in ((kk, serving.rope(k.double().cpu().numpy().reshape(T, HKV, D), pos, D, SECTIONS, interleaved=True)),
                              (vv, v.double().cpu().numpy().reshape(T, HKV, D))):
                amax = np.abs(want).reshape(T, HKV, D // 16, 16).max(-1).repeat(16, -1)
                assert (np.abs(got - want) <= amax / 6 * (1 + 2.0 ** -4) + 1e-5).all()
            at = 0
            for s in ids:
                self.held[layer][s] += [(kk[at + i], vv[at + i]) for i in range(n_new[s])]
                at += n_new[s]
            qs.append(q_out)
        return qs

    def check_attention(self, layer, q, o, n_tok):
        q, o = q.double().cpu().numpy(), o.double().cpu().numpy()
        for s in range(self.S):
            rows = self.held[layer][s]
            for w in range(n_tok):
                end = len(rows) - n_tok + 1 + w
                first = max(0, end - W) if layer else 0
                k, v = (np.stack([r[i] for r in rows[first:end]]) for i in range(2))
                g = np.arange(HQ) * HKV // HQ
                x = np.einsum("hd,khd->hk", q[s * n_tok + w], k[:, g]) * SCALE
                e = np.exp(x - x.max(1, keepdims=True))
                exp = np.einsum("hk,khd->hd", e / e.sum(1, keepdims=True), v[:, g])
                assert (np.abs(o[s * n_tok + w] - exp) <= tolerance(exp, q[s * n_tok + w], k, v, SCALE, end)).all()

    def tokens(self, ids):
        """The texts of the sequences as padded rows."""
        rows = np.full((len(ids), max(1, max(len(self.text[s]) for s in ids))), -1, np.int32)
        for i, s in enumerate(ids):
            rows[i, :len(self.text[s])] = self.text[s]
        return rows

    def check_counts(self):
        want = serving.count_tokens(self.tokens(range(self.S)), self.prompts, VOCAB, None)
        assert np.array_equal(self.counts.cpu().numpy().view(np.uint16), want)

    def prompt(self, n):
        for s in range(self.S):
            self.text[s] = self.rng.integers(0, VOCAB, n[s]).tolist()
        self.prompts = n.copy()
        rows = torch.as_tensor(self.tokens(range(self.S)), device="cuda")
        self.sess.count_tokens(self.counts, rows, torch.as_tensor(n.astype(np.int32), device="cuda"), clear=True)
        self.check_counts()
        qs = self.append(n)
        start = torch.as_tensor(np.concatenate([[0], np.cumsum(n)]).astype(np.int32), device="cuda")
        zero = torch.zeros(self.S, dtype=torch.int32, device="cuda")
        for layer, q in enumerate(qs):
            o = torch.empty_like(q)
            self.sess.prefill(layer, q, o, zero, start, self.S, int(n.max()), SCALE)
            last = np.cumsum(n) - 1
            self.check_attention(layer, q[last], o[last], 1)
        self.sess.release(range(self.S))

    def step(self, n_tok):
        S = self.S
        self.sess.release(range(S))
        qs = self.append(np.full(S, n_tok))
        for layer, q in enumerate(qs):
            o = torch.empty_like(q)
            if n_tok == 1:
                self.sess.decode(layer, q, o, S, SCALE)
            else:
                self.sess.decode_multi(layer, q, o, S, n_tok, SCALE)
            self.check_attention(layer, q, o, n_tok)
        logits = (o.float().view(S, n_tok, -1) @ self.head) * 8
        draft = torch.randint(0, VOCAB, (S, n_tok - 1), generator=self.g, device="cuda", dtype=torch.int32) if n_tok > 1 else None
        if n_tok > 1:  # some that will stay
            draft = torch.where(torch.rand(S, n_tok - 1, generator=self.g, device="cuda") < 0.6, logits[:, :-1].argmax(-1).int(), draft)
        allowed = self.rng.random((S * n_tok, VOCAB)) < 0.8
        p = torch.empty_like(logits)
        args = (self.params, self.counts, draft, self.bias_token, self.bias)
        self.sess.probs(logits, p, *args, bits(allowed))
        assert self.sess.check() == 0
        check(p, logits, *args, allowed)
        assert not p.view(S * n_tok, VOCAB)[torch.as_tensor(~allowed, device="cuda")].any()
        u = torch.rand(S, n_tok, generator=self.g, device="cuda")
        acc = torch.empty(S, dtype=torch.int32, device="cuda")
        tok = torch.empty(S, n_tok, dtype=torch.int32, device="cuda")
        self.sess.verify(p, None, draft, None, u, acc, tok)
        self.sess.count_tokens(self.counts, tok)
        assert self.sess.check() == 0
        acc, tok = acc.cpu().numpy(), tok.cpu().numpy()
        exp = serving.verify(p.double().cpu().numpy(), None, None if draft is None else draft.cpu().numpy(), None, u.double().cpu().numpy())
        assert np.array_equal(acc, exp[0]) and np.array_equal(tok, exp[1])
        for s in range(S):
            self.text[s] += tok[s, :acc[s] + 1].tolist()
        self.check_counts()
        back = n_tok - 1 - acc
        _, _, lens = self.sess.tables()
        self.sess.truncate(range(S), lens - back)
        for layer in range(2):
            for s in range(S):
                del self.held[layer][s][len(self.held[layer][s]) - back[s]:]
        self.sess.sync()
        return acc

    def readmit(self, s, n):
        """Sequence s ends; another takes its place with a prompt of n tokens."""
        self.sess.seq_free([s])
        for layer in range(2):
            self.held[layer][s] = []
        self.text[s], self.prompts[s] = self.rng.integers(0, VOCAB, n).tolist(), n
        row = torch.as_tensor(self.tokens([s]), device="cuda")
        self.sess.count_tokens(self.counts[s:s + 1], row, torch.tensor([n], dtype=torch.int32, device="cuda"), clear=True)
        self.check_counts()


@pytest.mark.gpu
def test_draft_probs_verify_count_and_take_back():
    loop = Loop(5, seed=71)
    loop.prompt(np.array([3, 64, 200, 450, 700]))
    accepted = 0
    for step in range(9):
        accepted += int(loop.step(1 + step % 6).sum())
        if step == 5:
            loop.readmit(2, 17)
    assert accepted > 0
    H.hswa_rope_destroy(loop.rope)


@pytest.mark.gpu
@pytest.mark.parametrize("n_tok", [2, 6])
def test_step_captured_once_and_replayed(n_tok):
    """One graph holds the device side of a step, from projections to counts; it
    is replayed as the sequences grow, beside an eager run of the same. Two
    more graphs on two streams, with pools and workspaces of their own, change
    nothing."""
    S = 3
    T = S * n_tok
    rope = H.hswa_rope_create(D, SECTIONS)
    g = torch.Generator(device="cuda")
    g.manual_seed(90)
    x = torch.empty(T, (HQ + 2 * HKV) * D, dtype=torch.bfloat16, device="cuda")
    q, k, v = x.split([HQ * D, HKV * D, HKV * D], 1)
    pos, slots = torch.zeros(3, T, dtype=torch.int32, device="cuda"), torch.zeros(T, dtype=torch.int32, device="cuda")
    head = torch.randn(HQ * D, VOCAB, generator=g, device="cuda") * 0.3
    draft, u = torch.zeros(S, n_tok - 1, dtype=torch.int32, device="cuda"), torch.zeros(S, n_tok, device="cuda")
    params = torch.tensor([[0.8, 1.2, 0.3, 0.1], [0, 1.1, 0.2, 0], [1, 1, 0, 0]], device="cuda")

    def step(s, o):
        s.rope_append(0, rope, q, k, v, pos, slots, o["q"])
        s.decode_multi(0, o["q"], o["o"], S, n_tok, SCALE)
        s.probs((o["o"].float().view(S, n_tok, -1) @ head), o["p"], params, o["counts"], draft)
        s.verify(o["p"], None, draft, None, u, o["acc"], o["tok"])
        s.count_tokens(o["counts"], o["tok"])
        s.read(0, slots, o["k"], o["v"])

    sess = [session(S, 5, kinds=[wl.KIND_FULL], pages=40) for _ in range(3)]
    outs = []
    for s in sess:
        s.workspace(S, n_tok)
        outs.append(dict(q=torch.zeros(T, HQ, D, dtype=torch.bfloat16, device="cuda"), o=torch.zeros(T, HQ, D, dtype=torch.bfloat16, device="cuda"),
                         p=torch.zeros(S, n_tok, VOCAB, device="cuda"), counts=torch.zeros(S, VOCAB, dtype=torch.int16, device="cuda"),
                         acc=torch.zeros(S, dtype=torch.int32, device="cuda"), tok=torch.zeros(S, n_tok, dtype=torch.int32, device="cuda"),
                         k=torch.zeros(T, HKV, D, dtype=torch.bfloat16, device="cuda"), v=torch.zeros(T, HKV, D, dtype=torch.bfloat16, device="cuda")))
        s.reserve(range(S), [1, 100, 200])
        s.sync()
        for pool in (s.k[0], s.v[0], s.ks[0], s.vs[0]):
            pool.zero_()
    x.normal_(generator=g)
    slots.fill_(-1)
    step(sess[0], {name: t.clone() for name, t in outs[0].items()})  # the first set-up of every kernel
    graphs = []
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for i, side in enumerate(streams):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            sess[1 + i].stream = torch.cuda.current_stream()
            step(sess[1 + i], outs[1 + i])
        sess[1 + i].stream = None
        graphs.append(graph)
    for o in outs:
        o["counts"].zero_()
    for i in range(3):
        x.normal_(generator=g)
        draft.random_(0, VOCAB, generator=g)
        u.uniform_(generator=g)
        for s in sess:
            s.release(range(S))
            where = s.reserve(range(S), [n_tok] * S)[0]
            s.sync()
        slots.copy_(torch.as_tensor(where, device="cuda"))
        pos.random_(0, 500, generator=g)
        torch.cuda.synchronize()
        step(sess[0], outs[0])
        for graph, side in zip(graphs, streams):
            with torch.cuda.stream(side):
                graph.replay()
        torch.cuda.synchronize()
        assert all(s.check() == 0 for s in sess)
        for o in outs[1:]:
            for name, t in o.items():
                assert torch.equal(t, outs[0][name]), name
        assert outs[0]["counts"].sum() > 0
    H.hswa_rope_destroy(rope)
