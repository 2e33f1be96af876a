"""FP4 KV cache on the GPU against the oracle.

Codes and scales that the library writes equal the oracle's quantizer bit for
bit, and hswa_read_kv gives back exactly their values. Attention over FP4
pools is compared with 64-bit attention over the exactly dequantized pools,
within what its roundings can add up to (see tolerance)."""
import math

import numpy as np
import pytest
import torch

import hswa_workloads as wl
import oracle
from oracle import fp4, serving
import hybrid_sliding_window_dual_gb300 as H
from hybrid_sliding_window_dual_gb300.session import DualPoolSession

FULL, SWA = wl.KIND_FULL, wl.KIND_SWA


class Case:
    """Sequences with cached tokens, the pools filled with what the quantizer
    makes of seeded normal values (of many magnitudes with `wild`)."""

    def __init__(self, cached, seed, kinds=(FULL, SWA), extra=8, hq=64, hkv=8, d=128, P=64, W=128, wild=False):
        B = len(cached)
        self.hq, self.hkv, self.d, self.P, self.W = hq, hkv, d, P, W
        full = sum(math.ceil((L + extra) / P) for L in cached) + 4
        swa = B * (math.ceil((W + extra) / P) + 3) + 4096 // P + 16
        mp = max(math.ceil((L + extra) / P) for L in cached) + 1
        self.cfg = H.Config(window=W, page_size=P, n_q_heads=hq, n_kv_heads=hkv, head_dim=d, dtype=H.HSWA_DTYPE_FP4, full_pages=full, swa_pages=swa, max_seqs=B,
                            max_pages_per_seq=mp)
        self.sess = DualPoolSession(self.cfg, kinds, wl.permutation(full, seed), wl.permutation(swa, seed + 1))
        self.kinds, self.B, self.scale = list(kinds), B, 1 / math.sqrt(d)
        for s, L in enumerate(cached):
            for start in range(0, L, 4096):
                self.sess.reserve([s], [min(4096, L - start)])
                self.sess.release([s])
        self.sess.sync()
        rng = np.random.default_rng(seed)
        for i in range(len(kinds)):
            for codes, scales in ((self.sess.k[i], self.sess.ks[i]), (self.sess.v[i], self.sess.vs[i])):
                x = rng.standard_normal((1 << 10, d)).astype(np.float32)
                if wild:
                    x *= np.exp(rng.uniform(-3, 1, (1 << 10, d // 16, 1)).astype(np.float32)).repeat(16, 2).reshape(1 << 10, d)
                c, s = (torch.as_tensor(y, device="cuda") for y in fp4.quantize_blocks(x))
                rows = torch.as_tensor(rng.integers(0, 1 << 10, codes[..., 0].numel()), device="cuda")
                codes.copy_(c[rows].view(codes.shape))
                scales.copy_(s[rows].view(scales.shape))

    def values(self, layer):
        """K and V of the layer's pages in fp32, which holds them exactly."""
        return [fp4.dequantize_blocks(c.cpu().numpy(), s.cpu().numpy()).astype(np.float32)
                for c, s in ((self.sess.k[layer], self.sess.ks[layer]), (self.sess.v[layer], self.sess.vs[layer]))]

    def table(self, layer):
        full, swa, _ = self.sess.tables()
        return full if self.kinds[layer] == FULL else swa

    def window(self, layer):
        return 0 if self.kinds[layer] == FULL else self.W


def tolerance(exp, q, k, v, scale, n):
    """What the roundings of an attention over n keys can add up to.

    Scores: sums of d products in fp32, whose additions round (or cut) by at most
    2^-23 of the partial sums of magnitudes A: d 2^-23 A; q as fp16 and the
    products with scale and log2 e a few 2^-23 more; A is at most |q| |k| scale. A relative error e of every
    weight moves the result by at most 2 e vmax. Weights are rounded to fp16
    (2^-11, and 2^-25 of the reference where they are below its normal range)
    after an exponential good to 2^-21; sums over keys go 16 at a time, 2^-23 each. The output is
    rounded to bf16."""
    d = q.shape[-1]
    a = float(np.linalg.norm(q, axis=-1).max() * np.linalg.norm(k, axis=-1).max()) * scale
    e = (d + 8) * 2.0 ** -23 * a + d * 2.0 ** -25 * float(np.abs(k).max()) * scale + 2.0 ** -21
    vmax = float(np.abs(v).max())
    return 2.0 ** -8 * np.abs(exp) + vmax * (2 * e + 2.0 ** -11 + (n / 16 + 32) * 2.0 ** -23 + n * 2.0 ** -25)


def compare(c, layer, q, o, seq, pos):
    """Rows of o against attention of the rows of q at positions pos."""
    q, got = q.float().cpu().numpy(), o.float().cpu().numpy()
    assert np.isfinite(got).all()
    before = pos < 0
    assert np.all(got[before] == 0)
    k, v = c.values(layer)
    exp = oracle.attention(q[~before], k, v, c.table(layer), seq[~before], pos[~before], c.window(layer), c.scale)
    off = np.abs(got[~before] - exp) / tolerance(exp, q, k, v, c.scale, int(pos.max()) + 1)
    assert off.max() <= 1, (layer, off.max(), np.unravel_index(off.argmax(), off.shape))


def step(c, n_tok, seed, fused=False, gain=1.0):
    """n_tok new tokens of every sequence: append, decode, compare."""
    slots = c.sess.reserve(range(c.B), [n_tok] * c.B)
    c.sess.sync()
    _, _, lens = c.sess.tables()
    names = set()
    for layer, kind in enumerate(c.kinds):
        kn = wl.normal((c.B * n_tok, c.hkv, c.d), seed + 10 * layer + 1, wl.DTYPE_BF16) * gain
        vn = wl.normal((c.B * n_tok, c.hkv, c.d), seed + 10 * layer + 2, wl.DTYPE_BF16)
        q = wl.normal((c.B * n_tok, c.hq, c.d), seed + 10 * layer, wl.DTYPE_BF16).cuda()
        o = torch.full_like(q, float("nan"))
        ds = torch.as_tensor(slots[0 if kind == FULL else 1], device="cuda")
        before = [x.cpu().numpy().copy() for x in (c.sess.k[layer], c.sess.ks[layer], c.sess.v[layer], c.sess.vs[layer])]
        if fused:
            c.sess.decode_append(layer, q, kn.cuda(), vn.cuda(), ds, o, c.B, c.scale)
        else:
            c.sess.append(layer, kn.cuda(), vn.cuda(), ds)
            if n_tok == 1:
                c.sess.decode(layer, q, o, c.B, c.scale)
            else:
                c.sess.decode_multi(layer, q, o, c.B, n_tok, c.scale)
        assert c.sess.check() == 0
        names.add(H.hswa_last_kernel())
        fp4.append_kv_fp4(*before, kn.float().numpy(), vn.float().numpy(), slots[0 if kind == FULL else 1])
        for want, got in zip(before, (c.sess.k[layer], c.sess.ks[layer], c.sess.v[layer], c.sess.vs[layer])):
            assert np.array_equal(got.cpu().numpy(), want)
        pos = (lens[:, None] - n_tok + np.arange(n_tok)[None]).reshape(-1)
        compare(c, layer, q, o, np.repeat(np.arange(c.B), n_tok), pos)
    return names


EDGES = [0, 1, 62, 63, 64, 65, 126, 127, 128, 129, 191, 700, 3000]


@pytest.mark.gpu
@pytest.mark.parametrize("d,P,hkv", [(16, 16, 1), (48, 16, 3), (64, 16, 2), (80, 64, 1), (96, 64, 4), (128, 64, 8), (256, 16, 2)])
def test_append_and_read_bits(d, P, hkv):
    """Rows of every magnitude, zeros, ties, infinities: the quantizer's bits,
    read back as their values; skipped slots stay as they were."""
    rng = np.random.default_rng(d + P)
    T, pages = 517, 40
    x = rng.standard_normal((2, T, hkv, d)).astype(np.float32) * np.exp(rng.uniform(-14, 12, (2, T, hkv, 1))).astype(np.float32)
    x[0, 0] = 0
    x[0, 1] = np.inf
    x[0, 2, :, ::3] = -np.inf
    x[1, 3] = -0.0
    x[1, 4] = 1e-38
    grid = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 6, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5, -6], np.float32)
    for t in range(5, 40):  # every border between codes, under scales of many magnitudes
        x[1, t] = np.tile(grid, d // 16) * np.float32(2.0 ** (t - 25)) * np.float32(1 + (t % 8) / 8)
    for t in range(40, 80):  # blocks whose largest is 6 times a border between scales
        x[1, t] = np.float32(6 * (1 + (2 * (t % 8) + 1) / 16) * 2.0 ** (t - 60)) * rng.choice([-1, 0.5, 0.25, 1], (hkv, d)).astype(np.float32)
    b = torch.as_tensor(x).bfloat16()
    slots = rng.permutation(pages * P)[:T].astype(np.int32)
    slots[rng.integers(80, T, 20)] = -1
    cfg = H.Config(window=128, page_size=P, n_q_heads=hkv, n_kv_heads=hkv, head_dim=d, dtype=H.HSWA_DTYPE_FP4, full_pages=pages, swa_pages=pages, max_seqs=1, max_pages_per_seq=pages)
    for kind in (FULL, SWA):
        s = DualPoolSession(cfg, [kind])
        pools = [s.k[0], s.ks[0], s.v[0], s.vs[0]]
        for p in pools:
            p.random_(0, 0x60)
        want = [p.cpu().numpy().copy() for p in pools]
        ds = torch.as_tensor(slots, device="cuda")
        s.append(0, b[0].cuda(), b[1].cuda(), ds)
        assert s.check() == 0 and H.hswa_last_kernel() == "append_kv_fp4"
        fp4.append_kv_fp4(*want, b[0].float().numpy(), b[1].float().numpy(), slots)
        for w, p in zip(want, pools):
            assert np.array_equal(p.cpu().numpy(), w)
        k, v = (torch.full((T, hkv, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        s.read(0, ds, k, v)
        assert s.check() == 0
        at = np.maximum(slots, 0)
        for codes, scales, got in ((want[0], want[1], k), (want[2], want[3], v)):
            exp = fp4.dequantize_blocks(codes[at // P, :, at % P], scales[at // P, :, at % P]) * (slots >= 0)[:, None, None]
            assert np.array_equal(got.double().cpu().numpy(), exp)
        s.close()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [H.HSWA_DTYPE_F32, H.HSWA_DTYPE_BF16, H.HSWA_DTYPE_FP8_E4M3])
def test_read_of_other_pools(dtype):
    """Rows read back from the other pool types; slots twice, negative, and past the pool."""
    hkv, d, P, pages, T = 2, 128, 64, 6, 90
    cfg = H.Config(window=128, page_size=P, n_q_heads=hkv, n_kv_heads=hkv, head_dim=d, dtype=dtype, full_pages=pages, swa_pages=pages, max_seqs=1, max_pages_per_seq=pages)
    s = DualPoolSession(cfg, [FULL])
    t = torch.float32 if dtype == H.HSWA_DTYPE_F32 else torch.bfloat16
    x = wl.normal((2, T, hkv, d), 5, wl.DTYPE_BF16).to(t).cuda()
    slots = torch.randperm(pages * P)[:T].int().cuda()
    s.append(0, x[0], x[1], slots)
    again = torch.cat((slots, slots[:7], torch.tensor([-1, -5], dtype=torch.int32, device="cuda")))
    k, v = (torch.full((T + 9, hkv, d), float("nan"), dtype=t, device="cuda") for _ in range(2))
    s.read(0, again, k, v)
    assert s.check() == 0
    for which, got in enumerate((k, v)):
        if dtype == H.HSWA_DTYPE_FP8_E4M3:
            pool, scales = (s.k[0], s.ks[0]) if which == 0 else (s.v[0].transpose(2, 3), s.vs[0])
            page, row = slots.long() // P, slots.long() % P
            exp = (pool[page, :, row].contiguous().view(torch.float8_e4m3fn).float() * scales[page, :, row]).bfloat16()
        else:
            exp = x[which]
        assert torch.equal(got[:T], exp) and torch.equal(got[T:T + 7], exp[:7]) and not got[T + 7:].any()
    again[3] = pages * P
    s.read(0, again, k, v)
    assert s.check() == H.HSWA_ERR_BOUNDS and not k[3].any()
    s.close()


@pytest.mark.gpu
@pytest.mark.parametrize("fused", [False, True])
def test_decode_at_the_edges(fused):
    names = step(Case(EDGES, seed=101), 1, seed=2000, fused=fused)
    assert names == {"append_kv_fp4+decode_mma_fp4_d128" if fused else "decode_mma_fp4_d128"}


@pytest.mark.gpu
@pytest.mark.parametrize("n_tok", [2, 3, 4, 5, 7, 8, 9, 16])
def test_multi_token_decode_at_the_edges(n_tok):
    names = step(Case(EDGES, seed=102, extra=24), n_tok, seed=2100 + n_tok)
    assert names == {"decode_mma_fp4_d128" if n_tok < 5 else "decode_tc_fp4_d128"}


@pytest.mark.gpu
@pytest.mark.parametrize("n_tok", [1, 2, 4, 6])
@pytest.mark.parametrize("hkv", [1, 3])
def test_decode_head_counts_and_magnitudes(n_tok, hkv):
    """Other numbers of kv heads; blocks whose scales differ by up to e^4; keys
    that grow with the step, so that every piece rescales; over steps with releases."""
    c = Case([40, 300, 1500, 0, 5000], seed=103 + hkv, extra=3 * n_tok + 8, hq=8 * hkv, hkv=hkv, wild=True)
    for i in range(3):
        c.sess.release(range(c.B))
        c.sess.sync()
        step(c, n_tok, seed=2200 + 40 * i + n_tok, gain=1.0 + 3 * i)


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv,d,P,W", [(4, 1, 64, 16, 128), (6, 2, 96, 16, 40), (32, 8, 128, 64, 128), (8, 8, 16, 64, 16), (5, 1, 256, 32, 100), (16, 2, 128, 16, 128)])
def test_other_shapes(hq, hkv, d, P, W):
    """The shapes off the tensor cores: decode, several tokens, and a prefill chunk."""
    c = Case([0, 1, 15, 16, 63, 200], seed=104, extra=40, hq=hq, hkv=hkv, d=d, P=P, W=W)
    assert step(c, 1, seed=2300) == {"decode_fp4_any"}
    assert step(c, 3, seed=2310) == {"decode_fp4_any"}
    prefill(c, [1, 5, 17, 3, 9, 20], seed=2320)


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv,d,P", [(4, 1, 64, 16), (10, 2, 80, 16), (3, 1, 256, 64)])
@pytest.mark.parametrize("cached", [[9000, 4100, 3], [5 + 37 * i for i in range(45)]])
def test_other_shapes_long_and_many(cached, hq, hkv, d, P):
    """Several tiles of keys a warp; one CTA a row and eight."""
    c = Case(cached, seed=140, extra=30, hq=hq, hkv=hkv, d=d, P=P, W=1000, wild=True)
    step(c, 1, seed=3400)
    c.sess.release(range(c.B))
    step(c, 4, seed=3410)


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv,d,P", [(4, 1, 64, 16), (6, 2, 96, 16)])
def test_other_shapes_nan_stays_in_its_head(hq, hkv, d, P):
    """A NaN in a head's query makes that head's output NaN and no other's."""
    c = Case([0, 5, 40, 700], seed=130, extra=10, hq=hq, hkv=hkv, d=d, P=P)
    c.sess.reserve(range(c.B), [1] * c.B)
    c.sess.sync()
    q = wl.normal((c.B, hq, d), 3300, wl.DTYPE_BF16).cuda()
    out = []
    for bad in (False, True):
        if bad:
            q[1, 0, 3] = q[3, hq - 1, d - 1] = float("nan")
        for layer in range(2):
            o = torch.zeros_like(q)
            c.sess.decode(layer, q, o, c.B, c.scale)
            out.append(o)
    assert c.sess.check() == 0
    for clean, got in zip(out[:2], out[2:]):
        nan = torch.zeros_like(got, dtype=torch.bool)
        nan[1, 0] = nan[3, hq - 1] = True
        assert torch.equal(got.isnan(), nan)
        assert torch.equal(got[~nan], clean[~nan])


def prefill(c, chunk, seed):
    _, _, cached = c.sess.tables()
    slots = c.sess.reserve(range(c.B), chunk)
    c.sess.sync()
    q_start = np.concatenate([[0], np.cumsum(chunk)]).astype(np.int32)
    names = []
    for layer, kind in enumerate(c.kinds):
        T = int(q_start[-1])
        q = wl.normal((T, c.hq, c.d), seed + 10 * layer, wl.DTYPE_BF16).cuda()
        kn, vn = (wl.normal((T, c.hkv, c.d), seed + 10 * layer + i, wl.DTYPE_BF16).cuda() for i in (1, 2))
        c.sess.append(layer, kn, vn, torch.as_tensor(slots[0 if kind == FULL else 1], device="cuda"))
        o = torch.full_like(q, float("nan"))
        c.sess.prefill(layer, q, o, torch.as_tensor(cached, device="cuda"), torch.as_tensor(q_start, device="cuda"), c.B, max(chunk), c.scale, prefix_host=cached,
                       q_start_host=q_start)
        assert c.sess.check() == 0
        names.append(H.hswa_last_kernel())
        pos = np.concatenate([np.arange(L, L + n) for L, n in zip(cached, chunk)])
        compare(c, layer, q, o, np.repeat(np.arange(c.B), chunk), pos)
    return names


@pytest.mark.gpu
def test_prefill_chunk():
    """A ragged chunk: pages staged as exact fp16 copies."""
    chunk = [1, 60, 64, 65, 128, 200, 7, 129, 300]
    c = Case([0, 5, 63, 64, 127, 128, 129, 700, 3000], seed=105, extra=max(chunk) + 8)
    assert prefill(c, chunk, seed=2400) == ["prefill_stage_fp4+prefill_tc_bf16_d128<f16>", "prefill_stage_fp4+prefill_swa_tc_d128<f16>"]


@pytest.mark.gpu
@pytest.mark.parametrize("n_tok", [1, 2, 3, 6])
def test_bad_table_entries(n_tok):
    """Entries outside the pool: HSWA_ERR_BOUNDS, the pages skipped, zeros where no key is left."""
    c = Case([300, 300, 60], seed=106, extra=16)
    c.sess.reserve(range(c.B), [n_tok] * c.B)
    c.sess.sync()
    c.sess.d_full_bt[0, 0] = -1
    c.sess.d_full_bt[1, 3] = 1 << 30
    c.sess.d_full_bt[2, :2] = -1
    q = wl.normal((c.B * n_tok, c.hq, c.d), 2500, wl.DTYPE_BF16).cuda()
    o = torch.full_like(q, float("nan"))
    c.sess.decode_multi(0, q, o, c.B, n_tok, c.scale)
    assert c.sess.check() == H.HSWA_ERR_BOUNDS and c.sess.check() == 0
    assert torch.isfinite(o).all() and not o[2 * n_tok:].any()


@pytest.mark.gpu
def test_decode_batch_long_and_many():
    """More units than workers, and long sequences cut among many of them."""
    step(Case([40000, 17, 9001], seed=107, kinds=(FULL,)), 1, seed=2600)
    step(Case([100 + 61 * i for i in range(40)], seed=108, kinds=(FULL,)), 1, seed=2610)
    step(Case([20000, 17, 9001], seed=109, kinds=(FULL,), extra=16), 2, seed=2620)


@pytest.mark.gpu
@pytest.mark.parametrize("n_tok", [1, 2, 4])
@pytest.mark.parametrize("B", [1, 31, 32, 33])
def test_decode_where_the_plan_changes_hands(B, n_tok):
    """Up to 32 sequences of one or two tokens have no launch for the plan; some are empty."""
    rng = np.random.default_rng(B)
    cached = [0 if i % 5 == 3 else int(x) for i, x in enumerate(rng.integers(0, 900, B))]
    c = Case(cached, seed=120 + B, extra=16)
    for i in range(2):
        step(c, n_tok, 3100 + 100 * i)
        c.sess.release(range(B))


@pytest.mark.gpu
def test_equal_inputs_equal_bits_captured_and_on_a_stream():
    """The same call again, from a graph, and on a side stream."""
    c = Case([700, 3000, 0, 65], seed=110, extra=16)
    c.sess.reserve(range(c.B), [2] * c.B)
    c.sess.sync()
    q = wl.normal((c.B * 2, c.hq, c.d), 2700, wl.DTYPE_BF16).cuda()
    outs = []

    def call():
        o = torch.full_like(q, float("nan"))
        c.sess.decode_multi(0, q, o, c.B, 2, c.scale)
        return o
    outs.append(call())
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    c.sess.stream = side
    with torch.cuda.stream(side):
        outs.append(call())
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            o = call()
    c.sess.stream = side
    for _ in range(3):
        o.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        outs.append(o.clone())
    for o in outs[1:]:
        assert torch.equal(o, outs[0])
    assert c.sess.check() == 0


def turned_and_quantized(x, pos, rot, sections, adjacent):
    return fp4.quantize_blocks(serving.rope(x.double().cpu().numpy(), pos, rot, sections, adjacent=adjacent).astype(np.float32))


@pytest.mark.gpu
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("hq,hkv,d,rot,P,T", [(64, 8, 128, 128, 64, 3), (64, 8, 128, 64, 64, 700), (16, 2, 128, 32, 16, 2000), (8, 1, 64, 64, 16, 100), (4, 2, 96, 96, 64, 50),
                                              (4, 2, 96, 48, 64, 50), (2, 1, 80, 20, 16, 33), (2, 2, 256, 128, 64, 40), (8, 1, 128, 96, 64, 4000)])
def test_rope_append(hq, hkv, d, rot, P, T, adjacent):
    """Rotated rows as codes: each value within what one step of its block's
    scale allows of the rotated one, V's codes bit for bit."""
    if adjacent and rot % 2:
        pytest.skip("pairs")
    pages = -(-T // P) + 2
    cfg = H.Config(window=128, page_size=P, n_q_heads=hq, n_kv_heads=hkv, head_dim=d, dtype=H.HSWA_DTYPE_FP4, full_pages=pages, swa_pages=pages, max_seqs=1, max_pages_per_seq=pages)
    s = DualPoolSession(cfg, [FULL])
    rope = H.hswa_rope_create(rot, [rot // 2], adjacent=adjacent)
    x = wl.normal((T, (hq + 2 * hkv) * d), 3000 + T, wl.DTYPE_BF16).cuda()
    q, k, v = x.split([hq * d, hkv * d, hkv * d], 1)
    rng = np.random.default_rng(T)
    pos = rng.integers(0, 1 << 20, (1, T)).astype(np.int32)
    slots = rng.permutation(pages * P)[:T].astype(np.int32)
    slots[T // 2] = -1
    q_out = torch.full((T, hq, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    s.rope_append(0, rope, q, k, v, torch.as_tensor(pos, device="cuda"), torch.as_tensor(slots, device="cuda"), q_out)
    assert s.check() == 0
    fast = d % 32 == 0 and (adjacent or rot % 32 == 0) and rot % (8 if adjacent else 16) == 0
    assert H.hswa_last_kernel() == ("rope_append_fp4" if fast else "rope_append_any_fp4")
    exp_q = serving.rope(q.double().cpu().numpy().reshape(T, hq, d), pos, rot, [rot // 2], adjacent=adjacent)
    assert np.abs(q_out.double().cpu().numpy() - exp_q).max() <= 2.0 ** -8 * np.abs(exp_q).max() + 1e-5
    there = slots >= 0
    at = slots[there]
    vc, vs = fp4.quantize_blocks(v.float().cpu().numpy().reshape(T, hkv, d)[there])
    assert np.array_equal(s.v[0].cpu().numpy()[at // P, :, at % P], vc) and np.array_equal(s.vs[0].cpu().numpy()[at // P, :, at % P], vs)
    kc, ks = s.k[0].cpu().numpy()[at // P, :, at % P], s.ks[0].cpu().numpy()[at // P, :, at % P]
    turned = serving.rope(k.double().cpu().numpy().reshape(T, hkv, d), pos, rot, [rot // 2], adjacent=adjacent)[there]
    # fp32 arithmetic and angles to 1e-7 put the rotated value off by at most 1e-6 of its pair's
    # length: the largest of a block moves its scale by a step of E5M3 at most (1 in 8), and a
    # code is the nearest under the scale that was taken
    wc, ws = fp4.quantize_blocks(turned.astype(np.float32))
    assert np.abs(ks.astype(int) - ws.astype(int)).max() <= 1 and (ks != ws).mean() <= 1e-3
    scale = fp4.E5M3[ks].repeat(16, -1)
    off = np.abs(fp4.dequantize_blocks(kc, ks) - np.clip(turned, -6 * scale, 6 * scale))
    half = np.where(np.abs(turned) > 4 * scale, 1.0, np.where(np.abs(turned) > 2 * scale, 0.5, 0.25)) * scale
    assert (off <= half + 1e-5).all()
    untouched = np.ones(pages * P, bool)
    untouched[at] = False
    free = np.flatnonzero(untouched)
    assert not s.k[0].cpu().numpy()[free // P, :, free % P].any()
    H.hswa_rope_destroy(rope)
    s.close()


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [-0.4, -3.0, 0.0])
@pytest.mark.parametrize("n_tok", [1, 2, 4, 5, 9, 16])
@pytest.mark.parametrize("hq,hkv,d,P", [(64, 8, 128, 64), (6, 2, 96, 16)])
def test_decode_under_scales_that_are_not_positive(hq, hkv, d, P, n_tok, scale):
    """The softmax of scores times a negative scale, and the mean under 0: scores of
    sequences that begin inside a page, of masked keys and of whole masked pages among them."""
    c = Case([1, 63, 64, 200, 900, 4000], seed=150, extra=n_tok + 8, hq=hq, hkv=hkv, d=d, P=P)
    c.sess.reserve(range(c.B), [n_tok] * c.B)
    c.sess.sync()
    _, _, lens = c.sess.tables()
    pos = (lens[:, None] - n_tok + np.arange(n_tok)[None]).reshape(-1)
    for layer in range(2):
        q = wl.normal((c.B * n_tok, hq, d), 3500 + layer, wl.DTYPE_BF16).cuda()
        o = torch.full_like(q, float("nan"))
        if n_tok == 1:
            c.sess.decode(layer, q, o, c.B, scale)
        else:
            c.sess.decode_multi(layer, q, o, c.B, n_tok, scale)
        assert c.sess.check() == 0
        k, v = c.values(layer)
        qh = q.float().cpu().numpy()
        exp = oracle.attention(qh, k, v, c.table(layer), np.repeat(np.arange(c.B), n_tok), pos, c.window(layer), scale)
        off = np.abs(o.float().cpu().numpy() - exp) / tolerance(exp, qh, k, v, abs(scale), int(pos.max()) + 1)
        assert off.max() <= 1, (layer, off.max())  # not for a NaN either


@pytest.mark.gpu
@pytest.mark.parametrize("most", [5, 7, 4, 3])
def test_a_workspace_serves_fewer_tokens(most):
    """The workspace that the most tokens ask for serves fewer: a captured call keeps it."""
    c = Case([300, 5000, 64, 3], seed=160, extra=80)
    step(c, most, seed=3600)
    ws = c.sess.ws
    assert ws.numel() == H.hswa_decode_multi_workspace_size(c.sess.pool, c.B, most)
    for n_tok in range(most - 1, 0, -1):
        c.sess.release(range(c.B))
        step(c, n_tok, seed=3610 + n_tok)
        assert c.sess.ws is ws


@pytest.mark.gpu
@pytest.mark.parametrize("n_tok", [1, 3])
def test_other_shapes_of_lengths_past_the_table(n_tok):
    """Positions behind a table's last page are left out and reported, whatever
    the length says; those that the window still holds are attended."""
    hq, hkv, d, P, W = 6, 2, 96, 16, 100
    c = Case([200, 60, 200, 200, 200, 200], seed=170, extra=0, hq=hq, hkv=hkv, d=d, P=P, W=W)
    cap = c.cfg.max_pages_per_seq * P
    c.sess.release(range(c.B))
    c.sess.reserve([0], [cap - 200])  # a row without a free entry
    c.sess.sync()
    for layer in range(2):
        table = c.table(layer)
        k, v = (x.astype(np.float64) for x in c.values(layer))
        q = wl.normal((c.B * n_tok, hq, d), 3700 + layer, wl.DTYPE_BF16).cuda()
        qh = q.double().cpu().numpy()
        for lens in ([cap + 1, 60, cap + 50, 200, 200, 200], [cap + W + 20, 60, (1 << 31) - 1, 200, cap + (1 << 20), (1 << 31) - 200]):
            c.sess.d_seq_len.copy_(torch.tensor(lens, dtype=torch.int32))
            o = torch.full_like(q, float("nan"))
            c.sess.decode_multi(layer, q, o, c.B, n_tok, c.scale)
            assert c.sess.check() == H.HSWA_ERR_BOUNDS
            got = o.double().cpu().numpy()
            for row in range(c.B * n_tok):
                s, t = row // n_tok, lens[row // n_tok] - n_tok + row % n_tok
                first = max(0, t - W + 1) if c.kinds[layer] == SWA else 0
                at = [j for j in range(first, min(t + 1, cap)) if table[s, j // P] >= 0]
                for h in range(hq):
                    if not at:
                        assert not got[row, h].any()
                        continue
                    pages, rows, g = [table[s, j // P] for j in at], [j % P for j in at], h // (hq // hkv)
                    x = k[pages, g, rows] @ qh[row, h] * c.scale
                    w = np.exp(x - x.max())
                    exp = w @ v[pages, g, rows] / w.sum()
                    assert (np.abs(got[row, h] - exp) <= tolerance(exp, qh, k, v, c.scale, cap)).all(), (layer, lens[s], row, h)


@pytest.mark.gpu
@pytest.mark.parametrize("P", [16, 48])
@pytest.mark.parametrize("dtype", [H.HSWA_DTYPE_F32, H.HSWA_DTYPE_BF16, H.HSWA_DTYPE_FP8_E4M3])
def test_read_of_other_pages(dtype, P):
    """Rows read back from pools of other pages, from the last slot too."""
    hkv, d, pages = 3, 128, 9
    cfg = H.Config(window=128, page_size=P, n_q_heads=hkv, n_kv_heads=hkv, head_dim=d, dtype=dtype, full_pages=pages, swa_pages=pages, max_seqs=1, max_pages_per_seq=pages)
    s = DualPoolSession(cfg, [FULL])
    t = torch.float32 if dtype == H.HSWA_DTYPE_F32 else torch.bfloat16
    x = wl.normal((2, pages * P, hkv, d), 7, wl.DTYPE_BF16).to(t).cuda()
    slots = torch.randperm(pages * P).int().cuda()
    s.append(0, x[0], x[1], slots)
    k, v = (torch.full((pages * P, hkv, d), float("nan"), dtype=t, device="cuda") for _ in range(2))
    s.read(0, slots, k, v)
    assert s.check() == 0
    for which, got in enumerate((k, v)):
        exp = x[which]
        if dtype == H.HSWA_DTYPE_FP8_E4M3:  # K rows of 128 codes, V columns of a page
            pool, scales = (s.k[0], s.ks[0]) if which == 0 else (s.v[0].view(pages, hkv, d, P).transpose(2, 3), s.vs[0])
            page, row = slots.long() // P, slots.long() % P
            exp = (pool[page, :, row].contiguous().view(torch.float8_e4m3fn).float() * scales[page, :, row]).bfloat16()
            # these rows: off by half a code's step (2^-4 of the value, 2^-10 of the scale below the normal codes) and the bf16's
            y, most = x[which].float(), scales.max() * 2.0 ** -10
            assert ((exp.float() - y).abs() <= (2.0 ** -4 + 2.0 ** -8 + 2.0 ** -12) * y.abs() + 1.01 * most).all()
        assert torch.equal(got, exp)
    s.close()
