"""FP4 pools and the step from logits to probabilities on the CPU: pins of the
oracle (quantizer, penalties, counts) and the library's refusals, each of which
comes before a launch."""
import gc
import math
import weakref

import numpy as np
import pytest
import torch

import oracle
from oracle import fp4, serving
import hybrid_sliding_window_dual_gb300 as H
from hybrid_sliding_window_dual_gb300.session import DualPoolSession

INVALID, UNSUPPORTED = H.HSWA_ERR_INVALID_ARG, H.HSWA_ERR_UNSUPPORTED
X = 1 << 20  # an address that is never followed


def refused(status, f, *args):
    with pytest.raises(H.HswaError) as e:
        f(*args)
    assert e.value.status == status, e.value


# ------------------------------------------------------------------ oracle
def test_oracle_scales_are_halves_without_their_last_bits():
    half = (np.arange(0xF8, dtype=np.uint16) << 7).view(np.float16).astype(np.float64)
    assert np.array_equal(fp4.E5M3, half) and fp4.E5M3[0xE2] == fp4.MAX_SCALE and 6 * fp4.E5M3[0xE2] < 65504 < 6 * fp4.E5M3[0xE3]


def test_oracle_quantizer_by_hand():
    def of(*x):
        c, s = fp4.quantize_blocks(np.array(list(x) + [0.0] * (16 - len(x)), np.float32))
        return [int(v) for v in np.stack((c & 15, c >> 4), -1).reshape(-1)[:len(x)]], int(s[0])

    one = 15 << 3  # the scale 1
    assert of(6, 4, 3, 2, 1.5, 1, 0.5, 0) == ([7, 6, 5, 4, 3, 2, 1, 0], one)
    assert of(-6, -4, -3, -2, -1.5, -1, -0.5, -0.0) == ([15, 14, 13, 12, 11, 10, 9, 8], one)
    # borders go to the even code, what is beside them to the nearer one
    assert of(6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5) == ([7, 0, 2, 2, 4, 4, 6, 6], one)
    up = [np.nextafter(np.float32(x), np.float32(9)) for x in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5)]
    down = [np.nextafter(np.float32(x), np.float32(0)) for x in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5)]
    assert of(6, *up) == ([7, 1, 2, 3, 4, 5, 6, 7], one) and of(6, *down) == ([7, 0, 1, 2, 3, 4, 5, 6], one)
    # scales: 6.375 / 6 = 1.0625 lies between 1 and 1.125 and goes to the even byte, 7.125 / 6 = 1.1875 to 1.25
    assert of(6.375) == ([7], one) and of(7.125) == ([7], one + 2)
    assert of(0.0) == ([0], 0) and of(-0.0) == ([0], 0)
    # 6 * 2^-18 is half of the smallest scale's: to 0, and codes with it; more than that is kept
    assert of(6 * 2.0 ** -18) == ([0], 0) and of(-6.5 * 2.0 ** -18) == ([13], 1)  # 3.25 under the scale 2^-17: -3
    assert of(np.inf, -np.inf, 70000) == ([7, 15, 7], 0xE2)


def test_oracle_dequantized_values_are_16_bit_floats():
    c, s = np.meshgrid(np.arange(256), np.arange(0xE3), indexing="ij")
    codes = np.repeat(c.reshape(-1, 1), 8, 1).astype(np.uint8)
    v = fp4.dequantize_blocks(codes, s.reshape(-1, 1).astype(np.uint8))
    assert np.array_equal(v, v.astype(np.float16).astype(np.float64))
    t = torch.as_tensor(v)
    assert torch.equal(t, t.bfloat16().double())


def test_oracle_quantizer_is_the_nearest_of_all_values():
    rng = np.random.default_rng(1)
    x = (rng.standard_normal((500, 32)) * np.exp(rng.uniform(-8, 8, (500, 1)))).astype(np.float32)
    c, s = fp4.quantize_blocks(x)
    v = fp4.dequantize_blocks(c, s)
    scale = fp4.E5M3[s].repeat(16, -1)
    every = np.concatenate((-fp4.E2M1[:0:-1], fp4.E2M1))
    best = np.abs(x[..., None] - scale[..., None] * every).min(-1)
    assert np.allclose(np.abs(x - v), best, rtol=0, atol=0)
    amax = np.abs(x.reshape(500, 2, 16)).max(-1)
    assert (np.abs(fp4.E5M3[s] - amax / 6) <= np.abs(fp4.E5M3 - (amax / 6)[..., None]).min(-1) + 1e-12).all()


def test_oracle_attention_over_an_fp4_pool_by_hand():
    """One key: its value; equal scores: the mean."""
    k, v = np.zeros((1, 1, 16, 16), np.float32), np.zeros((1, 1, 16, 16), np.float32)
    codes, scales = (np.zeros((1, 1, 16, n), np.uint8) for n in (8, 1))
    kc, ks = codes.copy(), scales.copy()
    rows = np.zeros((2, 1, 16), np.float32)
    rows[0, 0, :4], rows[1, 0, :4] = [6, 3, -1, 0.5], [12, 4, 0, 1]
    fp4.append_kv_fp4(kc, ks, codes, scales, np.zeros_like(rows), rows, [0, 1])
    v = fp4.dequantize_blocks(codes, scales).astype(np.float32)
    q = np.ones((2, 1, 16), np.float32)
    o = oracle.attention(q, k, v, np.array([[0]], np.int32), np.array([0, 0]), np.array([0, 1]), 0, 1.0)
    assert np.allclose(o[0, 0, :4], [6, 3, -1, 0.5]) and np.allclose(o[1, 0, :4], [9, 3.5, -0.5, 0.75])


def test_oracle_probs_by_hand():
    e = math.exp
    z = np.array([[[2.0, -1.0, 0.5, 0.0]]])
    p, _ = serving.logits_probs(z)
    w = np.exp(z[0, 0])
    assert np.allclose(p[0, 0], w / w.sum())
    counts = np.array([[1, 1 << 15 | 0, 0, 2]], np.uint16)
    # token 0 generated once, 1 in the prompt, 3 generated twice
    p, got = serving.logits_probs(z, [[0.5, 2.0, 0.25, 0.125]], counts)
    assert np.allclose(got[0, 0], [1.0 - 0.25 - 0.125, -2.0, 0.5, 0.0 - 0.5 - 0.125])
    w = [e(x / 0.5) for x in got[0, 0]]
    assert np.allclose(p[0, 0], np.array(w) / sum(w))
    # a draft counts from the next row on
    _, got = serving.logits_probs(np.repeat(z, 3, 1), [[1.0, 1.0, 1.0, 0.0]], np.zeros((1, 4), np.uint16), np.array([[2, 2]]))
    assert got[0, :, 2].tolist() == [0.5, -0.5, -1.5]
    _, got = serving.logits_probs(z, bias_token=np.array([[1, 3, 1, -1]]), bias=np.array([[9.0, 1.0, 2.0, 5.0]]))
    assert got[0, 0].tolist() == [2.0, 1.0, 0.5, 1.0]
    p, _ = serving.logits_probs(z, [[0.0, 1, 0, 0]], allowed=np.array([[False, True, True, True]]))
    assert p[0, 0].tolist() == [0, 0, 1, 0]
    p, _ = serving.logits_probs(z, allowed=np.zeros((1, 4), bool))
    assert not p.any()
    p, _ = serving.logits_probs(np.array([[[np.inf, 1.0, np.inf, np.nan]]]))
    assert p[0, 0].tolist() == [0.5, 0, 0.5, 0]


def test_oracle_counts_by_hand():
    c = serving.count_tokens([[1, 2, 2, -1, 2, 9]], [2], 4)
    assert c.tolist() == [[0, 1 << 15, 1 << 15 | 2, 0]]
    assert serving.count_tokens([[0, 1]], None, 2, np.array([[32767, 1 << 15 | 32767]], np.uint16)).tolist() == [[32767, 65535]]


# --------------------------------------------------------------- refusals
def layer(kind=None, **over):
    f = dict(kind=H.HSWA_KIND_FULL if kind is None else kind, window=128, k_pool=X, v_pool=X, k_scale=X, v_scale=X)
    f.update(over)
    return H.Layer(**f)


def pool(dtype=H.HSWA_DTYPE_FP4, d=128, hq=16, hkv=2, P=64, S=4, MP=8, pages=16):
    return H.hswa_pool_create(H.Config(window=128, page_size=P, n_q_heads=hq, n_kv_heads=hkv, head_dim=d, dtype=dtype, full_pages=pages, swa_pages=pages, max_seqs=S, max_pages_per_seq=MP))


def test_fp4_append_and_read_refusals():
    p, odd = pool(), pool(d=72)
    for f, args in ((H.hswa_append_kv, lambda o: (o["pool"], o["layer"], o["k"], o["v"], o["slots"], o["n"])),
                    (H.hswa_read_kv, lambda o: (o["pool"], o["layer"], o["slots"], o["n"], o["k"], o["v"]))):
        ok = dict(pool=p, layer=layer(), k=X, v=X, slots=X, n=5)

        def bad(status, **over):
            refused(status, f, *args({**ok, **over}))

        for name in ("pool", "k", "v", "slots"):
            bad(INVALID, **{name: None})
        bad(INVALID, n=-1)
        bad(INVALID, layer=layer(kind=7))
        bad(INVALID, layer=layer(k_pool=None))
        bad(INVALID, layer=layer(k_scale=None))
        bad(INVALID, layer=layer(v_scale=None))
        bad(UNSUPPORTED, k=X + 8)
        bad(UNSUPPORTED, v=X + 2)
        bad(UNSUPPORTED, layer=layer(v_pool=X + 4))
        bad(UNSUPPORTED, pool=odd)
        f(*args({**ok, "n": 0, "k": None, "v": None, "slots": None}))
    for x in (p, odd):
        H.hswa_pool_destroy(x)
    for dtype, d, status, over in ((H.HSWA_DTYPE_FP8_E4M3, 64, UNSUPPORTED, {}), (H.HSWA_DTYPE_FP8_E4M3, 128, INVALID, dict(k_scale=None)), (H.HSWA_DTYPE_BF16, 4, UNSUPPORTED, {}),
                                   (H.HSWA_DTYPE_BF16, 64, UNSUPPORTED, dict(k_pool=X + 8))):
        p = pool(dtype, d)
        refused(status, H.hswa_read_kv, p, layer(**over), X, 5, X, X)
        H.hswa_pool_destroy(p)


def test_fp4_attention_refusals():
    p, odd, wide = pool(), pool(d=72), pool(d=272)
    ws = 1 << 30
    for x, status in ((odd, UNSUPPORTED), (wide, UNSUPPORTED)):
        refused(status, H.hswa_decode, x, layer(), X, X, X, X, 4, 1.0, X, ws)
        refused(status, H.hswa_decode_multi, x, layer(), X, X, X, X, 4, 3, 1.0, X, ws)
        refused(status, H.hswa_prefill_chunk, x, layer(), X, X, X, X, X, 1, 4, 4, 1.0)
        assert H.hswa_prefill_workspace_size(x, layer(), 2, 64) == 0
    for over in (dict(k_scale=None), dict(v_scale=None)):
        refused(INVALID, H.hswa_decode, p, layer(**over), X, X, X, X, 4, 1.0, X, ws)
        refused(INVALID, H.hswa_prefill_chunk_ws, p, layer(**over), X, X, X, X, X, 1, 4, 4, 1.0, X, ws)
    refused(INVALID, H.hswa_decode, p, layer(), X, X, X, X, 5, 1.0, X, ws)
    refused(INVALID, H.hswa_decode_multi, p, layer(), X, X, X, X, 4, 17, 1.0, X, ws)
    # what FP4 pools have no call for
    refused(UNSUPPORTED, H.hswa_decode_weights, p, layer(), X, X, X, X, 4, 1.0, None, 0.0, X, X, ws)
    refused(UNSUPPORTED, H.hswa_decode_noalloc, p, layer(), X, X, X, X, 4, 1.0)
    swa = layer(kind=H.HSWA_KIND_SWA)
    refused(UNSUPPORTED, H.hswa_swa_gather, p, swa, X, X, X, 1, X)
    refused(UNSUPPORTED, H.hswa_swa_scatter, p, swa, X, X, X, 1, X)
    refused(UNSUPPORTED, H.hswa_swa_window_offsets, p, swa, 1)
    assert H.hswa_decode_multi_workspace_size(p, 4, 1) >= H.hswa_decode_workspace_size(p, 1) > 0
    assert H.hswa_prefill_workspace_size(p, layer(), 2, 64) > 0
    rope = H.hswa_rope_create(64, [32])
    refused(UNSUPPORTED, H.hswa_rope_append, odd, layer(), rope, X, 16 * 72, X << 4, 144, X << 5, 144, X, X, X << 6, 3)
    refused(INVALID, H.hswa_rope_append, p, layer(k_scale=None), rope, X, 2048, X << 4, 256, X << 5, 256, X, X, X << 6, 3)
    H.hswa_rope_destroy(rope)
    for x in (p, odd, wide):
        H.hswa_pool_destroy(x)


def test_logits_probs_refusals():
    ok = dict(ldt=H.HSWA_DTYPE_F32, logits=X, ls=100, pdt=H.HSWA_DTYPE_F32, p=X << 3, ps=100, params=X, counts=X, cs=100, draft=X, bt=X, bias=X, nb=3, mask=X, ms=4, n=2, n_tok=4, vocab=100)

    def bad(status, **over):
        refused(status, H.hswa_logits_probs, *{**ok, **over}.values())

    for name in ("logits", "p", "bt", "bias"):
        bad(INVALID, **{name: None})
    bad(INVALID, n=-1)
    bad(INVALID, n_tok=0)
    bad(INVALID, n_tok=17)
    bad(INVALID, vocab=0)
    bad(INVALID, nb=-1)
    bad(INVALID, ls=99)
    bad(INVALID, ps=99)
    bad(INVALID, cs=99)
    bad(INVALID, ms=3)
    bad(INVALID, logits=X + 2)
    bad(INVALID, p=X + 1)
    bad(INVALID, counts=X + 1)
    for name in ("params", "draft", "bt", "bias", "mask"):
        bad(INVALID, **{name: X + 2})
    bad(UNSUPPORTED, ldt=H.HSWA_DTYPE_FP8_E4M3)
    bad(UNSUPPORTED, pdt=H.HSWA_DTYPE_FP4)
    bad(UNSUPPORTED, nb=1025)
    big = 1 << 21
    bad(UNSUPPORTED, vocab=(1 << 20) + 1, ls=big, ps=big, cs=big, ms=big)
    # p over the logits, but not each value in its own place
    row = 100 * 4
    for at, over in ((X + 4, {}), (X - 4, {}), (X + 7 * row, {}), (X - 8 * row + 4, {}), (X, dict(ps=101)), (X, dict(pdt=H.HSWA_DTYPE_BF16))):
        bad(INVALID, p=at, **over)
    H.hswa_logits_probs(*{**ok, "n": 0, "logits": None}.values())


def test_count_tokens_refusals():
    ok = dict(counts=X, cs=100, tokens=X, ts=7, prompt=X, n=2, n_tokens=7, vocab=100, clear=0)

    def bad(status, **over):
        refused(status, H.hswa_count_tokens, *{**ok, **over}.values())

    for name in ("counts", "tokens"):
        bad(INVALID, **{name: None})
    bad(INVALID, n=-1)
    bad(INVALID, n_tokens=-1)
    bad(INVALID, vocab=0)
    bad(INVALID, cs=99)
    bad(INVALID, ts=6)
    bad(INVALID, counts=X + 1)
    bad(INVALID, tokens=X + 2)
    bad(INVALID, prompt=X + 2)
    bad(UNSUPPORTED, vocab=(1 << 20) + 1, cs=1 << 21)
    for over in (dict(n=0), dict(n_tokens=0)):
        H.hswa_count_tokens(*{**ok, "counts": None, "tokens": None, **over}.values())


def test_session_shapes():
    cfg = H.Config(window=128, page_size=64, n_q_heads=4, n_kv_heads=2, head_dim=32, dtype=H.HSWA_DTYPE_FP4, full_pages=4, swa_pages=5, max_seqs=2, max_pages_per_seq=4)
    s = DualPoolSession(cfg, [H.HSWA_KIND_FULL, H.HSWA_KIND_SWA], device="cpu")
    assert s.k[0].shape == s.v[0].shape == (4, 2, 64, 16) and s.ks[1].shape == s.vs[1].shape == (5, 2, 64, 2) and s.ks[0].dtype == s.k[0].dtype == torch.uint8
    f, i16, i32 = torch.zeros, dict(dtype=torch.int16), dict(dtype=torch.int32)
    logits = f(2, 3, 50)
    for args in (dict(logits=logits.double(), p=logits), dict(logits=logits, p=f(2, 3, 49)), dict(logits=logits, p=logits, params=f(2, 3)), dict(logits=logits, p=logits, counts=f(2, 50, **i32)),
                 dict(logits=logits, p=logits, counts=f(3, 50, **i16)), dict(logits=logits, p=logits, counts=f(2, 100, **i16)[:, ::2]), dict(logits=logits, p=logits, d_draft=f(2, 3, **i32)),
                 dict(logits=logits, p=logits, bias_token=f(2, 4, **i32)), dict(logits=logits, p=logits, bias_token=f(2, 4, **i32), bias=f(2, 5)),
                 dict(logits=logits, p=logits, mask=f(2, 2, **i32)), dict(logits=logits, p=logits, mask=f(6, 3, **i32)), dict(logits=f(2, 3, 100)[:, :, ::2], p=logits),
                 dict(logits=logits, p=logits, params=f(2, 4).double()), dict(logits=logits, p=logits, d_draft=f(2, 2).long()),
                 dict(logits=logits, p=logits, bias_token=f(2, 4).long(), bias=f(2, 4)), dict(logits=logits, p=logits, bias_token=f(2, 4, **i32), bias=f(2, 4).half())):
        with pytest.raises(ValueError):
            s.probs(**args)
    for counts, tokens in ((f(2, 50, **i32), f(2, 7, **i32)), (f(3, 50, **i16), f(2, 7, **i32)), (f(2, 50, **i16), f(2, 7)), (f(2, 100, **i16)[:, ::2], f(2, 7, **i32)),
                           (f(2, 50, **i16), f(2, 14, **i32)[:, ::2])):
        with pytest.raises(ValueError):
            s.count_tokens(counts, tokens)
    for prompt in (f(2), f(3, **i32), f(4, **i32)[::2]):
        with pytest.raises(ValueError):
            s.count_tokens(f(2, 50, **i16), f(2, 7, **i32), prompt)
    for k, v in ((f(3, 2, 32), f(3, 2, 32)), (f(3, 2, 32).bfloat16(), f(2, 2, 32).bfloat16()), (f(3, 32, 2).bfloat16().transpose(1, 2), f(3, 2, 32).bfloat16())):
        with pytest.raises(ValueError):
            s.read(0, f(3, **i32), k, v)
    s.close()


@pytest.mark.parametrize("dtype", [H.HSWA_DTYPE_F32, H.HSWA_DTYPE_BF16, H.HSWA_DTYPE_FP4])
def test_fused_decode_is_refused_before_its_append(dtype):
    """Heads that no decode takes: the call comes back before the pool is written."""
    p = pool(dtype, d=272)
    for kind in (H.HSWA_KIND_FULL, H.HSWA_KIND_SWA):
        refused(UNSUPPORTED, H.hswa_decode_append, p, layer(kind), X, X, X, X, X, X, X, 4, 1.0, X, 1 << 30)
    H.hswa_pool_destroy(p)


@pytest.mark.parametrize("dtype", [H.HSWA_DTYPE_F32, H.HSWA_DTYPE_BF16, H.HSWA_DTYPE_FP8_E4M3, H.HSWA_DTYPE_FP4])
def test_a_decode_workspace_serves_fewer_tokens_and_sequences(dtype):
    p = pool(dtype, S=64)
    for n in (1, 64):
        sizes = [H.hswa_decode_multi_workspace_size(p, n, t) for t in range(1, H.HSWA_DECODE_MAX_TOKENS + 1)]
        assert sizes == sorted(sizes) and sizes[0] == H.hswa_decode_workspace_size(p, n)
        assert all(a <= b for a, b in zip(sizes, (H.hswa_decode_multi_workspace_size(p, 64, t) for t in range(1, 17))))
    H.hswa_pool_destroy(p)


def test_session_keeps_the_workspaces_that_captured_calls_may_hold():
    cfg = H.Config(window=128, page_size=64, n_q_heads=16, n_kv_heads=2, head_dim=128, dtype=H.HSWA_DTYPE_FP4, full_pages=4, swa_pages=5, max_seqs=40, max_pages_per_seq=4)
    s = DualPoolSession(cfg, [H.HSWA_KIND_FULL], device="cpu")
    one = s.workspace(1, 1)
    assert s.workspace(40, 1) is one  # more sequences need no other
    held = [weakref.ref(one)]
    del one
    for n_tok in (4, 16):
        held.append(weakref.ref(s.workspace(3, n_tok)))
    at = s.ws.data_ptr()
    for n_tok in (16, 5, 4, 2, 1):
        assert s.workspace(40, n_tok).data_ptr() == at
    gc.collect()
    assert all(x() is not None for x in held)
    s.close()
