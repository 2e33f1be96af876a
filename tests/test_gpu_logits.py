"""hswa_logits_probs and hswa_count_tokens on the GPU against the oracle in 64
bits: probabilities within what the fp32 steps can add up to, greedy rows,
zeros and counts exactly."""
import numpy as np
import pytest
import torch

from oracle import serving
import hybrid_sliding_window_dual_gb300 as H

CODE = {torch.float32: H.HSWA_DTYPE_F32, torch.bfloat16: H.HSWA_DTYPE_BF16}


def run(logits, p, params=None, counts=None, draft=None, bias_token=None, bias=None, mask=None, stream=None, expect=0):
    S, n, V = logits.shape
    row = lambda x: x.stride(1) if n > 1 else x.stride(0) if S > 1 else V  # noqa: E731
    H.hswa_logits_probs(CODE[logits.dtype], logits, row(logits), CODE[p.dtype], p, row(p), params, counts, 0 if counts is None else counts.stride(0), draft, bias_token, bias,
                        0 if bias is None else bias.shape[1], mask, 0 if mask is None else mask.stride(0), S, n, V, stream)
    assert H.hswa_check(stream) == expect
    return p


def host(x):
    return None if x is None else x.double().cpu().numpy() if x.is_floating_point() else x.cpu().numpy()


def bits(allowed):
    """bool [rows][V] as int32 words."""
    V = allowed.shape[1]
    x = np.pad(allowed, ((0, 0), (0, -V % 32))).reshape(len(allowed), -1, 32)
    return torch.as_tensor((x.astype(np.uint64) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32).view(np.int32), device="cuda")


def check(got, logits, params=None, counts=None, draft=None, bias_token=None, bias=None, allowed=None):
    """Four steps make z, each off by at most 2^-24 of the largest value Z that
    occurs (Z: logits times or over the repetition, plus penalties and bias); the
    difference from the top, its product with log2 e / T (whose own roundings are
    two) and the exponential's 2 ulp give each weight; a sum adds at most 160 in
    a thread's, a block's and a cluster's order; then one product of two quotients."""
    exp, z = serving.logits_probs(host(logits), host(params), None if counts is None else counts.cpu().numpy().view(np.uint16), host(draft), host(bias_token), host(bias), allowed)
    got_dtype, got = got.dtype, host(got)
    assert np.isfinite(got).all()
    eps = 2.0 ** -24
    for i in range(exp.shape[0]):
        T, rep, freq, pres = (1, 1, 0, 0) if params is None else host(params)[i]
        if not T > 0:
            assert np.array_equal(got[i], exp[i])
            continue
        rep = rep if rep > 0 else 1
        x = host(logits)[i]
        most = 0 if counts is None else (counts[i].cpu().numpy().view(np.uint16) & 0x7fff).max() + 16
        Z = np.abs(x[np.isfinite(x)]).max(initial=0) * max(rep, 1 / rep) + abs(freq) * most + abs(pres) + (0 if bias is None else np.abs(host(bias)[i]).max())
        for w in range(exp.shape[1]):
            finite = z[i, w][np.isfinite(z[i, w])]
            top = z[i, w].max()
            assert np.array_equal(got[i, w] == 0, exp[i, w] == 0) or (exp[i, w][got[i, w] == 0] < 1e-30).all()
            if not finite.size or top == np.inf:
                tol = 2 * eps * exp[i, w]
            else:
                down = np.where(np.isfinite(z[i, w]), top - z[i, w], 0)
                tol = exp[i, w] * (2 * 8 * eps * Z / T + 6 * eps * down / T + 2 * 6 * eps * 20 + 200 * eps) + 1e-37
            if got_dtype == torch.bfloat16:
                tol = tol + exp[i, w] * 2.0 ** -8 + 2.0 ** -134
            assert (np.abs(got[i, w] - exp[i, w]) <= tol).all(), (i, w, np.abs(got[i, w] - exp[i, w]).max(), (np.abs(got[i, w] - exp[i, w]) / np.maximum(tol, 1e-45)).max())
            s = got[i, w].sum()
            assert s == 0 or abs(s - 1) <= (2.0 ** -8 if got_dtype == torch.bfloat16 else 1e-4)


def inputs(S, n, V, dtype, seed, pad=0, m=5, share=0.7, greedy=0.3):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rng = np.random.default_rng(seed)
    logits = torch.zeros(S, n, V + pad, dtype=dtype, device="cuda")[:, :, :V]
    logits.copy_(torch.randn(S, n, V, generator=g, device="cuda") * 4)
    params = np.stack((rng.uniform(0.3, 2, S), rng.uniform(0.7, 1.5, S), rng.uniform(-1, 1, S), rng.uniform(-1, 1, S)), 1)
    params[rng.random(S) < greedy, 0] = 0
    draft = torch.as_tensor(rng.integers(0, V, (S, n - 1)).astype(np.int32), device="cuda") if n > 1 else None
    if n > 3:  # a draft drawn twice, one outside
        draft[:, 2] = draft[:, 0]
        draft[0, 1] = -1
    counts = torch.zeros(S, V + pad, dtype=torch.int16, device="cuda")[:, :V]
    counts.copy_(torch.as_tensor(np.where(rng.random((S, V)) < 0.2, rng.integers(-(1 << 15), 1 << 15, (S, V)) & -32768 | rng.integers(0, 6, (S, V)), 0).astype(np.int16)))
    bt = torch.as_tensor(rng.integers(-1, V, (S, m)).astype(np.int32), device="cuda")
    if m > 2:
        bt[:, 2] = bt[:, 0]  # the last entry counts
    bias = torch.randn(S, m, generator=g, device="cuda") * 5
    allowed = rng.random((S * n, V)) < share
    return logits, torch.as_tensor(params.astype(np.float32), device="cuda"), counts, draft, bt, bias, allowed


SHAPES = [(1, 1, 1), (2, 1, 2), (3, 2, 7), (1, 3, 8), (5, 4, 31), (4, 16, 33), (9, 3, 1000), (3, 5, 4099), (40, 4, 2048), (2, 8, 32001), (200, 2, 5000), (2, 3, 131072), (1, 2, 163840), (1, 2, 163841),
          (2, 1, 262144), (1, 1, 327681), (1, 2, 1 << 20)]


@pytest.mark.gpu
@pytest.mark.parametrize("p_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("S,n,V", SHAPES)
def test_probs_match_oracle(S, n, V, dtype, p_dtype):
    if V >= 262144 and dtype != p_dtype:
        pytest.skip("the oracle's time")
    logits, params, counts, draft, bt, bias, allowed = inputs(S, n, V, dtype, seed=S * 100 + n)
    p = torch.full(logits.shape, float("nan"), dtype=p_dtype, device="cuda")
    check(run(logits, p), logits)
    check(run(logits, p, params, counts, draft, bt, bias, bits(allowed)), logits, params, counts, draft, bt, bias, allowed)


@pytest.mark.gpu
@pytest.mark.parametrize("pad", [1, 2, 3, 8, 61])
def test_probs_padded_rows_and_in_place(pad):
    for V in (1003, 1008):
        for dtype in CODE:
            logits, params, counts, draft, bt, bias, allowed = inputs(6, 3, V, dtype, seed=pad, pad=pad)
            store = torch.full((6, 3, V + pad), float("nan"), dtype=dtype, device="cuda")
            check(run(logits, store[:, :, :V], params, counts, draft, bt, bias, bits(allowed)), logits, params, counts, draft, bt, bias, allowed)
            assert store[:, :, V:].isnan().all()  # between the rows nothing is written
            same = torch.empty_like(store)[:, :, :V]
            same.copy_(logits)
            run(same, same, params, counts, draft, bt, bias, bits(allowed))
            assert torch.equal(same, store[:, :, :V])


@pytest.mark.gpu
@pytest.mark.parametrize("V", [40, 5000, 200000])
def test_probs_each_option_alone(V):
    logits, params, counts, draft, bt, bias, allowed = inputs(5, 4, V, torch.float32, seed=3, m=300 if V > 300 else 20)
    p = torch.empty_like(logits)
    check(run(logits, p, params), logits, params)
    check(run(logits, p, params, counts), logits, params, counts)
    check(run(logits, p, params, counts, draft), logits, params, counts, draft)
    check(run(logits, p, None, counts, draft), logits, None, counts, draft)  # nothing to penalize with
    check(run(logits, p, None, None, None, bt, bias), logits, bias_token=bt, bias=bias)
    check(run(logits, p, mask=bits(allowed)), logits, allowed=allowed)
    check(run(logits, p, params, None, draft, mask=bits(allowed)), logits, params, None, draft, allowed=allowed)


@pytest.mark.gpu
@pytest.mark.parametrize("V", [100, 30000])
def test_probs_infinities_nan_and_empty_rows(V):
    inf, nan = float("inf"), float("nan")
    logits, _, counts, draft, bt, bias, allowed = inputs(8, 2, V, torch.float32, seed=9)
    logits[0, 0] = -inf
    logits[0, 1] = nan
    logits[1, 0, 3] = nan
    logits[1, 1, 5] = inf
    logits[2, 0, ::7] = inf
    logits[2, 1] = torch.finfo(torch.float32).min
    logits[3, 0, 1:] = -inf
    logits[3, 1, 0] = 3e38
    allowed[8] = False                  # nothing allowed
    allowed[9] = False
    allowed[9, V - 1] = True            # one token
    logits[5, 0, ~torch.as_tensor(allowed[10], device="cuda")] = nan  # NaN and infinity where nothing is allowed
    logits[5, 1, ~torch.as_tensor(allowed[11], device="cuda")] = inf
    for T in (1.0, 0.0, 1e-30, inf, nan, -1.0):
        params = torch.tensor([[T, 1.3, 0.1, 0.1]], device="cuda").repeat(8, 1)
        params[7] = torch.tensor([T, nan, 0.0, 0.0])  # a repetition that counts as 1
        p = torch.full_like(logits, nan)
        run(logits, p, params, None, None, None, None, bits(allowed))
        check(p, logits, params, allowed=allowed)
        assert not p[0].any() and not p[4, 0].any() and p[4, 1, V - 1] == 1
        run(logits, p, params, counts, draft, bt, bias, bits(allowed))
        assert torch.isfinite(p).all() and not p[0].any()


@pytest.mark.gpu
def test_probs_ties_go_to_the_first():
    """Greedy rows of whole-number logits with many equal largest ones, on every CTA of a cluster."""
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    for V in (9, 4096, 70001, 150000):
        logits = torch.randint(0, 3, (6, 2, V), generator=g, device="cuda").float()
        logits[1] = 0
        logits[2, 0, : V // 2] = -1
        params = torch.tensor([[0.0, 1.0, 0.0, 0.0]], device="cuda").repeat(6, 1)
        p = run(logits, torch.empty_like(logits), params)
        first = (logits == logits.amax(-1, keepdim=True)).float().argmax(-1)
        assert torch.equal(p.sum(-1), torch.ones(6, 2, device="cuda")) and torch.equal(p.argmax(-1), first)


@pytest.mark.gpu
def test_probs_biases_outside_and_full_list():
    V = 2000
    logits, *_ = inputs(2, 1, V, torch.float32, seed=4)
    bt = torch.arange(1024, device="cuda").int().repeat(2, 1) * 7 % V
    bias = torch.randn(2, 1024, device="cuda")
    p = torch.empty_like(logits)
    check(run(logits, p, bias_token=bt, bias=bias), logits, bias_token=bt, bias=bias)
    bt[1, 5] = V
    run(logits, p, bias_token=bt, bias=bias, expect=H.HSWA_ERR_BOUNDS)
    bt[1, 5] = -1
    check(p, logits, bias_token=bt, bias=bias)


@pytest.mark.gpu
def test_probs_captured_replayed_and_on_a_stream():
    logits, params, counts, draft, bt, bias, allowed = inputs(7, 4, 50000, torch.bfloat16, seed=5)
    p = torch.empty(logits.shape, device="cuda")
    mask = bits(allowed)
    first = run(logits, p, params, counts, draft, bt, bias, mask).clone()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        again = run(logits, torch.empty_like(p), params, counts, draft, bt, bias, mask, stream=side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            H.hswa_logits_probs(H.HSWA_DTYPE_BF16, logits, 50000, H.HSWA_DTYPE_F32, p, 50000, params, counts, 50000, draft, bt, bias, 5, mask, mask.stride(0), 7, 4, 50000, side)
    assert torch.equal(first, again)
    other = inputs(7, 4, 50000, torch.bfloat16, seed=6)[0]
    logits.copy_(other)
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    check(p, logits, params, counts, draft, bt, bias, allowed)


def count(tokens, n_prompt, V, before=None, clear=True, pad=0, expect=0):
    S, n = tokens.shape
    store = torch.full((S, V + pad), -21555, dtype=torch.int16, device="cuda")
    counts = store[:, :V]
    if before is not None:
        counts.copy_(before)
    d = torch.as_tensor(tokens, device="cuda")
    np_ = None if n_prompt is None else torch.as_tensor(n_prompt, device="cuda")
    H.hswa_count_tokens(counts, V + pad, d, d.stride(0), np_, S, n, V, clear)
    assert H.hswa_check() == expect
    assert (store[:, V:] == -21555).all()
    want = serving.count_tokens(tokens, n_prompt, V, None if clear else before.cpu().numpy().view(np.uint16))
    assert np.array_equal(counts.cpu().numpy().view(np.uint16), want)


@pytest.mark.gpu
@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("S,n,V", [(1, 1, 1), (3, 4, 17), (5, 64, 8192), (5, 65, 8193), (2, 1000, 20000), (64, 4, 1000), (3, 40000, 131072), (2, 3, 1 << 20), (2, 5000, 393217), (2, 40000, 200000), (2, 5000, 390000), (1, 65537, 9000), (9, 33000, 1001)])
def test_count_tokens(S, n, V, pad):
    rng = np.random.default_rng(S + n)
    tokens = np.where(rng.random((S, n)) < 0.1, -1, np.minimum(rng.exponential(V / 50 + 1, (S, n)), V - 1)).astype(np.int32)
    prompt = rng.integers(0, n + 1, S).astype(np.int32)
    before = torch.as_tensor(np.where(rng.random((S, V)) < 0.3, rng.integers(-(1 << 15), 1 << 15, (S, V)), 0).astype(np.int16), device="cuda")
    before[:, 0] = 32767  # stays there
    if V > 1:
        before[:, 1] = -2  # 32766 and in the prompt
    for clear in (True, False):
        count(tokens, prompt, V, before, clear, pad)
        count(tokens, None, V, before, clear, pad)


@pytest.mark.gpu
def test_count_tokens_many_of_one_and_outside():
    """More than 32767 times one token; tokens past the vocabulary."""
    zero = torch.zeros(2, 300, dtype=torch.int16, device="cuda")
    for clear in (True, False):
        for n in (40000, 32768, 32767):
            count(np.full((2, n), 5, np.int32), None, 300, zero, clear)
            count(np.full((2, n), 4, np.int32), np.array([1, n], np.int32), 300, zero, clear)
        few = np.array([[299, 300, 2, 2, 2], [1 << 30, -(1 << 31), 0, 0, 1]], np.int32)
        count(few, np.array([3, 9], np.int32), 300, zero, clear, expect=H.HSWA_ERR_BOUNDS)
    empty = torch.empty(2, 0, dtype=torch.int32, device="cuda")
    counts = torch.ones(2, 300, dtype=torch.int16, device="cuda")
    H.hswa_count_tokens(counts, 300, empty, 0, None, 2, 0, 300, False)
    assert (counts == 1).all()
    H.hswa_count_tokens(counts, 300, None, 0, None, 2, 0, 300, True)
    assert H.hswa_check() == 0 and not counts.any()


@pytest.mark.gpu
@pytest.mark.parametrize("V", [2, 8])
def test_probs_repetition_divides_as_fp32_does(V):
    """A token that occurred against one that has the fp32 quotient (or product)
    already: greedy rows with the one first and with the other first both
    choose the first exactly where the two are equal, infinities, subnormal
    values and zeros among them. (Rows of 2 are off the boundary, of 8 on it.)"""
    rng = np.random.default_rng(V)
    S = 60000
    a = (rng.uniform(1, 2, S) * 2.0 ** rng.integers(-149, 128, S)).astype(np.float32)
    a[::5] = rng.uniform(2e38, 3.4e38, len(a[::5]))
    a[::7] = np.ldexp(rng.integers(1, 1 << 23, len(a[::7])), -149)
    a[::11] *= -1
    a[:4] = np.finfo(np.float32).max, np.finfo(np.float32).tiny, 0, np.inf
    rep = rng.uniform(0.5, 2, S)
    rep[::13] = 2.0 ** rng.uniform(-120, 120, len(rep[::13]))
    rep = rep.astype(np.float32)
    with np.errstate(over="ignore", under="ignore"):
        b = np.where(a > 0, a / rep, a * rep).astype(np.float32)
    keep = b > -np.inf  # a row of nothing but -inf chooses none
    a, b, rep = a[keep], b[keep], rep[keep]
    assert (b == np.inf).sum() > 1000 and (np.abs(b) < np.finfo(np.float32).tiny).sum() > 1000
    S = len(a)
    params = np.stack((np.zeros(S), rep, np.zeros(S), np.zeros(S)), 1).astype(np.float32)
    for at in (0, 1):
        logits = np.full((S, 1, V), -np.inf, np.float32)
        logits[:, 0, at], logits[:, 0, 1 - at] = a, b
        counts = np.zeros((S, V), np.int16)
        counts[:, at] = 1
        x = torch.as_tensor(logits, device="cuda")
        p = run(x, torch.empty_like(x), torch.as_tensor(params, device="cuda"), torch.as_tensor(counts, device="cuda"))
        wrong = (p[:, 0, 0] != 1).cpu().numpy()
        assert not wrong.any(), (at, wrong.sum(), a[wrong][:5], rep[wrong][:5], b[wrong][:5])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [37, 30000, 400000])
def test_probs_of_quotients_past_the_largest_value(V, dtype):
    """Logits whose quotient by a repetition below 1 is +inf take the probability, in equal shares."""
    most = torch.finfo(dtype).max
    logits = torch.randn(6, 2, V, device="cuda").to(dtype)
    counts = torch.zeros(6, V, dtype=torch.int16, device="cuda")
    params = torch.tensor([[1.0, r, 0.3, -0.2] for r in (0.5, 0.6, 0.7, 0.8, 0.9, 0.99)], device="cuda")
    logits[:, :, 3] = most
    logits[:, 1, V - 1] = most
    counts[:, 3] = 2
    counts[:, V - 1] = -32768  # in the prompt
    want = torch.zeros(6, 2, V, device="cuda")
    want[:, 0, 3], want[:, 1, 3], want[:, 1, V - 1] = 1, 0.5, 0.5
    assert torch.equal(run(logits, torch.empty_like(want), params, counts), want)
    params[:, 0] = 0
    want[:, 1, 3], want[:, 1, V - 1] = 1, 0
    assert torch.equal(run(logits, torch.empty_like(want), params, counts), want)


@pytest.mark.gpu
@pytest.mark.parametrize("first", [0, 1, 2, 3])
@pytest.mark.parametrize("S,V,pad", [(1, 1, 0), (1, 2, 0), (1, 9, 0), (3, 17, 0), (3, 16, 0), (2, 33, 2), (5, 1000, 1), (5, 1001, 1)])
def test_count_tokens_in_an_array_between_others(S, V, pad, first):
    """Counts that begin and end within a 32-bit word: the array's own values
    only change, its first and last counts are often met, up to 32767."""
    rng = np.random.default_rng(S * V + first)
    size = (S - 1) * (V + pad) + V
    n = 700
    tokens = rng.choice([0, 0, V - 1, V - 1, V // 2, -1], (S, n)).astype(np.int32)
    prompt = rng.integers(0, 9, S).astype(np.int32)
    for start in (0, 32400, 32767):
        for clear in (True, False):
            store = torch.as_tensor(rng.integers(-(1 << 15), 1 << 15, first + size + 3).astype(np.int16), device="cuda")
            counts = store[first:first + size].as_strided((S, V), (V + pad, 1))
            counts.copy_(torch.as_tensor(np.where(rng.random((S, V)) < 0.5, start, 5).astype(np.int16)))
            mine = torch.zeros(first + size + 3, dtype=torch.bool, device="cuda")
            mine[first:first + size].as_strided((S, V), (V + pad, 1)).fill_(True)
            before = store.clone()
            want = serving.count_tokens(tokens, prompt, V, None if clear else counts.cpu().numpy().view(np.uint16))
            H.hswa_count_tokens(counts, V + pad, torch.as_tensor(tokens, device="cuda"), n, torch.as_tensor(prompt, device="cuda"), S, n, V, clear)
            assert H.hswa_check() == 0
            assert np.array_equal(counts.cpu().numpy().view(np.uint16), want)
            assert torch.equal(store[~mine], before[~mine])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("S,n,V", [(80, 1, 50021), (40, 2, 131071), (170, 1, 9999)])
def test_probs_of_odd_vocabularies_in_batches(S, n, V, dtype):
    """Rows off every boundary, more of them than an SM each."""
    logits, params, counts, draft, bt, bias, allowed = inputs(S, n, V, dtype, seed=S + n)
    p = torch.full(logits.shape, float("nan"), device="cuda")
    check(run(logits, p, params, counts, draft, bt, bias, bits(allowed)), logits, params, counts, draft, bt, bias, allowed)


@pytest.mark.gpu
@pytest.mark.parametrize("V", [1003, 30001, 400001, 400000])
def test_probs_in_place_of_long_rows(V):
    """p is the logits: rows in registers and rows read three times, on and off a boundary."""
    for dtype in CODE:
        logits, params, counts, draft, bt, bias, allowed = inputs(3, 2, V, dtype, seed=V)
        apart = run(logits, torch.empty_like(logits), params, counts, draft, bt, bias, bits(allowed))
        same = logits.clone()
        run(same, same, params, counts, draft, bt, bias, bits(allowed))
        assert torch.equal(same, apart)
