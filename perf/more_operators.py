"""A KV cache in 4 bits and the step from logits to probabilities, as cases that can be timed.

Four operators:
  decode   attention of 1 to 4 query tokens per sequence over pools held in 4 bits (hswa_decode, hswa_decode_multi on HSWA_DTYPE_FP4 pools)
  store    K and V rows quantized into their slots, and those slots read back as values (hswa_append_kv, hswa_read_kv)
  probs    logits to the probabilities that the verification takes: penalties, biases, grammar masks, temperature (hswa_logits_probs)
  count    how often each token occurs in each sequence, which the penalties need (hswa_count_tokens)

The 4-bit format: blocks of 16 elements of a row share one scale, a byte of 5 exponent and 3 mantissa bits (a 16-bit float without its sign and
its last 7 bits); an element is a 4-bit code of sign, 2 exponent and 1 mantissa bit (0, 0.5, 1, 1.5, 2, 3, 4, 6), element 2 i in the lower half of byte i.

With `own` false, run() computes them with elementary torch operations; with `own` true it makes the library's calls.
"""
import math

import numpy as np
import torch

own = False

TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}
CODE = {"f32": 0, "bf16": 1, "fp4": 3}
BLOCK = 16
VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a short conversation or two: one Full layer, where latency counts
        dict(name="decode_few", op="decode", seqs=3, lo=700, hi=2500, n_tok=1, window=0, hq=64, hkv=8, d=128, page=64),
        # the decode batch: 64 sequences of 1K to 32K tokens
        dict(name="decode_batch", op="decode", seqs=64, lo=1024, hi=32768, n_tok=1, window=0, hq=64, hkv=8, d=128, page=64),
        # two contexts of some hundred thousand tokens
        dict(name="decode_long", op="decode", seqs=2, lo=200003, hi=300007, n_tok=1, window=0, hq=64, hkv=8, d=128, page=64),
        # the decode batch with three drafts each to verify
        dict(name="decode_verify", op="decode", seqs=64, lo=1024, hi=32768, n_tok=4, window=0, hq=64, hkv=8, d=128, page=64),
        # one new token of each of 64 sequences: latency
        dict(name="store_step", op="store", tokens=64, run=1, hkv=8, d=128, page=64),
        # a chunked-prefill chunk: 8 sequences of 4096 new tokens
        dict(name="store_chunk", op="store", tokens=32768, run=4096, hkv=8, d=128, page=64),
        # a ragged chunk of smaller heads on small pages
        dict(name="store_odd", op="store", tokens=9999, run=1111, hkv=4, d=96, page=16),
        # one sequence with three drafts, an odd vocabulary, every penalty: latency
        dict(name="probs_one", op="probs", seqs=1, n_tok=4, vocab=100003, dtype="f32", out="f32", counts=True, bias=16, mask="none"),
        # the decode batch with three drafts each, 16-bit logits, penalties
        dict(name="probs_batch", op="probs", seqs=64, n_tok=4, vocab=150000, dtype="bf16", out="f32", counts=True, bias=0, mask="none"),
        # a large batch under grammars, with penalties and biases
        dict(name="probs_grammar", op="probs", seqs=256, n_tok=1, vocab=131000, dtype="f32", out="f32", counts=True, bias=100, mask="grammar"),
        # 8 requests of up to 32K tokens admitted: their counts from nothing
        dict(name="count_admit", op="count", seqs=8, lo=501, hi=32768, vocab=131000),
        # a batch of short requests admitted
        dict(name="count_batch", op="count", seqs=64, lo=1, hi=2048, vocab=150000),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "store", "probs", "count"])
    if op == "decode":
        if rng.random() < 0.2:  # the small configuration: 4 query heads on one kv head, d 64, pages of 16
            lo = _log_int(rng, 1, 1000)
            return dict(op=op, seqs=_log_int(rng, 1, 16), lo=lo, hi=lo + _log_int(rng, 1, 1000), n_tok=rng.randint(1, 4), window=rng.choice([0, 128]), hq=4, hkv=1, d=64, page=16)
        lo, hkv = _log_int(rng, 1, 8192), rng.choice([1, 4, 8])
        return dict(op=op, seqs=_log_int(rng, 1, 64), lo=lo, hi=lo + _log_int(rng, 1, 16384), n_tok=rng.choice([1, 1, 2, 3, 4]), window=rng.choice([0, 0, 0, 128]), hq=8 * hkv, hkv=hkv, d=128, page=64)
    if op == "store":
        tokens = _log_int(rng, 1, 32768)
        return dict(op=op, tokens=tokens, run=rng.choice([1 if tokens <= 2048 else 16, max(1, tokens // 8), tokens]), hkv=rng.choice([1, 2, 4, 8]), d=rng.choice([64, 96, 128]), page=rng.choice([16, 64]))
    if op == "probs":
        return dict(op=op, seqs=_log_int(rng, 1, 64), n_tok=rng.randint(1, 4), vocab=_log_int(rng, 1000, 150000), dtype=rng.choice(["f32", "bf16"]), out=rng.choice(["f32", "f32", "bf16"]),
                    counts=rng.random() < 0.75, bias=rng.choice([0, 7, 300]), mask=rng.choice(["none", "few", "grammar"]))
    lo = _log_int(rng, 1, 16384)
    return dict(op=op, seqs=_log_int(rng, 1, 32), lo=lo, hi=lo + _log_int(rng, 1, 16384), vocab=_log_int(rng, 1000, 150000))


# ----------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _i32(a):
    return torch.as_tensor(np.ascontiguousarray(a, np.int32), device="cuda")


def _lengths(case):
    """The lengths of a case, evenly spread from lo to hi."""
    return np.rint(np.linspace(case["lo"], case["hi"], case["seqs"])).astype(np.int64)


def _scale_of(quotient):
    """The nearest scale to each value (ties to the even one), as a value: 4 significant bits, steps of 2^-17 below 2^-14, at most 10240."""
    x = quotient.clamp(max=10240)
    m, e = torch.frexp(x)
    return torch.where(x < 2.0 ** -14, torch.round(x * 2.0 ** 17) * 2.0 ** -17, torch.ldexp(torch.round(m * 16), e - 4))


def _quantize(x):
    """Blocks of 16 fp32 values [..., d] as (codes [..., d / 2], scales [..., d / 16]), both bytes."""
    x = x.unflatten(-1, (-1, BLOCK))
    top = x.abs().amax(-1)
    s = _scale_of(top / torch.full_like(top, 6))  # a division, as a product with 1 / 6 would be rounded twice
    q = x.abs() / torch.where(s > 0, s, torch.ones_like(s))[..., None]
    code = (q > 0.25).byte() + (q >= 0.75) + (q > 1.25) + (q >= 1.75) + (q > 2.5) + (q >= 3.5) + (q > 5)
    code = torch.where((s > 0)[..., None], code + 8 * torch.signbit(x).byte(), torch.zeros_like(code)).flatten(-2)
    return code[..., 0::2] + 16 * code[..., 1::2], (s.half().view(torch.int16) >> 7).byte()


def _values(codes, scales, dtype):
    """The values of codes [..., d / 2] under scales [..., d / 16]."""
    table = torch.tensor(VALUES, dtype=dtype, device="cuda")
    x = torch.stack((table[(codes & 15).int()], table[(codes >> 4).int()]), -1).flatten(-2)
    s = (scales.to(torch.int16) << 7).view(torch.float16).to(dtype)
    return (x.unflatten(-1, (-1, BLOCK)) * s[..., None]).flatten(-2)


def _config(case, H, **over):
    c = dict(window=128, page_size=case["page"], n_q_heads=case.get("hq", case["hkv"]), n_kv_heads=case["hkv"], head_dim=case["d"], dtype=CODE["fp4"],
             full_pages=1, swa_pages=1, max_seqs=1, max_pages_per_seq=1)
    c.update(over)
    return H.Config(**c)


def _layer(s, H, window=0):
    return H.Layer(kind=H.HSWA_KIND_SWA if window else H.HSWA_KIND_FULL, window=window, k_pool=s["k_pool"].data_ptr(), v_pool=s["v_pool"].data_ptr(),
                   k_scale=s["k_scale"].data_ptr(), v_scale=s["v_scale"].data_ptr())


def prepare(case, seed):
    return {"decode": _prepare_decode, "store": _prepare_store, "probs": _prepare_probs, "count": _prepare_count}[case["op"]](case, seed)


def _prepare_decode(case, seed):
    g, rng = _gen(seed), np.random.default_rng(seed)
    n, t, hq, hkv, d, P, W = (case[x] for x in ("seqs", "n_tok", "hq", "hkv", "d", "page", "window"))
    lens = rng.permutation(_lengths(case))
    npg = -(-lens // P)
    first = np.maximum(0, lens - t + 1 - W) // P if W else np.zeros(n, np.int64)  # pages before it have left the window
    pages, mp = int((npg - first).sum()), int(npg.max())
    perm, bt, at = rng.permutation(pages), np.full((n, mp), -1, np.int64), 0
    for i in range(n):
        m = npg[i] - first[i]
        bt[i, first[i]:npg[i]] = perm[at:at + m]
        at += m
    s = dict(case=case, bt=_i32(bt), lens=_i32(lens), q=torch.randn(n * t, hq, d, generator=g, device="cuda", dtype=torch.bfloat16),
             o=torch.empty(n * t, hq, d, dtype=torch.bfloat16, device="cuda"), scale=1 / math.sqrt(d))
    for which in ("k", "v"):
        codes = torch.empty(pages, hkv, P, d // 2, dtype=torch.uint8, device="cuda")
        scales = torch.empty(pages, hkv, P, d // BLOCK, dtype=torch.uint8, device="cuda")
        step = max(1, (1 << 26) // (hkv * P * d))
        for i in range(0, pages, step):
            m = min(step, pages - i)
            codes[i:i + m], scales[i:i + m] = _quantize(torch.randn(m, hkv, P, d, generator=g, device="cuda"))
        s[which + "_pool"], s[which + "_scale"] = codes, scales
    if own:
        import hybrid_sliding_window_dual_gb300 as H
        s["H"] = H
        s["pool"] = H.hswa_pool_create(_config(case, H, full_pages=pages, swa_pages=pages, max_seqs=n, max_pages_per_seq=mp))
        s["layer"] = _layer(s, H, W)
        s["ws"] = torch.empty(H.hswa_decode_multi_workspace_size(s["pool"], n, t), dtype=torch.uint8, device="cuda")
    return s


def _prepare_store(case, seed):
    g, rng = _gen(seed), np.random.default_rng(seed)
    n, hkv, d, P, run_ = case["tokens"], case["hkv"], case["d"], case["page"], case["run"]
    # rows as projections leave them: K with a few channels much larger than the others
    k = torch.randn(n, hkv, d, generator=g, device="cuda") * (1 + 15 * (torch.rand(hkv, d, generator=g, device="cuda") < 0.04))
    v = torch.randn(n, hkv, d, generator=g, device="cuda") * 0.3
    starts, pages = [], 0
    for at in range(0, n, run_):  # runs of consecutive tokens of a sequence, each starting anywhere on its first page
        m = min(run_, n - at)
        starts.append((at, m, int(rng.integers(0, P)), pages))
        pages += -(-(P - 1 + m) // P)  # enough wherever it starts
    perm, slots = rng.permutation(pages), np.empty(n, np.int64)
    for at, m, off, page in starts:
        t = off + np.arange(m)
        slots[at:at + m] = perm[page + t // P] * P + t % P
    s = dict(case=case, k=k.bfloat16(), v=v.bfloat16(), slots=_i32(slots))
    for which in ("k", "v"):
        s[which + "_pool"] = torch.zeros(pages, hkv, P, d // 2, dtype=torch.uint8, device="cuda")
        s[which + "_scale"] = torch.zeros(pages, hkv, P, d // BLOCK, dtype=torch.uint8, device="cuda")
        s[which + "_out"] = torch.empty(n, hkv, d, dtype=torch.bfloat16, device="cuda")
    if own:
        import hybrid_sliding_window_dual_gb300 as H
        s["H"] = H
        s["pool"] = H.hswa_pool_create(_config(case, H, full_pages=pages))
        s["layer"] = _layer(s, H)
    return s


def _tokens(g, shape, vocab):
    """Tokens as texts have them: a few of them often."""
    x = torch.exp(torch.rand(shape, generator=g, device="cuda") * math.log(vocab)) - 1
    return (x.long() * 7919 % vocab).int()


def _prepare_probs(case, seed):
    g, rng = _gen(seed), np.random.default_rng(seed)
    n, t, V = case["seqs"], case["n_tok"], case["vocab"]
    s = dict(case=case, logits=(torch.randn(n, t, V, generator=g, device="cuda") * 3 - 1).to(TORCH[case["dtype"]]), p=torch.empty(n, t, V, dtype=TORCH[case["out"]], device="cuda"),
             counts=None, draft=_tokens(g, (n, t - 1), V) if t > 1 else None, bias_token=None, bias=None, mask=None)
    temperature = rng.uniform(0.6, 1.3, n)
    temperature[rng.random(n) < 0.1] = 0  # some requests are greedy
    s["params"] = torch.as_tensor(np.stack((temperature, rng.uniform(1.0, 1.3, n), rng.uniform(0, 0.5, n), rng.uniform(0, 0.5, n)), 1).astype(np.float32), device="cuda")
    if case["counts"]:
        counts = torch.zeros(n, V, device="cuda").scatter_add_(1, _tokens(g, (n, 700), V).long(), torch.ones(n, 700, device="cuda")).int()
        prompt = torch.zeros(n, V, dtype=torch.int32, device="cuda").scatter_(1, _tokens(g, (n, 2000), V).long(), 1)
        s["counts"] = (counts - 32768 * prompt).to(torch.int16)
    if case["bias"]:  # distinct tokens, the lists of some sequences shorter
        s["bias_token"] = torch.argsort(torch.rand(n, min(V, 8192), generator=g, device="cuda"), 1)[:, :case["bias"]].int() * (V // min(V, 8192))
        s["bias_token"] = torch.where(torch.rand(n, 1, generator=g, device="cuda") * case["bias"] < torch.arange(case["bias"], device="cuda"), -1, s["bias_token"]).int().contiguous()
        s["bias"] = torch.randn(n, case["bias"], generator=g, device="cuda") * 4
    if case["mask"] != "none":  # bits of allowed tokens: nearly all, or what a grammar leaves
        share = torch.full((n * t, 1), 0.98, device="cuda") if case["mask"] == "few" else torch.exp(torch.rand(n * t, 1, generator=g, device="cuda") * math.log(2e-4))
        words, bits = -(-V // 32), torch.arange(32, device="cuda")
        mask = torch.zeros(n * t, words, dtype=torch.int64, device="cuda")
        for i in range(0, n * t, 64):
            on = torch.rand(min(64, n * t - i), words, 32, generator=g, device="cuda") < share[i:i + 64, :, None]
            mask[i:i + 64] = (on.long() << bits).sum(-1)
        s["mask"] = torch.where(mask >= 1 << 31, mask - (1 << 32), mask).int()
    if own:
        import hybrid_sliding_window_dual_gb300 as H
        s["H"] = H
    return s


def _prepare_count(case, seed):
    g, rng = _gen(seed), np.random.default_rng(seed)
    n, V = case["seqs"], case["vocab"]
    lens = rng.permutation(_lengths(case))
    width = int(lens.max())
    tokens = torch.where(torch.arange(width, device="cuda") < torch.as_tensor(lens, device="cuda")[:, None], _tokens(g, (n, width), V), -1).int()
    s = dict(case=case, tokens=tokens, n_prompt=_i32(np.rint(lens * rng.uniform(0.3, 1.0, n))), counts=torch.empty(n, V, dtype=torch.int16, device="cuda"))
    if own:
        import hybrid_sliding_window_dual_gb300 as H
        s["H"] = H
    return s


# -------------------------------------------------------------------- run
def run(s):
    if own:
        return _own(s)
    return {"decode": _plain_decode, "store": _plain_store, "probs": _plain_probs, "count": _plain_count}[s["case"]["op"]](s)


def _own(s):
    H, c = s["H"], s["case"]  # on the default stream, as a session's calls are
    if c["op"] == "decode":
        if c["n_tok"] == 1:
            H.hswa_decode(s["pool"], s["layer"], s["q"], s["o"], s["bt"], s["lens"], c["seqs"], s["scale"], s["ws"], s["ws"].numel())
        else:
            H.hswa_decode_multi(s["pool"], s["layer"], s["q"], s["o"], s["bt"], s["lens"], c["seqs"], c["n_tok"], s["scale"], s["ws"], s["ws"].numel())
        return s["o"]
    if c["op"] == "store":
        H.hswa_append_kv(s["pool"], s["layer"], s["k"], s["v"], s["slots"], c["tokens"])
        H.hswa_read_kv(s["pool"], s["layer"], s["slots"], c["tokens"], s["k_out"], s["v_out"])
        return dict(k=s["k_out"], v=s["v_out"])
    if c["op"] == "probs":
        V = c["vocab"]
        H.hswa_logits_probs(CODE[c["dtype"]], s["logits"], V, CODE[c["out"]], s["p"], V, s["params"], s["counts"], V, s["draft"], s["bias_token"], s["bias"], c["bias"],
                            s["mask"], -(-V // 32), c["seqs"], c["n_tok"], V)
        return s["p"]
    H.hswa_count_tokens(s["counts"], c["vocab"], s["tokens"], s["tokens"].shape[1], s["n_prompt"], c["seqs"], s["tokens"].shape[1], c["vocab"], True)
    return s["counts"]


def _plain_decode(s):
    c = s["case"]
    n, t, hq, hkv, d, P = (c[x] for x in ("seqs", "n_tok", "hq", "hkv", "d", "page"))
    table, mp = s["bt"].long().clamp(min=0), s["bt"].shape[1]
    q = s["q"].float().view(n, 1, t, hkv, hq // hkv, d).transpose(2, 3).reshape(n, 1, hkv, -1, d)  # rows of a kv head: token, query head
    scores = torch.matmul(q, _values(s["k_pool"][table], s["k_scale"][table], torch.float32).transpose(-1, -2)) * s["scale"]  # [n][mp][hkv][t G][P]
    scores = scores.view(n, mp, hkv, t, -1, P)
    key = torch.arange(mp * P, device="cuda").view(1, mp, 1, 1, 1, P)
    at = s["lens"].view(n, 1, 1, 1, 1, 1) - t + torch.arange(t, device="cuda").view(1, 1, 1, t, 1, 1)
    seen = key <= at
    if c["window"]:
        seen = seen & (key > at - c["window"])
    scores = scores.masked_fill(~seen, -math.inf)
    top = scores.amax((1, 5), keepdim=True)
    e = torch.exp(scores - torch.where(top > -math.inf, top, torch.zeros_like(top)))
    total = e.sum((1, 5), keepdim=True)
    e = (e / torch.where(total > 0, total, torch.ones_like(total))).view(n, mp, hkv, -1, P)
    o = torch.matmul(e, _values(s["v_pool"][table], s["v_scale"][table], torch.float32)).sum(1)
    s["o"].copy_(o.view(n, hkv, t, -1, d).transpose(1, 2).reshape(n * t, hq, d))
    return s["o"]


def _plain_store(s):
    P = s["case"]["page"]
    slots = s["slots"].long()
    page, row = slots // P, slots % P
    for which in ("k", "v"):
        codes, scales = _quantize(s[which].float())
        s[which + "_pool"][page, :, row] = codes
        s[which + "_scale"][page, :, row] = scales
    for which in ("k", "v"):
        s[which + "_out"].copy_(_values(s[which + "_pool"][page, :, row], s[which + "_scale"][page, :, row], torch.float32))
    return dict(k=s["k_out"], v=s["v_out"])


def _allowed(mask, V):
    v = torch.arange(V, device="cuda")
    return (mask[:, v // 32] >> (v % 32).int()) & 1 > 0


def _plain_probs(s):
    c = s["case"]
    n, t, V = c["seqs"], c["n_tok"], c["vocab"]
    z = s["logits"].float()
    temperature, repetition, frequency, presence = (s["params"][:, i].view(n, 1, 1) for i in range(4))
    if s["counts"] is not None:
        times = (s["counts"].int() & 0x7fff).float()[:, None].expand(n, t, V)
        if t > 1:  # the drafts before a row's own token have been generated, as far as that row goes
            before = (torch.arange(t - 1, device="cuda")[None] < torch.arange(t, device="cuda")[:, None]).float().expand(n, t, t - 1)
            times = times.clone().scatter_add_(2, s["draft"].long()[:, None].expand(n, t, t - 1), before.contiguous())
        seen = (times > 0) | (s["counts"] < 0)[:, None]
        z = torch.where(seen, torch.where(z > 0, z / repetition, z * repetition), z)
        z = z - frequency * times
        z = torch.where(times > 0, z - presence, z)
    if s["bias"] is not None:
        to = torch.where(s["bias_token"] >= 0, s["bias_token"], V).long()
        z = z + torch.zeros(n, V + 1, device="cuda").scatter_(1, to, s["bias"])[:, None, :V]
    if s["mask"] is not None:
        z = torch.where(_allowed(s["mask"], V).view(n, t, V), z, torch.full_like(z, -math.inf))
    top = z.amax(2, keepdim=True)
    there = top > -math.inf
    warm = torch.where(temperature > 0, temperature, torch.ones_like(temperature))
    e = torch.exp((z - torch.where(there, top, torch.zeros_like(top))) / warm)
    total = e.sum(2, keepdim=True)
    p = e / torch.where(there, total, torch.ones_like(total))
    greedy = (torch.arange(V, device="cuda") == z.argmax(2, keepdim=True)) & there
    s["p"].copy_(torch.where(temperature > 0, p, greedy.float()))
    return s["p"]


def _plain_count(s):
    V = s["case"]["vocab"]
    tokens = s["tokens"].long()
    n, width = tokens.shape
    prompt = torch.arange(width, device="cuda")[None] < s["n_prompt"][:, None]
    to = torch.where(tokens >= 0, tokens, V)
    times = torch.zeros(n, V + 1, dtype=torch.int32, device="cuda").scatter_add_(1, torch.where(prompt, V, to), torch.ones_like(tokens, dtype=torch.int32))[:, :V].clamp(max=32767)
    inside = torch.zeros(n, V + 1, dtype=torch.int32, device="cuda").scatter_(1, torch.where(prompt, to, V), 1)[:, :V]
    s["counts"].copy_(times - 32768 * inside)
    return s["counts"]


# ------------------------------------------------------------------- work
def work(case):
    if case["op"] == "decode":
        n, t, hq, hkv, d, P, W = (case[x] for x in ("seqs", "n_tok", "hq", "hkv", "d", "page", "window"))
        lens = _lengths(case)
        keys = int(np.minimum(lens, W + t - 1).sum() if W else lens.sum())
        return {"bytes": keys * 2 * hkv * (d // 2 + d // BLOCK) + 2 * n * t * hq * d * 2 + keys // P * 4, "flops": keys * 4 * hq * d * t}
    if case["op"] == "store":
        n, hkv, d = case["tokens"], case["hkv"], case["d"]
        return {"bytes": n * 2 * hkv * (2 * d + 2 * (d // 2 + d // BLOCK) + 2 * d), "flops": n * 2 * hkv * d * 3}
    if case["op"] == "probs":
        n, t, V = case["seqs"], case["n_tok"], case["vocab"]
        size = {"f32": 4, "bf16": 2}
        b = n * t * V * (size[case["dtype"]] + size[case["out"]]) + (n * V * 2 if case["counts"] else 0) + (n * t * V // 8 if case["mask"] != "none" else 0) + n * case["bias"] * 8
        return {"bytes": b, "flops": n * t * V * 6}
    lens = _lengths(case)
    return {"bytes": int(lens.sum()) * 4 + case["seqs"] * case["vocab"] * 2, "flops": int(lens.sum())}


# ------------------------------------------------------------------ exact
def exact(case, seed):
    s = prepare(case, seed)
    return {"decode": _exact_decode, "store": _exact_store, "probs": _exact_probs, "count": _exact_count}[case["op"]](s)


def _exact_decode(s):
    """One sequence after another, its keys in a row."""
    c = s["case"]
    t, hq, hkv, d, P, W = (c[x] for x in ("n_tok", "hq", "hkv", "d", "page", "window"))
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for i, L in enumerate(s["lens"].tolist()):
        first = max(0, L - t + 1 - W) // P if W else 0
        table = s["bt"][i, first:-(-L // P)].long()
        k, v = (_unpacked(s[x + "_pool"][table], s[x + "_scale"][table]).transpose(0, 1).reshape(hkv, -1, d)[:, :L - first * P] for x in ("k", "v"))
        for w in range(t):
            at = L - t + w
            lo = max(0, at - W + 1) if W else 0
            if at < 0:
                continue
            kw, vw = k[:, lo - first * P:at + 1 - first * P], v[:, lo - first * P:at + 1 - first * P]
            prob = torch.softmax(torch.einsum("ghd,gkd->ghk", s["q"][i * t + w].double().view(hkv, -1, d), kw) * s["scale"], -1)
            o[i * t + w] = torch.einsum("ghk,gkd->ghd", prob, vw).reshape(hq, d)
    return o


def _scales():
    """The value of each scale byte in 64 bits, from its fields (powers by the host, whose are exact)."""
    return torch.tensor([math.ldexp(b if b < 8 else 8 + b % 8, max(b // 8, 1) - 18) for b in range(256)], dtype=torch.float64, device="cuda")


def _unpacked(codes, scales):
    """Values in 64 bits from the fields of the codes and of the scales."""
    c = torch.stack((codes % 16, codes // 16), -1).flatten(-2).to(torch.int64)
    sign, e, m = 1.0 - 2.0 * (c // 8), c // 2 % 4, c % 2
    x = sign * torch.where(e == 0, m, (2 + m) << (e - 1).clamp(min=0)) / 2
    return x * _scales()[scales.int()].repeat_interleave(BLOCK, -1)


def _exact_store(s):
    """Each value the nearest of the sixteen that its block's scale allows, that scale the nearest one to a sixth of the largest."""
    every = _scales()[:0xE2 + 1]  # up to 10240
    steps = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")

    def nearest(x, table):  # the even index of two that are equally near
        hi = torch.searchsorted(table, x.contiguous()).clamp(1, table.numel() - 1)
        lo = hi - 1
        below, above = x - table[lo], table[hi] - x
        return torch.where((above < below) | ((above == below) & (hi % 2 == 0)), hi, lo)

    out = {}
    for which in ("k", "v"):
        x = s[which].double().unflatten(-1, (-1, BLOCK))
        scale = every[nearest(x.abs().amax(-1) / 6, every)][..., None]
        y = steps[nearest((x.abs() / torch.where(scale > 0, scale, torch.ones_like(scale))), steps)] * scale
        out[which] = (torch.sign(x) * y).flatten(-2)
    return out


def _exact_probs(s):
    """One row after another."""
    c = s["case"]
    n, t, V = c["seqs"], c["n_tok"], c["vocab"]
    p = torch.zeros(n, t, V, dtype=torch.float64, device="cuda")
    params = s["params"].double().tolist()
    v = torch.arange(V, device="cuda")
    for i in range(n):
        T, rep, freq, pres = params[i]
        for w in range(t):
            z = s["logits"][i, w].double()
            if s["counts"] is not None:
                times = (s["counts"][i].int() & 0x7fff).double()
                if w:
                    times = times + torch.bincount(s["draft"][i, :w].long(), minlength=V)
                seen = (times > 0) | (s["counts"][i] < 0)
                z = torch.where(seen & (z > 0), z / rep, torch.where(seen, z * rep, z)) - freq * times - pres * (times > 0)
            if s["bias"] is not None:
                use = s["bias_token"][i] >= 0
                z = z.index_add(0, s["bias_token"][i][use].long(), s["bias"][i][use].double())
            if s["mask"] is not None:
                bits = torch.remainder(s["mask"][i * t + w].long(), 1 << 32)
                z = torch.where(bits[v // 32] // 2 ** (v % 32) % 2 == 1, z, torch.full_like(z, -math.inf))
            if not torch.isfinite(z.max()):
                continue
            if T > 0:
                p[i, w] = torch.softmax(z / T, 0)
            else:
                p[i, w, int(torch.nonzero(z == z.max())[0])] = 1
    return p


def _exact_count(s):
    """By hand, one sequence after another."""
    V = s["case"]["vocab"]
    tokens, n_prompt = s["tokens"].cpu().numpy(), s["n_prompt"].tolist()
    out = np.zeros((len(n_prompt), V), np.int64)
    for i, m in enumerate(n_prompt):
        later = tokens[i, m:]
        out[i] = np.minimum(np.bincount(later[later >= 0], minlength=V), 32767)
        before = tokens[i, :m]
        out[i, before[before >= 0]] -= 32768
    return torch.as_tensor(out.astype(np.int16))
