"""The operators of a serving step around the dual KV pool, as cases that can be timed.

Four operators:
  rope     rotary positions with several axes on q and k, K and V written to their pool slots (hswa_rope_append)
  weights  one decode step of a Full layer that also accumulates each page's attention weight (hswa_decode_weights)
  select   which pages of each sequence stay under a budget, by accumulated weight (hswa_evict_select)
  verify   drafted tokens against the target's probabilities, from given random numbers (hswa_verify_draft)

With `own` false, run() computes them with elementary torch operations; with `own` true it makes the library's calls.
"""
import math

import numpy as np
import torch

own = False

WINDOW = 128
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}
CODE = {"f32": 0, "bf16": 1, "fp8": 2}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one new token of each of 64 sequences: the rotary step of a decode step, where latency counts
        dict(name="rope_decode", op="rope", tokens=64, run=1, hq=64, hkv=8, d=128, page=64, dtype="bf16", rotary=128, axes=3, interleaved=False, adjacent=False, packed=True),
        # a chunked-prefill chunk: 8 sequences of 4096 new tokens, text and images
        dict(name="rope_chunk", op="rope", tokens=32768, run=4096, hq=64, hkv=8, d=128, page=64, dtype="bf16", rotary=128, axes=3, interleaved=True, adjacent=False, packed=True),
        # the same over an FP8 pool, ragged, half of each head rotated
        dict(name="rope_chunk_fp8", op="rope", tokens=9999, run=1111, hq=64, hkv=8, d=128, page=64, dtype="fp8", rotary=64, axes=3, interleaved=False, adjacent=True, packed=False),
        # a short conversation or two: one Full layer, latency
        dict(name="weights_few", op="weights", seqs=3, lo=700, hi=2500, hq=64, hkv=8, d=128, page=64, dtype="bf16"),
        # the decode batch: 64 sequences of 1K to 32K tokens
        dict(name="weights_batch", op="weights", seqs=64, lo=1024, hi=32768, hq=64, hkv=8, d=128, page=64, dtype="bf16"),
        # the same over FP8 pools, an odd number of sequences
        dict(name="weights_batch_fp8", op="weights", seqs=49, lo=1001, hi=32700, hq=64, hkv=8, d=128, page=64, dtype="fp8"),
        # a decode batch that gives back half of its pages
        dict(name="select_batch", op="select", seqs=64, lo=17, hi=512, page=64, sink=1, keep=0.5),
        # 128 sequences of up to 128K tokens, an eighth kept
        dict(name="select_long", op="select", seqs=128, lo=300, hi=2048, page=64, sink=4, keep=0.125),
        # a few contexts of up to a million tokens
        dict(name="select_million", op="select", seqs=5, lo=4001, hi=16384, page=64, sink=1, keep=0.25),
        # one sequence with three drafts, an odd vocabulary: latency
        dict(name="verify_one", op="verify", seqs=1, n_tok=4, vocab=100003, dtype="f32", draft="sampled"),
        # the decode batch with three drafts each
        dict(name="verify_batch", op="verify", seqs=64, n_tok=4, vocab=150000, dtype="f32", draft="sampled"),
        # a large batch with 7 drafts each taken greedily (no draft probabilities), 16-bit probabilities
        dict(name="verify_greedy", op="verify", seqs=256, n_tok=8, vocab=131000, dtype="bf16", draft="greedy"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "weights", "select", "verify"])
    if op == "rope":
        tokens = _log_int(rng, 1, 32768)
        dtype = rng.choice(["bf16", "bf16", "fp8", "f32"])
        d = 128 if dtype == "fp8" else rng.choice([64, 128])
        hkv = rng.choice([1, 2, 4, 8])
        axes = rng.choice([1, 2, 3])
        return dict(op=op, tokens=tokens, run=rng.choice([1 if tokens <= 2048 else 16, max(1, tokens // 8), tokens]), hq=8 * hkv, hkv=hkv, d=d, page=rng.choice([16, 64]), dtype=dtype,
                    rotary=rng.choice([d, d // 2]), axes=axes, interleaved=rng.random() < 0.5, adjacent=rng.random() < 0.5, packed=rng.random() < 0.5)
    if op == "weights":
        dtype = rng.choice(["bf16", "bf16", "fp8", "f32"])
        if dtype == "f32":  # the small configuration: 4 query heads on one kv head, d 64, pages of 16
            lo = _log_int(rng, 1, 1000)
            return dict(op=op, seqs=_log_int(rng, 1, 16), lo=lo, hi=lo + _log_int(rng, 1, 1000), hq=4, hkv=1, d=64, page=16, dtype=dtype)
        lo = _log_int(rng, 1, 8192)
        hkv = rng.choice([1, 4, 8])
        return dict(op=op, seqs=_log_int(rng, 1, 64), lo=lo, hi=lo + _log_int(rng, 1, 16384), hq=8 * hkv, hkv=hkv, d=128, page=64, dtype=dtype)
    if op == "select":
        lo = _log_int(rng, 1, 4000)
        return dict(op=op, seqs=_log_int(rng, 1, 128), lo=lo, hi=lo + _log_int(rng, 1, 4000), page=rng.choice([16, 64]), sink=rng.randint(0, 8), keep=round(rng.uniform(0.02, 0.95), 4))
    return dict(op=op, seqs=_log_int(rng, 1, 256), n_tok=rng.randint(1, 8), vocab=_log_int(rng, 1000, 150000), dtype=rng.choice(["f32", "f32", "bf16"]),
                draft=rng.choice(["sampled", "greedy"]))


# ----------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32 if dtype != "bf16" else torch.bfloat16).to(TORCH.get(dtype, torch.bfloat16))


def _codes(g, shape):
    """E4M3 codes of normal values at the scale a quantizer gives them (amax of a row near 448)."""
    flat = torch.empty(math.prod(shape), dtype=torch.uint8, device="cuda")
    for i in range(0, flat.numel(), 1 << 28):
        part = flat[i:i + (1 << 28)]
        part.copy_((torch.randn(part.numel(), generator=g, device="cuda", dtype=torch.bfloat16) * 150).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
    return flat.view(shape)


def _i32(a):
    return torch.as_tensor(np.ascontiguousarray(a, np.int32), device="cuda")


def _lengths(case):
    """The sequence lengths (or page counts) of a case, evenly spread from lo to hi."""
    return np.rint(np.linspace(case["lo"], case["hi"], case["seqs"])).astype(np.int64)


def _sections(case):
    """Pairs of each axis: half of the pairs for time, the rest shared by height and width."""
    half, axes = case["rotary"] // 2, case["axes"]
    if axes == 1:
        return [half]
    rest = (half // 2) // (axes - 1)
    return [half - rest * (axes - 1)] + [rest] * (axes - 1)


def _axis_of_pair(case):
    sec, half, axes = _sections(case), case["rotary"] // 2, case["axes"]
    if not case["interleaved"]:
        return np.repeat(np.arange(axes), sec)
    i = np.arange(half)
    axis = i % axes
    return np.where(i // axes < np.array(sec)[axis], axis, 0)


def _positions(case, rng):
    """[axes][tokens]: each run of tokens starts at a position up to a million; stretches of text (the same position on every axis) and images (time fixed, rows and columns)."""
    axes, n, pos, at = case["axes"], case["tokens"], [], 0
    out = np.empty((axes, n), np.int64)
    while at < n:
        p = int(np.exp(rng.uniform(0, np.log(1 << 20))))
        end = min(n, at + case["run"])
        while at < end:
            m = min(end - at, int(rng.integers(1, 400)))
            out[:, at:at + m] = p + np.arange(m)
            p += m
            at += m
            if at < end and axes > 1:  # an image of w columns
                w = int(rng.integers(4, 32))
                m = min(end - at, w * int(rng.integers(4, 32)))
                i = np.arange(m)
                out[:, at:at + m] = p
                out[-1, at:at + m] = p + i % w
                if axes > 2:
                    out[1, at:at + m] = p + i // w
                p += 32
                at += m
    return out


def _slots(case, rng):
    """Slots of the tokens: runs of consecutive tokens of a sequence on pages in random order, each run starting anywhere on its first page; and the pages of the pool."""
    n, run, P = case["tokens"], case["run"], case["page"]
    starts, pages = [], 0
    for at in range(0, n, run):
        off = int(rng.integers(0, P))
        starts.append((at, min(n, at + run), off, pages))
        pages += -(-(P - 1 + min(n, at + run) - at) // P)  # enough wherever it starts
    perm = rng.permutation(pages)
    slots = np.empty(n, np.int64)
    for at, end, off, page in starts:
        t = off + np.arange(end - at)
        slots[at:end] = perm[page + t // P] * P + t % P
    return slots, pages


def _config(case, H, **over):
    c = dict(window=WINDOW, page_size=case["page"], n_q_heads=case.get("hq", 8), n_kv_heads=case.get("hkv", 1), head_dim=case.get("d", 128), dtype=CODE[case.get("dtype", "bf16")],
             full_pages=1, swa_pages=1, max_seqs=1, max_pages_per_seq=1)
    c.update(over)
    return H.Config(**c)


def prepare(case, seed):
    return {"rope": _prepare_rope, "weights": _prepare_weights, "select": _prepare_select, "verify": _prepare_verify}[case["op"]](case, seed)


def _prepare_rope(case, seed):
    g, rng = _gen(seed), np.random.default_rng(seed)
    n, hq, hkv, d, P, dt = case["tokens"], case["hq"], case["hkv"], case["d"], case["page"], case["dtype"]
    if case["packed"]:  # the output rows of one projection: q, k and v beside each other
        rows = _normal(g, (n, (hq + 2 * hkv) * d), dt)
        q, k, v = rows[:, :hq * d], rows[:, hq * d:(hq + hkv) * d], rows[:, (hq + hkv) * d:]
    else:
        q, k, v = _normal(g, (n, hq * d), dt), _normal(g, (n, hkv * d), dt), _normal(g, (n, hkv * d), dt)
    slots, pages = _slots(case, rng)
    s = dict(case=case, q=q, k=k, v=v, q_out=torch.empty(n, hq, d, dtype=q.dtype, device="cuda"), pos=_i32(_positions(case, rng)), slots=_i32(slots),
             inv_freq=10000.0 ** (-2.0 * torch.arange(case["rotary"] // 2, dtype=torch.float64, device="cuda") / case["rotary"]),
             axis=torch.as_tensor(_axis_of_pair(case), device="cuda"))
    pool = torch.uint8 if dt == "fp8" else TORCH[dt]
    s["k_pool"] = torch.zeros(pages, hkv, P, d, dtype=pool, device="cuda")
    s["v_pool"] = torch.zeros((pages, hkv, d, P) if dt == "fp8" else (pages, hkv, P, d), dtype=pool, device="cuda")
    if dt == "fp8":
        s["k_scale"] = torch.ones(pages, hkv, P, device="cuda")
        s["v_scale"] = torch.ones(pages, hkv, P, device="cuda")
    if own:
        import hybrid_sliding_window_dual_gb300 as H
        s["H"] = H
        s["pool"] = H.hswa_pool_create(_config(case, H, full_pages=pages))
        s["layer"] = _layer(s, H)
        s["rope"] = H.hswa_rope_create(rotary_dim=case["rotary"], sections=_sections(case), theta=10000.0, interleaved=case["interleaved"], adjacent=case["adjacent"])
    return s


def _layer(s, H):
    return H.Layer(kind=H.HSWA_KIND_FULL, window=0, k_pool=s["k_pool"].data_ptr(), v_pool=s["v_pool"].data_ptr(),
                   k_scale=s["k_scale"].data_ptr() if "k_scale" in s else None, v_scale=s["v_scale"].data_ptr() if "v_scale" in s else None)


def _prepare_weights(case, seed):
    g, rng = _gen(seed), np.random.default_rng(seed)
    n, hq, hkv, d, P, dt = case["seqs"], case["hq"], case["hkv"], case["d"], case["page"], case["dtype"]
    lens = rng.permutation(_lengths(case))
    npg = -(-lens // P)
    pages, mp = int(npg.sum()), int(npg.max())
    perm, bt, at = rng.permutation(pages), np.full((n, mp), -1, np.int64), 0
    for i, m in enumerate(npg):
        bt[i, :m] = perm[at:at + m]
        at += m
    s = dict(case=case, bt=_i32(bt), lens=_i32(lens), q=_normal(g, (n, hq, d), dt), o=torch.empty(n, hq, d, dtype=TORCH.get(dt, torch.bfloat16), device="cuda"),
             w_in=torch.rand(n, mp, generator=g, device="cuda") * 4, w_out=torch.empty(n, mp, device="cuda"), decay=0.875, scale=1 / math.sqrt(d))
    if dt == "fp8":
        s["k_pool"], s["v_pool"] = _codes(g, (pages, hkv, P, d)), _codes(g, (pages, hkv, d, P))
        s["k_scale"] = 0.005 + 0.005 * torch.rand(pages, hkv, P, generator=g, device="cuda")
        s["v_scale"] = 0.005 + 0.005 * torch.rand(pages, hkv, P, generator=g, device="cuda")
    else:
        s["k_pool"], s["v_pool"] = _normal(g, (pages, hkv, P, d), dt), _normal(g, (pages, hkv, P, d), dt)
    if own:
        import hybrid_sliding_window_dual_gb300 as H
        s["H"] = H
        s["pool"] = H.hswa_pool_create(_config(case, H, full_pages=pages, max_seqs=n, max_pages_per_seq=mp))
        s["layer"] = _layer(s, H)
        s["ws"] = torch.empty(H.hswa_decode_weights_workspace_size(s["pool"], n), dtype=torch.uint8, device="cuda")
    return s


def _prepare_select(case, seed):
    g, rng = _gen(seed), np.random.default_rng(seed)
    n, P = case["seqs"], case["page"]
    npg = rng.permutation(_lengths(case))
    mp = int(npg.max())
    lens = npg * P - rng.integers(0, P, n)  # the last page ends anywhere
    w = torch.exp(2.5 * torch.randn(n, mp, generator=g, device="cuda"))
    w = torch.where(torch.rand(n, mp, generator=g, device="cuda") < 0.05, torch.zeros_like(w), w)  # pages that no query looked at
    s = dict(case=case, lens=_i32(lens), w_in=w, budget=_i32(np.maximum(1, np.rint(npg * case["keep"]))), recent=WINDOW + 64,
             keep=torch.empty(n, mp, dtype=torch.int32, device="cuda"), n_keep=torch.empty(n, dtype=torch.int32, device="cuda"), w_out=torch.empty(n, mp, device="cuda"))
    if own:
        import hybrid_sliding_window_dual_gb300 as H
        s["H"] = H
        s["pool"] = H.hswa_pool_create(_config(case, H, max_seqs=n, max_pages_per_seq=mp))
    return s


def _prepare_verify(case, seed):
    g, rng = _gen(seed), np.random.default_rng(seed)
    n, t, V = case["seqs"], case["n_tok"], case["vocab"]
    dt = TORCH[case["dtype"]]
    logits = torch.randn(n, t, V, generator=g, device="cuda") * 3
    s = dict(case=case, p=torch.softmax(logits, -1).to(dt), q=None, u=torch.rand(n, t, generator=g, device="cuda"),
             n_draft=_i32(np.where(rng.random(n) < 0.75, t - 1, rng.integers(0, t, n))), n_accept=torch.empty(n, dtype=torch.int32, device="cuda"),
             tokens=torch.empty(n, t, dtype=torch.int32, device="cuda"))
    # the draft model: the target's logits with an error of its own
    logits = logits[:, :t - 1]
    logits += torch.randn(n, t - 1, V, generator=g, device="cuda") * 0.7
    if case["draft"] == "sampled":
        q = torch.softmax(logits, -1)
        s["q"] = q.to(dt)
        c = torch.cumsum(q.view(-1, V), -1)
        s["draft"] = torch.searchsorted(c, torch.rand(n * (t - 1), 1, generator=g, device="cuda") * c[:, -1:]).clamp_(max=V - 1).view(n, t - 1).int()
    else:
        s["draft"] = logits.argmax(-1).int() if t > 1 else torch.empty(n, 0, dtype=torch.int32, device="cuda")
    if own:
        import hybrid_sliding_window_dual_gb300 as H
        s["H"] = H
    return s


# -------------------------------------------------------------------- run
def run(s):
    if own:
        return _own(s)
    return {"rope": _plain_rope, "weights": _plain_weights, "select": _plain_select, "verify": _plain_verify}[s["case"]["op"]](s)


def _own(s):
    H, case = s["H"], s["case"]  # on the default stream, as a session's calls are
    if case["op"] == "rope":
        H.hswa_rope_append(s["pool"], s["layer"], s["rope"], s["q"], s["q"].stride(0), s["k"], s["k"].stride(0), s["v"], s["v"].stride(0), s["pos"], s["slots"], s["q_out"], case["tokens"])
        return _rope_outputs(s)
    if case["op"] == "weights":
        H.hswa_decode_weights(s["pool"], s["layer"], s["q"], s["o"], s["bt"], s["lens"], case["seqs"], s["scale"], s["w_in"], s["decay"], s["w_out"], s["ws"], s["ws"].numel())
        return dict(o=s["o"], w=s["w_out"])
    if case["op"] == "select":
        H.hswa_evict_select(s["pool"], s["lens"], s["w_in"], s["budget"], case["seqs"], case["sink"], s["recent"], s["keep"], s["n_keep"], s["w_out"])
        return dict(keep=s["keep"], n_keep=s["n_keep"], w=s["w_out"])
    H.hswa_verify_draft(CODE[case["dtype"]], s["p"], case["vocab"], s["q"], case["vocab"], s["draft"], s["n_draft"], s["u"], case["seqs"], case["n_tok"], case["vocab"], s["n_accept"], s["tokens"])
    return dict(n_accept=s["n_accept"], tokens=s["tokens"])


def _rope_outputs(s):
    out = dict(q=s["q_out"], k=s["k_pool"], v=s["v_pool"])
    if s["case"]["dtype"] == "fp8":  # codes as the values they stand for, beside their scales
        out.update(k=s["k_pool"].view(torch.float8_e4m3fn), v=s["v_pool"].view(torch.float8_e4m3fn), k_scale=s["k_scale"], v_scale=s["v_scale"])
    return out


def _plain_rope(s):
    c = s["case"]
    n, hq, hkv, d, P, R = c["tokens"], c["hq"], c["hkv"], c["d"], c["page"], c["rotary"]
    angle = s["pos"].double()[s["axis"]].T * s["inv_freq"]  # [tokens][R/2], far positions need 64 bits
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def rotate(x, heads):
        x = x.float().view(n, heads, d)
        if c["adjacent"]:
            a, b = x[..., 0:R:2], x[..., 1:R:2]
            y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
        else:
            a, b = x[..., :R // 2], x[..., R // 2:R]
            y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        return torch.cat((y, x[..., R:]), -1)

    s["q_out"].copy_(rotate(s["q"], hq))
    k, v = rotate(s["k"], hkv), s["v"].float().view(n, hkv, d)
    slots = s["slots"].long()
    page, row = slots // P, slots % P
    if c["dtype"] == "fp8":
        for x, pool, scales in ((k, s["k_pool"], s["k_scale"]), (v, s["v_pool"].transpose(2, 3), s["v_scale"])):
            amax = x.abs().amax(-1)
            scale = torch.where(amax > 0, amax / 448, torch.ones_like(amax))
            pool[page, :, row] = (x / scale[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            scales[page, :, row] = scale
    else:
        s["k_pool"][page, :, row] = k.to(s["k_pool"].dtype)
        s["v_pool"][page, :, row] = v.to(s["v_pool"].dtype)
    return _rope_outputs(s)


def _values(s, which, table, dtype):
    """Pages of a pool as values, [..., hkv, P, d]."""
    x = s[which + "_pool"][table]
    if s["case"]["dtype"] == "fp8":
        x = x.view(torch.float8_e4m3fn).to(dtype)
        if which == "v":
            x = x.transpose(-1, -2)
        return x * s[which + "_scale"][table].to(dtype)[..., None]
    return x.to(dtype)


def _plain_weights(s):
    c = s["case"]
    n, hq, hkv, d, P = c["seqs"], c["hq"], c["hkv"], c["d"], c["page"]
    table, mp = s["bt"].long().clamp(min=0), s["bt"].shape[1]
    q = s["q"].float().view(n, 1, hkv, hq // hkv, d)
    k = _values(s, "k", table, torch.float32)  # [n][mp][hkv][P][d]
    scores = torch.matmul(q, k.transpose(-1, -2)) * s["scale"]  # [n][mp][hkv][G][P]
    del k
    key = torch.arange(mp * P, device="cuda").view(1, mp, 1, 1, P)
    scores = scores.masked_fill(key >= s["lens"].view(n, 1, 1, 1, 1), -math.inf)
    top = scores.amax((1, 4), keepdim=True)
    e = torch.exp(scores - torch.where(top > -math.inf, top, torch.zeros_like(top)))
    total = e.sum((1, 4), keepdim=True)
    prob = e / torch.where(total > 0, total, torch.ones_like(total))
    s["o"].copy_(torch.matmul(prob, _values(s, "v", table, torch.float32)).sum(1).view(n, hq, d))
    used = torch.arange(mp, device="cuda")[None] * P < s["lens"][:, None]
    s["w_out"].copy_(torch.where(used, s["decay"] * s["w_in"] + prob.sum((2, 3, 4)), torch.zeros_like(s["w_in"])))
    return dict(o=s["o"], w=s["w_out"])


def _plain_select(s):
    c, mp = s["case"], s["w_in"].shape[1]
    P = c["page"]
    p, L = torch.arange(mp, device="cuda")[None], s["lens"].long()[:, None]
    there = p * P < L
    fixed = there & ((p < c["sink"]) | ((p + 1) * P > L - s["recent"]))
    n_pages = there.sum(1)
    n_keep = torch.minimum(n_pages, torch.maximum(s["budget"].long(), fixed.sum(1)))
    # the order in which pages are kept: fixed ones, then by weight, the lower page first among equals, then what is not there
    key = torch.where(fixed, torch.full_like(s["w_in"], math.inf), torch.where(there, s["w_in"], torch.full_like(s["w_in"], -math.inf)))
    order = torch.sort(key, dim=1, descending=True, stable=True)[1]
    kept = torch.zeros_like(there).scatter_(1, order, p < n_keep[:, None])
    pages = torch.sort(torch.where(kept, p, mp), 1)[0]
    inside = p < n_keep[:, None]
    s["keep"].copy_(torch.where(inside, pages, -1))
    s["n_keep"].copy_(n_keep)
    s["w_out"].copy_(torch.where(inside, s["w_in"].gather(1, pages.clamp(max=mp - 1)), torch.zeros_like(s["w_in"])))
    return dict(keep=s["keep"], n_keep=s["n_keep"], w=s["w_out"])


def _plain_verify(s):
    c = s["case"]
    n, t, V = c["seqs"], c["n_tok"], c["vocab"]
    w = torch.arange(t, device="cuda")[None]
    draft, last, at = s["draft"].long(), s["n_draft"].long(), torch.arange(n, device="cuda")
    u = s["u"].double()
    px = s["p"][:, :t - 1].gather(2, draft[..., None])[..., 0].double()
    qx = torch.ones_like(px) if s["q"] is None else s["q"].gather(2, draft[..., None])[..., 0].double()
    taken = (u[:, :t - 1] * qx < px) & (w[:, :t - 1] < last[:, None])
    a = taken.long().cumprod(1).sum(1)
    target = s["p"][at, a].double()  # values next to a border of the distribution: 64 bits
    left = target
    if t > 1:
        row = a.clamp(max=t - 2)
        if s["q"] is None:
            less = torch.zeros_like(target).scatter_(1, draft.gather(1, row[:, None]), 2.0)
        else:
            less = s["q"][at, row].double()
        left = (target - less * (a < last)[:, None]).clamp(min=0)
        left = torch.where(left.sum(1, keepdim=True) > 0, left, target)
    cdf = left.cumsum(1)
    token = (cdf <= u[:, t - 1:] * cdf[:, -1:]).sum(1)
    drafts = torch.cat((draft, draft.new_full((n, 1), -1)), 1)
    s["n_accept"].copy_(a)
    s["tokens"].copy_(torch.where(w < a[:, None], drafts, torch.where(w == a[:, None], token[:, None], -1)))
    return dict(n_accept=s["n_accept"], tokens=s["tokens"])


# ------------------------------------------------------------------- work
def work(case):
    if case["op"] == "rope":
        n, hq, hkv, d = case["tokens"], case["hq"], case["hkv"], case["d"]
        e = 4 if case["dtype"] == "f32" else 2
        read = n * ((hq + 2 * hkv) * d * e + 4 * case["axes"] + 4)
        kv = n * 2 * hkv * ((d + 4) if case["dtype"] == "fp8" else d * e)
        return {"bytes": read + n * hq * d * e + kv, "flops": n * (hq + hkv) * case["rotary"] * 3}
    if case["op"] == "weights":
        hq, hkv, d, P = case["hq"], case["hkv"], case["d"], case["page"]
        lens = _lengths(case)
        tokens, n, mp = int(lens.sum()), case["seqs"], -(-int(lens.max()) // P)
        row = {"f32": 4 * d, "bf16": 2 * d, "fp8": d + 4}[case["dtype"]]
        e = 4 if case["dtype"] == "f32" else 2
        return {"bytes": tokens * 2 * hkv * row + 2 * n * hq * d * e + int((-(-lens // P)).sum()) * 8 + n * mp * 4, "flops": tokens * 4 * hq * d}
    if case["op"] == "select":
        npg = _lengths(case)
        return {"bytes": int(npg.sum()) * 4 + case["seqs"] * (int(npg.max()) * 8 + 12), "flops": int(npg.sum())}
    e = 4 if case["dtype"] == "f32" else 2
    rows = 2 if case["draft"] == "sampled" and case["n_tok"] > 1 else 1
    return {"bytes": case["seqs"] * (rows * case["vocab"] * e + case["n_tok"] * 20), "flops": case["seqs"] * case["vocab"] * 2}


# ------------------------------------------------------------------ exact
def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "weights": _exact_weights, "select": _exact_select, "verify": _exact_verify}[case["op"]](s)


def _exact_rope(s):
    """Each pair as a complex number times exp(i angle)."""
    c = s["case"]
    n, d, P, R = c["tokens"], c["d"], c["page"], c["rotary"]
    half = R // 2
    i = torch.arange(half, dtype=torch.float64, device="cuda")
    angle = torch.stack([s["pos"][int(a)].double() for a in s["axis"]], 1) * torch.exp(-math.log(10000.0) * 2 * i / R)
    turn = torch.polar(torch.ones_like(angle), angle)
    first, second = (torch.arange(0, R, 2, device="cuda"), torch.arange(1, R, 2, device="cuda")) if c["adjacent"] else (torch.arange(half, device="cuda"), torch.arange(half, R, device="cuda"))

    def rotated(x, heads):
        x = x.double().reshape(n, heads, d).clone()
        z = torch.complex(x[:, :, first], x[:, :, second]) * turn[:, None]
        x[:, :, first], x[:, :, second] = z.real, z.imag
        return x

    out = dict(q=rotated(s["q"], c["hq"]))
    page, row = (s["slots"].long() // P), (s["slots"].long() % P)
    for name, x in (("k", rotated(s["k"], c["hkv"])), ("v", s["v"].double().reshape(n, c["hkv"], d))):
        pool = s[name + "_pool"]
        if c["dtype"] == "fp8":
            step = x.abs().amax(-1) / 448
            step[step == 0] = 1
            values = torch.zeros(pool.shape, dtype=torch.float64, device="cuda")
            view = values if name == "k" else values.transpose(2, 3)
            view[page, :, row] = x / step[..., None]
            scales = torch.ones(s[name + "_scale"].shape, dtype=torch.float64, device="cuda")
            scales[page, :, row] = step
            out[name], out[name + "_scale"] = values, scales
        else:
            values = torch.zeros(pool.shape, dtype=torch.float64, device="cuda")
            values[page, :, row] = x
            out[name] = values
    return out


def _exact_weights(s):
    """One sequence after another, its keys in a row."""
    c = s["case"]
    hq, hkv, d, P = c["hq"], c["hkv"], c["d"], c["page"]
    o = torch.zeros(c["seqs"], hq, d, dtype=torch.float64, device="cuda")
    w = torch.zeros(s["w_in"].shape, dtype=torch.float64, device="cuda")
    for i, L in enumerate(s["lens"].tolist()):
        if L == 0:
            continue
        table = s["bt"][i, :-(-L // P)].long()
        k = _values(s, "k", table, torch.float64).transpose(0, 1).reshape(hkv, -1, d)[:, :L]
        v = _values(s, "v", table, torch.float64).transpose(0, 1).reshape(hkv, -1, d)[:, :L]
        prob = torch.softmax(torch.einsum("ghd,gkd->ghk", s["q"][i].double().view(hkv, -1, d), k) * s["scale"], -1)
        o[i] = torch.einsum("ghk,gkd->ghd", prob, v).reshape(hq, d)
        key = torch.nn.functional.pad(prob.sum((0, 1)), (0, table.numel() * P - L))
        w[i, :table.numel()] = s["decay"] * s["w_in"][i, :table.numel()].double() + key.view(-1, P).sum(1)
    return dict(o=o, w=w)


def _exact_select(s):
    """By hand, one sequence after another."""
    c, P = s["case"], s["case"]["page"]
    w, lens, budget = s["w_in"].cpu().numpy(), s["lens"].tolist(), s["budget"].tolist()
    n, mp = w.shape
    keep, n_keep, out = np.full((n, mp), -1, np.int32), np.zeros(n, np.int32), np.zeros((n, mp))
    for i in range(n):
        pages = -(-lens[i] // P)
        fixed = [p for p in range(pages) if p < c["sink"] or (p + 1) * P > lens[i] - s["recent"]]
        others = sorted(set(range(pages)) - set(fixed), key=lambda p: (-w[i, p], p))
        stay = sorted(fixed + others[:max(0, budget[i] - len(fixed))])
        n_keep[i] = len(stay)
        keep[i, :len(stay)], out[i, :len(stay)] = stay, w[i, stay]
    return dict(keep=torch.as_tensor(keep), n_keep=torch.as_tensor(n_keep), w=torch.as_tensor(out))


def _exact_verify(s):
    """One sequence after another, on the host."""
    c = s["case"]
    t = c["n_tok"]
    draft, last, u = s["draft"].tolist(), s["n_draft"].tolist(), s["u"].double().cpu().numpy()
    accepted, tokens = [], []
    for i in range(c["seqs"]):
        a = 0
        while a < last[i]:
            x = draft[i][a]
            qx = 1.0 if s["q"] is None else float(s["q"][i, a, x])
            if not u[i, a] * qx < float(s["p"][i, a, x]):
                break
            a += 1
        p = s["p"][i, a].double().cpu().numpy()
        left = p
        if a < last[i]:
            if s["q"] is None:
                left = p.copy()
                left[draft[i][a]] = 0
            else:
                left = np.maximum(p - s["q"][i, a].double().cpu().numpy(), 0)
            if not left.any():
                left = p
        cdf = np.cumsum(left)
        accepted.append(a)
        tokens.append(draft[i][:a] + [int(np.searchsorted(cdf, u[i, t - 1] * cdf[-1], side="right"))] + [-1] * (t - 1 - a))
    return dict(n_accept=torch.tensor(accepted, dtype=torch.int32), tokens=torch.tensor(tokens, dtype=torch.int32))
