"""Queries with NaN, infinities and values beyond fp16 over every type of pool.

A head whose query holds a NaN has no softmax: its output is NaN, and nothing
else changes. So is that of a head with a score of NaN or +inf; keys whose
score is -inf have no weight, and a head with no others gives 0. Where a kernel works
on fp16 queries (FP8 and FP4 pools), finite values beyond +-65504 count as that and
infinities as NaN."""
import math

import numpy as np
import pytest
import torch

import hswa_workloads as wl
import hybrid_sliding_window_dual_gb300 as H
from hybrid_sliding_window_dual_gb300.session import DualPoolSession

FULL, SWA = wl.KIND_FULL, wl.KIND_SWA
BF16, FP8, FP4 = H.HSWA_DTYPE_BF16, H.HSWA_DTYPE_FP8_E4M3, H.HSWA_DTYPE_FP4
LENGTHS = [40, 64, 700, 9000]  # the last is cut among many CTAs


def session(dtype, lengths, seed, extra, hq=64, hkv=8, d=128, P=64, W=128):
    """A Full and an SWA layer with the sequences' tokens in both."""
    pages = [math.ceil((L + extra) / P) for L in lengths]
    cfg = H.Config(window=W, page_size=P, n_q_heads=hq, n_kv_heads=hkv, head_dim=d, dtype=dtype, full_pages=sum(pages) + 2, swa_pages=sum(pages) + 2, max_seqs=len(lengths),
                   max_pages_per_seq=max(pages))
    s = DualPoolSession(cfg, [FULL, SWA])
    full, swa = s.reserve(range(len(lengths)), lengths)
    s.sync()
    for layer, slots in enumerate((full, swa)):
        k, v = (wl.normal((sum(lengths), hkv, d), seed + 2 * layer + i, wl.DTYPE_BF16).cuda() for i in (0, 1))
        s.append(layer, k, v, torch.as_tensor(slots, device="cuda"))
    return s


def decode(s, layer, q, n_tok):
    o = torch.zeros_like(q)
    n = q.shape[0] // n_tok
    if n_tok == 1:
        s.decode(layer, q, o, n, 1 / math.sqrt(q.shape[2]))
    else:
        s.decode_multi(layer, q, o, n, n_tok, 1 / math.sqrt(q.shape[2]))
    assert s.check() == 0
    return o


def only_there(got, clean, rows, zero=()):
    """NaN in all of the given (row, head)s (0 in some) and what was there everywhere else."""
    nan = torch.zeros_like(got, dtype=torch.bool)
    want = clean.clone()
    for row, head in rows:
        if (row, head) in zero:
            want[row, head] = 0
        else:
            nan[row, head] = True
    assert torch.equal(got.isnan(), nan)
    assert torch.equal(got[~nan], want[~nan])


@pytest.mark.gpu
@pytest.mark.parametrize("n_tok", [1, 2, 3, 4, 5, 8, 9, 16])
@pytest.mark.parametrize("dtype", [BF16, FP8, FP4])
def test_decode_of_bad_queries(dtype, n_tok):
    s = session(dtype, LENGTHS, 4000, 0)
    q = wl.normal((len(LENGTHS) * n_tok, 64, 128), 4100, wl.DTYPE_BF16).cuda()
    bad = [(0, 0), (n_tok, 9), (3 * n_tok - 1, 31), (4 * n_tok - 1, 63)]
    for layer in range(2):
        clean = decode(s, layer, q, n_tok)
        assert torch.isfinite(clean).all()
        for values in ([float("nan")] * 4, [float("inf"), -float("inf"), float("inf"), -float("inf")]):
            x = q.clone()
            for i, (row, head) in enumerate(bad):
                x[row, head, (3 + 41 * i) % 128] = values[i]
            only_there(decode(s, layer, x, n_tok), clean, bad)
        if dtype == FP4 or (dtype == FP8 and n_tok > 2):  # finite values beyond fp16's
            outs = []
            for big in (65536.0, 1e20, torch.finfo(torch.bfloat16).max):
                x = q.clone()
                x[n_tok - 1, 5, 7], x[-1, 40, 100] = big, -big
                outs.append(decode(s, layer, x, n_tok))
            assert torch.isfinite(outs[0]).all() and torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    s.close()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, FP8, FP4])
def test_prefill_of_bad_queries(dtype):
    chunk = [30, 64, 200, 1]
    s = session(dtype, LENGTHS, 4200, 0)  # the chunks' keys are there already
    prefix = np.array([L - n for L, n in zip(LENGTHS, chunk)], np.int32)
    q_start = np.concatenate([[0], np.cumsum(chunk)]).astype(np.int32)
    q = wl.normal((int(q_start[-1]), 64, 128), 4300, wl.DTYPE_BF16).cuda()

    def prefill(layer, x):
        o = torch.zeros_like(x)
        s.prefill(layer, x, o, torch.as_tensor(prefix, device="cuda"), torch.as_tensor(q_start, device="cuda"), 4, max(chunk), 1 / math.sqrt(128), prefix_host=prefix,
                  q_start_host=q_start)
        assert s.check() == 0
        return o

    first = []  # K of the second sequence's first token
    for layer in range(2):
        k, v = (torch.empty(1, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        s.read(layer, s.bt(layer)[1, :1] * 64, k, v)
        first.append(k[0])
    assert prefix[1] == 0
    bad = [(20, 0), (30, 7), (200, 31), (294, 63)]
    for layer in range(2):
        clean = prefill(layer, q)
        assert torch.isfinite(clean).all()
        for values in ([float("nan")] * 4, [float("inf"), -float("inf"), float("inf"), -float("inf")]):
            x = q.clone()
            for i, (row, head) in enumerate(bad):
                x[row, head, (3 + 41 * i) % 128] = values[i]
            # the second row sees one key: its score is that key's element times an infinity
            alone = (x[30, 7, 44] * first[layer][0, 44]).item()
            only_there(prefill(layer, x), clean, bad, [bad[1]] if dtype == BF16 and alone == -math.inf else [])
    s.close()


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [-0.4, -3.0, 0.0])
@pytest.mark.parametrize("n_tok", [1, 3, 4, 8, 16])
def test_decode_under_scales_that_are_not_positive(n_tok, scale):
    """bf16 pools: against 64-bit attention over the rows read back. Weights are
    rounded to bf16 (2^-8 of each, so at most that of the largest value), scores
    summed and scaled in fp32 (d + 8 roundings of at most 2^-23 of |q| |k| scale, twice
    that of the largest value), the output rounded to bf16."""
    lengths, W = [16, 63, 64, 200, 900, 4000], 128
    s = session(BF16, lengths, 4400, 0)
    for layer in range(2):
        q = wl.normal((len(lengths) * n_tok, 64, 128), 4500 + layer, wl.DTYPE_BF16).cuda()
        o = torch.full_like(q, float("nan"))
        s.decode_multi(layer, q, o, len(lengths), n_tok, scale)
        assert s.check() == 0
        for i, L in enumerate(lengths):
            pos = torch.arange(L, device="cuda")
            slots = (s.bt(layer)[i, pos // 64] * 64 + pos % 64).int()
            k, v = (torch.empty(L, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
            s.read(layer, slots, k, v)
            k, v = (x.double().repeat_interleave(8, 1) for x in (k, v))
            for w in range(n_tok):
                t = L - n_tok + w
                first = max(0, t - W + 1) if layer else 0
                x = q[i * n_tok + w].double()
                z = torch.einsum("hd,lhd->hl", x, k[first:t + 1]) * scale
                exp = torch.einsum("hl,lhd->hd", z.softmax(1), v[first:t + 1])
                score = (128 + 8) * 2.0 ** -23 * x.norm(dim=1).max() * k.norm(dim=2).max() * abs(scale) + 2.0 ** -20
                tol = 2.0 ** -8 * exp.abs() + v.abs().max() * (2.0 ** -8 + 2 * score)
                assert ((o[i * n_tok + w].double() - exp).abs() <= tol).all(), (layer, L, w)
    s.close()


@pytest.mark.gpu
@pytest.mark.parametrize("n_tok", [1, 2, 3, 4, 5, 9, 16])
@pytest.mark.parametrize("dtype", [FP8, FP4])
def test_a_negative_scale_is_that_of_the_negative_query(dtype, n_tok):
    """Equal bits: products and sums of the one are those of the other."""
    s = session(dtype, LENGTHS, 4600, 0)
    for layer in range(2):
        q = wl.normal((len(LENGTHS) * n_tok, 64, 128), 4700 + layer, wl.DTYPE_BF16).cuda()
        outs = []
        for x, scale in ((q, -0.3), (-q, 0.3)):
            o = torch.full_like(q, float("nan"))
            s.decode_multi(layer, x, o, len(LENGTHS), n_tok, scale)
            outs.append(o)
        assert s.check() == 0 and torch.isfinite(outs[0]).all() and torch.equal(outs[0], outs[1])
    s.close()
