"""Decode at batch sizes that a 32-way search does not divide evenly: the
CTA that starts inside the last sequence has to find it. (Between 33 and 61
sequences, and in most of every later span up to a multiple of 32, the probes
past the last sequence repeat it.)"""
import numpy as np
import pytest
import torch

import hswa_workloads as wl
import hybrid_sliding_window_dual_gb300 as H
from scenario import Scenario
from test_gpu_decode import run_decode_step
from test_gpu_fp8 import Fp8Case, fp8_multi_step
from test_gpu_multi import run_multi_step


def lengths(n):
    """Short sequences with one long enough for many CTAs at the end."""
    return [(37 * i) % 150 + 1 for i in range(n - 1)] + [9000]


@pytest.mark.gpu
@pytest.mark.parametrize("n", [32, 33, 40, 49, 61, 62, 65, 90, 123, 200, 278])
def test_decode_starts_inside_the_last_sequence(n):
    sc = Scenario(64, 8, 128, 64, 128, wl.DTYPE_BF16, lengths(n), seed=n)
    run_decode_step(sc, [0, n // 2, n - 2, n - 1], seed=60 + n, expect_kernel="decode_mma_bf16_d128")


@pytest.mark.gpu
@pytest.mark.parametrize("n_tok", [2, 3, 8])
def test_multi_token_decode_starts_inside_the_last_sequence(n_tok):
    sc = Scenario(64, 8, 128, 64, 128, wl.DTYPE_BF16, lengths(49), seed=49)
    run_multi_step(sc, n_tok, seed=70 + n_tok, samples=[0, 47, 48])


@pytest.mark.gpu
@pytest.mark.parametrize("n_tok", [1, 4])
def test_fp8_decode_starts_inside_the_last_sequence(n_tok):
    fp8_multi_step(Fp8Case(lengths(49), seed=75, extra=8), n_tok, seed=80 + n_tok, samples=[0, 47, 48])


FEW = [[1566, 14213], [64, 65, 3000, 1], [30000], [304 * 64], [305 * 64 - 1, 2], [20000, 20000, 63]]


@pytest.mark.gpu
@pytest.mark.parametrize("lens", FEW, ids=str)
@pytest.mark.parametrize("hkv", [1, 2])
def test_decode_of_few_segments(lens, hkv):
    # a segment's pieces, up to one a CTA, with and without CTAs between that have no page
    sc = Scenario(8 * hkv, hkv, 128, 64, 128, wl.DTYPE_BF16, lens, seed=len(lens))
    run_decode_step(sc, list(range(len(lens))), seed=90 + hkv, expect_kernel="decode_mma_bf16_d128")


@pytest.mark.gpu
@pytest.mark.parametrize("n_tok", [2, 3, 8])
@pytest.mark.parametrize("lens", FEW[:3], ids=str)
def test_multi_token_decode_of_few_segments(lens, n_tok):
    sc = Scenario(8, 1, 128, 64, 128, wl.DTYPE_BF16, [max(x, n_tok) for x in lens], seed=n_tok)
    run_multi_step(sc, n_tok, seed=95 + n_tok, samples=list(range(len(lens))))


@pytest.mark.gpu
@pytest.mark.parametrize("fused", [False, True])
def test_decode_by_both_register_splits(fused):
    """Tables with room for more than 1 GB of K and V take the other
    instantiation of the one-token kernel: equal bits."""
    hkv, P, d, pages = 8, 64, 128, 4200  # 1.1 GB
    lens = np.array([5, 700, 0, 3000, 64])
    S, g = len(lens), torch.Generator(device="cuda")
    g.manual_seed(17)
    rows = -(-lens // P)
    table = np.full((S, 50), -1, np.int32)
    perm = np.random.default_rng(17).permutation(pages)[:rows.sum()]
    for i, at in enumerate(np.cumsum(rows) - rows):
        table[i, :rows[i]] = perm[at:at + rows[i]]
    k, v = (torch.randn(pages, hkv, P, d, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    q = torch.randn(S, 8 * hkv, d, generator=g, device="cuda", dtype=torch.bfloat16)
    new = torch.randn(2, S, hkv, d, generator=g, device="cuda", dtype=torch.bfloat16)
    slots = torch.as_tensor(np.where(lens > 0, table[np.arange(S), np.maximum(lens - 1, 0) // P] * P + (lens - 1) % P, -1).astype(np.int32), device="cuda")
    outs = []
    for mp in (50, 5000):  # 50: at most 250 pages
        pool = H.hswa_pool_create(H.Config(window=128, page_size=P, n_q_heads=8 * hkv, n_kv_heads=hkv, head_dim=d, dtype=H.HSWA_DTYPE_BF16,
                                           full_pages=pages, swa_pages=1, max_seqs=S, max_pages_per_seq=mp))
        kk, vv = (k.clone(), v.clone()) if fused else (k, v)
        layer = H.Layer(kind=H.HSWA_KIND_FULL, window=0, k_pool=kk.data_ptr(), v_pool=vv.data_ptr())
        bt = torch.full((S, mp), -1, dtype=torch.int32, device="cuda")
        bt[:, :50] = torch.as_tensor(table, device="cuda")
        o, n = torch.full_like(q, float("nan")), torch.as_tensor(lens.astype(np.int32), device="cuda")
        ws = torch.empty(H.hswa_decode_workspace_size(pool, S), dtype=torch.uint8, device="cuda")
        if fused:
            H.hswa_decode_append(pool, layer, q, new[0], new[1], slots, o, bt, n, S, 0.088, ws, ws.numel())
        else:
            H.hswa_decode(pool, layer, q, o, bt, n, S, 0.088, ws, ws.numel())
        assert H.hswa_check() == 0
        outs.append((o, kk, vv))
        H.hswa_pool_destroy(pool)
    assert torch.isfinite(outs[0][0]).all() and (outs[0][0][2] == 0).all() and outs[0][0][[0, 1, 3, 4]].abs().sum() > 0
    for a, b in zip(*outs):
        assert torch.equal(a, b)
