"""Decode at batch sizes that a 32-way search does not divide evenly: the
CTA that starts inside the last sequence has to find it. (Between 33 and 61
sequences, and in most of every later span up to a multiple of 32, the probes
past the last sequence repeat it.)"""
import pytest

import hswa_workloads as wl
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
