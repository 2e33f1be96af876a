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
