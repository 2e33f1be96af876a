"""hswa_rope_append on the GPU against the 64-bit oracle.

Tolerances. fp32: a result is x cos - y sin. The angle is within pi 2^-25
(its rounding to fp32) + 3e-7 (64-bit frequencies at positions up to 2^31) of
the exact one, at positions up to 2^22 within 1e-7; sincospif adds 2^-23 at
most and the two products and their difference 2^-24 each: below
5e-7 (|x| + |y|) at ordinary positions, 9e-7 (|x| + |y|) at the far ones.
bf16: half a step, 2^-8 of the value, on top. E4M3: half a step of the code,
2^-4 of the value or 2^-10 of the scale, on top. Elements that do not turn,
and V, are copied bit for bit; V's codes are the oracle quantizer's."""
import numpy as np
import pytest
import torch

import hswa_workloads as wl
import oracle
from oracle import serving
from oracle.fp8 import e4m3_decode
import hybrid_sliding_window_dual_gb300 as H

F32, BF16, FP8 = wl.DTYPE_F32, wl.DTYPE_BF16, H.HSWA_DTYPE_FP8_E4M3
HALF_STEP = {F32: 0.0, BF16: 2.0 ** -8}


class Case:
    """T tokens of one layer; tensors as a caller has them."""

    def __init__(self, T, hq, hkv, d, P, dtype, rotary, sections, seed=0, far=False, packed=True, pages=None, run=1 << 30, **rope):
        rng = np.random.default_rng(seed)
        self.T, self.hq, self.hkv, self.d, self.P, self.dtype = T, hq, hkv, d, P, dtype
        self.rotary, self.sections, self.rope_args = rotary, sections, rope
        dt = torch.float32 if dtype == F32 else torch.bfloat16
        rows = wl.normal((T, (hq + 2 * hkv) * d), seed, dt, "cuda")
        cut = [x for x in rows.split([hq * d, hkv * d, hkv * d], 1)]
        self.q, self.k, self.v = cut if packed else [x.clone() for x in cut]
        top = 2 ** 31 - 1 if far else 1 << 20
        self.pos_h = rng.integers(-top if far else 0, top, (len(sections), T))
        self.pages = pages or -(-T // P) + 3
        slots = np.full(T, -1)
        for at in range(0, T, run):  # runs of consecutive slots, in a permuted order of pages
            n = min(run, T - at)
            slots[at:at + n] = at + np.arange(n)
        perm = rng.permutation(self.pages)
        self.slots_h = perm[slots // P] * P + slots % P
        self.make_pool()

    def make_pool(self):
        dt = {F32: torch.float32, BF16: torch.bfloat16, FP8: torch.uint8}[self.dtype]
        shape = (self.pages, self.hkv, self.P, self.d)
        self.k_pool = torch.full(shape, 7, dtype=dt, device="cuda")
        self.v_pool = torch.full((self.pages, self.hkv, self.d, self.P) if self.dtype == FP8 else shape, 7, dtype=dt, device="cuda")
        self.ks = torch.full((self.pages, self.hkv, self.P, 1), 3.0, device="cuda")
        self.vs = torch.full((self.pages, self.hkv, self.P, 1), 3.0, device="cuda")

    def run(self, kind=H.HSWA_KIND_FULL, q_out=None, stream=None):
        cfg = H.Config(window=128, page_size=self.P, n_q_heads=self.hq, n_kv_heads=self.hkv, head_dim=self.d, dtype=self.dtype,
                       full_pages=self.pages if kind == H.HSWA_KIND_FULL else 1, swa_pages=self.pages if kind == H.HSWA_KIND_SWA else 1,
                       max_seqs=1, max_pages_per_seq=1)
        pool = H.hswa_pool_create(cfg)
        layer = H.Layer(kind=kind, window=128, k_pool=self.k_pool.data_ptr(), v_pool=self.v_pool.data_ptr(), k_scale=self.ks.data_ptr(), v_scale=self.vs.data_ptr())
        rope = H.hswa_rope_create(self.rotary, self.sections, **self.rope_args)
        self.q_out = torch.full((self.T, self.hq, self.d), 5, dtype=self.q.dtype, device="cuda") if q_out is None else q_out
        pos = torch.as_tensor(self.pos_h.astype(np.int32), device="cuda")
        slots = torch.as_tensor(self.slots_h.astype(np.int32), device="cuda")
        H.hswa_rope_append(pool, layer, rope, self.q, self.q.stride(0) if self.T > 1 else self.hq * self.d, self.k,
                           self.k.stride(0) if self.T > 1 else self.hkv * self.d, self.v, self.v.stride(0) if self.T > 1 else self.hkv * self.d,
                           pos, slots, self.q_out, self.T, stream)
        status = H.hswa_check(stream)
        H.hswa_pool_destroy(pool)
        H.hswa_rope_destroy(rope)
        return status

    def turned(self, x, heads):
        """(exact rotation, |x| + |y| of each element's pair) in 64 bits."""
        x = x.double().cpu().numpy().reshape(self.T, heads, self.d)
        exact = serving.rope(x, self.pos_h, self.rotary, self.sections, **self.rope_args)
        half, size = self.rotary // 2, np.zeros_like(x)
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if self.rope_args.get("adjacent") else (i, i + half)
            size[:, :, a] = size[:, :, b] = np.abs(x[:, :, a]) + np.abs(x[:, :, b])
        return exact, size

    def check(self, q_in=None, far=False):
        angle = 9e-7 if far else 5e-7
        step = HALF_STEP[F32 if self.dtype == F32 else BF16]
        exact, size = self.turned(self.q if q_in is None else q_in, self.hq)
        got = self.q_out.double().cpu().numpy()
        assert (np.abs(got - exact) <= angle * size + step * np.abs(exact) * (1 + 1e-6) + (size > 0) * 1e-37).all()
        there = (self.slots_h >= 0) & (self.slots_h < self.pages * self.P)
        slots = self.slots_h[there]
        page, row = slots // self.P, slots % self.P
        exact, size = [x[there] for x in self.turned(self.k, self.hkv)]
        v = self.v.reshape(self.T, self.hkv, self.d)[torch.as_tensor(there, device="cuda")]
        touched = np.zeros((self.pages, self.P), bool)
        touched[page, row] = True
        if self.dtype == FP8:
            codes = self.k_pool.cpu().numpy()
            scale = self.ks.cpu().numpy()[page, :, row, 0].astype(np.float64)
            amax = np.abs(exact).max(-1)
            assert (np.abs(scale - np.where(amax > 0, amax / 448, 1)) <= (angle * size.max(-1) + 2.0 ** -23 * amax) / 448).all()
            got = e4m3_decode(codes[page, :, row]) * scale[..., None]
            assert (np.abs(got - exact) <= angle * size + np.maximum(2.0 ** -4 * np.abs(exact), 2.0 ** -10 * scale[..., None]) * (1 + 1e-5)).all()
            exp = [np.full(self.k_pool.shape, 7, np.uint8), np.full(self.ks.shape, 3, np.float32), np.full(self.v_pool.shape, 7, np.uint8), np.full(self.vs.shape, 3, np.float32)]
            rows = v.float().cpu().numpy()
            oracle.append_kv_fp8(*exp, rows, rows, slots)
            same = (self.v_pool.cpu().numpy() == exp[2]).all(), (self.vs.cpu().numpy() == exp[3]).all()
            assert all(same)
            assert (codes.transpose(0, 2, 1, 3)[~touched] == 7).all() and (self.ks.cpu().numpy().transpose(0, 2, 1, 3)[~touched] == 3).all()
        else:
            k = self.k_pool.double().cpu().numpy().transpose(0, 2, 1, 3)  # [page][row][head][d]
            assert (np.abs(k[page, row] - exact) <= angle * size + step * np.abs(exact) * (1 + 1e-6)).all()
            vp = self.v_pool.transpose(1, 2)
            assert torch.equal(vp[torch.as_tensor(page), torch.as_tensor(row)], v)
            keep = torch.as_tensor(~touched, device="cuda")
            assert (k[~touched] == 7).all() and (vp[keep] == 7).all()


SHAPES = [  # T, hq, hkv, d, P, rotary, sections, rope
    (1, 64, 8, 128, 64, 128, [64], {}),
    (2, 64, 8, 128, 64, 128, [16, 24, 24], {}),
    (67, 64, 8, 128, 64, 128, [24, 20, 20], dict(interleaved=True)),
    (130, 16, 2, 128, 64, 64, [16, 8, 8], dict(adjacent=True)),
    (200, 24, 3, 128, 16, 128, [64, 0], {}),
    (33, 8, 8, 128, 64, 128, [24, 16, 12, 12], dict(adjacent=True, interleaved=True, theta=5e6)),
    (77, 4, 1, 128, 7, 2, [1], {}),
    (65, 6, 2, 128, 64, 20, [4, 6], {}),      # a rotary dim that no vector divides
    (65, 6, 2, 128, 64, 16, [8], {}),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32, FP8])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "T%d-h%d-R%d" % (s[0], s[1], s[5]))
def test_rope_append_matches_oracle(shape, dtype):
    T, hq, hkv, d, P, rotary, sections, rope = shape
    c = Case(T, hq, hkv, d, P, dtype, rotary, sections, seed=T, **rope)
    assert c.run() == 0
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d,rotary", [(64, 64), (64, 32), (96, 96), (256, 256), (40, 24), (20, 20), (5, 4), (1, 0)])
def test_rope_append_head_dims(dtype, d, rotary):
    if rotary == 0:
        d, rotary = 2, 2
    c = Case(50, 4, 2, d, 16, dtype, rotary, [rotary // 2], seed=d)
    assert c.run() == 0
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32, FP8])
def test_rope_append_far_positions_and_given_frequencies(dtype):
    c = Case(90, 8, 2, 128, 64, dtype, 128, [32, 32], seed=5, far=True)
    assert c.run() == 0
    c.check(far=True)
    # a table of its own: turning faster than once a position, backwards, not at all
    f = np.concatenate([[7.0, -0.5, 0.0, 6.283185307179586], np.geomspace(1, 1e-6, 60)])
    c = Case(90, 8, 2, 128, 64, dtype, 128, [64], seed=6, inv_freq=f)
    c.pos_h = c.pos_h % 5000
    assert c.run() == 0
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, FP8])
@pytest.mark.parametrize("kind", [H.HSWA_KIND_FULL, H.HSWA_KIND_SWA])
def test_rope_append_padding_and_bad_slots(dtype, kind):
    """Tokens without a slot still get their q; a slot past the pool is
    reported and skipped."""
    c = Case(300, 16, 2, 128, 64, dtype, 128, [32, 16, 16], seed=8)
    c.slots_h[[0, 5, 64, 65, 66, 299]] = -1
    assert c.run(kind) == 0
    c.check()
    c.make_pool()
    c.slots_h[[3, 190]] = c.pages * c.P, 2 ** 31 - 1
    c.slots_h[191] = -2 ** 31
    assert c.run(kind) == H.HSWA_ERR_BOUNDS
    c.check()
    c.make_pool()
    c.slots_h[:] = -1
    assert c.run(kind) == 0
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, FP8])
@pytest.mark.parametrize("order", ["scattered", "backwards", "holes"])
def test_rope_append_slot_orders(dtype, order):
    """Slots in any order: tokens of many sequences, descending, with gaps."""
    c = Case(257, 8, 4, 128, 64, dtype, 128, [64], seed=9, pages=9)
    rng = np.random.default_rng(10)
    if order == "scattered":
        c.slots_h = rng.permutation(9 * 64)[:257]
    elif order == "backwards":
        c.slots_h = np.arange(300, 300 - 257, -1)
    else:
        c.slots_h = np.arange(257) * 2 + (np.arange(257) > 100)
    assert c.run() == 0
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("adjacent,rotary", [(False, 128), (True, 64), (False, 20)])
def test_rope_append_in_place(dtype, adjacent, rotary):
    c = Case(70, 16, 2, 128, 64, dtype, rotary, [rotary // 2], seed=11, packed=False, adjacent=adjacent)
    before = c.q.clone()
    c.q = c.q.view(70, 16, 128)
    assert c.run(q_out=c.q) == 0
    c.check(q_in=before)


@pytest.mark.gpu
@pytest.mark.parametrize("shift", [1, 3, 4])
def test_rope_append_unaligned_rows(shift):
    """Rows that start anywhere: bases and strides off the vector width."""
    for dtype in (BF16, F32, FP8):
        c = Case(40, 8, 2, 128, 64, dtype, 128, [64], seed=12 + shift)
        wide = torch.zeros(40, 12 * 128 + 1 + shift, dtype=c.q.dtype, device="cuda")
        cut = []
        for at, x in ((shift, c.q), (shift + 1024, c.k), (shift + 1280, c.v)):
            wide[:, at:at + x.shape[1]] = x
            cut.append(wide[:, at:at + x.shape[1]])
        c.q, c.k, c.v = cut
        assert c.run() == 0
        c.check()


@pytest.mark.gpu
def test_rope_append_special_values():
    """Zero rows get scale 1 and zero codes; infinities and NaN stay in their
    own pairs and rows."""
    c = Case(70, 8, 2, 128, 64, FP8, 128, [64], seed=13, packed=False)
    c.k[3] = 0
    c.v[3] = 0
    assert c.run() == 0
    c.check()
    at = int(c.slots_h[3])
    assert (c.ks[at // 64, :, at % 64] == 1).all() and (c.k_pool[at // 64, :, at % 64] & 0x7f == 0).all()
    c = Case(70, 8, 2, 128, 64, BF16, 128, [64], seed=14, packed=False)
    c.q[5, 128 + 7] = float("inf")
    c.k[6, 9] = float("nan")
    clean = Case(70, 8, 2, 128, 64, BF16, 128, [64], seed=14, packed=False)
    assert c.run() == 0 and clean.run() == 0
    odd = ~torch.isfinite(c.q_out)
    odd[5, 1, [7, 71]] = False
    assert not odd.any()
    same = torch.ones_like(odd)
    same[5, 1, [7, 71]] = False
    assert torch.equal(c.q_out[same], clean.q_out[same])
    bad = (~torch.isfinite(c.k_pool)).nonzero()
    at = int(c.slots_h[6])
    assert bad.tolist() == [[at // 64, 0, at % 64, 9], [at // 64, 0, at % 64, 73]]


@pytest.mark.gpu
def test_rope_append_codes_of_extreme_rows():
    """V's codes are the oracle quantizer's for rows of every magnitude, with
    zeros of both signs, subnormals, and quotients next to the middles between
    codes."""
    c = Case(256, 8, 2, 128, 64, FP8, 128, [64], seed=18, packed=False)
    v = c.v.view(256, 2, 128)
    g = torch.Generator(device="cuda")
    g.manual_seed(18)
    size = torch.logspace(-39, 38, 256, device="cuda", dtype=torch.float64)
    v.copy_((torch.randn(256, 2, 128, generator=g, device="cuda", dtype=torch.float64) * size[:, None, None]).clamp(-3e38, 3e38))
    v[:, 0, 5], v[:, 0, 6], v[:, 1, 7] = 0.0, -0.0, 1e-40
    # rows whose quotients are exact halves of steps, and just off them
    steps = torch.arange(1, 129, device="cuda", dtype=torch.float64) * 3.5
    v[100, 0], v[100, 1] = steps, steps * (1 + 2.0 ** -8)
    v[101, 0], v[101, 1] = -steps / 7, steps * 2.0 ** -60
    c.k.copy_(c.v)
    # nothing turns: K has the same values, but for the sign of a zero: the
    # turned -0 1 - y 0 is +0 for a negative y
    c.pos_h[:] = 0
    assert c.run() == 0
    rows = v.float().cpu().numpy()
    exp = [np.full(c.k_pool.shape, 7, np.uint8), np.full(c.ks.shape, 3, np.float32), np.full(c.v_pool.shape, 7, np.uint8), np.full(c.vs.shape, 3, np.float32)]
    oracle.append_kv_fp8(*exp, rows, rows, c.slots_h)
    for name, e in (("ks", exp[1]), ("vs", exp[3]), ("v_pool", exp[2])):
        assert (getattr(c, name).cpu().numpy() == e).all(), name
    assert (e4m3_decode(c.k_pool.cpu().numpy()) == e4m3_decode(exp[0])).all()


@pytest.mark.gpu
def test_rope_append_long_pool_offsets():
    """Slots whose elements lie past 2^31 bytes and 2^31 elements of the pool."""
    pages = 33000  # x 8 heads x 64 x 128 elements = 2.16e9
    c = Case(200, 16, 8, 128, 64, BF16, 128, [64], seed=15, pages=pages)
    c.slots_h = np.concatenate([np.arange(100), np.arange(100) + (pages - 3) * 64 + 30])
    assert c.run() == 0
    exact, size = c.turned(c.k, 8)
    page, row = c.slots_h // 64, c.slots_h % 64
    k = c.k_pool[torch.as_tensor(page, device="cuda"), :, torch.as_tensor(row, device="cuda")].double().cpu().numpy()
    assert (np.abs(k - exact) <= 5e-7 * size + 2.0 ** -8 * np.abs(exact) * (1 + 1e-6)).all()
    assert int((c.k_pool[100:pages - 10] != 7).sum()) == 0


@pytest.mark.gpu
def test_rope_append_on_a_stream_and_in_a_graph():
    c = Case(64, 16, 2, 128, 64, FP8, 128, [24, 20, 20], seed=16)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    assert c.run(stream=side) == 0
    c.check()
    # captured once, replayed on new inputs
    cfg = H.Config(window=128, page_size=64, n_q_heads=16, n_kv_heads=2, head_dim=128, dtype=FP8, full_pages=c.pages, swa_pages=1, max_seqs=1, max_pages_per_seq=1)
    pool, rope = H.hswa_pool_create(cfg), H.hswa_rope_create(128, [24, 20, 20])
    layer = H.Layer(kind=0, window=0, k_pool=c.k_pool.data_ptr(), v_pool=c.v_pool.data_ptr(), k_scale=c.ks.data_ptr(), v_scale=c.vs.data_ptr())
    pos = torch.as_tensor(c.pos_h.astype(np.int32), device="cuda")
    slots = torch.as_tensor(c.slots_h.astype(np.int32), device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        H.hswa_rope_append(pool, layer, rope, c.q, c.q.stride(0), c.k, c.k.stride(0), c.v, c.v.stride(0), pos, slots, c.q_out, 64, torch.cuda.current_stream())
    H.hswa_rope_destroy(rope)  # nothing of it is needed any more
    other = Case(64, 16, 2, 128, 64, FP8, 128, [24, 20, 20], seed=17)
    for name in ("q", "k", "v"):
        getattr(c, name).copy_(getattr(other, name))
    c.pos_h = other.pos_h
    pos.copy_(torch.as_tensor(c.pos_h.astype(np.int32)))
    g.replay()
    assert H.hswa_check() == 0
    c.check()
    H.hswa_pool_destroy(pool)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32, FP8])
@pytest.mark.parametrize("T,hq,hkv", [(639, 8, 1), (643, 8, 1), (1023, 32, 4), (1025, 32, 4)])
@pytest.mark.parametrize("adjacent", [False, True])
def test_rope_append_around_the_tiles(T, hq, hkv, dtype, adjacent):
    # one token a CTA and four, the last CTA's tokens fewer
    c = Case(T, hq, hkv, 128, 64, dtype, 128, [24, 20, 20], adjacent=adjacent, seed=T)
    assert c.run() == 0
    c.check()
