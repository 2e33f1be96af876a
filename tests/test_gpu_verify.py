"""hswa_verify_draft on the GPU against the oracle, whose decisions are made
in exact rational arithmetic: every count and token is equal."""
import numpy as np
import pytest
import torch

from oracle import serving
import hybrid_sliding_window_dual_gb300 as H

CODE = {torch.float32: H.HSWA_DTYPE_F32, torch.bfloat16: H.HSWA_DTYPE_BF16}


def verify(p, q, draft, n_draft, u, stream=None, expect=0):
    S, n, V = p.shape
    acc = torch.full((S,), -7, dtype=torch.int32, device="cuda")
    tok = torch.full((S, n), -7, dtype=torch.int32, device="cuda")
    H.hswa_verify_draft(CODE[p.dtype], p, p.stride(1), q, 0 if q is None else q.stride(1), draft, n_draft, u, S, n, V, acc, tok, stream)
    assert H.hswa_check(stream) == expect
    return acc.cpu().numpy(), tok.cpu().numpy()


def host(x):
    return None if x is None else x.double().cpu().numpy() if x.is_floating_point() else x.cpu().numpy()


def check(p, q, draft, n_draft, u, **kw):
    got = verify(p, q, draft, n_draft, u, **kw)
    exp = serving.verify(host(p), host(q), host(draft), host(n_draft), host(u), bits=50 if p.dtype == torch.float32 else 45)
    assert np.array_equal(got[0], exp[0])
    assert np.array_equal(got[1], exp[1])
    return got


def make(S, n, V, dtype, greedy, seed, sharp=3.0, pad=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    logits = torch.randn(S, n, V, generator=g, device="cuda") * sharp
    p = torch.zeros(S, n, V + pad, dtype=dtype, device="cuda")[:, :, :V]
    p.copy_(torch.softmax(logits, -1))
    logits = logits[:, :n - 1] + torch.randn(S, n - 1, V, generator=g, device="cuda") * 0.7
    q, draft = None, torch.zeros(S, 0, dtype=torch.int32, device="cuda")
    if n > 1:
        soft = torch.softmax(logits, -1)
        if greedy:
            draft = soft.argmax(-1).int()
        else:
            q = torch.zeros(S, n - 1, V + pad, dtype=dtype, device="cuda")[:, :, :V]
            q.copy_(soft)
            draft = torch.multinomial(soft.view(-1, V), 1, generator=g).view(S, n - 1).int()
    u = torch.rand(S, n, generator=g, device="cuda")
    n_draft = torch.randint(0, n, (S,), generator=g, device="cuda", dtype=torch.int32)
    return p, q, draft.contiguous(), n_draft, u


@pytest.mark.gpu
@pytest.mark.parametrize("greedy", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("S,n,V", [(1, 1, 1), (1, 2, 1), (3, 1, 7), (5, 4, 2), (9, 3, 127), (4, 16, 129), (6, 5, 1000), (40, 4, 4099), (2, 8, 32001),
                                   (3, 4, 131072), (2, 2, 262145), (1, 2, 1 << 20)])
def test_verify_matches_oracle(S, n, V, dtype, greedy):
    p, q, draft, n_draft, u = make(S, n, V, dtype, greedy, seed=S * 1000 + n)
    check(p, q, draft, n_draft, u)
    check(p, q, draft, None, u)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("pad", [1, 2, 3, 5, 8, 61])
def test_verify_padded_rows(dtype, pad):
    """Rows further apart than the vocabulary, starting anywhere."""
    for V in (1003, 1004):
        p, q, draft, n_draft, u = make(12, 4, V, dtype, False, seed=pad, pad=pad)
        assert p.stride(1) == V + pad
        check(p, q, draft, n_draft, u)


@pytest.mark.gpu
def test_verify_acceptance_borders():
    """u q against p where they are equal, one step apart, zero."""
    V = 64
    p = torch.full((6, 2, V), 1 / 64, device="cuda")
    q = torch.full((6, 1, V), 1 / 32, device="cuda")
    draft = torch.full((6, 1), 5, dtype=torch.int32, device="cuda")
    half = np.float32(0.5)
    u = torch.tensor([[half, 0.3], [np.nextafter(half, np.float32(0)), 0.3], [np.nextafter(half, np.float32(1)), 0.3], [0, 0.3], [0.7, 0.3], [0, 0.3]], device="cuda")
    p[3, 0, 5] = 0       # the target cannot say it
    q[4, 0, 5] = 0       # the draft could not have drawn it
    q[5, 0, 5], p[5, 0, 5] = 0, 0
    acc, _ = check(p, q, draft, None, u)
    assert acc.tolist() == [0, 1, 0, 0, 1, 0]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_verify_draw_borders(dtype):
    """Draws at the very edges of the distribution: u = 0, the largest u below
    1, exact cumulative sums, one token with everything, weight at either end."""
    V = 5000
    rows = []
    one = torch.zeros(V)
    for at in (0, 1, 2499, V - 1):
        x = one.clone()
        x[at] = 1
        rows.append(x)
    x = one.clone()
    x[[0, V - 1]] = 0.5
    rows.append(x)
    rows.append(torch.full((V,), 2.0 ** -12))      # adds up to more than 1
    rows.append(torch.full((V,), 2.0 ** -20))      # and to less
    x = one.clone()
    x[100:116] = 2.0 ** -4
    rows.append(x)
    us = [0.0, 2.0 ** -149, 2.0 ** -126, 2.0 ** -24, 2.0 ** -4, 0.5, 0.5 - 2.0 ** -25, 0.75, 1 - 2.0 ** -24]
    p = torch.stack([r for r in rows for _ in us])[:, None].to(dtype).cuda()
    u = torch.tensor(us * len(rows), device="cuda")[:, None].contiguous()
    _, tok = check(p, None, None, None, u)
    assert (tok[:4 * len(us), 0].reshape(4, -1) == np.array([0, 1, 2499, V - 1])[:, None]).all()


@pytest.mark.gpu
def test_verify_nothing_left_and_empty_rows():
    """Equal distributions refused by u (the difference is empty: the target is
    drawn from), rows without any probability, greedy drafts with all of it."""
    V = 777
    p, q, draft, _, u = make(5, 3, V, torch.float32, False, seed=3)
    q.copy_(p[:, :2])
    q.scatter_(2, draft.long()[..., None], 1.0)  # refused nearly always; elsewhere p - q is 0
    p.scatter_(2, torch.nn.functional.pad(draft, (0, 1)).long()[..., None], 0.0)
    u[:, :2] = 0.9
    acc, tok = check(p, q, draft, None, u)
    assert (acc == 0).all() and (tok[:, 0] >= 0).all()
    p.zero_()
    acc, tok = check(p, q, draft, None, u)
    assert (tok == -1).all()
    p[:, 0, 4] = 1  # a greedy draft of the only token there is, refused by its u alone
    draft[:, 0] = 4
    u[:, 0] = 1.0   # outside [0, 1): not below p
    acc, tok = check(p, None, draft, None, u)
    assert (acc == 0).all() and (tok[:, 0] == 4).all()


@pytest.mark.gpu
def test_verify_odd_values():
    """NaN, negative, infinite and large values, u outside [0, 1)."""
    V = 3001
    p, q, draft, _, u = make(8, 4, V, torch.float32, False, seed=4)
    p[0, :, 10:20] = float("nan")
    p[1, :, ::3] = -1
    p[2, :, 7] = 5.0
    q[3, :, ::2] = float("nan")
    q[4, :, ::2] = -0.5
    u[5] = float("nan")
    u[6] = -0.25
    u[7] = 1.5
    u[0, 3], u[1, 3] = 1.0, -1.0
    p[2, :, 9] = 2.5
    # the same once more with everything accepted up to the last row
    check(p, q, draft, None, u)
    u[:, :3] = 0
    check(p, q, draft, None, u)
    big = torch.ones(2, 1, 1 << 20, device="cuda")  # the largest sum there can be
    u = torch.tensor([[0.3], [1 - 2.0 ** -24]], device="cuda")
    _, tok = verify(big, None, None, None, u)
    assert tok[:, 0].tolist() == [int(np.floor(float(np.float32(0.3)) * (1 << 20))), (1 << 20) - 1]


@pytest.mark.gpu
def test_verify_reports_bad_drafts():
    p, q, draft, n_draft, u = make(4, 4, 500, torch.float32, False, seed=5)
    u[:, :3] = 0
    draft[1, 1], draft[2, 0] = 500, -1
    got = verify(p, q, draft, None, u, expect=H.HSWA_ERR_BOUNDS)
    exp = serving.verify(host(p), host(q), host(draft), None, host(u))
    assert np.array_equal(got[0], exp[0]) and got[0].tolist() == [3, 1, 0, 3]
    assert np.array_equal(got[1], exp[1])
    draft.clamp_(0, 499)
    n_draft = torch.tensor([-3, 9, 3, 0], dtype=torch.int32, device="cuda")
    got = verify(p, q, draft, n_draft, u, expect=H.HSWA_ERR_BOUNDS)
    exp = serving.verify(host(p), host(q), host(draft), host(n_draft), host(u))
    assert np.array_equal(got[0], exp[0]) and np.array_equal(got[1], exp[1])


@pytest.mark.gpu
def test_verify_large_batch_streams_and_graph():
    p, q, draft, n_draft, u = make(700, 3, 2000, torch.bfloat16, False, seed=6)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    exp = check(p, q, draft, n_draft, u, stream=side)
    acc = torch.zeros(700, dtype=torch.int32, device="cuda")
    tok = torch.zeros(700, 3, dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        H.hswa_verify_draft(H.HSWA_DTYPE_BF16, p, p.stride(1), q, q.stride(1), draft, n_draft, u, 700, 3, 2000, acc, tok, torch.cuda.current_stream())
    for _ in range(3):
        acc.fill_(-7)
        g.replay()
        assert H.hswa_check() == 0
        assert np.array_equal(acc.cpu().numpy(), exp[0]) and np.array_equal(tok.cpu().numpy(), exp[1])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sampled", [True, False])
def test_verify_infinities(dtype, sampled):
    """Infinities in p, q and u, at drafted values and others: the acceptance
    test is the inequality as it stands (0 times infinity is no number and
    refuses), the draw clamps them to [0, 1]."""
    V, inf = 1003, float("inf")
    p, q, draft, _, u = make(12, 4, V, dtype, not sampled, seed=8)
    u[:, :3] *= 0.01
    at = draft.long()
    for i, x in enumerate((inf, -inf)):
        p[i, 0, at[i, 0]] = x
        p[2 + i, :, 40:44] = x
        if sampled:
            q[4 + i, 0, at[4 + i, 0]] = x
            q[6 + i, :, 100:900:7] = x
        u[8 + i, 0] = x
    p[10, 1, at[10, 1]], u[10, 1] = inf, inf
    p[11, 2, at[11, 2]], u[11, 2] = -inf, -inf
    if sampled:
        q[4, 1, at[4, 1]], u[4, :2] = inf, 0.0
        q[11, 2, at[11, 2]] = inf
    acc, _ = check(p, q if sampled else None, draft, None, u)
    assert acc[0] > 0 and acc[1] == 0 and acc[8] == 0
    u[:, :3] = 0.9
    check(p, q if sampled else None, draft, None, u)
    u[:, 3] = torch.tensor([inf, -inf] * 6, device="cuda")
    check(p, q if sampled else None, draft, None, u)
