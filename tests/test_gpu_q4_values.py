"""Values of very different scales over the paged 4-bit cache, and values that are NaN."""
import numpy as np
import pytest
import torch

import sparse_decode_attention_gb300 as kvr
from oracle import quant4 as q4
from test_gpu_q4 import BF, DEV, F32, U, Batch, i32, word

pytestmark = pytest.mark.gpu


def params(b):
    """Parameters [page, head, token, 4 (K s, K z, V s, V z), groups] of a batch's pages, to be written."""
    NG = b.d // 32
    return b.np_pages[:, :, b.ps * b.d:].reshape(-1, b.H, b.ps * b.d // 4).view(np.float16).reshape(-1, b.H, b.ps, 4, NG)


def one_heavy_token(N, ps, d, tiny, weight, ordinary, seed=31):
    """A request whose logits are 0 but for one token's, which has `weight` times another token's
    probability and no value in group 0; group 0's values of the others are codes times `tiny`, group 1's
    have the scale `ordinary`, the rest of them are 0 (scale 0)."""
    b = Batch([N], 1, ps, d, seed=seed)
    par = params(b)
    heavy = N // 2 + 5
    for t in range(N):
        p = par[b.table[0, t // ps], 0, t % ps]
        p[0], p[1] = 0.0, 0.0
        if t == heavy:
            p[1, 0] = np.log(weight)
        p[2], p[3] = 0.0, 0.0
        p[2, 0] = 0.0 if t == heavy else tiny
        p[2, 1], p[3, 1] = ordinary, -7.5 * ordinary
    b.pages.copy_(torch.from_numpy(b.np_pages))
    return b


def product_tolerance(b, K, V, qn, scale, out, want):
    """Bound of every channel. With p the probabilities and P the largest: relative errors of logits and powers
    (72 u (A + 1) of a probability), fp16's half steps for bf16 outputs and two terms (2^-22 each) for fp32 ones, sums of
    n terms, the output's rounding; p itself is held to 2^-36 P; and the product of p and a scale, to 2^-25 in units
    of which the largest p has 2^11 at least: where a group's scales are under 2^-11 (fp32 outputs:
    2^-7), or pass 2, the units are such that the largest product of 32 tokens has 2^13 at least."""
    n = len(K)
    x = (K @ qn) * scale
    p = np.exp(x - x.max())
    P = 1.0 / p.sum()
    p = p * P
    A = abs(scale) * np.max(np.abs(qn) @ np.abs(K).T)
    g = V.reshape(n, -1, 32)
    R, top = g.max(-1) - g.min(-1), np.abs(g).max(-1)           # of every token and group
    rel = 2 * 72 * U * (A + 1) + n * U / 4 + (3 * 2.0 ** -11 if out == BF else 3 * 2.0 ** -22)
    tol = rel * (p[:, None] * (R + top)).sum(0) + 2.0 ** -36 * P * (top + R).sum(0)
    S = np.zeros_like(R)                                        # the largest scale of 32 tokens
    for i in range(0, n, 32):
        S[i:i + 32] = R[i:i + 32].max(0) / 15
    lifted = S < (2.0 ** -11 if out == BF else 2.0 ** -7)
    tol += 15 * P * np.where(lifted, 2.0 ** -38 * S, np.maximum(2.0 ** -36, 2.0 ** -38 * S)).sum(0)
    return np.repeat(tol, 32) + (2.0 ** -8 if out == BF else U) * np.abs(want)


@pytest.mark.parametrize("ot", [F32, BF])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("ps", [16, 64])
@pytest.mark.parametrize("tiny", [2.0 ** -12, 2.0 ** -15, 2.0 ** -18, 2.0 ** -21, 2.0 ** -24])
@pytest.mark.parametrize("weight,ordinary", [(3000.0, 0.1), (3000.0, 300.0), (300000.0, 0.1)])
def test_a_group_of_small_scales_beside_an_ordinary_one(ot, d, ps, tiny, weight, ordinary):
    N = 2976                      # whole spans of 32 tokens
    b = one_heavy_token(N, ps, d, tiny, weight, ordinary)
    q = torch.ones((1, 1, 12, d), dtype=BF, device=DEV)
    K, V = b.kv(0, 0, np.arange(N))
    want = q4.attend_row(np.ones(d), K, V, 1 / 32)
    tol = product_tolerance(b, K, V, np.ones(d), 1 / 32, ot, want)
    for rows in (q[:, :, :4], q):  # single blocks of query rows, and pairs of them
        for o in b.attend(rows.contiguous(), ot, 1 / 32):
            off = np.abs(o.double().cpu().numpy()[0, 0] - want)
            assert np.all(off <= tol), (off / tol).max(-1)


@pytest.mark.parametrize("ot", [F32, BF])
@pytest.mark.parametrize("d", [64, 128])
def test_scales_of_every_size_token_by_token(ot, d):
    """Scales of all fp16 sizes side by side, drafted tokens, a last span that is not whole."""
    N, ps = 1003, 32
    b = Batch([N], 1, ps, d, seed=33)
    par, rng = params(b), np.random.default_rng(34)
    for t in range(N):
        p = par[b.table[0, t // ps], 0, t % ps]
        p[2] = 2.0 ** rng.uniform(-24, 12 if t % 7 == 0 else -3, d // 32)
        p[3] = -7.5 * p[2].astype(np.float64)
    b.pages.copy_(torch.from_numpy(b.np_pages))
    for Lq, G in ((1, 4), (3, 5)):
        b.dense(Lq, G, BF, ot)
    idx = np.sort(rng.permutation(N - 40)[:500]).astype(np.int32)[None, None]
    q = b.query(1, 4, BF)[:, 0].contiguous()
    o, err = torch.full(q.shape, float("nan"), dtype=ot, device=DEV), word()
    kvr.kvr_sparse_attend_q4(b.cache, q, i32(b.table), i32(idx), i32([[500]]), i32(b.lens), 37, 0.1, o, b.ws(1, 4), err=err)
    assert kvr.kvr_read_error(err) == 0
    sel = q4.token_list(idx[0, 0], 500, N, 37)
    K, V = b.kv(0, 0, sel)
    for g in range(4):
        qn = q[0, g].double().cpu().numpy()
        want = q4.attend_row(qn, K, V, 0.1)
        tol = product_tolerance(b, K, V, qn, 0.1, ot, want)
        assert np.all(np.abs(o[0, g].double().cpu().numpy() - want) <= tol)


@pytest.mark.parametrize("ot", [F32, BF])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N", [64, 90, 899, 3000])
def test_a_nan_value_of_a_vanishing_probability(ot, d, N):
    """0 times NaN is NaN: a row that sees such a token has it, wherever the token lies; a row that does not, has not."""
    ps, Lq, NG = 32, 3, d // 32
    spots = {0, 17, 31, 32, N - 26, N - 4, N - 3, N - 1}
    for tok in sorted(t for t in spots if 0 <= t < N):
        b = Batch([N], 1, ps, d, seed=35)
        p = params(b)[b.table[0, tok // ps], 0, tok % ps]
        p[0], p[1] = 0.0, -100.0                    # a logit 100s under the others
        p[2, NG - 1], p[3, NG - 1] = np.nan, np.nan  # as kvr_append_q4 writes a group that fp16 cannot hold
        b.pages.copy_(torch.from_numpy(b.np_pages))
        for G in (1, 4):
            q = torch.ones((1, Lq, G, d), dtype=BF, device=DEV)
            want = np.zeros((Lq, G, d), bool)
            for t in range(Lq):
                if tok <= N - Lq + t:
                    want[t, :, 32 * (NG - 1):] = True
            for o in b.attend(q, ot, 0.1):
                assert np.array_equal(torch.isnan(o[0]).cpu().numpy(), want), (tok, G)
        idx = np.arange(0, N - 20, 3, dtype=np.int32)[None, None]
        o = torch.zeros((1, 4, d), dtype=ot, device=DEV)
        kvr.kvr_sparse_attend_q4(b.cache, torch.ones((1, 4, d), dtype=BF, device=DEV), i32(b.table), i32(idx),
                                 i32([[idx.size]]), i32([N]), 20, 0.1, o, b.ws(1, 4))
        seen = tok in q4.token_list(idx[0, 0], idx.size, N, 20)
        bad = torch.isnan(o[0]).cpu().numpy()
        assert not bad[:, :32 * (NG - 1)].any() and (bad[:, 32 * (NG - 1):] == seen).all(), tok
