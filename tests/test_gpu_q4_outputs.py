"""fp32 outputs over the paged 4-bit cache are held to fp32's errors, not to those of fp16 products; and the
long runs of one warp: lists of many spans, sums folded on the way."""
import numpy as np
import pytest
import torch

import sparse_decode_attention_gb300 as kvr
from oracle import quant4 as q4
from test_gpu_q4 import BF, DEV, F32, U, Batch, i32, tolerance, word

pytestmark = pytest.mark.gpu


def many(b, B):
    """The batch's one request B times over: tables may share pages."""
    b.lens = b.lens * B
    b.table, b.wide = (np.repeat(t, B, 0) for t in (b.table, b.wide))
    return b


def value_parts(b, n):
    """Scales and zeros of the values of the first n tokens of request 0, head 0: [n, d] each."""
    NG, t = b.d // 32, np.arange(n)
    par = np.ascontiguousarray(b.np_pages[:, 0, b.ps * b.d:]).view(np.float16).astype(np.float64).reshape(-1, b.ps, 4, NG)
    return tuple(np.repeat(par[b.table[0, t // b.ps], t % b.ps, i], 32, -1) for i in (2, 3))


def with_fp16_products(p, s, code, z, first, second):
    """The output with probabilities and (or) their products with scales rounded to fp16, as the bf16 form has them."""
    w = p / p.max() * 2.0 ** 11
    w = w.astype(np.float16).astype(np.float64) if first else w
    u = w[:, None] * s
    u = u.astype(np.float16).astype(np.float64) if second else u
    return ((u * code).sum(0) + w @ z) / w.sum()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("qt", [BF, F32])
@pytest.mark.parametrize("N,B,G", [(3000, 1, 4), (2500, 160, 4), (6000, 160, 4), (3000, 1, 16)])
def test_fp32_outputs_have_the_errors_of_fp32(d, qt, N, B, G):
    """Values are independent of queries and keys, with mean 0, so relative errors e of the probabilities move an
    output by max(e) of itself (root of the mean square over its channels): 72 u (A + 1). The codes' part C = p (s c)
    and the zeros' part, which cancel but for the output, come from products that truncate by 4 u of the parts
    at most, two for each. Products as pairs of fp16 terms: 2^-22. One fp16 term in place of either pair
    has 2^-12 and more, and would fail: such outputs, made here, are over the bound."""
    scale = 0.02
    b = many(Batch([N], 1, 64, d, seed=51), B)
    q = b.query(1, G, qt)
    K, V = b.kv(0, 0, np.arange(N))
    s, z = value_parts(b, N)
    code = np.rint((V - z) / s)
    outs = [o.double().cpu().numpy() for o in b.attend(q, F32, scale)]
    qn = q.double().cpu().numpy()
    norm = lambda x: np.sqrt((x ** 2).mean())  # noqa: E731
    for r in sorted({0, B // 2, B - 1}):
        for g in range(G):
            x = (K @ qn[r, 0, g]) * float(np.float32(scale))
            p = np.exp(x - x.max())
            p /= p.sum()
            want = p @ V
            A = scale * np.max(np.abs(qn[r, 0, g]) @ np.abs(K).T)
            tol = (72 * U * (A + 1) + 2.0 ** -21) * norm(want) + 8 * U * (norm(p @ (s * code)) + norm(p @ np.abs(z)))
            for o in outs:
                off = norm(o[r, 0, g] - want)
                assert off <= tol, (r, g, off / norm(want), tol / norm(want))
            for rounded in ((True, False), (False, True)):
                planted = with_fp16_products(p, s, code, z, *rounded)
                assert norm(planted - want) > tol, (rounded, norm(planted - want) / norm(want), tol / norm(want))


@pytest.mark.parametrize("ot", [F32, BF])
@pytest.mark.parametrize("d", [64, 128])
def test_many_spans_of_a_warp(ot, d):
    """160 requests of 13000 tokens: a CTA to each, sums folded every 32 spans (bf16 outputs); all tokens, and the
    same tokens as a region, and as lists of 12500."""
    N, B, G, scale = 13000, 160, 4, 0.1
    b = many(Batch([N], 1, 64, d, seed=52), B)
    q = b.query(1, G, BF)
    K, V = b.kv(0, 0, np.arange(N))
    qn = q.double().cpu().numpy()
    rng = np.random.default_rng(53)
    picked = np.sort(rng.permutation(N)[:12500]).astype(np.int32)
    err, ws, table, lens = word(), b.ws(1, G), i32(b.table), i32(b.lens)
    idx = i32(np.broadcast_to(picked, (B, 1, 12500)).copy())
    got = {}
    o = torch.full(q.shape, float("nan"), dtype=ot, device=DEV)
    kvr.kvr_attend_q4(b.cache, q, table, lens, scale, o, ws, err)
    got["all"] = (o, np.arange(N))
    rows = q[:, 0].contiguous()
    for name, count, end in (("region", 0, 0), ("list", 12500, N)):
        o = torch.full(rows.shape, float("nan"), dtype=ot, device=DEV)
        kvr.kvr_sparse_attend_q4(b.cache, rows, table, idx, i32([[count]] * B), lens, 0, scale, o, ws,
                                 region_end=i32([end] * B), err=err)
        got[name] = (o[:, None], np.arange(N) if name == "region" else picked)
    assert kvr.kvr_read_error(err) == 0
    for r in (0, 1, 77, 151, 152, 159):
        for g in range(G):
            for name, (o, sel) in got.items():
                want = q4.attend_row(qn[r, 0, g], K[sel], V[sel], scale)
                tol = tolerance(qn[r, 0, g], K[sel], V[sel], scale, len(sel), ot, want)
                assert np.all(np.abs(o[r, 0, g].double().cpu().numpy() - want) <= tol), (name, r, g)


@pytest.mark.parametrize("qt,ot", [(BF, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("d", [64, 128])
def test_long_lists_of_more_units_than_sms(d, qt, ot):
    """160 units with lists of up to 2100 tokens: CTAs of twelve warps, several turns of their rings."""
    rng = np.random.default_rng(54)
    b = many(Batch([2600], 2, 32, d, seed=55), 80)
    b.lens = rng.integers(2000, 2601, 80).tolist()
    b.lens[:2] = 2600, 3
    k, W, sink, G = 2000, 90, 5, 4
    idx, cnt = np.full((80, 2, k), -1, np.int32), np.zeros((80, 2), np.int32)
    for r, n in enumerate(b.lens):
        for h in range(2):
            c = max(0, min(k - 37 * h, n - W - sink))
            idx[r, h, :c] = np.sort(rng.permutation(np.arange(sink, max(sink, n - W)))[:c])
            cnt[r, h] = c
    q = b.query(1, 2 * G, qt)[:, 0].contiguous()
    o, err = torch.full(q.shape, float("nan"), dtype=ot, device=DEV), word()
    kvr.kvr_sparse_attend_q4(b.cache, q, i32(b.table), i32(idx), i32(cnt), i32(b.lens), W, 0.1, o, b.ws(1, 2 * G),
                             sink=sink, err=err)
    assert kvr.kvr_read_error(err) == 0
    qn, on = q.double().cpu().numpy(), o.double().cpu().numpy()
    for r in range(0, 80, 1 if ot == BF else 5):
        for h in range(2):
            pos = q4.token_list(idx[r, h], cnt[r, h], b.lens[r], W, sink)
            K, V = b.kv(r, h, pos)
            for g in range(h * G, (h + 1) * G):
                want = q4.attend_row(qn[r, g], K, V, 0.1)
                tol = tolerance(qn[r, g], K, V, 0.1, len(pos), ot, want)
                assert np.all(np.abs(on[r, g] - want) <= tol), (r, g)
