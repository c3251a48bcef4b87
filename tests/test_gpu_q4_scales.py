"""Scales of groups whose range is a few fp32 steps of their offset: 15 s + z rounds at the size of z
there, so the smallest fp16 scale that covers the maximum lies many fp16 steps under the quotient
(maximum - z) / 15. Bytes and values equal the oracle's, which searches all of fp16."""
import numpy as np
import pytest
import torch

import sparse_decode_attention_gb300 as kvr
from oracle import quant4 as q4

pytestmark = pytest.mark.gpu

DEV = "cuda"


def narrow_rows(rng, n, H, d):
    """fp32 rows, every group an offset and up to 2000 fp32 steps more; the minimum is an fp16 value or,
    in every third token, between two."""
    x = np.empty((n, H, d // 32, 32), np.float32)
    base = np.float16([1000.0, -1000.0, 32.0, -32.0, 100.0, 0.1, -0.1, 3.0, 60000.0, -60000.0, 2.0 ** -20, -(2.0 ** -24)])
    for t in range(n):
        lo = np.float32(base[rng.integers(0, len(base), (H, d // 32))])
        if t % 3 == 2:
            lo = lo * np.float32(1.0 + rng.uniform(0, 2.0 ** -11))
        steps = [1, 2, 3, 20, 100, 2000][t % 6]
        at = rng.integers(0, steps + 1, (H, d // 32, 32))
        at[..., 5], at[..., 17] = 0, steps
        x[t] = lo[..., None] + at * np.spacing(np.abs(lo))[..., None]
    return x.reshape(n, H, d)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H", [1, 2])
def test_groups_of_a_few_steps_at_an_offset(d, H):
    rng = np.random.default_rng(d + H)
    n, ps = 240, 16
    K, V = narrow_rows(rng, n, H, d), narrow_rows(rng, n, H, d)
    want = np.zeros((n // ps, H, ps * q4.token_bytes(d)), np.uint8)
    for t in range(n):
        for h in range(H):
            q4.write_token(want, ps, d, t, h, K[t, h], V[t, h])
    pages, slot = torch.zeros(want.shape, dtype=torch.uint8, device=DEV), torch.arange(n, device=DEV)
    cache, err = kvr.Q4Cache(pages, ps, d), torch.zeros(1, dtype=torch.int32, device=DEV)
    kvr.kvr_append_q4(cache, torch.from_numpy(K).to(DEV), torch.from_numpy(V).to(DEV), slot, err)
    assert kvr.kvr_read_error(err) == 0
    assert np.array_equal(pages.cpu().numpy(), want)
    Ko, Vo = torch.zeros((n, H, d), device=DEV), torch.zeros((n, H, d), device=DEV)
    kvr.kvr_read_q4(cache, slot, Ko, Vo)
    for got, x in ((Ko, K), (Vo, V)):
        assert torch.equal(got.cpu(), torch.from_numpy(q4.values(*q4.quantise(x))).float())


def test_every_few_steps_above_every_binade():
    """One group per row: minima on fp16's grid in all its binades, maxima 1 to 40 fp32 steps above."""
    rng = np.random.default_rng(3)
    lo = np.concatenate([rng.integers(1024 * e, 1024 * e + 1024, 16) for e in range(31)]).astype(np.uint16).view(np.float16)
    lo = np.concatenate([lo, -lo]).astype(np.float32)
    x = np.repeat(lo[:, None], 40, 1)
    top = x + np.arange(1, 41, dtype=np.float32) * np.spacing(np.abs(x))
    rows = np.repeat(x.reshape(-1, 1), 64, 1)
    rows[:, 9], rows[:, 40] = top.reshape(-1), top.reshape(-1)
    n = len(rows)
    cache = kvr.Q4Cache.empty(-(-n // 64), 64, 1, 64)
    X, slot = torch.from_numpy(rows[:, None]).to(DEV), torch.arange(n, device=DEV)
    kvr.kvr_append_q4(cache, X, X, slot)
    Ko, Vo = torch.zeros_like(X), torch.zeros_like(X)
    kvr.kvr_read_q4(cache, slot, Ko, Vo)
    c, s, z = q4.quantise(rows)
    par = cache.pages.cpu().numpy()[:, 0, 64 * 64:].reshape(-1, 16)[:n].copy().view(np.float16).astype(np.float64)
    assert np.array_equal(par[:, 0:2], s) and np.array_equal(par[:, 4:6], s)
    want = torch.from_numpy(q4.values(c, s, z)).float()
    assert torch.equal(Ko[:, 0].cpu(), want) and torch.equal(Vo[:, 0].cpu(), want)
