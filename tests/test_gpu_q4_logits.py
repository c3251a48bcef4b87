"""Large logits over the paged 4-bit cache, all output types.

A logit's error counts absolutely, as exp turns it into a relative one of the probability. The bound is the one
of tests/test_gpu_q4.py: with A = |scale| sum |q_c k_c| and u = 2^-24, 68 u A for the logit and 4 u (A + 1) for the
power, for bf16 outputs as for fp32 ones."""
import numpy as np
import pytest
import torch

import sparse_decode_attention_gb300 as kvr
from test_gpu_q4 import BF, DEV, F32, TYPES, U, Batch, i32, word

pytestmark = pytest.mark.gpu


def twins(rng, B, d, G, big, A):
    """B requests of two tokens with values +1 and -1 whose keys s c (s = 1/8, z = 0) agree in one channel
    of code 1, where the query is `big` times its other channels, and queries that are
    nearly orthogonal to the keys' difference: (K, V, q, scales of the heads' logits)."""
    out = rng.integers(0, d, B)
    code = rng.integers(0, 16, (B, 2, d))
    for b in range(B):
        for t in range(2):
            for g in range(d // 32):
                own = 32 * g + rng.permutation([i for i in range(32) if 32 * g + i != out[b]])
                code[b, t, own[0]], code[b, t, own[1]] = 0, 15
        code[b, :, out[b]] = 1
    K = code / 8.0
    diff = K[:, 0] - K[:, 1]
    q = rng.standard_normal((B, G, d))
    q -= (np.einsum("bgd,bd->bg", q, diff) / (diff ** 2).sum(-1)[:, None])[..., None] * diff[:, None]
    q[np.arange(B), :, out] *= big
    q = torch.from_numpy(q.astype(np.float32)).to(BF)
    qn = q.double().numpy()
    scale = A / np.median(np.einsum("bgd,btd->bgt", np.abs(qn), K))
    V = np.stack([np.ones((B, d)), -np.ones((B, d))], 1)
    return K, V, q, float(scale)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("big", [1.0, 30.0, 300.0])
@pytest.mark.parametrize("qt,ot", TYPES)
@pytest.mark.parametrize("G", [4, 16])
def test_two_keys_with_nearly_equal_large_logits(d, big, qt, ot, G):
    """The output is tanh of half of the logits' difference, so it shows their errors as they are."""
    rng = np.random.default_rng(int(big) + d + G)
    B, ps = 24, 16
    K, V, q, scale = twins(rng, B, d, G, big, 3000.0)
    cache = kvr.Q4Cache.empty(B, ps, 1, d)
    slot = torch.arange(B, device=DEV)[:, None] * ps + torch.arange(2, device=DEV)
    rows = [torch.from_numpy(x.astype(np.float32)).reshape(2 * B, 1, d).to(DEV) for x in (K, V)]
    kvr.kvr_append_q4(cache, *rows, slot.reshape(-1).contiguous())
    held = [torch.zeros_like(x) for x in rows]
    kvr.kvr_read_q4(cache, slot.reshape(-1).contiguous(), *held)
    assert torch.equal(held[0], rows[0]) and torch.equal(held[1], rows[1])   # the cache holds them exactly
    qn = q.double().numpy()
    logit = np.einsum("bgd,btd->bgt", qn, K) * float(np.float32(scale))
    A = np.einsum("bgd,btd->bgt", np.abs(qn), K).max(-1) * scale
    want = np.tanh((logit[..., 0] - logit[..., 1]) / 2)
    assert np.median(np.abs(want)) < 0.9
    # each logit 68 u A, each power 4 u (A + 1); half of the difference. bf16: each probability half a step of fp16
    tol = 72 * U * (A + 1) + (2.0 ** -11 + 2.0 ** -8 * np.abs(want) if ot == BF else 2.0 ** -21)
    for P in (1, 25000 // ps):
        table = np.full((B, P), -1, np.int32)
        table[:, 0] = np.arange(B)
        o, err = torch.full((B, G, d), float("nan"), dtype=ot, device=DEV), word()
        ws = kvr.workspace(kvr.kvr_attend_q4_workspace_size(cache, B, 1, G))
        kvr.kvr_attend_q4(cache, q.to(qt).to(DEV), i32(table), i32([2] * B), scale, o, ws, err)
        assert kvr.kvr_read_error(err) == 0
        off = np.abs(o.double().cpu().numpy() - want[..., None]).max(-1)
        assert np.all(off <= tol), (P, (off / tol).max(), off.max())


@pytest.mark.parametrize("scale", [3.0, 0.0, -0.5])
def test_sharp_and_flat_logits_bf16_outputs(scale):
    Batch([2000, 130], 2, 64, 128, seed=7).dense(1, 4, BF, BF, scale=scale)
    Batch([2000, 130], 1, 64, 64, seed=8).dense(1, 8, F32, BF, scale=scale)


def test_queries_of_extreme_size_bf16_outputs():
    b = Batch([300], 1, 32, 128, seed=12)
    for mag in (1e-30, 1e-6, 1e6, 1e30):
        q = (b.query(1, 4, F32) * mag).to(BF)
        q[0, 0, 1] = 0
        for o in b.attend(q, BF, 0.088 / mag):
            b.check_dense(q, o, 0.088 / mag)
    q = b.query(1, 4, F32)
    q[..., 5] *= 1e6
    for o in b.attend(q, BF, 1e-7):
        b.check_dense(q, o, 1e-7)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("qt,ot", TYPES)
@pytest.mark.parametrize("size", [2.0 ** 26, 3e8, 1e10, -1e20, 1e35])
def test_logits_far_beyond_the_softmax_reference(d, qt, ot, size):
    """Logits whose fp32 steps are larger than the differences a softmax sees: the largest one's value, where it
    leads by more than their errors."""
    b = Batch([1, 2, 33, 300, 2100], 2, 64, d, seed=19)
    scale = size / (0.3 * d)
    q = b.query(1, 8, qt)
    qn, rows = q.double().cpu().numpy(), 0
    for o in b.attend(q, ot, scale):
        on = o.double().cpu().numpy()
        for r, N in enumerate(b.lens):
            for h in range(2):
                K, V = b.kv(r, h, np.arange(N))
                for g in range(4 * h, 4 * h + 4):
                    x = (K @ qn[r, 0, g]) * float(np.float32(scale))
                    A = abs(scale) * np.max(np.abs(qn[r, 0, g]) @ np.abs(K).T)
                    at = np.argsort(x)
                    if N > 1 and x[at[-1]] - x[at[-2]] <= 2 * 72 * U * (A + 1) + 60:
                        continue
                    rows += 1
                    want, v = V[at[-1]], np.abs(V).max()
                    R = V.reshape(N, -1, 32).max() - V.reshape(N, -1, 32).min()
                    # one token: its probability cancels but for the roundings of the products and the quotient
                    tol = 8 * U * v + (2.0 ** -8 * np.abs(want) + 2.0 ** -11 * (3 * R + v) if ot == BF else U * np.abs(want) + 2.0 ** -21 * (R + v))
                    assert np.all(np.abs(on[r, 0, g] - want) <= tol), (N, g, on[r, 0, g][:4], want[:4])
    assert rows > 40


def test_a_zero_query_under_the_largest_scale():
    """All logits are 0: the mean of the values."""
    b = Batch([1, 90, 700], 1, 32, 128, seed=20)
    for qt in (BF, F32):
        q = torch.zeros((3, 1, 4, 128), dtype=qt, device=DEV)
        for ot in (BF, F32):
            for o in b.attend(q, ot, 3e38):
                b.check_dense(q, o, 3e38)


def test_the_largest_scales_of_the_smallest_queries():
    """Ordinary logits of a scale of 3.3e38, which times log2 e would pass fp32."""
    b = Batch([1, 90, 700], 2, 32, 128, seed=22)
    for qt in (BF, F32):
        q = (b.query(2, 8, F32).double() * 1e-39).to(qt)
        for ot in (BF, F32):
            for o in b.attend(q, ot, 3.3e38):
                b.check_dense(q, o, 3.3e38)
