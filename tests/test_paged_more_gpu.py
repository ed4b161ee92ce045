"""Paged attention whose running maximum moves from tile to tile, in every
kernel, scores that overflow to -inf, and eviction of sequences longer than
the selection keeps in shared memory."""
import math

import pytest

from test_paged_gpu import (Batch, S, check_evict, check_forward, check_scores,  # noqa: F401
                            forward, hook)

pytestmark = pytest.mark.gpu

# rows of a sequence and kv head: up to 4, 8 and 16, 17 to 128, more
KINDS = [([1, 1], 4, 2), ([1, 1], 12, 2), ([1, 1], 28, 2), ([2, 1], 8, 1), ([9, 30], 4, 2),
         ([150, 90], 4, 2)]


def rewrite(t):
    """The cache's rows from t.K and t.V."""
    for b, n in enumerate(t.ks):
        pos = t.torch.arange(n, device="cuda")
        pg = t.table[b, pos // t.page].long()
        t.k_pages[pg, :, pos % t.page] = t.K[b]
        t.v_pages[pg, :, pos % t.page] = t.V[b]


@pytest.mark.parametrize("ctas", [0, 1, 7])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("page", [16, 12])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kind", KINDS, ids=str)
def test_scores_that_grow(cuda, S, hook, kind, D, page, dtype, ctas):
    """Each run of 64 keys larger than the one before: the maximum moves
    tile after tile, and pieces of a cut unit are far apart."""
    hook("paged_ctas", ctas)
    qs, hq, hkv = kind
    t = Batch(cuda, qs, [1300, 800], hq, hkv, D, dtype, page)
    for b, n in enumerate(t.ks):
        grow = 1 + cuda.arange(n, device="cuda").div(64, rounding_mode="floor")
        t.K[b] = (t.K[b].float() * grow[:, None, None] / 2).to(t.dtype)
    rewrite(t)
    scale = 4 / D
    o, lse = forward(S, t, scale=scale)
    check_forward(t, o, lse, scale)
    base = cuda.zeros(2, hkv, 1300, device="cuda")
    got = base.clone()
    S.sdpa_paged_scores(t.q, t.k_pages, lse, got, t.table, t.lens, cu_seqlens_q=t.cu, scale=scale)
    check_scores(t, got, base, lse, scale)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("page", [16, 12])
@pytest.mark.parametrize("kind", KINDS, ids=str)
def test_scores_of_minus_infinity(cuda, S, kind, page, dtype):
    """Keys of the type's lowest values, whose scores overflow to -inf, add
    exactly what keys of vanishing weight add: nothing."""
    qs, hq, hkv = kind
    results = []
    for value in (cuda.finfo(getattr(cuda, "float32" if dtype == "f32" else "bfloat16")).min, -1e5):
        t = Batch(cuda, qs, [1300, 800], hq, hkv, 64, dtype, page)
        t.q[:, :, 0] = t.q[:, :, 0].abs() + 2
        for b in range(2):
            for j in (0, 5, 130, 131, 132, 600, t.ks[b] - 200):
                t.K[b][j] = 0
                t.K[b][j, :, 0] = value
        rewrite(t)
        o, lse = forward(S, t)
        sc = cuda.zeros(2, hkv, 1300, device="cuda")
        S.sdpa_paged_scores(t.q, t.k_pages, lse, sc, t.table, t.lens, cu_seqlens_q=t.cu)
        results.append((o, lse, sc))
    for a, b in zip(*results):
        assert a.isfinite().all() and cuda.equal(a, b)
    assert (results[0][2][:, :, [0, 5, 130, 131, 132, 600]] == 0).all()


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("ks,keep,recent", [
    ([60001, 49152, 49153], 20000, 500), ([70000], 300, 0), ([49153, 1000], 49152, 49152),
    ([131072], 65000, 64)], ids=str)
@pytest.mark.parametrize("kind", ["uniform", "ties", "special"])
def test_evict_of_very_long_sequences(cuda, S, kind, ks, keep, recent, inplace):
    """More positions than the selection keeps in shared memory (49152)."""
    t = Batch(cuda, [0] * len(ks), ks, 1, 1, 64, "bf16", 64)
    g = cuda.Generator(device="cuda").manual_seed(7)
    s = cuda.rand(len(ks), 1, max(ks), generator=g, device="cuda")
    if kind == "ties":
        s = (s * 5).floor()
    elif kind == "special":
        s = cuda.where(s < 0.1, float("nan"), s - 0.5)
        s = cuda.where(s > 0.4, float("inf"), s)
    check_evict(cuda, S, t, s, keep, recent, inplace)
