"""Softmax weights of fp32 calls over the 4-bit cache: one key far above a long tail of equal ones.

The first key scores `gap` above every other and its value is zero, so O is the tail's alone and a
relative error of the tail's weights is one of O.  Queries have one element, 1, and the keys' products
with it are exact, so a weight 2^((s - m) log2 e) differs from the exact one by the rounding of scale *
log2 e (2 units of 2^-24), of its product with the score and of the reference (2 more), times gap *
log2 e * ln 2, and by its exponential's 2^-22:  gap 2^-22 + 2^-22.  A weight enters the value product as
two fp16 parts, the second scaled so that it holds what the first leaves to 2^-22 of the weight or to
2^-41 of the largest.  The product adds up nk / 16 terms in fp32, one unit each; O is rounded once.
"""
import math

import pytest

from test_fp4_gpu import S, values_of  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


def tail_cache(torch, n, D, page=64, seed=0):
    """A kv head of n keys: the first one's first element is 1, all others are 0; values positive,
    but for the first, which is 0."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    pages = -(-n // page)
    kc, vc = (torch.zeros(pages, 1, page, D // 2, device="cuda", dtype=torch.uint8) for _ in "kv")
    ks, vs = (torch.full((pages, 1, page, D // 16), 0x38, device="cuda", dtype=torch.uint8)
              for _ in "kv")
    kc[0, 0, 0, 0] = 2  # code 2: 1
    digits = torch.randint(1, 8, (2,) + vc.shape, generator=g, device="cuda", dtype=torch.uint8)
    vc[:] = digits[0] | (digits[1] << 4)
    vc[0, 0, 0] = 0
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    v = values_of(torch, vc, vs)[:, 0].flatten(0, 1)[:n]
    return kc, vc, ks, vs, table, v


@pytest.mark.parametrize("bits", [20.3, 24.6, 26.3, 28.85, 29.2, 33.0])
@pytest.mark.parametrize("n,nq,heads", [(32769, 1, 4), (32769, 3, 4), (32769, 50, 4), (5000, 1, 1),
                                        (5000, 140, 1)])
@pytest.mark.parametrize("D", [64, 128])
def test_long_tail_under_one_key(cuda, S, D, n, nq, heads, bits):  # noqa: F811
    kc, vc, ks, vs, table, v = tail_cache(cuda, n, D)
    q = cuda.zeros(nq, heads, D, device="cuda")
    q[:, :, 0] = 1.0
    gap = bits * math.log(2.0)
    scale = float(cuda.tensor(gap, dtype=cuda.float32))
    o, lse = S.sdpa_paged_forward_fp4(
        q, kc, vc, ks, vs, table, cuda.tensor([n], dtype=cuda.int32, device="cuda"),
        cu_seqlens_q=cuda.tensor([0, nq], dtype=cuda.int32, device="cuda"), scale=scale)
    sums = v.cumsum(0)
    for i in range(nq):
        seen = n - nq + i + 1
        w = math.exp(-scale)
        total = 1.0 + (seen - 1) * w
        ref = sums[seen - 1] * (w / total)
        rel = 2 * (gap + 1) * 2.0**-22 + 2.0**-22 + (seen / 16 + 8) * 2.0**-23 + 2.0**-23
        tol = rel * 1.01 * ref + 2.0**-41 / total * sums[seen - 1]
        err = (o[i].double() - ref).abs()
        assert (err <= tol).all(), (i, float((err / ref).max()), float((tol / ref).min()))
        z = scale + math.log(total)
        assert ((lse[i].double() - z).abs() <= (gap + 1) * 2.0**-22 + z * 2.0**-22 + 2.0**-21).all()
