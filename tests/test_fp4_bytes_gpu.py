"""Every byte of codes at every place of a row, in each kernel of the attention over the 4-bit
cache.

A sequence of one key: O is its value row, whatever the query, and LSE the key's element that a query
of a single 1 picks, times the scale.  The key's weight, its sum and the quotient are off by a few
roundings of numbers up to 2^5 (scores below 17 in units of ln 2): less than 2^-18 in all, which the
rounding of O to 16 bits removes, element values having six significant bits.  LSE is off by less
than 2^-20 of itself and 2^-20.  Codes of one scale differ by 0.5 and more.
"""
import pytest

from test_fp4_gpu import DT, S, values_of  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("tokens,heads", [(1, 8), (1, 16), (64, 1), (32, 8)])
@pytest.mark.parametrize("page", [16, 4])
def test_every_byte_at_every_place(cuda, S, page, tokens, heads, D, dtype):  # noqa: F811
    dt, B = getattr(cuda, DT[dtype]), 256
    b = cuda.arange(B, device="cuda")[:, None]
    j = cuda.arange(D // 2, device="cuda")[None]
    rows = [((b * m + 37 * j + 5) & 255).to(cuda.uint8) for m in (1, 3)]  # (odd: every byte)
    group = cuda.arange(D // 16, device="cuda")[None]
    sc = [(0x30 + (b + 3 * group + i) % 16).to(cuda.uint8) for i in range(2)]

    def pages(x):
        p = cuda.zeros(B, 1, page, x.shape[1], device="cuda", dtype=cuda.uint8)
        p[:, 0, 0] = x
        return p

    cache = [pages(x) for x in rows + sc]
    k, v = (values_of(cuda, x, y) for x, y in zip(rows, sc))
    table = cuda.arange(B, dtype=cuda.int32, device="cuda")[:, None]
    lens = cuda.ones(B, dtype=cuda.int32, device="cuda")
    cu = cuda.arange(B + 1, dtype=cuda.int32, device="cuda") * tokens
    per = tokens * heads  # elements that a call picks, one a row
    for first in range(0, D, per):
        pick = (first + cuda.arange(per, device="cuda")) % D
        q = cuda.zeros(per, D, device="cuda", dtype=dt)
        q[cuda.arange(per), pick] = 1.0
        q = q.view(1, tokens, heads, D).expand(B, tokens, heads, D).reshape(B * tokens, heads, D)
        o, lse = S.sdpa_paged_forward_fp4(q, *cache, table, lens, cu_seqlens_q=cu, scale=1.0,
                                          causal=False)
        want = v[:, None, None].expand(B, tokens, heads, D).reshape(o.shape)
        off = (o.double() - want).abs()
        assert (off <= (want.abs() * 2.0**-18 if dtype == "f32" else 0.0)).all()
        want = k[:, pick].reshape(lse.shape)
        assert ((lse.double() - want).abs() <= want.abs() * 2.0**-20 + 2.0**-20).all()
