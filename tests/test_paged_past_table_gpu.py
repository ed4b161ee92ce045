"""Lengths that pass the end of a sequence's page-table row.

Positions at or past max_pages * page_size have no page.  New tokens there
are not written (and move nothing that is), no query sees them, and every
token keeps its own position: one at or past the end sees all keys that have
a place, one before it the keys up to itself.
"""
import math

import pytest

from test_paged_gpu import Batch, S, check_forward, check_scores, forward, hook  # noqa: F401

pytestmark = pytest.mark.gpu

END = 320  # keys that the table has places for
LAST = 2**31 - 1 - END  # a length of 2^31 - 1


class Past(Batch):
    """Sequence b has ks[b] keys with a place and over[b] positions behind
    them (only where ks[b] is the table's end)."""

    def __init__(self, torch, qs, ks, over, *args, **kw):
        super().__init__(torch, qs, ks, *args, extra_cols=0, **kw)
        assert self.table.shape[1] * self.page == END
        assert all(k == END for k, x in zip(ks, over) if x)
        self.over = over
        self.lens = torch.tensor([k + x for k, x in zip(ks, over)], dtype=torch.int32,
                                 device="cuda")

    def weights(self, b, h, scale, causal, sinks=None):
        torch = self.torch
        nq, nk = self.qs[b], self.ks[b]
        q = self.q[self.rows(b), h].double()
        k = self.K[b][:, h // (self.hq // self.hkv)].double()
        x = q @ k.T * scale
        c = float((q.abs() @ k.abs().T).max() * abs(scale))
        if causal:
            place = nk + self.over[b] - nq + torch.arange(nq, device="cuda")
            x = x.masked_fill(torch.arange(nk, device="cuda")[None] > place[:, None], -math.inf)
        y = x if sinks is None else torch.cat([x, sinks[h].double().expand(nq, 1)], 1)
        z = torch.logsumexp(y, 1)
        return x, z, (x - z[:, None]).exp(), c


CASES = [  # qs, ks, over
    ([1, 1, 1, 1], [END, END, 100, END], [1, 7, 0, LAST]),
    ([3, 2, 1], [END, END, END], [1, 2, 0]),
    ([40, 70, 9], [END, END, 12], [30, 100, 0]),
    ([300, 200, 1], [END, END, END], [150, 1, 5]),
    ([500], [END], [330]),
]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("page", [16, 5, 64])
@pytest.mark.parametrize("hq,hkv,D", [(4, 1, 64), (14, 2, 128), (20, 1, 64)])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_tokens_keep_their_positions(cuda, S, case, hq, hkv, D, page, dtype):
    t = Past(cuda, *case, hq, hkv, D, dtype, page, pad=2)
    for causal in (True, False):
        o, lse = forward(S, t, causal=causal)
        check_forward(t, o, lse, 1 / math.sqrt(D), causal)
        base = cuda.rand(len(t.ks), hkv, END + 3, device="cuda")
        got = base.clone()
        S.sdpa_paged_scores(t.q, t.k_pages, lse, got, t.table, t.lens, cu_seqlens_q=t.cu,
                            causal=causal)
        check_scores(t, got, base, lse, 1 / math.sqrt(D), causal)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("ctas", [1, 3, 29])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_shared_out_differently(cuda, S, hook, case, ctas, dtype):
    hook("paged_ctas", ctas)
    t = Past(cuda, *case, 8, 2, 64, dtype, 16)
    o, lse = forward(S, t, sinks=t.sinks)
    check_forward(t, o, lse, 1 / 8, True, t.sinks)
    base = cuda.rand(len(t.ks), 2, END - 9, device="cuda")
    got = base.clone()
    S.sdpa_paged_scores(t.q, t.k_pages, lse, got, t.table, t.lens, cu_seqlens_q=t.cu)
    check_scores(t, got, base, lse, 1 / 8, True, t.sinks)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("page", [16, 5])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_write_drops_what_has_no_place(cuda, S, case, page, dtype):
    t = Past(cuda, *case, 2, 2, 64, dtype, page, poison=False, pad=1)
    want = [t.k_pages.clone(), t.v_pages.clone()]
    for b in range(len(t.qs)):
        for i in range(t.qs[b]):
            p = t.ks[b] + t.over[b] - t.qs[b] + i
            if 0 <= p < END:
                at = int(t.table[b, p // page])
                want[0][at, :, p % page] = t.k[t.rows(b)][i]
                want[1][at, :, p % page] = t.v[t.rows(b)][i]
    S.sdpa_paged_write(t.k, t.v, t.k_pages, t.v_pages, t.table, t.lens, cu_seqlens_q=t.cu)
    assert cuda.equal(t.k_pages, want[0]) and cuda.equal(t.v_pages, want[1])


@pytest.mark.parametrize("over", [1, LAST])
def test_write_of_single_tokens_without_offsets(cuda, S, over):
    t = Past(cuda, [1, 1], [END, 17], [over, 0], 2, 2, 64, "f16", 16, poison=False)
    k, v = t.k_pages.clone(), t.v_pages.clone()
    at = int(t.table[1, 1])
    k[at, :, 0], v[at, :, 0] = t.k[1], t.v[1]
    S.sdpa_paged_write(t.k, t.v, t.k_pages, t.v_pages, t.table, t.lens)
    assert cuda.equal(t.k_pages, k) and cuda.equal(t.v_pages, v)


def test_evict_of_a_length_past_the_table(cuda, S):
    """Only the keys that have a place compete."""
    from test_paged_gpu import check_evict
    t = Past(cuda, [0, 0], [END, 90], [4, 0], 2, 2, 64, "bf16", 16)
    check_evict(cuda, S, t, cuda.rand(2, 2, END + 4, device="cuda"), 100, 10)
