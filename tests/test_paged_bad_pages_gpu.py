"""Page-table entries outside the cache: such a page reads as zero keys and
values, rows written to it are dropped, and the device status word is set."""
import math

import numpy as np
import pytest

from test_paged_gpu import Batch, check_forward, check_scores, evict_reference, forward

pytestmark = pytest.mark.gpu


def status(cuda, S):
    return S.sdpa_device_status(cuda.cuda.current_stream().cuda_stream)


@pytest.fixture
def lib(cuda):
    import scaled_dot_product_fwd_gb300 as S
    status(cuda, S)
    yield S
    status(cuda, S)


def bad_columns(t, b, columns, value):
    """Columns of sequence b name no page; the plain rows read zero there."""
    for c in columns:
        t.table[b, c] = value
        for rows in (t.K, t.V):
            rows[b][c * t.page:(c + 1) * t.page] = 0


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("hq,qs,ks", [
    (8, [1, 1], [100, 700]), (24, [1, 1], [100, 700]), (8, [1, 40], [100, 700]),
    (8, [90, 300], [100, 700])], ids=str)
@pytest.mark.parametrize("page", [16, 12])
def test_attention_and_weights_read_zeros(cuda, lib, page, hq, qs, ks, dtype):
    t = Batch(cuda, qs, ks, hq, 2, 64, dtype, page)
    # one in the middle, the first, and the last (which the length ends in)
    bad_columns(t, 1, [0, 9, (ks[1] - 1) // page], t.k_pages.shape[0])
    bad_columns(t, 0, [2], -1)
    o, lse = forward(lib, t)
    assert status(cuda, lib) == 7
    check_forward(t, o, lse, 1 / 8)
    base = cuda.rand(2, 2, max(ks), device="cuda")
    got = base.clone()
    lib.sdpa_paged_scores(t.q, t.k_pages, lse, got, t.table, t.lens, cu_seqlens_q=t.cu)
    assert status(cuda, lib) == 7
    check_scores(t, got, base, lse, 1 / 8)


@pytest.mark.parametrize("value", [-1, None, 2**31 - 1, -2**31])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("keep", [60, 100, 300, 700, 1500])
def test_eviction(cuda, lib, keep, D, dtype, value):
    """The kept rows are those of the scores; one from a bad page arrives as
    zeros, one that would go to a bad page is dropped."""
    torch = cuda
    page, ks, hkv = 16, [3000, 1700, 40], 2
    t = Batch(torch, [0] * 3, ks, hkv, hkv, D, dtype, page)
    if value is None:
        value = t.k_pages.shape[0]
    scores = torch.rand(3, hkv, max(ks), device="cuda") ** 3
    kept = evict_reference(t, scores, keep, 20)
    # rows are taken from below and past the budget; rows go below it
    bad = {0: [1, keep // page // 2, keep // page + 3, 120, (ks[0] - 1) // page],
           1: [0, (ks[1] - 1) // page]}
    for b, columns in bad.items():
        for c in columns:
            t.table[b, c] = value
    want = [t.k_pages.clone(), t.v_pages.clone()]
    for b in range(3):
        if ks[b] <= keep:
            continue
        for h in range(hkv):
            src = torch.from_numpy(kept[b, h]).cuda()
            dst = torch.arange(keep, device="cuda")
            ps, pd = (t.table[b, x // page].long() for x in (src, dst))
            n = t.k_pages.shape[0]
            ok_s = (ps >= 0) & (ps < n)
            to = (pd >= 0) & (pd < n) & (src != dst)
            for w, pages in zip(want, (t.k_pages, t.v_pages)):
                rows = pages[ps.clamp(0, n - 1), h, src % page]
                rows = torch.where(ok_s[:, None], rows, torch.zeros_like(rows))
                w[pd[to], h, dst[to] % page] = rows[to]
    got, lens, out = lib.sdpa_paged_evict(t.k_pages, t.v_pages, scores, t.table, t.lens, keep, 20)
    assert status(cuda, lib) == 7
    assert np.array_equal(got.cpu().numpy(), kept)
    assert lens.tolist() == [min(k, keep) for k in ks]
    for w, pages in zip(want, (t.k_pages, t.v_pages)):
        assert torch.equal(w.nan_to_num(nan=77.0), pages.nan_to_num(nan=77.0))
