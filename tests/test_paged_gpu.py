"""The paged KV cache operators against their definitions in 64 bits.

Bounds, element by element.  With A = sum_j w_j |v_j| (w the softmax weights),
c = scale * max_j sum_d |q_d k_d| and eps the type's spacing:
  - a score is a sum of D products in fp32, off by at most D 2^-23 c, and its
    product with scale*log2(e), the subtraction of the maximum and the
    exponential add at most (4 + 4 |x|) 2^-22 relative to the weight, |x| the
    largest score; a weight and its share of the sum are each off by that, so
    O by at most twice it times A, plus the order of the sums (K / 32 + 64
    terms of 2^-24);
  - on the tensor cores the weights enter the value product rounded to the
    type: eps / 2 times A;
  - O is rounded once: eps / 2 times |O|.
LSE and the accumulated weights follow from the first item alone.
"""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

DT = {"f32": "float32", "f16": "float16", "bf16": "bfloat16"}


@pytest.fixture
def S(cuda):
    import scaled_dot_product_fwd_gb300 as S
    yield S
    cuda.cuda.synchronize()
    assert S.sdpa_device_status() == 0


@pytest.fixture
def hook(cuda):
    import scaled_dot_product_fwd_gb300 as S
    saved = {}

    def set_hook(name, value):
        prev = S.sdpa_debug_set_option(name, int(value))
        saved.setdefault(name, prev)

    yield set_hook
    for name, prev in saved.items():
        S.sdpa_debug_set_option(name, prev)


class Batch:
    """A cache with sequences of the given query and key counts."""

    def __init__(self, torch, qs, ks, hq, hkv, D, dtype, page, layout="nhd", pad=0, seed=0,
                 poison=True, extra_cols=1):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.torch, self.qs, self.ks, self.hq, self.hkv, self.D, self.page = (
            torch, qs, ks, hq, hkv, D, page)
        dt = self.dtype = getattr(torch, DT[dtype])

        def normal(*s):
            return torch.randn(s, generator=g, device="cuda").to(dt)

        T = sum(qs) + pad
        self.q, self.k, self.v = normal(T, hq, D), normal(T, hkv, D), normal(T, hkv, D)
        need = [-(-k // page) for k in ks]
        cols = max(need + [0]) + extra_cols
        pages = sum(need) + 2
        shape = (pages, page, hkv, D) if layout == "nhd" else (pages, hkv, page, D)
        # rows past a sequence's length hold NaN: nothing may read them into a result
        raw = [torch.full(shape, float("nan") if poison else 0.0, device="cuda", dtype=dt)
               for _ in range(2)]
        self.k_pages, self.v_pages = [r.transpose(1, 2) if layout == "nhd" else r for r in raw]
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        # entries that no key uses name no page
        self.table = torch.full((len(ks), cols), -7, dtype=torch.int32, device="cuda")
        at = 0
        self.K, self.V = [], []
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
            k, v = normal(ks[b], hkv, D), normal(ks[b], hkv, D)
            self.K.append(k)
            self.V.append(v)
            if ks[b]:
                pos = torch.arange(ks[b], device="cuda")
                pg = self.table[b, pos // page].long()
                self.k_pages[pg, :, pos % page] = k
                self.v_pages[pg, :, pos % page] = v
        self.lens = torch.tensor(ks, dtype=torch.int32, device="cuda")
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(qs)]), dtype=torch.int32,
                               device="cuda")
        self.sinks = torch.randn(hq, generator=g, device="cuda")

    def rows(self, b):
        t0 = sum(self.qs[:b])
        return slice(t0, t0 + self.qs[b])

    def weights(self, b, h, scale, causal, sinks=None):
        """x, z, w of query head h over sequence b in float64, and c."""
        torch = self.torch
        nq, nk = self.qs[b], self.ks[b]
        q = self.q[self.rows(b), h].double()
        k = self.K[b][:, h // (self.hq // self.hkv)].double()
        x = q @ k.T * scale
        c = float((q.abs() @ k.abs().T).max() * abs(scale)) if x.numel() else 0.0
        if causal:
            hidden = torch.arange(nk, device="cuda")[None] > (
                nk - nq + torch.arange(nq, device="cuda"))[:, None]
            x = x.masked_fill(hidden, -math.inf)
        y = x
        if sinks is not None:
            y = torch.cat([x, sinks[h].double().expand(nq, 1)], 1)
        z = torch.logsumexp(y, 1) if y.shape[1] else torch.full((nq,), -math.inf,
                                                               dtype=torch.float64,
                                                               device="cuda")
        w = (x - z[:, None]).exp().masked_fill(z[:, None] == -math.inf, 0.0)
        return x, z, w, c

    def weight_error(self, c, nk):
        return self.D * 2.0**-23 * c + (4 + 4 * c) * 2.0**-22 + (nk / 32 + 64) * 2.0**-24


def check_forward(t, o, lse, scale, causal=True, sinks=None, P_rounded=True):
    torch = t.torch
    eps = torch.finfo(t.dtype).eps
    for b in range(len(t.qs)):
        if t.qs[b] == 0:
            continue
        for h in range(t.hq):
            x, z, w, c = t.weights(b, h, scale, causal, sinks)
            v = t.V[b][:, h // (t.hq // t.hkv)].double()
            ref, A = w @ v, w @ v.abs()
            e = t.weight_error(c, t.ks[b])
            tol = eps / 2 * ref.abs() + (2 * e + (eps / 2 if P_rounded else 0)) * A * 1.01 + 1e-30
            if t.dtype == torch.float16:  # values below 2^-14 are spaced 2^-24
                tol = tol + 2.0**-25 + (2.0**-25 * v.abs().sum(0) if P_rounded else 0)
            got = o[t.rows(b), h].double()
            bad = ((got - ref).abs() > tol) | got.isnan()
            assert not bad.any(), (b, h, float((got - ref).abs().max()), float(tol.min()))
            gl = lse[t.rows(b), h].double()
            inf = z == -math.inf
            assert torch.equal(gl == -math.inf, inf)
            dl = (gl - z).abs()[~inf]
            assert (dl <= e + z[~inf].abs() * 2.0**-22 + 2.0**-21).all(), (b, h, float(dl.max()))
            assert (got[inf] == 0).all()


def forward(S, t, **kw):
    return S.sdpa_paged_forward(t.q, t.k_pages, t.v_pages, t.table, t.lens, cu_seqlens_q=t.cu, **kw)


SHAPES = [  # qs, ks, hq, hkv, D, page
    ([1], [1], 1, 1, 64, 16),
    ([1, 1, 1], [1, 17, 300], 8, 2, 128, 16),
    ([1] * 9, [5, 64, 128, 129, 1000, 31, 2, 640, 255], 32, 8, 128, 16),
    ([1, 1], [4097, 2000], 16, 1, 64, 32),
    ([3, 1, 0, 40, 17], [3, 9, 30, 400, 17], 12, 4, 64, 8),
    ([130, 257], [130, 700], 8, 8, 128, 64),
    ([100, 33], [612, 1033], 24, 8, 64, 48),
    ([5, 300], [2000, 311], 4, 1, 128, 128),
    ([64], [500], 38, 38, 64, 256),
    ([20, 7], [90, 33], 6, 3, 128, 24),
    ([2, 70], [150, 71], 160, 1, 64, 16),
]
ODD_PAGES = [([1, 5], [40, 33], 8, 2, 64, 1), ([9, 30], [100, 77], 6, 2, 128, 7),
             ([1, 1], [500, 61], 8, 2, 128, 20)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("layout", ["nhd", "hnd"])
@pytest.mark.parametrize("shape", SHAPES + ODD_PAGES, ids=str)
def test_forward(cuda, S, shape, layout, dtype):
    t = Batch(cuda, *shape[:5], dtype, shape[5], layout, pad=3)
    o = cuda.full_like(t.q, 7.0)
    lse = cuda.full(t.q.shape[:2], 7.0, device="cuda")
    forward(S, t, out=o, lse=lse)
    check_forward(t, o, lse, 1 / math.sqrt(t.D))
    # rows behind the last sequence are left as they were
    assert (o[-3:] == 7).all() and (lse[-3:] == 7).all()


@pytest.mark.parametrize("shape", SHAPES[:8], ids=str)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_forward_on_cuda_cores(cuda, S, hook, shape, dtype):
    hook("paged_simt", 1)
    t = Batch(cuda, *shape[:5], dtype, shape[5])
    o, lse = forward(S, t)
    check_forward(t, o, lse, 1 / math.sqrt(t.D), P_rounded=False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("ctas", [1, 2, 5, 37])
@pytest.mark.parametrize("shape", [SHAPES[2], SHAPES[3], SHAPES[4], SHAPES[7]], ids=str)
def test_forward_shared_out_differently(cuda, S, hook, shape, ctas, dtype):
    """Units cut at other places: the same results within the same bounds."""
    hook("paged_ctas", ctas)
    t = Batch(cuda, *shape[:5], dtype, shape[5])
    o, lse = forward(S, t, sinks=t.sinks)
    check_forward(t, o, lse, 1 / math.sqrt(t.D), sinks=t.sinks)


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("kw", [dict(causal=False), dict(scale=-0.2), dict(scale=0.0),
                                dict(sinks=True), dict(sinks=True, scale=0.5)], ids=str)
@pytest.mark.parametrize("shape", [SHAPES[2], SHAPES[6], SHAPES[7]], ids=str)
def test_forward_options(cuda, S, shape, kw, dtype):
    t = Batch(cuda, *shape[:5], dtype, shape[5])
    kw = dict(kw)
    sinks = t.sinks if kw.pop("sinks", False) else None
    o, lse = forward(S, t, sinks=sinks, **kw)
    check_forward(t, o, lse, kw.get("scale", 1 / math.sqrt(t.D)), kw.get("causal", True), sinks)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_forward_empty_rows(cuda, S, dtype):
    """More new tokens than keys: the first see none; a sequence of no keys."""
    t = Batch(cuda, [6, 3, 1, 200], [4, 0, 0, 150], 8, 2, 64, dtype, 16)
    for sinks in (None, t.sinks):
        o, lse = forward(S, t, sinks=sinks)
        if sinks is None:
            check_forward(t, o, lse, 1 / 8)
        else:
            assert (o[:2] == 0).all() and (o[6:10] == 0).all()
            # the sink itself, through log2 units and back: two roundings
            assert ((lse[6:10] - sinks).abs() <= sinks.abs() * 2.0**-21 + 2.0**-22).all()
    # no page at all
    o, lse = S.sdpa_paged_forward(t.q, t.k_pages, t.v_pages, t.table[:, :0], t.lens,
                                  cu_seqlens_q=t.cu)
    assert (o == 0).all() and (lse == -math.inf).all()


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("hq,nq", [(4, 1), (12, 1), (20, 3), (20, 40)])
@pytest.mark.parametrize("ctas", [1, 2, 0])
def test_sequences_without_keys_among_others(cuda, S, hook, ctas, hq, nq, D, dtype):
    """Units without a key, alone and several in a row, before and behind
    units with some in one CTA's share."""
    hook("paged_ctas", ctas)
    ks = [0, 300, 0, 5, 0, 0, 140, 128, 0, 0, 0, 17, 2, 0]
    t = Batch(cuda, [nq] * len(ks), ks, hq, 1, D, dtype, 16)
    for causal in (True, False):
        o, lse = forward(S, t, causal=causal)
        check_forward(t, o, lse, 1 / math.sqrt(D), causal)
    cuda.cuda.synchronize()
    assert S.sdpa_device_status() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [SHAPES[2], SHAPES[4], SHAPES[7]], ids=str)
def test_sink_of_minus_infinity_is_none(cuda, S, shape, dtype):
    t = Batch(cuda, *shape[:5], dtype, shape[5])
    t.lens[-1] = 0  # and a sequence whose tokens see nothing
    o, lse = forward(S, t)
    o2, lse2 = forward(S, t, sinks=cuda.full((t.hq,), -math.inf, device="cuda"))
    assert cuda.equal(o, o2) and cuda.equal(lse, lse2)
    assert (lse[t.rows(len(t.qs) - 1)] == -math.inf).all()


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_tokens_between_and_before_the_sequences(cuda, S, dtype):
    """Offsets that start behind row 0 and end before the last row."""
    t = Batch(cuda, [4, 50, 1], [60, 444, 9], 8, 2, 64, dtype, 16)
    ref, ref_lse = forward(S, t)
    q = cuda.cat([cuda.full_like(t.q[:5], float("nan")), t.q, cuda.full_like(t.q[:7], float("nan"))])
    o = cuda.full_like(q, 3.0)
    lse = cuda.full(q.shape[:2], 3.0, device="cuda")
    S.sdpa_paged_forward(q, t.k_pages, t.v_pages, t.table, t.lens, cu_seqlens_q=t.cu + 5, out=o,
                         lse=lse)
    assert cuda.equal(o[5:-7], ref) and cuda.equal(lse[5:-7], ref_lse)
    for x in (o, lse):
        assert (x[:5] == 3).all() and (x[-7:] == 3).all()
    k, v = (cuda.cat([x[:5], x, x[:7]]) for x in (t.k, t.v))
    before = t.k_pages.clone()
    S.sdpa_paged_write(k, v, t.k_pages, t.v_pages, t.table, t.lens, cu_seqlens_q=t.cu + 5)
    pos = 444 - 50 + 7
    assert cuda.equal(t.k_pages[int(t.table[1, pos // 16]), :, pos % 16], t.k[4 + 7])
    assert (before.nan_to_num() != t.k_pages.nan_to_num()).any(-1).sum() <= 55 * 2


def test_threads_on_one_stream(cuda, S):
    """Calls of several host threads on one stream: their kernels interleave,
    their workspaces are their own."""
    import threading
    ts = [Batch(cuda, [1, 9, 300], [3000, 900, 1500], 8, 2, 64, "bf16", 16, seed=i)
          for i in range(4)]
    refs = [forward(S, t) for t in ts]
    cuda.cuda.synchronize()
    bad = []

    def work(t, ref):
        for _ in range(30):
            o, lse = forward(S, t)
            if not (cuda.equal(o, ref[0]) and cuda.equal(lse, ref[1])):
                bad.append(1)

    th = [threading.Thread(target=work, args=x) for x in zip(ts, refs)]
    [x.start() for x in th]
    [x.join() for x in th]
    assert not bad


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_forward_one_token_each_without_offsets(cuda, S, dtype):
    t = Batch(cuda, [1] * 5, [3, 99, 1, 500, 64], 8, 4, 128, dtype, 16, pad=2)
    o, lse = forward(S, t)
    o2, lse2 = S.sdpa_paged_forward(t.q, t.k_pages, t.v_pages, t.table, t.lens)
    assert cuda.equal(o[:5], o2[:5]) and cuda.equal(lse[:5], lse2[:5])


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_forward_strides(cuda, S, dtype):
    """Query and output rows inside wider rows, a cache inside a wider one,
    a page table with spare columns."""
    t = Batch(cuda, [5, 40], [70, 300], 8, 2, 64, dtype, 16)
    wide = cuda.zeros(t.q.shape[0], 3, 8, 64, device="cuda", dtype=t.dtype)
    wide[:, 1] = t.q
    both = cuda.zeros(t.k_pages.shape[0], 16, 2, 2, 64, device="cuda", dtype=t.dtype)
    both[:, :, 0], both[:, :, 1] = t.k_pages.transpose(1, 2), t.v_pages.transpose(1, 2)
    kp, vp = both[:, :, 0].transpose(1, 2), both[:, :, 1].transpose(1, 2)
    out = cuda.zeros(8, t.q.shape[0], 64, device="cuda", dtype=t.dtype).transpose(0, 1)
    tab = cuda.full((2, 99), -1, dtype=cuda.int32, device="cuda")
    tab[:, :t.table.shape[1]] = t.table
    o, lse = S.sdpa_paged_forward(wide[:, 1], kp, vp, tab[:, :t.table.shape[1]], t.lens,
                                  cu_seqlens_q=t.cu, out=out)
    check_forward(t, o, lse, 1 / 8)


def test_forward_large_scores_and_infinite_keys(cuda, S):
    """Scores far apart from tile to tile (the running maximum moves), and a
    key of -inf weight for one sign of the query."""
    t = Batch(cuda, [1, 33], [900, 700], 4, 2, 64, "bf16", 16)
    for b in range(2):
        for i in range(0, t.ks[b], 128):
            n = min(128, t.ks[b] - i)
            f = cuda.tensor(1.0 + i / 64, device="cuda", dtype=t.dtype)
            t.K[b][i:i + n] *= f
        pos = cuda.arange(t.ks[b], device="cuda")
        t.k_pages[t.table[b, pos // 16].long(), :, pos % 16] = t.K[b]
    o, lse = forward(S, t, scale=1.0)
    check_forward(t, o, lse, 1.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_nan_query_stays_in_its_row(cuda, S, dtype):
    t = Batch(cuda, [4, 1], [300, 1000], 4, 1, 64, dtype, 16)
    ref, _ = forward(S, t)
    t.q[1, 2] = float("nan")
    t.q[4, 0] = float("nan")
    o, lse = forward(S, t)
    assert o[1, 2].isnan().all() and lse[1, 2].isnan()
    assert o[4, 0].isnan().all() and lse[4, 0].isnan()
    o[1, 2], o[4, 0] = ref[1, 2], ref[4, 0]
    assert cuda.equal(o, ref)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_bad_page_is_reported(cuda, dtype):
    import scaled_dot_product_fwd_gb300 as S
    t = Batch(cuda, [1, 40], [100, 200], 8, 2, 64, dtype, 16, poison=False)
    good = t.table.clone()
    for bad in (-1, t.k_pages.shape[0], 2**31 - 1, -2**31):
        t.table[1, 3] = bad
        o, lse = forward(S, t)
        assert S.sdpa_device_status(cuda.cuda.current_stream().cuda_stream) == 7
        assert o.isfinite().all() and lse.isfinite().all()
        sc = cuda.zeros(2, 2, 200, device="cuda")
        S.sdpa_paged_scores(t.q, t.k_pages, lse, sc, t.table, t.lens, cu_seqlens_q=t.cu)
        assert S.sdpa_device_status(cuda.cuda.current_stream().cuda_stream) == 7
        before = t.k_pages.clone()
        S.sdpa_paged_write(t.k, t.v, t.k_pages, t.v_pages, t.table[:, :4],
                           cuda.tensor([100, 60], dtype=cuda.int32, device="cuda"),
                           cu_seqlens_q=t.cu)
        assert S.sdpa_device_status(cuda.cuda.current_stream().cuda_stream) == 7
        t.k_pages.copy_(before)
        t.table.copy_(good)
    forward(S, t)
    cuda.cuda.synchronize()
    assert S.sdpa_device_status() == 0


# ---------------------------------------------------------------- score sums
def check_scores(t, got, base, lse, scale, causal=True, sinks=None):
    torch = t.torch
    G = t.hq // t.hkv
    for b in range(len(t.qs)):
        nk = min(t.ks[b], got.shape[2])
        for h in range(t.hkv):
            ref, tol = base[b, h, :nk].double(), 0.0
            tol = ref.abs() * 2.0**-24
            for e in range(G):
                if not t.qs[b]:
                    continue
                x, _, _, c = t.weights(b, h * G + e, scale, causal, sinks)
                z = lse[t.rows(b), h * G + e].double()
                w = (x - z[:, None]).exp().masked_fill(z[:, None] == -math.inf, 0.0)
                err = t.weight_error(c, t.ks[b]) + 4 * float(
                    z[z.isfinite()].abs().max() if z.isfinite().any() else 0) * 2.0**-23
                s = w.sum(0)[:nk]
                ref = ref + s
                # the order of the sum: rows in chains of a few hundred terms
                tol = tol + s * 1.01 * (err + (t.qs[b] * G / 4 + 64) * 2.0**-24)
            d = (got[b, h, :nk].double() - ref).abs()
            assert (d <= tol + ref * 2.0**-23 + 1e-30).all(), (b, h, float(d.max()))
        assert torch.equal(got[b, :, nk:], base[b, :, nk:])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES + ODD_PAGES, ids=str)
def test_scores(cuda, S, shape, dtype):
    t = Batch(cuda, *shape[:5], dtype, shape[5], pad=2)
    _, lse = forward(S, t)
    base = cuda.rand(len(t.ks), t.hkv, max(t.ks) + 5, device="cuda")
    got = base.clone()
    assert S.sdpa_paged_scores(t.q, t.k_pages, lse, got, t.table, t.lens, cu_seqlens_q=t.cu) is got
    check_scores(t, got, base, lse, 1 / math.sqrt(t.D))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("ctas", [1, 2, 5, 37])
@pytest.mark.parametrize("shape", [SHAPES[2], SHAPES[4], SHAPES[7], SHAPES[10]], ids=str)
def test_scores_shared_out_differently(cuda, S, hook, shape, ctas, dtype):
    hook("paged_ctas", ctas)
    t = Batch(cuda, *shape[:5], dtype, shape[5])
    _, lse = forward(S, t)
    base = cuda.zeros(len(t.ks), t.hkv, max(t.ks), device="cuda")
    got = base.clone()
    S.sdpa_paged_scores(t.q, t.k_pages, lse, got, t.table, t.lens, cu_seqlens_q=t.cu)
    check_scores(t, got, base, lse, 1 / math.sqrt(t.D))


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_scores_options(cuda, S, dtype):
    t = Batch(cuda, [5, 140, 9], [70, 300, 4], 8, 2, 64, dtype, 16)
    for kw, sinks in ((dict(causal=False), None), (dict(scale=-0.3), None), ({}, t.sinks)):
        _, lse = forward(S, t, sinks=sinks, **kw)
        base = cuda.rand(3, 2, 250, device="cuda")  # fewer columns than keys
        wide = cuda.zeros(3, 4, 260, device="cuda")
        got = wide[:, ::2, 3:253]  # rows inside wider ones
        got.copy_(base)
        S.sdpa_paged_scores(t.q, t.k_pages, lse, got, t.table, t.lens, cu_seqlens_q=t.cu, **kw)
        check_scores(t, got, base, lse, kw.get("scale", 1 / 8), kw.get("causal", True), sinks)
        wide[:, ::2, 3:253] = 0
        assert (wide == 0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("hq,D,page", [(2, 128, 16), (4, 64, 5), (14, 64, 8)])
@pytest.mark.parametrize("ctas", [0, 3])
def test_single_tokens_with_a_chunk(cuda, S, hook, ctas, hq, D, page, causal, dtype):
    """Few rows a sequence on average, one sequence with many: its keys'
    sums take several blocks of rows."""
    hook("paged_ctas", ctas)
    qs = [1, 1, 70 if hq == 4 else 9, 0, 2, 1, 1] + [1] * (120 if hq == 4 else 10)
    ks = [130, 64, 300, 77, 2, 0, 200] + [1 + 7 * i % 190 for i in range(len(qs) - 7)]
    t = Batch(cuda, qs, ks, hq, 2, D, dtype, page, pad=1)
    o, lse = forward(S, t, causal=causal)
    check_forward(t, o, lse, 1 / math.sqrt(D), causal)
    base = cuda.rand(len(ks), 2, 310, device="cuda")
    got = base.clone()
    S.sdpa_paged_scores(t.q, t.k_pages, lse, got, t.table, t.lens, cu_seqlens_q=t.cu,
                        causal=causal)
    check_scores(t, got, base, lse, 1 / math.sqrt(D), causal)


# --------------------------------------------------------------------- write
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("layout", ["nhd", "hnd"])
@pytest.mark.parametrize("shape", SHAPES[:8] + ODD_PAGES, ids=str)
def test_write(cuda, S, shape, layout, dtype):
    t = Batch(cuda, *shape[:5], dtype, shape[5], layout, pad=4, poison=False)
    k, v = t.k_pages.clone(), t.v_pages.clone()
    for b in range(len(t.qs)):
        for i in range(t.qs[b]):
            pos = t.ks[b] - t.qs[b] + i
            page = int(t.table[b, pos // t.page])
            k[page, :, pos % t.page] = t.k[t.rows(b)][i]
            v[page, :, pos % t.page] = t.v[t.rows(b)][i]
    S.sdpa_paged_write(t.k, t.v, t.k_pages, t.v_pages, t.table, t.lens, cu_seqlens_q=t.cu)
    assert cuda.equal(t.k_pages, k) and cuda.equal(t.v_pages, v)


def test_write_drops_rows_without_a_place(cuda, S):
    """Tokens before position 0, many sequences (some without tokens), and
    new rows inside wider ones."""
    qs = [(7 * i) % 4 for i in range(1100)]
    ks = [q + (i % 5) for i, q in enumerate(qs)]
    ks[1] = 1  # of its three tokens only the last has a place
    t = Batch(cuda, qs, ks, 2, 2, 64, "bf16", 8, poison=False)
    k = t.k_pages.clone()
    cu = np.concatenate([[0], np.cumsum(qs)])
    table = t.table.cpu().numpy()
    for b in range(len(qs)):
        for i in range(qs[b]):
            pos = ks[b] - qs[b] + i
            if pos >= 0:
                k[int(table[b, pos // 8]), :, pos % 8] = t.k[int(cu[b]) + i]
    kv = cuda.stack([t.k, t.v], 1)
    S.sdpa_paged_write(kv[:, 0], kv[:, 1], t.k_pages, t.v_pages, t.table, t.lens,
                       cu_seqlens_q=t.cu)
    assert cuda.equal(t.k_pages, k)


# ------------------------------------------------------------------ eviction
def evict_reference(t, scores, keep, recent):
    """Positions kept by each sequence and head."""
    kept = np.full((len(t.ks), t.hkv, keep), -1, dtype=np.int64)
    sc = scores.double().cpu().numpy()
    for b, n in enumerate(t.ks):
        for h in range(t.hkv):
            w = np.zeros(n)
            m = min(n, sc.shape[2])
            w[:m] = sc[b, h, :m]
            w[np.isnan(w)] = -np.inf
            if n <= keep:
                kept[b, h, :n] = np.arange(n)
                continue
            r = min(recent, keep)
            order = np.argsort(-w[:n - r], kind="stable")[:keep - r]
            kept[b, h] = np.sort(np.concatenate([order, np.arange(n - r, n)]))
    return kept


def check_evict(cuda, S, t, scores, keep, recent, inplace=False):
    kept = evict_reference(t, scores, keep, recent)
    old = scores.clone()
    out = scores if inplace else None
    lens = t.lens if inplace else None
    old_k, old_v = t.k_pages.clone(), t.v_pages.clone()
    got, n, sc = S.sdpa_paged_evict(t.k_pages, t.v_pages, scores, t.table, t.lens, keep, recent,
                                    scores_out=out, seq_lens_out=lens)
    assert np.array_equal(got.cpu().numpy(), kept)
    assert n.tolist() == [min(x, keep) for x in t.ks]
    if inplace:
        assert sc is scores and n is t.lens
    else:
        assert cuda.equal(old, scores) or old.isnan().any()
    for b in range(len(t.ks)):
        for h in range(t.hkv):
            m = min(t.ks[b], keep)
            src = cuda.from_numpy(kept[b, h, :m]).cuda()
            dst = cuda.arange(m, device="cuda")
            pd = t.table[b, dst // t.page].long()
            for pages, rows in ((t.k_pages, t.K), (t.v_pages, t.V)):
                assert cuda.equal(pages[pd, h, dst % t.page], rows[b][src, h])
            want = cuda.zeros(sc.shape[2], device="cuda")
            i = cuda.arange(min(m, sc.shape[2]), device="cuda")
            s = src[:len(i)]
            want[i] = cuda.where(s < old.shape[2], old[b, h, s.clamp(max=old.shape[2] - 1)],
                                 cuda.zeros((), device="cuda"))
            assert cuda.equal(sc[b, h].nan_to_num(nan=123.0), want.nan_to_num(nan=123.0))
            # rows at or past `keep` are as they were
            dst = cuda.arange(m, t.ks[b], device="cuda")
            pd = t.table[b, dst // t.page].long()
            for pages, was in ((t.k_pages, old_k), (t.v_pages, old_v)):
                assert cuda.equal(pages[pd, h, dst % t.page].nan_to_num(),
                                  was[pd, h, dst % t.page].nan_to_num())


EVICT = [  # ks, hkv, D, page, keep, recent
    ([5, 1, 9], 2, 64, 16, 4, 1), ([1], 1, 128, 16, 1, 0), ([2, 3, 0], 3, 64, 8, 1, 5),
    ([1000, 300, 4000], 2, 128, 16, 300, 50), ([2500, 2049], 8, 64, 64, 2048, 0),
    ([700, 123], 4, 128, 7, 128, 128), ([9000], 1, 64, 48, 4500, 1000),
    ([5000, 5000], 38, 64, 256, 129, 300), ([7, 3, 20] * 40, 4, 64, 8, 5, 2),
    ([4000, 2600], 3, 128, 32, 1500, 0), ([130], 2, 64, 16, 129, 4),
]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("case", EVICT, ids=str)
def test_evict(cuda, S, case, dtype):
    ks, hkv, D, page, keep, recent = case
    t = Batch(cuda, [0] * len(ks), ks, hkv, hkv, D, dtype, page, "nhd" if hkv % 2 else "hnd")
    scores = cuda.rand(len(ks), hkv, max(ks) + 3, device="cuda") ** 4
    check_evict(cuda, S, t, scores, keep, recent)


@pytest.mark.parametrize("kind", ["ties", "zeros", "special", "negative", "short", "sorted",
                                  "reversed"])
@pytest.mark.parametrize("inplace", [False, True])
def test_evict_score_values(cuda, S, kind, inplace):
    t = Batch(cuda, [0, 0], [3001, 1500], 2, 2, 64, "bf16", 16)
    g = cuda.Generator(device="cuda").manual_seed(1)
    shape = (2, 2, 3001)
    s = cuda.rand(shape, generator=g, device="cuda")
    if kind == "ties":
        s = (s * 7).floor()
    elif kind == "zeros":
        s = cuda.where(s < 0.5, 0.0, -0.0)
    elif kind == "special":
        s = cuda.where(s < 0.1, float("nan"), s)
        s = cuda.where((s > 0.1) & (s < 0.2), float("inf"), s)
        s = cuda.where((s > 0.2) & (s < 0.3), -float("inf"), s)
        s = cuda.where((s > 0.3) & (s < 0.32), 1e-42, s)  # a denormal number
    elif kind == "negative":
        s = s - 0.5
    elif kind == "short":
        s = s[:, :, :900].contiguous()
    else:
        s = s.sort(dim=-1, descending=kind == "reversed").values.contiguous()
    check_evict(cuda, S, t, s, 1000, 64, inplace)


# ------------------------------------------------- together, streams, graphs
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_serving_loop(cuda, S, dtype):
    """Prompt chunks, then single tokens, with the cache cut back when it
    outgrows its budget: each step against the definition over what a plain
    model of the cache holds."""
    torch, B, hq, hkv, D, page, keep = cuda, 3, 8, 2, 64, 16, 90
    dt = getattr(torch, DT[dtype])
    g = torch.Generator(device="cuda").manual_seed(3)
    t = Batch(torch, [0] * B, [0] * B, hq, hkv, D, dtype, page)
    t.k_pages = torch.full((40, hkv, page, D), float("nan"), device="cuda", dtype=dt)
    t.v_pages = t.k_pages.clone()
    t.table = torch.randperm(40, generator=g, device="cuda")[:39].reshape(3, 13).to(torch.int32)
    scores = torch.zeros(B, hkv, 13 * page, device="cuda")
    # rows held by each sequence and head, in order
    t.K = [torch.zeros(0, hkv, D, device="cuda", dtype=dt) for _ in range(B)]
    t.V = [x.clone() for x in t.K]
    t.ks = [0] * B
    for step, qs in enumerate([[60, 33, 100], [40, 50, 7]] + [[1, 1, 1]] * 4):
        T = sum(qs)
        q, k, v = (torch.randn(T, h, D, generator=g, device="cuda").to(dt)
                   for h in (hq, hkv, hkv))
        t.qs, t.q = qs, q
        t.cu = torch.tensor(np.concatenate([[0], np.cumsum(qs)]), dtype=torch.int32,
                            device="cuda")
        for b in range(B):
            t.K[b] = torch.cat([t.K[b], k[t.rows(b)]])
            t.V[b] = torch.cat([t.V[b], v[t.rows(b)]])
            t.ks[b] += qs[b]
        t.lens = torch.tensor(t.ks, dtype=torch.int32, device="cuda")
        S.sdpa_paged_write(k, v, t.k_pages, t.v_pages, t.table, t.lens, cu_seqlens_q=t.cu)
        o, lse = forward(S, t)
        check_forward(t, o, lse, 1 / 8)
        base = scores.clone()
        S.sdpa_paged_scores(q, t.k_pages, lse, scores, t.table, t.lens, cu_seqlens_q=t.cu)
        check_scores(t, scores, base, lse, 1 / 8)
        if max(t.ks) > keep:
            kept = evict_reference(t, scores, keep, 16)
            S.sdpa_paged_evict(t.k_pages, t.v_pages, scores, t.table, t.lens, keep, 16,
                               scores_out=scores, seq_lens_out=t.lens)
            for b in range(B):
                m = min(t.ks[b], keep)
                idx = torch.from_numpy(kept[b, :, :m]).cuda()
                for rows in (t.K, t.V):
                    rows[b] = torch.stack([rows[b][idx[h], h] for h in range(hkv)], 1)
                t.ks[b] = m
            assert t.lens.tolist() == t.ks


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_graphs_and_streams(cuda, S, dtype):
    """Two captured graphs replayed on two streams at once (each has its own
    workspace), new lengths between replays, and eager calls beside them."""
    torch = cuda
    ts = [Batch(torch, [1, 3, 70], [200, 900, 333], 16, 2, 128, dtype, 16, seed=i)
          for i in range(2)]
    graphs, outs, scs = [], [], []
    for t in ts:
        forward(S, t)  # first call outside a capture
        sc = torch.zeros(3, 2, 900, device="cuda")
        S.sdpa_paged_scores(t.q, t.k_pages, forward(S, t)[1], sc, t.table, t.lens,
                            cu_seqlens_q=t.cu)
        torch.cuda.synchronize()
        sc.zero_()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o, lse = forward(S, t)
            S.sdpa_paged_scores(t.q, t.k_pages, lse, sc, t.table, t.lens, cu_seqlens_q=t.cu)
        graphs.append(g)
        outs.append((o, lse))
        scs.append(sc)
    streams = [torch.cuda.Stream() for _ in ts]
    for lens in ([200, 900, 333], [50, 601, 70], [17, 3, 129]):
        for t, sc in zip(ts, scs):
            t.lens.copy_(torch.tensor(lens, dtype=torch.int32))
            sc.zero_()
        torch.cuda.synchronize()
        for _ in range(3):
            for g, s, t, sc in zip(graphs, streams, ts, scs):
                with torch.cuda.stream(s):
                    sc.zero_()
                    g.replay()
            eager = [forward(S, t) for t in ts]
        torch.cuda.synchronize()
        for t, (o, lse), (eo, el), sc in zip(ts, outs, eager, scs):
            assert torch.equal(o, eo) and torch.equal(lse, el)
            keep = t.ks, t.K, t.V
            t.ks, t.K, t.V = lens, [k[:n] for k, n in zip(t.K, lens)], [
                v[:n] for v, n in zip(t.V, lens)]
            check_forward(t, o, lse, 1 / math.sqrt(128))
            check_scores(t, sc, torch.zeros_like(sc), lse, 1 / math.sqrt(128))
            t.ks, t.K, t.V = keep


def test_raw_stream_and_given_workspace(cuda, S):
    torch = cuda
    t = Batch(torch, [4, 90], [300, 2000], 8, 2, 64, "bf16", 16)
    ref = forward(S, t)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    o, lse = forward(S, t, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])
    ws = torch.full((S.sdpa_paged_workspace_size(params_of(S, t)),), 255, dtype=torch.uint8,
                    device="cuda")
    for _ in range(2):  # dirty workspaces change nothing
        o = forward(S, t, workspace=ws, return_lse=False)
        assert torch.equal(o, ref[0])
    with pytest.raises(S.SdpaError):
        forward(S, t, workspace=ws[:1024])


def params_of(S, t):
    p = S.SdpaPagedParams()
    p.num_seqs, p.num_tokens, p.num_q_heads, p.num_kv_heads = len(t.ks), len(t.q), t.hq, t.hkv
    p.head_dim, p.dtype, p.scale, p.page_size = t.D, S.dtype_code(t.dtype), 1.0, t.page
    return p


def test_many_sequences(cuda, S):
    """More sequences than a CTA has threads, most of them without tokens."""
    qs = [1 if i % 7 == 0 else 2 if i % 501 == 0 else 0 for i in range(1500)]
    ks = [(13 * i) % 40 + q for i, q in enumerate(qs)]
    for dtype in ("f32", "bf16"):
        t = Batch(cuda, qs, ks, 2, 1, 64, dtype, 8)
        o, lse = forward(S, t)
        check_forward(t, o, lse, 1 / 8)
        sc = cuda.zeros(len(ks), 1, 42, device="cuda")
        S.sdpa_paged_scores(t.q, t.k_pages, lse, sc, t.table, t.lens, cu_seqlens_q=t.cu)
        check_scores(t, sc, cuda.zeros_like(sc), lse, 1 / 8)


def test_offsets_past_32_bits(cuda, S):
    """A cache of more than 2^32 elements, its last pages in use."""
    torch = cuda
    pages = (1 << 32) // (2 * 64 * 64) + 5
    k = torch.empty(pages, 64, 2, 64, device="cuda", dtype=torch.float16)
    v = torch.empty_like(k)
    t = Batch(torch, [1, 70], [130, 200], 4, 2, 64, "f16", 64)
    n = t.k_pages.shape[0]
    k[-n:] = t.k_pages.transpose(1, 2)
    v[-n:] = t.v_pages.transpose(1, 2)
    t.k_pages, t.v_pages = k.transpose(1, 2), v.transpose(1, 2)
    t.table = torch.where(t.table >= 0, t.table + (pages - n), t.table)
    o, lse = forward(S, t)
    check_forward(t, o, lse, 1 / 8)
    sc = torch.zeros(2, 2, 200, device="cuda")
    S.sdpa_paged_scores(t.q, t.k_pages, lse, sc, t.table, t.lens, cu_seqlens_q=t.cu)
    check_scores(t, sc, torch.zeros_like(sc), lse, 1 / 8)
    t.lens = torch.tensor([130, 200], dtype=torch.int32, device="cuda")
    S.sdpa_paged_write(t.k, t.v, t.k_pages, t.v_pages, t.table, t.lens, cu_seqlens_q=t.cu)
    assert torch.equal(t.k_pages[int(t.table[0, 2]), :, 1], t.k[0])
    check_evict(torch, S, _reread(t), torch.rand(2, 2, 200, device="cuda"), 64, 10)


def _reread(t):
    """The plain rows as the cache now holds them."""
    for b, n in enumerate(t.ks):
        pos = t.torch.arange(n, device="cuda")
        pg = t.table[b, pos // t.page].long()
        t.K[b], t.V[b] = t.k_pages[pg, :, pos % t.page], t.v_pages[pg, :, pos % t.page]
    return t
