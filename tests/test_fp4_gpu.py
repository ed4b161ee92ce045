"""Attention over the 4-bit paged cache against its definition in 64 bits.

Bounds, element by element.  With A = sum_j w_j |v_j| (w the softmax weights),
c = scale * max_j sum_d |q_d k_d| and eps the spacing of q's type:
  - code * scale is exact in fp16, and so are fp16 queries; bf16 ones lose what
    is below 2^-39 of their row's largest, fp32 ones are held to 22 bits: c 2^-22;
  - a score is a sum of D products in fp32 (each addition off by at most one
    unit, 2^-23), its product with the factor, the subtraction of the reference
    and the exponential as for the 16-bit cache: e below;
  - a weight enters the value product in fp16: 2^-11 of itself, or 2^-29 of the
    largest where it is small (2^-25, the least step's half, against a largest
    of at least 2^4); fp32 calls add a second fp16 part, 2^-21 in all;
  - the value product adds up nk / 16 terms in fp32, one unit each;
  - O is rounded once: eps / 2 times |O|.
LSE follows from the first two items alone.
"""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

DT = {"f32": "float32", "f16": "float16", "bf16": "bfloat16"}
VALUES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
# every scale byte's value (a table: powers computed on the GPU are not exact)
SCALES = [math.ldexp(b & 7, -9) if not b >> 3 & 15 else math.ldexp(8 + (b & 7), (b >> 3 & 15) - 10)
          for b in range(128)]


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


def values_of(torch, codes, scales):
    """What rows of code and scale bytes stand for, in float64."""
    lut = torch.tensor(VALUES + [-v for v in VALUES], dtype=torch.float64, device=codes.device)
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    s = torch.tensor(SCALES + [-v for v in SCALES], dtype=torch.float64,
                     device=codes.device)[scales.long()]
    return lut[c.long()] * s.repeat_interleave(16, -1)


class Cache4:
    """A 4-bit cache with sequences of the given query and key counts."""

    def __init__(self, torch, qs, ks, hq, hkv, D, dtype, page, layout="nhd", pad=0, seed=0,
                 gains=True, extra_cols=1, top=0x40):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.torch, self.qs, self.ks, self.hq, self.hkv, self.D, self.page = (
            torch, qs, ks, hq, hkv, D, page)
        dt = self.dtype = getattr(torch, DT[dtype])
        T = sum(qs) + pad
        self.q = torch.randn(T, hq, D, generator=g, device="cuda").to(dt)
        need = [-(-k // page) for k in ks]
        cols, pages = max(need + [0]) + extra_cols, sum(need) + 2

        def raw(n, fill):
            shape = (pages, page, hkv, n) if layout == "nhd" else (pages, hkv, page, n)
            x = torch.full(shape, fill, device="cuda", dtype=torch.uint8)
            return x.transpose(1, 2) if layout == "nhd" else x

        # rows past a sequence's length: the largest codes, scales of NaN
        self.codes = [raw(D // 2, 0x7F) for _ in "kv"]
        self.scales = [raw(D // 16, 0x7F) for _ in "kv"]
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        self.table = torch.full((len(ks), cols), -7, dtype=torch.int32, device="cuda")
        self.gain = [0.25 + torch.rand(hkv, generator=g, device="cuda") if gains else None
                     for _ in "kv"]
        at = 0
        self.KV = []
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
            pos = torch.arange(ks[b], device="cuda")
            pg = self.table[b, pos // page].long()
            rows = []
            for i in range(2):
                c = torch.randint(0, 256, (ks[b], hkv, D // 2), generator=g, device="cuda",
                                  dtype=torch.uint8)
                # scales from the smallest subnormal to `top`, a few of both signs
                s = torch.randint(0x28, top, (ks[b], hkv, D // 16), generator=g, device="cuda",
                                  dtype=torch.uint8)
                u = torch.rand(s.shape, generator=g, device="cuda")
                s = torch.where(u < 0.05, torch.ones_like(s), s)
                s = torch.where(u > 0.95, s + 128, s)
                if ks[b]:
                    self.codes[i][pg, :, pos % page] = c
                    self.scales[i][pg, :, pos % page] = s
                x = values_of(torch, c, s)
                if gains:
                    x = x * self.gain[i].double()[:, None]
                rows.append(x)
            self.KV.append(rows)
        self.lens = torch.tensor(ks, dtype=torch.int32, device="cuda")
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(qs)]), dtype=torch.int32,
                               device="cuda")
        self.sinks = torch.randn(hq, generator=g, device="cuda")

    def rows(self, b):
        t0 = sum(self.qs[:b])
        return slice(t0, t0 + self.qs[b])


def forward(S, t, **kw):
    return S.sdpa_paged_forward_fp4(t.q, *t.codes, *t.scales, t.table, t.lens, cu_seqlens_q=t.cu,
                                    k_gain=t.gain[0], v_gain=t.gain[1], **kw)


def check(t, o, lse, scale, causal=True, sinks=None):
    torch = t.torch
    eps = torch.finfo(t.dtype).eps
    f32 = t.dtype == torch.float32
    G = t.hq // t.hkv
    for b in range(len(t.qs)):
        nq, nk = t.qs[b], t.ks[b]
        for h in range(t.hq if nq else 0):
            q = t.q[t.rows(b), h].double()
            k, v = (x[:, h // G] for x in t.KV[b])
            x = q @ k.T * scale
            c = float((q.abs() @ k.abs().T).max() * abs(scale)) if x.numel() else 0.0
            if causal:
                x = x.masked_fill(torch.arange(nk, device="cuda")[None] > (
                    nk - nq + torch.arange(nq, device="cuda"))[:, None], -math.inf)
            y = x if sinks is None else torch.cat([x, sinks[h].double().expand(nq, 1)], 1)
            z = torch.logsumexp(y, 1) if y.shape[1] else torch.full(
                (nq,), -math.inf, dtype=torch.float64, device="cuda")
            w = (x - z[:, None]).exp().masked_fill(z[:, None] == -math.inf, 0.0)
            ref, A = w @ v, w @ v.abs()
            e = t.D * 2.0**-23 * c + 2.0**-22 * c + (4 + 4 * c) * 2.0**-22 + (
                nk / 32 + 64) * 2.0**-24
            top = w.amax(1, keepdim=True) if nk else 0.0
            tol = (eps / 2 * ref.abs()
                   + (2 * e + (2.0**-21 if f32 else 2.0**-11) + (nk / 16 + 8) * 2.0**-23) * A * 1.01
                   + 2.0**-29 * top * v.abs().sum(0) + 1e-30)
            if t.dtype == torch.float16:
                tol = tol + 2.0**-25
            got = o[t.rows(b), h].double()
            bad = ((got - ref).abs() > tol) | got.isnan()
            assert not bad.any(), (b, h, int(bad.sum()), float((got - ref).abs().max()),
                                   float(tol.min()))
            gl = lse[t.rows(b), h].double()
            inf = z == -math.inf
            assert torch.equal(gl == -math.inf, inf)
            dl = (gl - z).abs()[~inf]
            assert (dl <= e + z[~inf].abs() * 2.0**-22 + 2.0**-21).all(), (b, h, float(dl.max()))
            assert (got[inf] == 0).all()


SHAPES = [  # qs, ks, hq, hkv, D, page
    ([1], [1], 1, 1, 64, 16),
    ([1, 1, 1], [1, 17, 300], 8, 2, 128, 16),
    ([1] * 9, [5, 64, 128, 129, 1000, 31, 2, 640, 255], 32, 8, 128, 16),
    ([1, 1], [4097, 2000], 16, 1, 64, 32),
    ([1, 1], [700, 33], 38, 38, 64, 64),
    ([2, 1, 2], [700, 33, 280], 24, 6, 128, 32),
    ([3, 1, 0, 40, 17], [3, 9, 30, 400, 17], 12, 4, 64, 8),
    ([130, 257], [130, 700], 8, 8, 128, 64),
    ([100, 33], [612, 1033], 24, 8, 64, 48),
    ([5, 300], [2000, 311], 4, 1, 128, 128),
    ([64], [500], 38, 38, 64, 256),
    ([20, 7], [90, 33], 6, 3, 128, 24),
    ([2, 70], [150, 71], 160, 1, 64, 16),
    ([1, 1], [3000, 71], 160, 1, 128, 16),
    # pages without whole groups of 8 rows
    ([1, 5], [40, 33], 8, 2, 64, 1),
    ([9, 30], [100, 77], 6, 2, 128, 7),
    ([1, 1], [500, 61], 8, 2, 128, 20),
    ([160, 300], [500, 310], 8, 2, 128, 12),
]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("layout", ["nhd", "hnd"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(cuda, S, shape, layout, dtype):
    t = Cache4(cuda, *shape[:5], dtype, shape[5], layout, pad=3, gains=layout == "nhd")
    o = cuda.full_like(t.q, 7.0)
    lse = cuda.full(t.q.shape[:2], 7.0, device="cuda")
    forward(S, t, out=o, lse=lse)
    check(t, o, lse, 1 / math.sqrt(t.D))
    # rows behind the last sequence are left as they were
    assert (o[-3:] == 7).all() and (lse[-3:] == 7).all()


OPTIONS = [dict(causal=False), dict(scale=-0.2), dict(scale=0.0), dict(sinks=True),
           dict(sinks=True, scale=0.5, causal=False)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("kw", OPTIONS, ids=str)
@pytest.mark.parametrize("shape", [SHAPES[2], SHAPES[5], SHAPES[8], SHAPES[9]], ids=str)
def test_options(cuda, S, shape, kw, dtype):
    t = Cache4(cuda, *shape[:5], dtype, shape[5])
    kw = dict(kw)
    sinks = t.sinks if kw.pop("sinks", False) else None
    o, lse = forward(S, t, sinks=sinks, **kw)
    check(t, o, lse, kw.get("scale", 1 / math.sqrt(t.D)), kw.get("causal", True), sinks)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("ctas", [1, 2, 5, 37])
@pytest.mark.parametrize("shape", [SHAPES[2], SHAPES[3], SHAPES[6], SHAPES[9]], ids=str)
def test_shared_out_differently(cuda, S, hook, shape, ctas, dtype):
    hook("paged_ctas", ctas)
    t = Cache4(cuda, *shape[:5], dtype, shape[5])
    o, lse = forward(S, t, sinks=t.sinks)
    check(t, o, lse, 1 / math.sqrt(t.D), sinks=t.sinks)


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("hq,hkv,nq", [(4, 1, 1), (12, 1, 1), (20, 1, 3), (20, 1, 40), (8, 8, 1)])
@pytest.mark.parametrize("ctas", [1, 2, 0])
def test_sequences_without_keys_among_others(cuda, S, hook, ctas, hq, hkv, nq, dtype):
    hook("paged_ctas", ctas)
    ks = [0, 300, 0, 5, 0, 0, 140, 128, 0, 0, 0, 17, 2, 0]
    t = Cache4(cuda, [nq] * len(ks), ks, hq, hkv, 64, dtype, 16)
    for causal in (True, False):
        o, lse = forward(S, t, causal=causal)
        check(t, o, lse, 1 / 8, causal)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_empty_rows(cuda, S, dtype):
    """More new tokens than keys: the first see none; a sequence of no keys; no page at all."""
    t = Cache4(cuda, [6, 3, 1, 200], [4, 0, 0, 150], 8, 2, 64, dtype, 16)
    o, lse = forward(S, t)
    check(t, o, lse, 1 / 8)
    o, lse = forward(S, t, sinks=t.sinks)
    assert (o[:2] == 0).all() and (o[6:10] == 0).all()
    assert ((lse[6:10] - t.sinks).abs() <= t.sinks.abs() * 2.0**-21 + 2.0**-22).all()
    o, lse = S.sdpa_paged_forward_fp4(t.q, *t.codes, *t.scales, t.table[:, :0], t.lens,
                                      cu_seqlens_q=t.cu)
    assert (o == 0).all() and (lse == -math.inf).all()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("nq", [1, 6, 150])
def test_growing_scores(cuda, S, nq, dtype):
    """Keys that grow along the sequence: the reference maximum moves again and again."""
    t = Cache4(cuda, [nq], [1500], 4, 2, 128, dtype, 16, gains=False)
    b, n = 0, 1500
    pos = cuda.arange(n, device="cuda")
    pg = t.table[0, pos // 16].long()
    step = (0x28 + pos * 0x20 // n).to(cuda.uint8)  # scales from 2^-2 to 2^2
    t.scales[0][pg, :, pos % 16] = step[:, None, None].expand(n, 2, 8).contiguous()
    codes = t.codes[0][pg, :, pos % 16] & 0x77  # all positive
    t.codes[0][pg, :, pos % 16] = codes
    t.KV[0][0] = values_of(cuda, codes, t.scales[0][pg, :, pos % 16])
    t.q = t.q.abs()
    o, lse = forward(S, t)
    check(t, o, lse, 1 / math.sqrt(128))


@pytest.mark.parametrize("nq", [1, 140])
def test_small_and_large_queries(cuda, S, nq):
    """bf16 rows whose elements lie far outside fp16's range, up and down."""
    for factor, scale in ((2.0**60, 2.0**-64), (2.0**-100, 2.0**96), (2.0**-130, 1.0)):
        t = Cache4(cuda, [nq], [300], 8, 2, 64, "bf16", 16)
        t.q = (t.q.float() * factor).to(cuda.bfloat16)
        o, lse = forward(S, t, scale=scale)
        check(t, o, lse, scale)


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("nq", [1, 40])
def test_strides(cuda, S, nq, dtype):
    """Rows inside wider rows, K and V of one tensor, a page table with spare columns."""
    t = Cache4(cuda, [nq, nq], [70, 300], 8, 2, 64, dtype, 16)
    wide = cuda.zeros(t.q.shape[0], 3, 8, 64, device="cuda", dtype=t.dtype)
    wide[:, 1] = t.q
    P = t.codes[0].shape[0]
    codes = cuda.zeros(P, 16, 2, 2, 48, device="cuda", dtype=cuda.uint8)
    scales = cuda.full((P, 16, 2, 2, 12), 0x7F, device="cuda", dtype=cuda.uint8)
    for i in range(2):
        codes[:, :, i, :, :32] = t.codes[i].transpose(1, 2)
        scales[:, :, i, :, 4:8] = t.scales[i].transpose(1, 2)
    kc, vc = (codes[:, :, i, :, :32].transpose(1, 2) for i in range(2))
    ks, vs = (scales[:, :, i, :, 4:8].transpose(1, 2) for i in range(2))
    out = cuda.zeros(8, t.q.shape[0], 64, device="cuda", dtype=t.dtype).transpose(0, 1)
    tab = cuda.full((2, 99), -1, dtype=cuda.int32, device="cuda")
    tab[:, :t.table.shape[1]] = t.table
    o, lse = S.sdpa_paged_forward_fp4(
        wide[:, 1], kc, vc, ks.view(cuda.float8_e4m3fn), vs.view(cuda.float8_e4m3fn),
        tab[:, :t.table.shape[1]], t.lens, cu_seqlens_q=t.cu, k_gain=t.gain[0], v_gain=t.gain[1],
        out=out)
    check(t, o, lse, 1 / 8)


@pytest.mark.parametrize("nq", [1, 40])
def test_offsets_past_32_bits(cuda, S, nq):
    """Pages further apart than 2^31 bytes, codes and scales."""
    t = Cache4(cuda, [nq], [3 * 64], 4, 2, 128, "bf16", 64, extra_cols=0)
    far = (2**31 + 4096) // 64 * 64
    room = cuda.zeros(2 * 4 * far + 2**20, dtype=cuda.uint8, device="cuda")
    big = []
    for i, (x, n) in enumerate(((t.codes[0], 64), (t.codes[1], 64))):
        v = room.as_strided((5, 2, 64, n), (far // 2, 64 * n, n, 1), i * 2**14)
        v.copy_(x)
        big.append(v)
    for i, x in enumerate(t.scales):
        v = room.as_strided((5, 2, 64, 8), (far // 2, 512, 8, 1), 2**16 + i * 2**14)
        v.copy_(x)
        big.append(v)
    assert 4 * big[0].stride(0) > 2**32
    o, lse = S.sdpa_paged_forward_fp4(t.q, *big, t.table, t.lens, cu_seqlens_q=t.cu,
                                      k_gain=t.gain[0], v_gain=t.gain[1])
    check(t, o, lse, 1 / math.sqrt(128))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("nq", [1, 40])
def test_cache_of_no_pages(cuda, nq, dtype):
    """Every entry of the table names no page then."""
    import scaled_dot_product_fwd_gb300 as S
    t = Cache4(cuda, [nq, nq], [100, 0], 8, 2, 64, dtype, 16)
    none = [x[:0] for x in t.codes + t.scales]
    for x in t.KV[0]:
        x[:] = 0
    o, lse = S.sdpa_paged_forward_fp4(t.q, *none, t.table, t.lens, cu_seqlens_q=t.cu)
    cuda.cuda.synchronize()
    assert S.sdpa_device_status() == 7
    check(t, o, lse, 1 / 8)
    assert S.sdpa_device_status() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("nq", [1, 40])
def test_bad_pages(cuda, nq, dtype):
    """An entry that names no page reads as zero keys and values and is reported."""
    import scaled_dot_product_fwd_gb300 as S
    for page in (16, 5):
        t = Cache4(cuda, [nq, nq], [100, 90], 8, 2, 64, dtype, page)
        t.table[0, 1] = 10**6
        t.table[1, 2] = -1
        for i in range(2):
            t.KV[0][i][page:2 * page] = 0
            t.KV[1][i][2 * page:3 * page] = 0
        o, lse = forward(S, t)
        cuda.cuda.synchronize()
        assert S.sdpa_device_status() == 7
        check(t, o, lse, 1 / 8)
    assert S.sdpa_device_status() == 0


def test_streams_graphs_and_repeats(cuda, S):
    """A call under capture and its replays, on other streams, again and again: the same bits."""
    ts = [Cache4(cuda, [1, 1], [3000, 900], 8, 2, 64, "bf16", 16),
          Cache4(cuda, [9, 300], [900, 1500], 8, 2, 128, "f16", 16),
          Cache4(cuda, [40], [700], 8, 2, 64, "f32", 16)]
    refs = [forward(S, t) for t in ts]
    for t, ref in zip(ts, refs):
        for _ in range(3):
            o, lse = forward(S, t)
            assert cuda.equal(o, ref[0]) and cuda.equal(lse, ref[1])
        side = cuda.cuda.Stream()
        side.wait_stream(cuda.cuda.current_stream())
        with cuda.cuda.stream(side):
            o, lse = forward(S, t)
        o2, lse2 = forward(S, t, stream=side.cuda_stream)
        side.synchronize()
        assert cuda.equal(o, ref[0]) and cuda.equal(o2, ref[0]) and cuda.equal(lse2, ref[1])
    graphs = []
    for t in ts:
        g = cuda.cuda.CUDAGraph()
        with cuda.cuda.graph(g):
            out = forward(S, t)
        graphs.append((g, out))
    for _ in range(3):
        for (g, out), ref in zip(graphs, refs):
            out[0].zero_()
            g.replay()
        for (g, out), ref in zip(graphs, refs):
            assert cuda.equal(out[0], ref[0]) and cuda.equal(out[1], ref[1])


def test_one_token_each_without_offsets(cuda, S):
    t = Cache4(cuda, [1] * 5, [3, 99, 1, 500, 64], 8, 4, 128, "bf16", 16, pad=2)
    o, lse = forward(S, t)
    o2, lse2 = S.sdpa_paged_forward_fp4(t.q, *t.codes, *t.scales, t.table, t.lens,
                                        k_gain=t.gain[0], v_gain=t.gain[1])
    assert cuda.equal(o[:5], o2[:5]) and cuda.equal(lse[:5], lse2[:5])


def test_long_sequence(cuda, S):
    t = Cache4(cuda, [1, 20], [70001, 33333], 4, 1, 128, "bf16", 64)
    o, lse = forward(S, t)
    check(t, o, lse, 1 / math.sqrt(128))


def test_against_the_16_bit_cache(cuda, S):
    """The same values in a 16-bit cache (exact there too: six significant bits) give the same
    results within both operators' bounds."""
    t = Cache4(cuda, [1, 30], [500, 300], 8, 2, 64, "f16", 16, gains=False)
    kp, vp = (values_of(cuda, c, cuda.where(s == 0x7F, cuda.zeros_like(s), s)).to(cuda.float16)
              for c, s in zip(t.codes, t.scales))
    o, lse = forward(S, t)
    o2, lse2 = S.sdpa_paged_forward(t.q, kp, vp, t.table, t.lens, cu_seqlens_q=t.cu)
    assert ((lse - lse2).abs() <= 2.0**-12).all()
    # 2^-11 of sum w |v| <= max |v| for each side's weights, and both roundings of o
    tol = 2 * 2.0**-11 * float(vp.abs().max()) + 2.0**-11 * o.abs().float() + 2.0**-10
    assert ((o.float() - o2.float()).abs() <= tol).all()
