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
    e, m = (scales >> 3 & 15).double(), (scales & 7).double()
    s = torch.where(e == 0, m * 2.0**-9, (1 + m / 8) * 2.0**(e - 7))
    s = torch.where(scales >= 128, -s, s)
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
