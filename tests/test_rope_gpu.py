"""Rotary positions, rotated appends to the paged caches, and a serving loop of them.

Bounds.  A rotated element is fma(x, c, y s): y s rounded (2^-24 |y s|), the sum
rounded (2^-24 |r|), then once to the type (eps / 2 |r|; below fp16's normal
range 2^-25).  Appends do the same arithmetic as sdpa_rope: equal bits.  What the
4-bit cache stores is pinned bit by bit: the rotated row in its type from the
exact sum (64 bits hold it to 2^-53), then y = x / g, max / 6 and y / scale in
fp32, each correctly rounded.
"""
import math

import numpy as np
import pytest

from test_fp4_gpu import DT, SCALES, check, values_of

pytestmark = pytest.mark.gpu


@pytest.fixture
def S(cuda):
    import scaled_dot_product_fwd_gb300 as S
    yield S
    cuda.cuda.synchronize()
    assert S.sdpa_device_status() == 0


def turned(torch, x, cs, interleaved, back=False):
    """x [..., D] and cs [..., R / 2, 2] in float64: (result, |y s| per element)."""
    h = cs.shape[-2]
    c, s = cs[..., 0].double(), cs[..., 1].double() * (-1 if back else 1)
    r, size = x.double().clone(), torch.zeros_like(x, dtype=torch.float64)
    i = torch.arange(h, device=x.device)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + h)
    xa, xb = x[..., a].double(), x[..., b].double()
    r[..., a], r[..., b] = xa * c - xb * s, xb * c + xa * s
    size[..., a], size[..., b] = (xb * s).abs(), (xa * s).abs()
    return r, size


def close(torch, got, ref, size, dtype):
    eps = torch.finfo(dtype).eps
    tol = 2.0**-24 * 1.01 * (size + ref.abs())
    if dtype != torch.float32:
        tol = tol + eps / 2 * (ref.abs() + tol)
    if dtype == torch.float16:
        tol = tol + 2.0**-25
    bad = ((got.double() - ref).abs() > tol + 1e-44) | got.isnan()
    assert not bad.any(), float((got.double() - ref).abs().max())


def rows(torch, shape, dtype, layout, g):
    B, H, L, D = shape
    x = torch.randn(shape if layout == "hnd" else (B, L, H, D), generator=g, device="cuda")
    x = x.to(getattr(torch, DT[dtype]))
    return x if layout == "hnd" else x.transpose(1, 2)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("layout", ["nhd", "hnd"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,hq,hkv,L,D,R", [
    (1, 1, 1, 1, 64, 64), (2, 8, 2, 33, 128, 128), (1, 38, 38, 100, 64, 32), (3, 5, 1, 7, 128, 96),
    (1, 3, 3, 50, 512, 512), (2, 2, 1, 19, 512, 48), (1, 40, 8, 300, 128, 16), (64, 4, 4, 1, 64, 48),
])
def test_rope(cuda, S, B, hq, hkv, L, D, R, interleaved, layout, dtype):
    g = cuda.Generator(device="cuda").manual_seed(1)
    q, k = rows(cuda, (B, hq, L, D), dtype, layout, g), rows(cuda, (B, hkv, L, D), dtype, layout, g)
    table = S.sdpa_rope_table(500, R)
    each = cuda.randint(0, 500, (B, L), generator=g, device="cuda").to(cuda.int32)
    for pos, at in ((None, cuda.arange(L, device="cuda")[None]), (each, each), (each[0], each[:1])):
        cs = table[at.long()][:, None]
        for back in (False, True):
            f = S.sdpa_rope_backward if back else S.sdpa_rope
            q2, k2 = f(q, k, table, positions=pos, interleaved=interleaved)
            assert q2.stride() == q.stride() and k2.stride() == k.stride()
            for x, y in ((q, q2), (k, k2)):
                close(cuda, y, *turned(cuda, x, cs, interleaved, back), x.dtype)
    # in place, and alone
    q3, none = S.sdpa_rope(q.clone(), None, table, positions=each, interleaved=interleaved)
    qi, ki = q.clone(), k.clone()
    S.sdpa_rope(qi, ki, table, positions=each, interleaved=interleaved, q_out=qi, k_out=ki)
    q4, k4 = S.sdpa_rope(q, k, table, positions=each, interleaved=interleaved)
    assert none is None and cuda.equal(q3, q4) and cuda.equal(qi, q4) and cuda.equal(ki, k4)


def test_rope_strided_and_broadcast(cuda, S):
    """Rows inside wider ones, an expanded input, outputs of another order."""
    g = cuda.Generator(device="cuda").manual_seed(2)
    qkv = cuda.randn(2, 40, 3, 8, 64, generator=g, device="cuda").to(cuda.bfloat16)
    q, k = qkv[:, :, 0].transpose(1, 2), qkv[:, :, 1].transpose(1, 2)
    table = S.sdpa_rope_table(40, 64)
    out = cuda.zeros(2, 8, 40, 64, device="cuda", dtype=cuda.bfloat16)
    q2, _ = S.sdpa_rope(q, k, table, q_out=out)
    cs = table[None, None]
    close(cuda, q2, *turned(cuda, q, cs, False), q.dtype)
    one = cuda.randn(1, 1, 40, 64, generator=g, device="cuda")
    wide = one.expand(3, 4, 40, 64)
    q3, _ = S.sdpa_rope(wide, None, table, q_out=cuda.empty(3, 4, 40, 64, device="cuda"))
    close(cuda, q3, *turned(cuda, wide, cs, False), q3.dtype)
    # the gradient of a broadcast input: the sum of its copies' gradients
    d, _ = S.sdpa_rope_backward(q3, None, table)
    ref = turned(cuda, q3, cs, False, True)[0].sum((0, 1))
    assert ((d.double().sum((0, 1)) - ref).abs() <= 12 * 2.0**-22 * q3.abs().max()).all()


def test_rope_gradient_is_the_transpose(cuda, S):
    """<R x, y> = <x, R^T y>, and differences of sum(R x * y) along each element."""
    g = cuda.Generator(device="cuda").manual_seed(3)
    x, y = (cuda.randn(1, 2, 9, 64, generator=g, device="cuda") for _ in range(2))
    table = S.sdpa_rope_table(9, 48, scaling="yarn", factor=4.0, original_length=64)
    for inter in (False, True):
        rx, _ = S.sdpa_rope(x, None, table, interleaved=inter)
        ry, _ = S.sdpa_rope_backward(y, None, table, interleaved=inter)
        a, b = (rx.double() * y).sum(), (x.double() * ry).sum()
        assert abs(float(a - b)) <= 1152 * 2.0**-22 * float((rx.abs() * y.abs()).max() + 1)
        # the map is linear: a difference over h = 1 has rounding errors alone
        for i in (0, 5, 30, 47, 48, 63):
            step = x.clone()
            step[0, 1, 4, i] += 1.0
            r2, _ = S.sdpa_rope(step, None, table, interleaved=inter)
            diff = float(((r2.double() - rx.double()) * y).sum())
            slack = 4 * 2.0**-23 * float(((rx.abs() + r2.abs()) * y.abs())[0, 1, 4].sum() + 1)
            assert abs(diff - float(ry[0, 1, 4, i])) <= slack


def test_rope_table(cuda, S):
    for kw in (dict(), dict(base=5e5), dict(scaling="linear", factor=8.0),
               dict(scaling="ntk", factor=4.0),
               dict(scaling="yarn", factor=16.0, original_length=4096)):
        freq, gain = S.rope_frequencies(128, **kw)
        t = S.sdpa_rope_table(3000, 128, **kw).cpu().numpy()
        a = np.arange(3000.0)[:, None] * np.array(freq)
        # the angle rounded once in 64 bits, its functions to a few units, then once to 32 bits
        tol = 2.0**-24 * gain + 2.0**-52 * (a + 4)
        assert (np.abs(t[..., 0] - gain * np.cos(a)) <= tol).all()
        assert (np.abs(t[..., 1] - gain * np.sin(a)) <= tol).all()
    far = S.sdpa_rope_table(2_000_001, 16, inv_freq=[1.0 / (i + 1) for i in range(8)], gain=2.0)
    a = 2e6 / np.arange(1.0, 9.0)
    assert np.abs(far[-1, :, 0].cpu().numpy() - 2 * np.cos(a)).max() <= 2.0**-23 + 1e-8
    assert S.sdpa_rope_table(0, 64).shape == (0, 32, 2)


def test_positions_outside_the_table(cuda):
    import scaled_dot_product_fwd_gb300 as S
    x = cuda.randn(1, 2, 4, 64, device="cuda")
    table = S.sdpa_rope_table(10, 64)
    pos = cuda.tensor([3, 10, -1, 2**31 - 1], dtype=cuda.int32, device="cuda")
    y, _ = S.sdpa_rope(x, None, table, positions=pos)
    cuda.cuda.synchronize()
    assert S.sdpa_device_status() == 8 and S.sdpa_device_status() == 0
    assert cuda.equal(y[:, :, 1:], x[:, :, 1:]) and not cuda.equal(y[:, :, 0], x[:, :, 0])
    S.sdpa_rope(x[:, :, :0], None, table)  # nothing to do
    S.sdpa_rope(x, None, S.sdpa_rope_table(0, 64))
    cuda.cuda.synchronize()
    assert S.sdpa_device_status() == 8


class Step:
    """New tokens of a step, packed, and empty 16- and 4-bit caches for them."""

    def __init__(self, torch, qs, ks, hq, hkv, D, dtype, page, layout="nhd", pad=0, seed=0,
                 gains=False):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.qs, self.ks, self.D, self.page, self.hkv = qs, ks, D, page, hkv
        dt = self.dtype = getattr(torch, DT[dtype])
        self.T = T = sum(qs) + pad
        self.q, self.k, self.v = (torch.randn(T, h, D, generator=g, device="cuda").to(dt)
                                  for h in (hq, hkv, hkv))
        need = [-(-k // page) for k in ks]
        pages = sum(need) + 2
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        self.table = torch.full((len(ks), max(need)), -7, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n

        def cache(n, dtype, fill):
            shape = (pages, page, hkv, n) if layout == "nhd" else (pages, hkv, page, n)
            x = torch.full(shape, fill, device="cuda", dtype=dtype)
            return x.transpose(1, 2) if layout == "nhd" else x

        self.pages = [cache(D, dt, 3.0) for _ in "kv"]
        self.codes = [cache(D // 2, torch.uint8, 0x5A) for _ in "kv"]
        self.scales = [cache(D // 16, torch.uint8, 0x11) for _ in "kv"]
        self.gain = [0.01 + torch.rand(hkv, generator=g, device="cuda") if gains else None
                     for _ in "kv"]
        self.lens = torch.tensor(ks, dtype=torch.int32, device="cuda")
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(qs)]), dtype=torch.int32,
                               device="cuda")
        self.seq = torch.cat([torch.full((n,), b) for b, n in enumerate(qs)]).long().cuda()
        self.pos = torch.cat([torch.arange(k - n, k) for n, k in zip(qs, ks)]).cuda()
        self.n = sum(qs)

    def places(self):
        """Token rows with a place, their pages and rows."""
        at = (self.pos >= 0).nonzero()[:, 0]
        pos = self.pos[at]
        return at, self.table[self.seq[at], pos // self.page].long(), pos % self.page


STEPS = [([1], [1], 1, 1, 64, 16), ([1] * 5, [3, 99, 1, 500, 64], 32, 8, 128, 16),
         ([30, 1, 0, 300], [30, 70, 4, 777], 12, 4, 64, 48), ([5, 9], [3, 20], 6, 3, 128, 7),
         ([17], [1000], 38, 38, 64, 8)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("layout", ["nhd", "hnd"])
@pytest.mark.parametrize("interleaved,R,shift", [(False, 64, 0), (True, 48, 900), (False, 16, 3)])
@pytest.mark.parametrize("shape", STEPS, ids=str)
def test_append(cuda, S, shape, interleaved, R, shift, layout, dtype):
    t = Step(cuda, *shape[:5], dtype, shape[5], layout, pad=3)
    table = S.sdpa_rope_table(2000, R)
    at, page, row = t.places()
    turn = (t.pos + shift).clamp(min=0).to(cuda.int32)
    positions = None
    if shift:
        positions = cuda.zeros(t.T, dtype=cuda.int32, device="cuda")
        positions[:t.n] = turn
    ref = [x.clone() for x in t.pages]
    q2, k2 = (x.transpose(0, 1) for x in [
        y[0] for y in S.sdpa_rope(t.q[:t.n].transpose(0, 1)[None], t.k[:t.n].transpose(0, 1)[None],
                                  table, positions=turn, interleaved=interleaved)])
    if not shift:  # tokens before their sequence's start stay as they are
        early = t.pos < 0
        q2, k2 = (cuda.where(early[:, None, None], x[:t.n], y) for x, y in ((t.q, q2), (t.k, k2)))
    ref[0][page, :, row], ref[1][page, :, row] = k2[at], t.v[at]
    out = cuda.full_like(t.q, 7.0)
    q3 = S.sdpa_paged_append(t.q, t.k, t.v, *t.pages, t.table, t.lens, table, cu_seqlens_q=t.cu,
                             positions=positions, interleaved=interleaved, q_out=out)
    assert q3 is out and cuda.equal(out[:t.n], q2) and (out[t.n:] == 7).all()
    assert cuda.equal(t.pages[0], ref[0]) and cuda.equal(t.pages[1], ref[1])
    # q in place, and none
    S.sdpa_paged_append(t.q, t.k, t.v, *t.pages, t.table, t.lens, table, cu_seqlens_q=t.cu,
                        positions=positions, interleaved=interleaved, q_out=t.q)
    assert cuda.equal(t.q[:t.n], q2)
    assert S.sdpa_paged_append(None, t.k, t.v, *t.pages, t.table, t.lens, table,
                               cu_seqlens_q=t.cu, positions=positions,
                               interleaved=interleaved) is None
    assert cuda.equal(t.pages[0], ref[0])


def to_e4m3(torch, x):
    """Positive float32 numbers as e4m3 bytes: nearest, ties to even, 1 .. 0x7E."""
    grid = torch.tensor(SCALES[:127], dtype=torch.float64, device="cuda")
    i = torch.searchsorted(grid, x.double().contiguous()).clamp(1, 126)
    lo, hi = x.double() - grid[i - 1], grid[i] - x.double()
    down = (lo < hi) | ((lo == hi) & (i % 2 == 1))
    return torch.where(down, i - 1, i).clamp(min=1).to(torch.uint8), grid


def quantised(torch, x, gain):
    """Codes, scales and values of rows [rows, heads, D] by the definition."""
    y = x.float() if gain is None else x.float() / gain[:, None]
    y = y.unflatten(-1, (-1, 16))
    top = y.abs().amax(-1).nan_to_num(posinf=3e38)
    sb, grid = to_e4m3(torch, top / 6.0)
    s = grid[sb.long()]
    t = y.double() / s[..., None]
    a = t.abs()
    # borders between codes; those whose lower code is even keep the tie
    n = sum(((a > b) if even else (a >= b)).int() for b, even in
            ((0.25, 1), (0.75, 0), (1.25, 1), (1.75, 0), (2.5, 1), (3.5, 0), (5.0, 1)))
    # (the sign of a number that rounds to 0 is kept, a zero's is not)
    code = (n + 8 * (y < 0).int()).to(torch.uint8).flatten(-2)
    codes = code[..., 0::2] | (code[..., 1::2] << 4)
    value = values_of(torch, codes, sb)
    value = value.float() if gain is None else value.float() * gain[:, None]
    return codes, sb, value.to(x.dtype)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("layout", ["nhd", "hnd"])
@pytest.mark.parametrize("interleaved,R,gains", [(False, 64, True), (True, 48, False),
                                                 (False, 16, True), (False, 48, False),
                                                 (False, 0, True)])
@pytest.mark.parametrize("shape", STEPS, ids=str)
def test_append_fp4(cuda, S, shape, interleaved, R, gains, layout, dtype):
    t = Step(cuda, *shape[:5], dtype, shape[5], layout, pad=3, gains=gains)
    table = S.sdpa_rope_table(2000, R) if R else None
    at, page, row = t.places()
    k, q = t.k[:t.n], t.q[:t.n]
    if R:
        cs = table[t.pos.clamp(min=0)][:, None]
        early = (t.pos < 0)[:, None, None]
        # (through 32 bits, as the row is rounded)
        k = cuda.where(early, k, turned(cuda, k, cs, interleaved)[0].float().to(t.dtype))
    kc, ks, kv = quantised(cuda, k, t.gain[0])
    vc, vs, vv = quantised(cuda, t.v[:t.n], t.gain[1])
    ref = [x.clone() for x in t.codes + t.scales]
    for x, y in zip(ref, (kc, vc, ks, vs)):
        x[page, :, row] = y[at]
    out, ko, vo = cuda.full_like(t.q, 7.0), cuda.full_like(t.k, 7.0), cuda.full_like(t.k, 7.0)
    S.sdpa_paged_append_fp4(t.q, t.k, t.v, *t.codes, *t.scales, t.table, t.lens, table,
                            cu_seqlens_q=t.cu, interleaved=interleaved, k_gain=t.gain[0],
                            v_gain=t.gain[1], q_out=out, k_out=ko, v_out=vo)
    for x, y in zip(t.codes + t.scales, ref):
        assert cuda.equal(x, y), int((x != y).sum())
    assert cuda.equal(ko[:t.n], kv) and cuda.equal(vo[:t.n], vv)
    for x in (out, ko, vo):
        assert (x[t.n:] == 7).all()
    if R:
        ok = ~early.expand(q.shape)
        r, size = turned(cuda, q, cs, interleaved)
        close(cuda, out[:t.n][ok], r[ok], size[ok], t.dtype)
        assert cuda.equal(out[:t.n][~ok], q[~ok])
    else:
        assert cuda.equal(out[:t.n], q)
    # values of K or V alone, no queries
    ko2 = cuda.zeros_like(t.k)
    S.sdpa_paged_append_fp4(None, t.k, t.v, *t.codes, *t.scales, t.table, t.lens, table,
                            cu_seqlens_q=t.cu, interleaved=interleaved, k_gain=t.gain[0],
                            v_gain=t.gain[1], k_out=ko2)
    assert cuda.equal(ko2[:t.n], ko[:t.n])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_quantisation_borders(cuda, S, dtype):
    """Ties between codes and between scales, every scale, magnitudes at the ends of the range."""
    dt = getattr(cuda, DT[dtype])
    T = 3000
    t = Step(cuda, [T], [T], 1, 2, 64, dtype, 16)
    g = cuda.Generator(device="cuda").manual_seed(5)
    grid = to_e4m3(cuda, cuda.ones(1, device="cuda"))[1]
    s = grid[cuda.randint(1, 127, (T, 2, 4, 1), generator=g, device="cuda")]
    quarter = cuda.randint(-24, 25, (T, 2, 4, 16), generator=g, device="cuda") * 0.25
    quarter[..., 3] = 6.0  # the largest: max / 6 is the scale itself
    t.v = (quarter * s).flatten(-2).to(dt)
    # scales at ties: 6 * (the middle of two neighbours) as the largest
    mid = (grid[1:126] + grid[2:127]) / 2
    x = mid[cuda.randint(0, 125, (T, 2, 4, 1), generator=g, device="cuda")] * 6
    t.k = (cuda.randn(T, 2, 4, 16, generator=g, device="cuda", dtype=cuda.float64).clamp(-1, 1)
           * x).to(dt)
    t.k[..., 0] = x[..., 0].to(dt)
    t.k = t.k.flatten(-2)
    tiny = 2.0**-24 if dtype == "f16" else 2.0**-100
    for i, v in enumerate((0.0, -0.0, tiny, 3e4, -6e4, 2.0**-12, 0.0117)):
        t.v[i], t.k[i] = v, -v
    for gains in (None, [cuda.tensor([0.7, 1.3], device="cuda")] * 2):
        S.sdpa_paged_append_fp4(None, t.k, t.v, *t.codes, *t.scales, t.table, t.lens,
                                cu_seqlens_q=t.cu, k_gain=gains and gains[0],
                                v_gain=gains and gains[1])
        at, page, row = t.places()
        for x, c, sc in ((t.k, t.codes[0], t.scales[0]), (t.v, t.codes[1], t.scales[1])):
            codes, sb, _ = quantised(cuda, x, gains and gains[0])
            assert cuda.equal(sc[page, :, row], sb)
            assert cuda.equal(c[page, :, row], codes)


def test_infinities_and_nans_are_stored_finite(cuda, S):
    t = Step(cuda, [4], [4], 1, 1, 64, "f32", 16)
    t.v[0, 0, 5], t.v[1, 0, 0], t.v[2, 0, 20], t.v[3] = math.inf, -math.inf, math.nan, math.nan
    for gain in (None, cuda.tensor([0.3], device="cuda")):
        vo = cuda.empty_like(t.v)
        S.sdpa_paged_append_fp4(None, t.k, t.v, *t.codes, *t.scales, t.table, t.lens,
                                cu_seqlens_q=t.cu, v_gain=gain, v_out=vo)
        f = 1.0 if gain is None else float(gain)
        assert vo.isfinite().all()
        assert vo[0, 0, 5] == 2688 * cuda.tensor(f) and vo[1, 0, 0] == -2688 * cuda.tensor(f)


def test_append_bad_pages_positions_and_lengths(cuda):
    import scaled_dot_product_fwd_gb300 as S
    table = S.sdpa_rope_table(40, 64)
    for four in (False, True):
        t = Step(cuda, [6, 3], [38, 3], 2, 2, 64, "bf16", 8)
        t.table[0, 4] = -3  # positions 32 .. 37
        before = [x.clone() for x in t.codes + t.scales + t.pages]

        def call(**kw):
            a = dict(cu_seqlens_q=t.cu) | kw
            if four:
                S.sdpa_paged_append_fp4(t.q, t.k, t.v, *t.codes, *t.scales, t.table, t.lens, table,
                                        **a)
            else:
                S.sdpa_paged_append(t.q, t.k, t.v, *t.pages, t.table, t.lens, table, **a)
            cuda.cuda.synchronize()
            return S.sdpa_device_status()

        assert call() == 7
        changed = [(x != y).any(-1).any(1).sum() for x, y in zip(t.codes + t.scales + t.pages,
                                                                 before)]
        assert all(int(n) <= 3 for n in changed)  # sequence 1's rows alone
        t.table[0, 4] = t.table[0, 0]
        assert call() == 0
        assert call(positions=cuda.full((9,), 40, dtype=cuda.int32, device="cuda")) == 8
        # past the table's end (of pages): q is rotated, k and v have no place
        t.lens[1] = 30
        before = [x.clone() for x in t.codes + t.scales + t.pages]
        cut = t.table[:, :3]
        t.table = cut.contiguous()
        t.lens[0] = 35
        assert call() == 0
        for x, y in zip(t.codes + t.scales + t.pages, before):
            assert cuda.equal(x, y)
        # more tokens than keys: the early ones have no place and stay as they are
        t.lens[0], t.lens[1] = 2, 3
        assert call() == 0


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_serving_loop(cuda, S, dtype):
    """Chunks, then single tokens, into both caches; each step's attention against its definition
    over what the cache holds, and the 16-bit loop against rotated keys."""
    torch, D, hq, hkv, page = cuda, 64, 8, 2, 16
    dt = getattr(torch, DT[dtype])
    g = torch.Generator(device="cuda").manual_seed(7)
    table = S.sdpa_rope_table(600, 64)
    B, cap = 2, 384
    cols = cap // page
    order = torch.randperm(B * cols, generator=g, device="cuda").to(torch.int32).view(B, cols)
    codes = [torch.zeros(B * cols, page, hkv, D // 2, device="cuda", dtype=torch.uint8).transpose(
        1, 2) for _ in "kv"]
    scales = [torch.full((B * cols, page, hkv, D // 16), 0x7F, device="cuda",
                         dtype=torch.uint8).transpose(1, 2) for _ in "kv"]
    gain = [torch.tensor([0.5, 0.25], device="cuda"), torch.tensor([0.3, 1.0], device="cuda")]
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    ks = [0, 0]
    for qs in ([200, 77], [1, 1], [1, 1], [5, 100], [1, 1]):
        ks = [a + b for a, b in zip(ks, qs)]
        lens.copy_(torch.tensor(ks, dtype=torch.int32))
        cu = torch.tensor([0, qs[0], sum(qs)], dtype=torch.int32, device="cuda")
        q, k, v = (torch.randn(sum(qs), h, D, generator=g, device="cuda").to(dt)
                   for h in (hq, hkv, hkv))
        q = S.sdpa_paged_append_fp4(q, k, v, *codes, *scales, order, lens, table, cu_seqlens_q=cu,
                                    k_gain=gain[0], v_gain=gain[1])
        o, lse = S.sdpa_paged_forward_fp4(q, *codes, *scales, order, lens, cu_seqlens_q=cu,
                                          k_gain=gain[0], v_gain=gain[1])

        class T:
            pass

        t = T()
        t.torch, t.dtype, t.hq, t.hkv, t.D, t.q, t.qs, t.ks = torch, dt, hq, hkv, D, q, qs, ks
        t.rows = lambda b: slice(sum(qs[:b]), sum(qs[:b + 1]))
        t.KV = []
        for b in range(B):
            pos = torch.arange(ks[b], device="cuda")
            pg = order[b, pos // page].long()
            t.KV.append([values_of(torch, codes[i][pg, :, pos % page], scales[i][pg, :, pos % page])
                         * gain[i].double()[:, None] for i in range(2)])
        check(t, o, lse, 1 / math.sqrt(D))


def test_training_step(cuda, S):
    """Rotation, attention and both backward passes in a row: the gradients of q, k and v against
    64 bits."""
    torch = cuda
    g = torch.Generator(device="cuda").manual_seed(8)
    B, hq, hkv, L, D = 2, 4, 2, 70, 64
    q, k, v, dy = (torch.randn(B, h, L, D, generator=g, device="cuda")
                   for h in (hq, hkv, hkv, hq))
    table = S.sdpa_rope_table(L, D)
    q2, k2 = S.sdpa_rope(q, k, table)
    o, lse = S.sdpa_forward(q2, k2, v, causal=True)
    dq2, dk2, dv = S.sdpa_backward(q2, k2, v, o, lse, dy, causal=True)
    dq, dk = S.sdpa_rope_backward(dq2, dk2, table)

    leaves = [x.double().requires_grad_() for x in (q, k, v)]

    def rot(x):
        c, s = table[:, :, 0].double(), table[:, :, 1].double()
        a, b = x[..., :D // 2], x[..., D // 2:]
        return torch.cat([a * c - b * s, b * c + a * s], -1)

    x = rot(leaves[0]) @ rot(leaves[1]).repeat_interleave(2, 1).transpose(2, 3) / math.sqrt(D)
    x = x.masked_fill(torch.ones(L, L, device="cuda", dtype=torch.bool).triu(1), -math.inf)
    y = x.softmax(-1) @ leaves[2].repeat_interleave(2, 1)
    y.backward(dy.double())
    for got, leaf in zip((dq, dk, dv), leaves):
        # sums of some 2 L D products of fp32 numbers of size 1, each off by a unit
        err = (got.double() - leaf.grad).abs().max()
        assert float(err) <= 2 * L * D * 2.0**-23, float(err)


def test_streams_and_graphs(cuda, S):
    t = Step(cuda, [1] * 6, [5, 60, 700, 33, 2, 90], 8, 2, 64, "bf16", 16, gains=True)
    table = S.sdpa_rope_table(1000, 64)

    def call():
        out, ko = cuda.zeros_like(t.q), cuda.zeros_like(t.k)
        S.sdpa_paged_append_fp4(t.q, t.k, t.v, *t.codes, *t.scales, t.table, t.lens, table,
                                cu_seqlens_q=t.cu, k_gain=t.gain[0], v_gain=t.gain[1], q_out=out,
                                k_out=ko)
        q2 = S.sdpa_paged_append(t.q, t.k, t.v, *t.pages, t.table, t.lens, table,
                                 cu_seqlens_q=t.cu)
        r, _ = S.sdpa_rope(t.q.transpose(0, 1)[None], None, table,
                           positions=t.pos.to(cuda.int32))
        return out, ko, q2, r

    ref = [x.clone() for x in call()]
    side = cuda.cuda.Stream()
    side.wait_stream(cuda.cuda.current_stream())
    with cuda.cuda.stream(side):
        got = call()
    side.synchronize()
    assert all(cuda.equal(a, b) for a, b in zip(got, ref))
    g = cuda.cuda.CUDAGraph()
    with cuda.cuda.graph(g):
        got = call()
    for x in t.codes + t.scales + t.pages:
        x.zero_()
    g.replay()
    cuda.cuda.synchronize()
    assert all(cuda.equal(a, b) for a, b in zip(got, ref))
    at, page, row = t.places()
    assert cuda.equal(t.pages[1][page, :, row], t.v[at])
    # a raw stream handle
    at = t.pos.to(cuda.int32)
    cuda.cuda.synchronize()
    r2, _ = S.sdpa_rope(t.q.transpose(0, 1)[None], None, table, positions=at,
                        stream=side.cuda_stream)
    side.synchronize()
    assert cuda.equal(r2, ref[3])
