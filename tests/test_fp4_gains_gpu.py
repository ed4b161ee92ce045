"""Gains at the ends of their range, 2^-100 and 2^100 in magnitude, over long sequences and in cut
units: neither a partial result nor a factor of it leaves fp32's range where the result does not.

The gains are powers of two, exact wherever they enter, so a call's O is that of a call without
them times the value gain, and LSE that of the same scores: equal bits, where O's type holds both
(the values are at least 2^-10 and at most 2688 in magnitude, so fp32 and bf16 do).
"""
import math

import pytest

from test_fp4_gpu import Cache4, S, check, forward  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("qs,ks", [([1], [40000]), ([1, 1], [50, 700]), ([3, 2], [9000, 20]),
                                   ([100], [40000]), ([130, 20], [3000, 200])], ids=str)
@pytest.mark.parametrize("power", [100, -100])
@pytest.mark.parametrize("D", [64, 128])
def test_gains_of_any_size(cuda, S, D, power, qs, ks, dtype):  # noqa: F811
    t = Cache4(cuda, qs, ks, 4, 2, D, dtype, 16, gains=False, top=0x7E)
    # the largest values throughout one kv head of V: its sums are as large as they can be
    live = t.scales[1][:, 1] != 0x7F
    t.codes[1][:, 1] = 0x77
    t.scales[1][:, 1] = cuda.where(live, 0x7E, 0x7F).to(cuda.uint8)
    for b in range(len(qs)):
        t.KV[b][1][:, 1] = 2688.0
    scale = 1e-4
    ref = forward(S, t, scale=scale)
    check(t, *ref, scale)
    g = 2.0**power
    t.gain = [cuda.tensor([g, -g], device="cuda"), cuda.tensor([-g, g], device="cuda")]
    q = t.q.clone()
    t.q[:, 2:] = -t.q[:, 2:]  # (of kv head 1, whose gain is negative)
    o, lse = forward(S, t, scale=scale / g)
    t.q = q
    # scale / g * log2 e * g rounds as scale * log2 e does
    assert cuda.equal(lse, ref[1])
    sign = cuda.tensor([-1.0, -1.0, 1.0, 1.0], device="cuda")[:, None]
    assert cuda.equal(o.double(), ref[0].double() * sign * g)


@pytest.mark.parametrize("power", [100, -100])
def test_append_with_gains_of_any_size(cuda, S, power):  # noqa: F811
    from test_rope_gpu import Step, quantised
    for dtype in ("f32", "bf16"):
        t = Step(cuda, [300], [300], 1, 2, 64, dtype, 16)
        gain = cuda.tensor([1.625, -1.3], device="cuda") * 2.0**power
        t.k, t.v = ((x.float() * 2.0**power).to(t.dtype) for x in (t.k, t.v))
        vo = cuda.empty_like(t.v)
        S.sdpa_paged_append_fp4(None, t.k, t.v, *t.codes, *t.scales, t.table, t.lens,
                                cu_seqlens_q=t.cu, k_gain=gain, v_gain=gain, v_out=vo)
        at, page, row = t.places()
        for x, c, s, out in ((t.k, t.codes[0], t.scales[0], None), (t.v, t.codes[1], t.scales[1], vo)):
            codes, sb, value = quantised(cuda, x, gain)
            assert cuda.equal(s[page, :, row], sb) and cuda.equal(c[page, :, row], codes)
            assert out is None or (cuda.equal(out, value) and math.isfinite(float(out.float().sum())))
