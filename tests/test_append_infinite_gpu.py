"""Rotated keys that are infinite or overflow, on their way to the 4-bit cache: a row holds what
sdpa_rope makes of it, and an infinity is stored as the largest value, 6 * 448, under its sign.

What is stored has no rounding here (largest codes, largest scale), so results are equal.  The
group's other elements are at most 2688 / 448 / 4 in size: under a scale of 448 they become code 0.
"""
import math

import pytest

from test_fp4_gpu import DT, values_of

pytestmark = pytest.mark.gpu


def append(cuda, k, R, interleaved, gain):
    import scaled_dot_product_fwd_gb300 as S
    T, H, D = k.shape
    codes = [cuda.zeros(1, H, T, D // 2, device="cuda", dtype=cuda.uint8) for _ in "kv"]
    scales = [cuda.zeros(1, H, T, D // 16, device="cuda", dtype=cuda.uint8) for _ in "kv"]
    # positions of one radian or less: every pair's cosine and sine are positive
    table = S.sdpa_rope_table(2, R, inv_freq=[1.0 / (1 + i) for i in range(R // 2)])
    ones = cuda.ones(T, dtype=cuda.int32, device="cuda")
    S.sdpa_paged_append_fp4(None, k, cuda.zeros_like(k), *codes, *scales,
                            cuda.zeros(1, 1, dtype=cuda.int32, device="cuda"),
                            cuda.tensor([T], dtype=cuda.int32, device="cuda"), table,
                            cu_seqlens_q=cuda.tensor([0, T], dtype=cuda.int32, device="cuda"),
                            positions=ones, interleaved=interleaved, k_gain=gain)
    kr, _ = S.sdpa_rope(k.transpose(0, 1)[None], None, table, positions=ones,
                        interleaved=interleaved)
    cuda.cuda.synchronize()
    assert S.sdpa_device_status() == 0
    return kr[0].transpose(0, 1), values_of(cuda, codes[0][0], scales[0][0]).transpose(0, 1), \
        scales[0][0].transpose(0, 1)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,R", [(64, 64), (128, 48)])
@pytest.mark.parametrize("gain", [None, 0.75])
def test_infinite_keys_under_rotation(cuda, gain, D, R, interleaved, dtype):
    dt = getattr(cuda, DT[dtype])
    g = cuda.Generator(device="cuda").manual_seed(11)
    big = {"f32": 3.3e38, "f16": 6e4, "bf16": 3.3e38}[dtype]
    k = (cuda.rand(6, 2, D, generator=g, device="cuda") - 0.5).to(dt)
    lo, hi = (4, 5) if interleaved else (2, 2 + R // 2)  # a pair, its first and second element
    k[0, :, lo] = math.inf
    k[1, :, lo] = -math.inf
    k[2, :, hi] = math.inf
    k[3, :, hi] = -math.inf
    k[4, :, lo], k[4, :, hi] = big, big      # its second element overflows
    k[5, :, lo], k[5, :, hi] = -big, big     # its first
    n = 1 / 3                                # the pair's angle
    c, s = math.cos(n), math.sin(n)
    assert c + s > 1.25 and big * 1.25 > float(cuda.finfo(dt).max)
    row, value, scale = append(cuda, k, R, interleaved,
                               None if gain is None else cuda.full((2,), gain, device="cuda"))
    inf = row.isinf()
    # the row itself: which elements are infinite, and no NaN
    assert not row.isnan().any()
    want = cuda.zeros_like(inf)
    want[:4, :, lo] = want[:4, :, hi] = True
    want[4, :, hi] = want[5, :, lo] = True
    assert cuda.equal(inf, want)
    assert (value[inf] == cuda.where(row[inf] > 0, 2688.0, -2688.0)).all()
    groups = inf.unflatten(-1, (-1, 16)).any(-1)
    assert (scale[groups] == 0x7E).all()
    rest = groups.repeat_interleave(16, -1) & (row.abs() < 1)
    assert int(rest.sum()) >= 6 * 2 * 14 and (value[rest] == 0).all()
