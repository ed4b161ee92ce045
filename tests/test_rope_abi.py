"""Host-side checks of the rotary and 4-bit cache entry points: argument errors
are found before any CUDA call (these tests run without a GPU)."""
import ctypes
import math

import pytest

import scaled_dot_product_fwd_gb300 as S
from scaled_dot_product_fwd_gb300 import _binding as B
from test_paged_abi import P, i64


def rotation(**kw):
    r = B.SdpaRotation()
    for k, v in dict(table=256, table_len=100, rotary_dim=64, interleaved=0, positions=512,
                     **{}).items():
        setattr(r, k, kw.get(k, v))
    return r


def R(**kw):
    p = B.SdpaRopeParams()
    d = dict(batch=2, num_q_heads=8, num_kv_heads=2, seq_len=5, head_dim=64, dtype=S.SDPA_BF16,
             transpose=0, flags=0, position_stride=5)
    for k, v in d.items():
        setattr(p, k, kw.get(k, v))
    p.rotation = rotation(**{k: v for k, v in kw.items() if hasattr(B.SdpaRotation, k)})
    for name, h in (("q", 8), ("k", 2)):
        for out in ("", "_out"):
            f = name + out + "_stride"
            getattr(p, f)[:] = kw.get(f, (h * 5 * 64, 5 * 64, 64))
    return p


def rope(lib, p, q=1024, k=2048, q_out=4096, k_out=8192):
    return lib.sdpa_rope(None if p is None else ctypes.byref(p), q, k, q_out, k_out, None)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), 1), (dict(num_q_heads=-1), 1), (dict(num_kv_heads=-1), 1),
    (dict(seq_len=-1), 1), (dict(flags=1), 1), (dict(dtype=3), 1), (dict(position_stride=-1), 1),
    (dict(head_dim=0), 1), (dict(head_dim=96), 2), (dict(head_dim=256), 2),
    (dict(rotary_dim=0), 1), (dict(rotary_dim=-16), 1), (dict(rotary_dim=80), 1),
    (dict(rotary_dim=24), 2), (dict(rotary_dim=63), 2), (dict(table=None), 1),
    (dict(table=264), 3), (dict(table_len=-1), 1), (dict(positions=514), 3),
    (dict(q_stride=(2560, 320, 3)), 3), (dict(k_out_stride=(640, 4, 64)), 3),
    (dict(q_stride=(-2560, 320, 64)), 1), (dict(q_out_stride=(2560, 0, 64)), 1),
    (dict(k_out_stride=(0, 320, 64)), 1), (dict(q_out_stride=(2560, 320, 0)), 1),
    (dict(batch=1 << 16, seq_len=1 << 15), 2),
])
def test_rope_rejects(sdpa_lib, kw, status):
    assert rope(sdpa_lib, R(**kw)) == status
    assert S.sdpa_last_launch_count() == 0


def test_rope_rejects_pointers(sdpa_lib):
    assert rope(sdpa_lib, None) == 1
    for name in ("q", "k", "q_out", "k_out"):
        assert rope(sdpa_lib, R(), **{name: None}) == 1
        assert rope(sdpa_lib, R(), **{name: 1032}) == 3
    # in place only with the input's own layout
    assert rope(sdpa_lib, R(q_out_stride=(2560, 64, 512)), q_out=1024) == 1


def test_rope_rejects_one_output_for_both(sdpa_lib):
    assert rope(sdpa_lib, R(), q_out=4096, k_out=4096) == 1
    assert rope(sdpa_lib, R(), q=1024, k=1024, q_out=1024, k_out=1024) == 1


def test_rope_nothing_to_do(sdpa_lib):
    for kw in (dict(batch=0), dict(seq_len=0), dict(num_q_heads=0, num_kv_heads=0)):
        assert rope(sdpa_lib, R(**kw), None, None, None, None) == 0


def test_rope_table_rejects(sdpa_lib):
    f = (ctypes.c_double * 32)(*[1.0] * 32)
    call = sdpa_lib.sdpa_rope_table
    assert call(256, -1, 64, f, 1.0, None) == 1
    assert call(256, 10, 0, f, 1.0, None) == 1
    assert call(256, 10, 24, f, 1.0, None) == 2
    assert call(256, 10, 528, f, 1.0, None) == 2
    assert call(256, 10, 64, None, 1.0, None) == 1
    assert call(256, 10, 64, f, math.inf, None) == 1
    assert call(None, 10, 64, f, 1.0, None) == 1
    assert call(260, 10, 64, f, 1.0, None) == 3
    f[3] = math.nan
    assert call(256, 10, 64, f, 1.0, None) == 1
    assert call(None, 0, 64, (ctypes.c_double * 32)(), 1.0, None) == 0


KN = (256, 128)


def append(lib, p, rot="own", q=1024, k=2048, v=6144, q_out=4096, kn=KN, vn=KN, kp=8192,
           vp=16384):
    r = rotation(rotary_dim=128) if rot == "own" else rot
    return lib.sdpa_paged_append(None if p is None else ctypes.byref(p),
                                 None if r is None else ctypes.byref(r), q, k, v, q_out,
                                 None if kn is None else i64(*kn), None if vn is None else i64(*vn),
                                 kp, vp, None)


def test_append_rejects(sdpa_lib):
    lib = sdpa_lib
    assert append(lib, None) == 1 and append(lib, P(), rot=None) == 1
    for kw, status in ((dict(num_q_heads=7), 1), (dict(num_q_heads=-2), 1), (dict(head_dim=96), 2),
                       (dict(flags=1), 1), (dict(q_stride=(1023, 128)), 3),
                       (dict(o_stride=(0, 128)), 1), (dict(o_stride=(1024, 0)), 1),
                       (dict(k_stride=(0, 128, 256)), 1), (dict(seq_lens_kv=None), 1),
                       (dict(seq_lens_kv=770), 3), (dict(page_table=None), 1)):
        assert append(lib, P(**kw)) == status, kw
    for name in ("q", "k", "v", "q_out", "kp", "vp"):
        assert append(lib, P(), **{name: None}) == 1, name
        assert append(lib, P(), **{name: 1032}) == 3, name
    assert append(lib, P(), kn=None) == 1 and append(lib, P(), vn=(256, 3)) == 3
    assert append(lib, P(), vp=8192) == 1  # one cache for both
    for kw, status in ((dict(rotary_dim=144), 1), (dict(rotary_dim=8), 2), (dict(table=None), 1),
                       (dict(table=4), 3)):
        assert append(lib, P(), rot=rotation(**kw)) == status, kw
    # in place only with q's own strides
    assert append(lib, P(o_stride=(2048, 128)), q_out=1024) == 1
    for kw in (dict(num_seqs=0), dict(num_tokens=0)):
        assert append(lib, P(**kw), q=None, k=None, v=None, q_out=None) == 0


def cache4(**kw):
    c = B.SdpaFp4Cache()
    d = dict(k_codes=1024, v_codes=2048, k_scales=4096, v_scales=8192, k_gain=256, v_gain=512)
    for k, v in d.items():
        setattr(c, k, kw.get(k, v))
    c.k_scale_stride[:] = kw.get("k_scale_stride", (16 * 16, 8, 16))
    c.v_scale_stride[:] = kw.get("v_scale_stride", (16 * 16, 8, 16))
    return c


def P4(**kw):
    d = dict(k_stride=(2048, 64, 128), v_stride=(2048, 64, 128))
    d.update(kw)
    return P(**d)


BAD4 = [(dict(k_codes=None), 1), (dict(v_scales=None), 1), (dict(k_codes=1032), 3),
        (dict(v_scales=8196), 3), (dict(k_gain=258), 3), (dict(k_scale_stride=(256, 8, 12)), 3),
        (dict(v_scale_stride=(256, -8, 16)), 1)]


def forward4(lib, p, c="own", q=256, o=512, lse=None, ws=256, n=1 << 40):
    c = cache4() if c == "own" else c
    return lib.sdpa_paged_forward_fp4(None if p is None else ctypes.byref(p),
                                      None if c is None else ctypes.byref(c), q, o, lse, ws, n,
                                      None)


def test_forward_fp4_rejects(sdpa_lib):
    lib = sdpa_lib
    assert forward4(lib, None) == 1 and forward4(lib, P4(), c=None) == 1
    for kw, status in ((dict(num_q_heads=7), 1), (dict(scale=math.nan), 1), (dict(head_dim=96), 2),
                       (dict(head_dim=512), 2), (dict(dtype=3), 1), (dict(flags=1), 1),
                       (dict(k_stride=(2048, 64, 100)), 3), (dict(v_stride=(-16, 64, 128)), 1),
                       (dict(q_stride=(1023, 128)), 3), (dict(o_stride=(0, 128)), 1),
                       (dict(max_pages=1 << 28), 2), (dict(seq_lens_kv=None), 1),
                       (dict(page_table=258), 3), (dict(sinks=6), 3)):
        assert forward4(lib, P4(**kw)) == status, kw
    for kw, status in BAD4:
        assert forward4(lib, P4(), cache4(**kw)) == status, kw
    for name in ("q", "o"):
        assert forward4(lib, P4(), **{name: None}) == 1
        assert forward4(lib, P4(), **{name: 264}) == 3
    assert forward4(lib, P4(), lse=258) == 3
    assert forward4(lib, P4(), n=100) == 4 and forward4(lib, P4(), ws=None) == 4
    assert forward4(lib, P4(), ws=257) == 3
    for kw in (dict(num_seqs=0), dict(num_tokens=0), dict(num_q_heads=0)):
        assert forward4(lib, P4(**kw), q=None, o=None, ws=None, n=0) == 0


def append4(lib, p, c="own", rot=None, q=1024, k=2048, v=6144, q_out=4096, kn=KN, vn=KN, ko=None,
            vo=None, os=None):
    c = cache4() if c == "own" else c
    return lib.sdpa_paged_append_fp4(None if p is None else ctypes.byref(p),
                                     None if rot is None else ctypes.byref(rot),
                                     None if c is None else ctypes.byref(c), q, k, v, q_out,
                                     i64(*kn), i64(*vn), ko, vo,
                                     None if os is None else i64(*os), None)


def test_append_fp4_rejects(sdpa_lib):
    lib = sdpa_lib
    assert append4(lib, None) == 1 and append4(lib, P4(), c=None) == 1
    for kw, status in BAD4 + [(dict(k_scale_stride=(0, 8, 16)), 1), (dict(v_codes=1024), 1),
                              (dict(v_scales=4096), 1)]:
        assert append4(lib, P4(), cache4(**kw)) == status, kw
    assert append4(lib, P4(k_stride=(0, 64, 128))) == 1
    assert append4(lib, P4(num_q_heads=7)) == 1
    assert append4(lib, P4(), rot=rotation(rotary_dim=20)) == 2
    assert append4(lib, P4(), k=None) == 1 and append4(lib, P4(), v=6152) == 3
    assert append4(lib, P4(), kn=(256, 3)) == 3
    assert append4(lib, P4(), ko=16384) == 1  # no strides
    assert append4(lib, P4(), ko=16384, vo=16384, os=(256, 128)) == 1
    assert append4(lib, P4(), ko=16384, os=(0, 128)) == 1
    assert append4(lib, P4(), ko=16392, os=(256, 128)) == 3
    assert append4(lib, P4(num_tokens=0), k=None, v=None) == 0


def test_struct_layouts():
    assert ctypes.sizeof(B.SdpaRotation) == 32 == B._ROTATION.size
    assert ctypes.sizeof(B.SdpaRopeParams) == 168 == B._ROPE.size
    assert ctypes.sizeof(B.SdpaFp4Cache) == 96 == B._FP4.size
    assert B.SdpaRopeParams.rotation.offset == 32
    assert B.SdpaRopeParams.q_stride.offset == 72
    assert B.SdpaFp4Cache.k_gain.offset == 80


def test_status_string(sdpa_lib):
    assert S.sdpa_status_string(8) == "position outside the rotation table"


def test_frequencies():
    f, g = S.rope_frequencies(8, base=16.0)
    assert g == 1.0 and f == [1.0, 0.5, 0.25, 0.125]
    f, g = S.rope_frequencies(8, base=16.0, scaling="linear", factor=4.0)
    assert g == 1.0 and f == [0.25, 0.125, 0.0625, 0.03125]
    # the slowest pair counts 1 / factor, the fastest stays
    f, g = S.rope_frequencies(64, scaling="ntk", factor=8.0)
    slow = 10000.0**(-62 / 64)
    assert f[0] == 1.0 and math.isclose(f[-1], slow / 8, rel_tol=1e-12)
    f, g = S.rope_frequencies(128, scaling="yarn", factor=16.0, original_length=4096)
    own, _ = S.rope_frequencies(128)
    assert math.isclose(g, 0.1 * math.log(16.0) + 1)
    assert f[0] == own[0] and math.isclose(f[-1], own[-1] / 16)
    assert all(b / 16 <= a <= b for a, b in zip(f, own))
    ratio = [a / b for a, b in zip(f, own)]
    assert ratio == sorted(ratio, reverse=True)
    for bad in (dict(rotary_dim=7), dict(rotary_dim=8, base=0.0), dict(rotary_dim=8, factor=0.0),
                dict(rotary_dim=8, scaling="no"), dict(rotary_dim=8, scaling="yarn"),
                dict(rotary_dim=2, scaling="ntk")):
        with pytest.raises(ValueError):
            S.rope_frequencies(**bad)


def test_binding_rejects_cpu_tensors(sdpa_lib):
    torch = pytest.importorskip("torch")
    x = torch.zeros(1, 2, 4, 64)
    table = torch.zeros(4, 32, 2)
    with pytest.raises(ValueError):
        S.sdpa_rope(x, x, table)
    with pytest.raises(ValueError):
        S.sdpa_rope_backward(x, None, table)
    with pytest.raises(ValueError):
        S.sdpa_rope_table(10, 64, device="cpu")
    q = torch.zeros(1, 2, 64)
    kp = torch.zeros(1, 2, 16, 64)
    c, s = torch.zeros(1, 2, 16, 32, dtype=torch.uint8), torch.zeros(1, 2, 16, 4,
                                                                     dtype=torch.uint8)
    t, n = torch.zeros(1, 1, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        S.sdpa_paged_append(q, q, q, kp, kp, t, n, table)
    with pytest.raises(ValueError):
        S.sdpa_paged_append_fp4(q, q, q, c, c, s, s, t, n)
    with pytest.raises(ValueError):
        S.sdpa_paged_forward_fp4(q, c, c, s, s, t, n)
    with pytest.raises(TypeError):
        S.sdpa_paged_forward_fp4(q, kp, kp, s, s, t, n)
