"""Host-side checks of the paged KV cache entry points: argument errors are
found before any CUDA call (these tests run without a GPU)."""
import ctypes

import pytest

import scaled_dot_product_fwd_gb300 as S
from scaled_dot_product_fwd_gb300 import _binding as B


def P(**kw):
    p = B.SdpaPagedParams()
    d = dict(num_seqs=2, num_tokens=5, num_q_heads=8, num_kv_heads=2, head_dim=128,
             dtype=S.SDPA_BF16, scale=0.1, causal=1, num_pages=9, page_size=16, max_pages=4,
             page_table=256, page_table_stride=4, cu_seqlens_q=512, seq_lens_kv=768)
    d.update({k: v for k, v in kw.items() if not k.endswith("_stride") or k == "page_table_stride"})
    for k, v in d.items():
        setattr(p, k, v)
    D = p.head_dim
    p.q_stride[:] = kw.get("q_stride", (p.num_q_heads * D, D))
    p.o_stride[:] = kw.get("o_stride", (p.num_q_heads * D, D))
    row = 2 * D
    p.k_stride[:] = kw.get("k_stride", (16 * row, D, row))
    p.v_stride[:] = kw.get("v_stride", (16 * row, D, row))
    return p


def forward(lib, p, q=256, k=256, v=256, o=512, lse=None, ws=256, n=1 << 40):
    return lib.sdpa_paged_forward(None if p is None else ctypes.byref(p), q, k, v, o, lse, ws, n,
                                  None)


def i64(*v):
    return (ctypes.c_int64 * len(v))(*v)


BAD = [
    (dict(num_seqs=-1), 1), (dict(num_tokens=-1), 1), (dict(num_kv_heads=0), 1),
    (dict(num_q_heads=7), 1), (dict(num_q_heads=-2), 1), (dict(page_size=0), 1),
    (dict(num_pages=-1), 1), (dict(max_pages=-1), 1), (dict(page_table_stride=-4), 1),
    (dict(flags=1), 1), (dict(dtype=3), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(head_dim=0), 1), (dict(head_dim=96), 2),
    (dict(head_dim=512), 2), (dict(max_pages=1 << 28), 2), (dict(num_tokens=(1 << 30) + 1), 2),
    (dict(k_stride=(4096, 128, 3)), 3), (dict(v_stride=(4096, 4, 256)), 3),
    (dict(q_stride=(1023, 128)), 3), (dict(o_stride=(1024, 12)), 3),
    (dict(q_stride=(-1024, 128)), 1), (dict(k_stride=(-8, 128, 256)), 1),
    (dict(o_stride=(0, 128)), 1), (dict(o_stride=(1024, 0)), 1),
    (dict(seq_lens_kv=None), 1), (dict(page_table=None), 1), (dict(seq_lens_kv=770), 3),
    (dict(cu_seqlens_q=513), 3), (dict(page_table=258), 3), (dict(sinks=6), 3),
]


@pytest.mark.parametrize("kw,status", BAD)
def test_forward_rejects(sdpa_lib, kw, status):
    assert forward(sdpa_lib, P(**kw)) == status
    assert S.sdpa_last_launch_count() == 0


def test_forward_rejects_pointers(sdpa_lib):
    p = P()
    assert forward(sdpa_lib, None) == 1
    for name in ("q", "k", "v", "o"):
        assert forward(sdpa_lib, p, **{name: None}) == 1
        assert forward(sdpa_lib, p, **{name: 264}) == 3
    assert forward(sdpa_lib, p, lse=258) == 3
    need = S.sdpa_paged_workspace_size(p)
    assert need > 0
    assert forward(sdpa_lib, p, n=need - 1) == 4
    assert forward(sdpa_lib, p, ws=None) == 4
    assert forward(sdpa_lib, p, ws=257) == 3


def test_nothing_to_compute(sdpa_lib):
    for kw in (dict(num_seqs=0), dict(num_tokens=0), dict(num_q_heads=0)):
        p = P(**kw)
        assert S.sdpa_paged_workspace_size(p) == 0
        assert forward(sdpa_lib, p, None, None, None, None, None, None, 0) == 0
    assert S.sdpa_paged_workspace_size(P(head_dim=96)) == 0


def test_workspace_is_independent_of_lengths(sdpa_lib):
    n = S.sdpa_paged_workspace_size(P())
    assert n == S.sdpa_paged_workspace_size(P(max_pages=4096, num_pages=9999))
    assert n % 256 == 0 and n < 1 << 28


def test_write_rejects(sdpa_lib):
    f = sdpa_lib.sdpa_paged_write
    kn = i64(256, 128)

    def call(p, k=256, v=256, ks=kn, vs=kn, kp=256, vp=256):
        return f(ctypes.byref(p), k, v, ks, vs, kp, vp, None)

    for kw, status in BAD:
        if not {"num_q_heads", "scale", "q_stride", "o_stride", "sinks"} & set(kw):
            assert call(P(**kw)) == status, kw
    p = P()
    for name in ("k", "v", "kp", "vp"):
        assert call(p, **{name: None}) == 1
        assert call(p, **{name: 264}) == 3
    assert call(p, ks=None) == 1 and call(p, vs=None) == 1
    assert call(p, ks=i64(257, 128)) == 3 and call(p, vs=i64(-256, 128)) == 1
    # a cache whose rows lie on one another cannot be written
    assert call(P(k_stride=(0, 128, 256))) == 1 and call(P(v_stride=(4096, 128, 0))) == 1
    assert call(P(num_tokens=0), None, None, None, None, None, None) == 0


def test_scores_rejects(sdpa_lib):
    f = sdpa_lib.sdpa_paged_scores
    st = i64(128, 64)

    def call(p, q=256, k=256, lse=256, sc=256, ss=st, n=64, ws=256, nb=1 << 40):
        return f(ctypes.byref(p), q, k, lse, sc, ss, n, ws, nb, None)

    for kw, status in BAD:
        if not {"v_stride", "o_stride"} & set(kw):
            assert call(P(**kw)) == status, kw
    p = P()
    for name in ("q", "k", "lse", "sc"):
        assert call(p, **{name: None}) == 1
    assert call(p, q=264) == 3 and call(p, k=264) == 3
    assert call(p, lse=257) == 3 and call(p, sc=258) == 3
    assert call(p, ss=None) == 1 and call(p, ss=i64(-1, 64)) == 1 and call(p, n=-1) == 1
    assert call(p, ss=i64(0, 64)) == 1 and call(p, ss=i64(128, 0)) == 1
    assert call(p, nb=64) == 4 and call(p, ws=264) == 3
    assert call(p, n=0, q=None) == 0


def test_evict_rejects(sdpa_lib):
    f = sdpa_lib.sdpa_paged_evict
    st = i64(128, 64)

    def call(p, keep=8, recent=2, k=256, v=256, sc=256, so=None, ss=st, n=64, kept=256, sl=None):
        return f(ctypes.byref(p), keep, recent, k, v, sc, so, ss, n, kept, sl, None)

    for kw, status in BAD:
        if not {"num_q_heads", "scale", "q_stride", "o_stride", "sinks", "num_tokens",
                "cu_seqlens_q"} & set(kw):
            assert call(P(**kw)) == status, kw
    p = P()
    assert call(p, keep=0) == 1 and call(p, recent=-1) == 1 and call(p, n=-1) == 1
    for name in ("k", "v", "sc", "kept", "ss"):
        assert call(p, **{name: None}) == 1
    assert call(p, k=264) == 3 and call(p, so=258) == 3 and call(p, kept=257) == 3
    assert call(p, sl=255) == 3
    assert call(p, so=256, ss=i64(0, 64)) == 1
    assert call(P(k_stride=(0, 128, 256))) == 1


def test_evict_rejects_counts_past_the_positions(sdpa_lib):
    """Loops over keep and score_len step past them: near 2^31 they would wrap."""
    f = sdpa_lib.sdpa_paged_evict
    p, st, big = P(), i64(128, 64), (1 << 30) + 1
    for keep, n in ((big, 64), ((1 << 31) - 1, 64), (8, big), (8, (1 << 31) - 1)):
        assert f(ctypes.byref(p), keep, 2, 256, 512, 256, None, st, n, 256, None, None) == 2


def test_one_cache_for_keys_and_values_is_not_written(sdpa_lib):
    p, st = P(), i64(128, 64)
    assert sdpa_lib.sdpa_paged_evict(ctypes.byref(p), 8, 2, 256, 256, 256, None, st, 64, 256,
                                     None, None) == 1
    kn = i64(256, 128)
    assert sdpa_lib.sdpa_paged_write(ctypes.byref(p), 256, 512, kn, kn, 1024, 1024, None) == 1


def test_binding_rejects_cpu_tensors(sdpa_lib):
    torch = pytest.importorskip("torch")
    q = torch.zeros(1, 2, 64)
    kp = torch.zeros(1, 2, 16, 64)
    t = torch.zeros(1, 1, dtype=torch.int32)
    n = torch.ones(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        S.sdpa_paged_forward(q, kp, kp, t, n)
    with pytest.raises(ValueError):
        S.sdpa_paged_write(q, q, kp, kp, t, n)


def test_params_struct_layout():
    assert ctypes.sizeof(B.SdpaPagedParams) == 168
    assert B.SdpaPagedParams.page_table.offset == 48
    assert B.SdpaPagedParams.q_stride.offset == 88
    assert B.SdpaPagedParams.v_stride.offset == 144
