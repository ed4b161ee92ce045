"""sdpa_paged_write with one cache for keys and values (runs without a GPU): the
rows written twice have to be the same, places and values."""
import ctypes

import pytest

from test_paged_abi import P, i64


@pytest.mark.parametrize("kw,kn,vn", [
    ({}, (256, 128), (128, 256)),                       # other rows of the same tensor
    ({}, (256, 128), (512, 128)),
    (dict(v_stride=(4096, 2048, 128)), (256, 128), (256, 128)),  # the same rows to other places
    (dict(k_stride=(8192, 128, 256)), (256, 128), (256, 128)),
], ids=str)
def test_one_cache_with_other_rows_is_refused(sdpa_lib, kw, kn, vn):
    assert sdpa_lib.sdpa_paged_write(ctypes.byref(P(**kw)), 256, 256, i64(*kn), i64(*vn), 1024,
                                     1024, None) == 1
