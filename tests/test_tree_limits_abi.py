"""More host-side refusals of the calls for branching decode: tables too wide for 32-bit entries.  (No GPU: every
call below is refused before anything is launched.)"""
import ctypes

import pytest

from linear_attention_fwd_gb300 import build as kbuild


@pytest.fixture(scope="module")
def K():
    kbuild.build()
    from linear_attention_fwd_gb300 import kda
    kda.lib()
    return kda


def dims(K, **kw):
    d = dict(rows=3, heads=8, kv_heads=2, head_dim=128, pages=10, page_size=16, max_pages=4, dtype=1)
    d.update(kw)
    return ctypes.byref(K.KdaPagedDims(*[d[f] for f, _ in K.KdaPagedDims._fields_]))


@pytest.mark.parametrize("width", [(1 << 30) + 1, (1 << 31) - (1 << 17) + 1, (1 << 31) - 65])
def test_fork_of_tables_too_wide(K, width):
    """A segment's end, or a step past it, would not fit 32 bits."""
    apart = [(i + 1) << 40 for i in range(10)]      # (never dereferenced; no two arrays overlap)
    assert K.lib().kda_paged_fork(*apart, dims(K, rows=1, page_size=1, max_pages=width), None) == K.KDA_ERR_SHAPE
