"""More host-side refusals of the calls for branching decode: tables too wide for 32-bit entries, lengths written over a call's own
inputs.  (No GPU: every call below is refused before anything is launched.)"""
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


def test_new_lengths_that_overlap_inputs(K):
    size = dict(table=3 * 4, lens=3, parents=3 * 8, num=3, accepted=3)
    at = {x: (i + 1) << 16 for i, x in enumerate(size)}

    def keep(new_lens, **kw):
        p = {**at, **kw}
        return K.lib().kda_paged_tree_commit(1 << 24, 1 << 25, p["table"], p["lens"], p["parents"], p["num"], p["accepted"], 8, new_lens, dims(K), None)
    for x in size:
        places = [at[x] + 4 * (size[x] - 1), at[x] + 4, at[x] - 4, at[x] - 8] + [at[x]] * (x != "lens")   # (seq_lens itself may be replaced)
        for place in places:
            assert keep(place) == K.KDA_ERR_SHAPE, (x, place - at[x])
    for x in ("parents", "num"):                    # what is not given overlaps nothing; the others still do
        assert keep(at["lens"] + 4, **{x: None}) == K.KDA_ERR_SHAPE


def test_the_smallest_attention_has_two_ctas(K):
    """The join, which also writes the outputs of tokens past a count, follows every call that is shared out."""
    need = K.lib().kda_paged_tree_attention_workspace_bytes
    for d in (64, 128):
        one = dims(K, rows=1, heads=1, kv_heads=1, head_dim=d, pages=1, page_size=1, max_pages=1, dtype=0)
        assert need(1, one) == 2 * 2 * 64 * (d + 2) * 4
        assert need(64, one) >= need(1, one)
    # bf16: the shortest rows that are not taken in one launch
    assert need(1, dims(K, rows=1, heads=1, kv_heads=1, max_pages=1 << 12)) >= 2 * 2 * 256 * (128 + 2) * 4
