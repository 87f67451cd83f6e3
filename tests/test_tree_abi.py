"""Host-side refusals of the calls for branching decode (no GPU: every call below fails validation, or has nothing to
do, before anything is launched)."""
import ctypes

import pytest
import torch

from linear_attention_fwd_gb300 import build as kbuild

FAKE = 1 << 20          # 16-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def K():
    kbuild.build()
    from linear_attention_fwd_gb300 import kda
    kda.lib()
    return kda


def ref(d):
    return ctypes.byref(d) if d is not None else None


def dims(K, **kw):
    d = dict(batch=2, seqlen=8, num_seqs=2, heads=4, dk=128, dv=64, dtype=1)
    d.update(kw)
    return K.KdaDims(*[d[f] for f, _ in K.KdaDims._fields_])


def paged(K, **kw):
    d = dict(rows=3, heads=8, kv_heads=2, head_dim=128, pages=10, page_size=16, max_pages=4, dtype=1)
    d.update(kw)
    return K.KdaPagedDims(*[d[f] for f, _ in K.KdaPagedDims._fields_])


def verify(K, d, q=FAKE, k=FAKE, v=FAKE, g=FAKE, beta=FAKE, state=FAKE, idx=None, parents=None, num=None, out=FAKE, eps=None):
    if eps is None:
        return K.lib().kda_recurrent_tree(q, k, v, g, beta, state, idx, parents, num, out, ref(d), None)
    return K.lib().kda_recurrent_tree_qknorm(q, k, v, g, beta, eps, state, idx, parents, num, out, ref(d), None)


def replay(K, d, k=FAKE, v=FAKE, g=FAKE, beta=FAKE, state=FAKE, idx=None, parents=None, num=None, accepted=FAKE, eps=None):
    if eps is None:
        return K.lib().kda_recurrent_tree_commit(k, v, g, beta, state, idx, parents, num, accepted, ref(d), None)
    return K.lib().kda_recurrent_tree_commit_qknorm(k, v, g, beta, eps, state, idx, parents, num, accepted, ref(d), None)


def attend(K, d, q=FAKE, kc=FAKE, vc=FAKE, table=FAKE, lens=FAKE, parents=None, num=None, tokens=8, scale=0.1, out=FAKE, lse=FAKE,
           ws=FAKE, wb=1 << 40):
    return K.lib().kda_paged_tree_attention(q, kc, vc, table, lens, parents, num, tokens, scale, out, lse, ws, wb, ref(d), None)


def keep(K, d, kc=FAKE, vc=FAKE, table=FAKE, lens=FAKE, parents=None, num=None, accepted=FAKE, tokens=8, new_lens=None):
    return K.lib().kda_paged_tree_commit(kc, vc, table, lens, parents, num, accepted, tokens, new_lens, ref(d), None)


PLACES = {x: FAKE + (i + 1) * 4096 for i, x in enumerate(
    ("table", "lens", "refs", "sources", "new", "new_table", "new_lens", "new_refs", "copies", "short"))}


def fork(K, d, **kw):
    p = {**PLACES, **kw}
    return K.lib().kda_paged_fork(*(p[x] for x in PLACES), ref(d), None)


def compact(K, d, **kw):
    p = {**PLACES, **kw}
    return K.lib().kda_paged_compact(*(p[x] for x in ("table", "refs", "new_table", "new_refs", "copies")), ref(d), None)


def copy(K, d, kc=FAKE, vc=FAKE, copies=FAKE, count=3):
    return K.lib().kda_paged_copy(kc, vc, copies, count, ref(d), None)


@pytest.mark.parametrize("kw,code", [
    (dict(dk=96), 3), (dict(dv=32), 3), (dict(dtype=2), 3), (dict(heads=0), 2), (dict(batch=0), 2), (dict(batch=-1), 2), (dict(seqlen=0), 2),
    (dict(seqlen=65), 2), (dict(num_seqs=0), 2), (dict(num_seqs=1), 2), (dict(batch=1 << 20, num_seqs=1 << 20, heads=1 << 12), 2),
    (dict(batch=1 << 20, num_seqs=1 << 20, heads=1 << 9), 2),
])
def test_state_dims(K, kw, code):
    for eps in (None, 1e-6):
        assert verify(K, dims(K, **kw), eps=eps) == code
        assert replay(K, dims(K, **kw), eps=eps) == code


def test_state_pointers(K):
    for eps in (None, 0.0):
        assert verify(K, None, eps=eps) == replay(K, None, eps=eps) == K.KDA_ERR_NULL
        for x in ("q", "k", "v", "g", "beta", "state", "out"):
            assert verify(K, dims(K), **{x: None}, eps=eps) == K.KDA_ERR_NULL
            assert verify(K, dims(K), **{x: FAKE + 8}, eps=eps) == K.KDA_ERR_ALIGN
        for x in ("k", "v", "g", "beta", "state"):
            assert replay(K, dims(K), **{x: None}, eps=eps) == K.KDA_ERR_NULL
            assert replay(K, dims(K), **{x: FAKE + 4}, eps=eps) == K.KDA_ERR_ALIGN
        assert replay(K, dims(K), accepted=None, eps=eps) == K.KDA_ERR_NULL
        for x in ("idx", "parents", "num"):
            assert verify(K, dims(K), **{x: FAKE + 2}, eps=eps) == K.KDA_ERR_ALIGN
            assert replay(K, dims(K), **{x: FAKE + 1}, eps=eps) == K.KDA_ERR_ALIGN
        assert replay(K, dims(K), accepted=FAKE + 2, eps=eps) == K.KDA_ERR_ALIGN
    for eps in (-1.0, float("nan"), float("inf")):
        assert verify(K, dims(K), eps=eps) == replay(K, dims(K), eps=eps) == K.KDA_ERR_SHAPE


@pytest.mark.parametrize("kw,code", [
    (dict(head_dim=96), 3), (dict(dtype=2), 3), (dict(rows=-1), 2), (dict(kv_heads=0), 2), (dict(pages=0), 2), (dict(page_size=0), 2),
    (dict(max_pages=0), 2), (dict(page_size=1 << 20, max_pages=1 << 12), 2), (dict(page_size=1, max_pages=(1 << 31) - 500), 2),
])
def test_cache_dims(K, kw, code):
    assert attend(K, paged(K, **kw)) == code
    assert keep(K, paged(K, **kw)) == code
    assert K.lib().kda_paged_tree_attention_workspace_bytes(8, ctypes.byref(paged(K, **kw))) == 0


def test_attention_refusals(K):
    assert attend(K, None) == K.KDA_ERR_NULL
    for kw in (dict(heads=0), dict(heads=7), dict(pages=1 << 27, page_size=16), dict(rows=1 << 20, heads=1 << 10)):
        assert attend(K, paged(K, **kw)) == K.KDA_ERR_SHAPE
    for tokens in (0, -1, 65):
        assert attend(K, paged(K), tokens=tokens) == K.KDA_ERR_SHAPE
        assert K.lib().kda_paged_tree_attention_workspace_bytes(tokens, ctypes.byref(paged(K))) == 0
    for scale in (float("nan"), float("inf")):
        assert attend(K, paged(K), scale=scale) == K.KDA_ERR_SHAPE
    for x in ("q", "kc", "vc", "table", "lens", "out"):
        assert attend(K, paged(K), **{x: None}) == K.KDA_ERR_NULL
    for x in ("q", "kc", "vc", "out"):
        assert attend(K, paged(K), **{x: FAKE + 8}) == K.KDA_ERR_ALIGN
    for x in ("table", "lens", "lse", "parents", "num"):
        assert attend(K, paged(K), **{x: FAKE + 2}) == K.KDA_ERR_ALIGN
    d = paged(K, max_pages=4096)      # rows that are cut: a workspace
    need = K.lib().kda_paged_tree_attention_workspace_bytes(8, ctypes.byref(d))
    assert need > 0
    assert attend(K, d, ws=None) == K.KDA_ERR_NULL
    assert attend(K, d, wb=need - 1) == K.KDA_ERR_WORKSPACE
    assert attend(K, d, ws=FAKE + 4) == K.KDA_ERR_ALIGN
    assert attend(K, paged(K, rows=0), q=None) == K.KDA_OK
    assert K.lib().kda_paged_tree_attention_workspace_bytes(8, None) == 0


def test_commit_refusals(K):
    assert keep(K, None) == K.KDA_ERR_NULL
    for tokens in (0, 65):
        assert keep(K, paged(K), tokens=tokens) == K.KDA_ERR_SHAPE
    for x in ("kc", "vc", "table", "lens", "accepted"):
        assert keep(K, paged(K), **{x: None}) == K.KDA_ERR_NULL
    for x in ("kc", "vc"):
        assert keep(K, paged(K), **{x: FAKE + 8}) == K.KDA_ERR_ALIGN
    for x in ("table", "lens", "parents", "num", "accepted", "new_lens"):
        assert keep(K, paged(K), **{x: FAKE + 2}) == K.KDA_ERR_ALIGN
    assert keep(K, paged(K, rows=0), kc=None) == K.KDA_OK


@pytest.mark.parametrize("kw", [dict(rows=-1), dict(rows=65537), dict(pages=0), dict(pages=(1 << 22) + 1), dict(page_size=0), dict(max_pages=0),
                                dict(page_size=1 << 20, max_pages=1 << 12), dict(rows=65536, max_pages=1 << 16, page_size=1)])
def test_pool_dims(K, kw):
    assert fork(K, paged(K, **kw)) == K.KDA_ERR_SHAPE
    assert compact(K, paged(K, **kw)) == K.KDA_ERR_SHAPE


def test_pool_refusals(K):
    assert fork(K, None) == compact(K, None) == K.KDA_ERR_NULL
    assert fork(K, paged(K, rows=0)) == K.KDA_ERR_SHAPE
    for x in PLACES:
        if x != "new":
            assert fork(K, paged(K), **{x: None}) == K.KDA_ERR_NULL
        assert fork(K, paged(K), **{x: FAKE + 2}) == K.KDA_ERR_ALIGN
    for x in ("new_table", "new_lens", "new_refs", "copies", "short"):
        for y in ("table", "lens", "refs", "sources", "new"):
            assert fork(K, paged(K), **{x: PLACES[y]}) == K.KDA_ERR_SHAPE
    for x in ("table", "refs", "new_table", "new_refs", "copies"):
        assert compact(K, paged(K), **{x: None}) == K.KDA_ERR_NULL
        assert compact(K, paged(K), **{x: FAKE + 2}) == K.KDA_ERR_ALIGN
    for x in ("new_table", "new_refs", "copies"):
        for y in ("table", "refs"):
            assert compact(K, paged(K), **{x: PLACES[y]}) == K.KDA_ERR_SHAPE


def test_outputs_that_overlap(K):
    """In part, too: an array that starts within another's last number, or ends within its first."""
    size = dict(table=12, lens=3, refs=10, sources=3, new=3, new_table=12, new_lens=3, new_refs=10, copies=6, short=1)
    outs = ("new_table", "new_lens", "new_refs", "copies", "short")
    for x in outs:
        for y in size:
            if x != y:
                assert fork(K, paged(K), **{x: PLACES[y] + 4 * (size[y] - 1)}) == K.KDA_ERR_SHAPE, (x, y)
                assert fork(K, paged(K), **{x: PLACES[y] - 4 * (size[x] - 1)}) == K.KDA_ERR_SHAPE, (x, y)
    size["copies"] = 10
    for x in ("new_table", "new_refs", "copies"):
        for y in ("table", "refs", "new_table", "new_refs", "copies"):
            if x != y:
                assert compact(K, paged(K), **{x: PLACES[y] + 4 * (size[y] - 1)}) == K.KDA_ERR_SHAPE, (x, y)
                assert compact(K, paged(K), **{x: PLACES[y] - 4 * (size[x] - 1)}) == K.KDA_ERR_SHAPE, (x, y)


def test_copy_refusals(K):
    assert copy(K, None) == K.KDA_ERR_NULL
    for kw in (dict(head_dim=96), dict(dtype=5)):
        assert copy(K, paged(K, **kw)) == K.KDA_ERR_UNSUPPORTED
    for kw in (dict(kv_heads=0), dict(pages=0), dict(page_size=0), dict(pages=1 << 22, page_size=1 << 11)):
        assert copy(K, paged(K, **kw)) == K.KDA_ERR_SHAPE
    assert copy(K, paged(K), count=-1) == copy(K, paged(K), count=1 << 31) == K.KDA_ERR_SHAPE
    for x in ("kc", "vc", "copies"):
        assert copy(K, paged(K), **{x: None}) == K.KDA_ERR_NULL
        assert copy(K, paged(K), **{x: FAKE + 2}) == K.KDA_ERR_ALIGN
    assert copy(K, paged(K), count=0, kc=None) == K.KDA_OK


def test_binding_refuses_host_tensors(K):
    x, i = torch.zeros(1, 4, 2, 64), torch.zeros(1, dtype=torch.int32)
    bad = (ValueError, RuntimeError, AssertionError)
    with pytest.raises(bad):
        K.kda_recurrent_tree(x, x, x, x, x[..., 0], torch.zeros(1, 2, 64, 64))
    with pytest.raises(bad):
        K.kda_paged_tree_attention(x, x, x, i[None], i, None, 1.0)
    with pytest.raises(bad):
        K.kda_paged_fork(i[None], i, i, i, page_size=1)
