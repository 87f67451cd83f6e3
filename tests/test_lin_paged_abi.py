"""Host-side refusals of the linear-attention and paged-cache calls (no GPU: every call below fails
validation, or has nothing to do, before anything is launched)."""
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


def lin(K, **kw):
    d = dict(batch=2, seqlen=100, num_seqs=2, heads=4, qk_heads=2, dk=128, dv=64, dtype=1)
    d.update(kw)
    return K.KdaLinDims(*[d[f] for f, _ in K.KdaLinDims._fields_])


def paged(K, **kw):
    d = dict(rows=3, heads=8, kv_heads=2, head_dim=128, pages=10, page_size=16, max_pages=4, dtype=1)
    d.update(kw)
    return K.KdaPagedDims(*[d[f] for f, _ in K.KdaPagedDims._fields_])


def chunk(K, d, q=FAKE, k=FAKE, v=FAKE, g=FAKE, head_g=FAKE, s0=None, cu=None, out=FAKE, sT=None, ws=FAKE, wb=1 << 40):
    return K.lib().kda_lin_chunk_fwd(q, k, v, g, head_g, s0, cu, out, sT, ws, wb, ctypes.byref(d) if d else None, None)


def step(K, d, q=FAKE, k=FAKE, v=FAKE, g=FAKE, head_g=FAKE, state=FAKE, idx=None, out=FAKE):
    return K.lib().kda_lin_recurrent_step(q, k, v, g, head_g, state, idx, out, ctypes.byref(d) if d else None, None)


def append(K, d, k=FAKE, v=FAKE, kc=FAKE, vc=FAKE, table=FAKE, pos=FAKE, cu=None, tokens=3):
    return K.lib().kda_paged_append(k, v, kc, vc, table, pos, cu, tokens, ctypes.byref(d) if d else None, None)


def attend(K, d, q=FAKE, kc=FAKE, vc=FAKE, table=FAKE, lens=FAKE, scale=0.1, out=FAKE, lse=FAKE, ws=FAKE, wb=1 << 40):
    return K.lib().kda_paged_attention(q, kc, vc, table, lens, scale, out, lse, ws, wb, ctypes.byref(d) if d else None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dk=96), 3), (dict(dv=32), 3), (dict(dtype=2), 3), (dict(heads=0), 2), (dict(qk_heads=0), 2),
    (dict(qk_heads=3), 2), (dict(qk_heads=8), 2), (dict(batch=0), 2), (dict(seqlen=-1), 2), (dict(num_seqs=3), 2), (dict(num_seqs=0), 2),
])
def test_chunk_dims(K, kw, code):
    assert chunk(K, lin(K, **kw)) == code


def test_chunk_pointers(K):
    assert chunk(K, None) == K.KDA_ERR_NULL
    for x in ("q", "k", "v", "out"):
        assert chunk(K, lin(K), **{x: None}) == K.KDA_ERR_NULL
        assert chunk(K, lin(K), **{x: FAKE + 8}) == K.KDA_ERR_ALIGN
    for x in ("s0", "sT"):
        assert chunk(K, lin(K), **{x: FAKE + 8}) == K.KDA_ERR_ALIGN
    for x in ("g", "head_g"):
        assert chunk(K, lin(K), **{x: FAKE + 2}) == K.KDA_ERR_ALIGN
    assert chunk(K, lin(K, batch=1, num_seqs=5), cu=FAKE + 2) == K.KDA_ERR_ALIGN
    assert chunk(K, lin(K), cu=FAKE) == K.KDA_ERR_SHAPE                     # packed needs batch == 1
    assert chunk(K, lin(K), s0=FAKE, sT=FAKE + 4096) == K.KDA_ERR_SHAPE     # partial overlap
    assert chunk(K, lin(K, seqlen=0), q=None, k=None, v=None, out=None) == K.KDA_OK


def test_chunk_workspace(K):
    d = lin(K, batch=1, num_seqs=1, seqlen=1 << 16, dv=128)
    slot = 128 * 128 * 4 + 8   # one slot of state and decay per head and part but the last; packed: lists of pieces too
    need = K.lib().kda_lin_chunk_fwd_workspace_bytes(ctypes.byref(d), 0)
    assert need > 0 and need % (4 * slot) == 0 and need <= 160 * slot
    assert 0 < K.lib().kda_lin_chunk_fwd_workspace_bytes(ctypes.byref(d), 1) <= 4 * 160 * (slot + 64) + 4 * 32 + 16
    assert K.lib().kda_lin_chunk_fwd_workspace_bytes(ctypes.byref(lin(K, dtype=0, batch=1, num_seqs=1, seqlen=1 << 16)), 1) == 0
    need = K.lib().kda_lin_chunk_fwd_workspace_bytes(ctypes.byref(d), 0)
    if need:
        assert chunk(K, d, ws=None) == K.KDA_ERR_NULL
        assert chunk(K, d, wb=need - 1) == K.KDA_ERR_WORKSPACE
        assert chunk(K, d, ws=FAKE + 8) == K.KDA_ERR_ALIGN
    assert K.lib().kda_lin_chunk_fwd_workspace_bytes(None, 0) == 0
    assert K.lib().kda_lin_chunk_fwd_workspace_bytes(ctypes.byref(lin(K, heads=0)), 1) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(dk=32), 3), (dict(dtype=9), 3), (dict(seqlen=2), 2), (dict(seqlen=0), 2), (dict(batch=-1), 2), (dict(batch=3), 2), (dict(qk_heads=3), 2),
])
def test_step_dims(K, kw, code):
    d = dict(seqlen=1)
    d.update(kw)
    assert step(K, lin(K, **d)) == code


def test_step_pointers(K):
    d = lin(K, seqlen=1)
    assert step(K, None) == K.KDA_ERR_NULL
    for x in ("q", "k", "v", "state", "out"):
        assert step(K, d, **{x: None}) == K.KDA_ERR_NULL
        assert step(K, d, **{x: FAKE + 4}) == K.KDA_ERR_ALIGN
    assert step(K, d, idx=FAKE + 1) == K.KDA_ERR_ALIGN
    assert step(K, lin(K, seqlen=1, batch=0), q=None) == K.KDA_OK


@pytest.mark.parametrize("kw,code", [
    (dict(head_dim=96), 3), (dict(dtype=2), 3), (dict(rows=-1), 2), (dict(kv_heads=0), 2), (dict(pages=0), 2), (dict(page_size=0), 2),
    (dict(max_pages=0), 2), (dict(page_size=1 << 20, max_pages=1 << 12), 2),
])
def test_paged_dims(K, kw, code):
    assert attend(K, paged(K, **kw)) == code
    assert append(K, paged(K, **kw)) == code


def test_attention_refusals(K):
    assert attend(K, None) == K.KDA_ERR_NULL
    assert attend(K, paged(K, heads=0)) == K.KDA_ERR_SHAPE
    assert attend(K, paged(K, heads=7)) == K.KDA_ERR_SHAPE
    for scale in (float("nan"), float("inf")):
        assert attend(K, paged(K), scale=scale) == K.KDA_ERR_SHAPE
    for x in ("q", "kc", "vc", "table", "lens", "out"):
        assert attend(K, paged(K), **{x: None}) == K.KDA_ERR_NULL
    for x in ("q", "kc", "vc", "out"):
        assert attend(K, paged(K), **{x: FAKE + 8}) == K.KDA_ERR_ALIGN
    for x in ("table", "lens", "lse"):
        assert attend(K, paged(K), **{x: FAKE + 2}) == K.KDA_ERR_ALIGN
    need = K.lib().kda_paged_attention_workspace_bytes(ctypes.byref(paged(K)))
    if need:
        assert attend(K, paged(K), ws=None) == K.KDA_ERR_NULL
        assert attend(K, paged(K), wb=need - 1) == K.KDA_ERR_WORKSPACE
        assert attend(K, paged(K), ws=FAKE + 4) == K.KDA_ERR_ALIGN
    assert attend(K, paged(K, rows=0), q=None) == K.KDA_OK
    assert K.lib().kda_paged_attention_workspace_bytes(None) == 0


def test_append_refusals(K):
    assert append(K, None) == K.KDA_ERR_NULL
    assert append(K, paged(K), tokens=-1) == K.KDA_ERR_SHAPE
    assert append(K, paged(K), tokens=4) == K.KDA_ERR_SHAPE        # no offsets: one token per row
    for x in ("k", "v", "kc", "vc", "table", "pos"):
        assert append(K, paged(K), **{x: None}) == K.KDA_ERR_NULL
    for x in ("k", "v", "kc", "vc"):
        assert append(K, paged(K), **{x: FAKE + 8}) == K.KDA_ERR_ALIGN
    for x in ("table", "pos", "cu"):
        assert append(K, paged(K), **{x: FAKE + 2}) == K.KDA_ERR_ALIGN
    assert append(K, paged(K), cu=FAKE, tokens=0, k=None) == K.KDA_OK
    assert append(K, paged(K, rows=0), tokens=0, k=None) == K.KDA_OK


def test_binding_refuses_host_tensors(K):
    x = torch.zeros(1, 4, 2, 64)
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        K.kda_lin_chunk_fwd(x, x, x)
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        K.kda_paged_append(x[0], x[0], x, x, torch.zeros(4, 1, dtype=torch.int32), torch.zeros(4, dtype=torch.int32))


def test_attention_workspace(K):
    """Tables wider than a cluster's rows take the shared-out form, which needs a workspace; narrow ones none."""
    d = paged(K, max_pages=1024)
    need = K.lib().kda_paged_attention_workspace_bytes(ctypes.byref(d))
    # 304 CTAs at most, two parts each, of 16 heads' 128 sums, a maximum and a sum
    assert 0 < need <= 304 * 2 * 16 * 130 * 4
    assert attend(K, d, ws=None) == K.KDA_ERR_NULL
    assert attend(K, d, wb=need - 1) == K.KDA_ERR_WORKSPACE
    assert attend(K, d, ws=FAKE + 4) == K.KDA_ERR_ALIGN
    assert K.lib().kda_paged_attention_workspace_bytes(ctypes.byref(paged(K))) == 0
    assert K.lib().kda_paged_attention_workspace_bytes(ctypes.byref(paged(K, max_pages=1024, rows=0))) == 0


def test_packed_chunk_workspace_is_checked(K):
    d = lin(K, batch=1, num_seqs=5, seqlen=1 << 14, dv=128)
    need = K.lib().kda_lin_chunk_fwd_workspace_bytes(ctypes.byref(d), 1)
    assert need > 0
    for s0, sT in ((None, None), (FAKE, FAKE)):           # in place too
        assert chunk(K, d, cu=FAKE, s0=s0, sT=sT, ws=None) == K.KDA_ERR_NULL
        assert chunk(K, d, cu=FAKE, s0=s0, sT=sT, wb=need - 1) == K.KDA_ERR_WORKSPACE
        assert chunk(K, d, cu=FAKE, s0=s0, sT=sT, ws=FAKE + 8) == K.KDA_ERR_ALIGN
