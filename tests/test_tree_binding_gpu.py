"""What the binding of the calls for branching decode refuses, and that a refused call leaves everything as it was; other
devices' streams, captured and eager calls beside one another."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF16, I32 = torch.bfloat16, torch.int32


@pytest.fixture(scope="module")
def K(cuda_device):
    from linear_attention_fwd_gb300 import build, kda
    build.build()
    return kda


def z(*s, dt=BF16):
    return torch.zeros(*s, dtype=dt, device="cuda")


def calls(K):
    tree = dict(k=z(2, 5, 3, 64), v=z(2, 5, 3, 128), g=z(2, 5, 3, 64), beta=z(2, 5, 3), state=z(4, 3, 64, 128, dt=torch.float32),
                parents=z(2, 5, dt=I32), state_indices=z(2, dt=I32), num_tokens=z(2, dt=I32))
    cache = dict(k_cache=z(9, 4, 2, 64), v_cache=z(9, 4, 2, 64), block_table=z(2, 6, dt=I32), seq_lens=z(2, dt=I32), parents=z(2, 5, dt=I32))
    pool = dict(block_table=z(2, 6, dt=I32), page_refs=z(9, dt=I32))
    return {
        "kda_recurrent_tree": dict(q=z(2, 5, 3, 64), **tree, out=z(2, 5, 3, 128)),
        "kda_recurrent_tree_commit": dict(**tree, accepted=z(2, dt=I32)),
        "kda_paged_tree_attention": dict(q=z(2, 5, 4, 64), **cache, scale=1.0, num_tokens=z(2, dt=I32), out=z(2, 5, 4, 64), lse=z(2, 5, 4, dt=torch.float32)),
        "kda_paged_tree_commit": dict(**cache, accepted=z(2, dt=I32), num_tokens=z(2, dt=I32), new_lens=z(2, dt=I32)),
        "kda_paged_fork": dict(**pool, seq_lens=z(2, dt=I32), sources=z(2, dt=I32), new_tokens=z(2, dt=I32), page_size=4, new_table=z(2, 6, dt=I32),
                               new_lens=z(2, dt=I32), new_refs=z(9, dt=I32), copies=z(2, 2, dt=I32), short_of=z(1, dt=I32)),
        "kda_paged_compact": dict(**pool, new_table=z(2, 6, dt=I32), new_refs=z(9, dt=I32), copies=z(4, 2, dt=I32)),
        "kda_paged_copy": dict(k_cache=z(9, 4, 2, 64), v_cache=z(9, 4, 2, 64), copies=z(3, 2, dt=I32)),
    }


NAMES = ["kda_recurrent_tree", "kda_recurrent_tree_commit", "kda_paged_tree_attention", "kda_paged_tree_commit", "kda_paged_fork",
         "kda_paged_compact", "kda_paged_copy"]


@pytest.mark.parametrize("name", NAMES)
def test_every_tensor_is_checked(K, name):
    """Another type, another shape, another device, not contiguous, not a tensor: refused, and nothing has changed."""
    good = calls(K)[name]
    tensors = [x for x, t in good.items() if isinstance(t, torch.Tensor)]
    for x in tensors:
        t = good[x]
        wrong = [t.to(torch.int16 if t.dtype == I32 else torch.float16), t.cpu(), t[None], torch.cat([t, t])[: t.shape[0] + 1], 3]
        if t.dim() > 1:
            wrong.append(torch.stack([t, t], -1)[..., 0])
        for w in wrong:
            bad = {y: u.clone() if isinstance(u, torch.Tensor) else u for y, u in good.items()}
            bad[x] = w
            # (a longer first dimension may be what the call's other tensors are measured by: some other one is then refused)
            before = {y: u.clone() for y, u in bad.items() if isinstance(u, torch.Tensor)}
            try:
                getattr(K, name)(**bad)
            except (TypeError, ValueError, K.KdaError):
                torch.cuda.synchronize()
                for y, u in before.items():
                    assert torch.equal(u, bad[y]), (x, y)
            else:
                assert isinstance(w, torch.Tensor) and w.dim() == t.dim() and w.dtype == t.dtype and w.is_cuda and x in (
                    "state", "k_cache", "v_cache", "page_refs", "copies"), (x, w if w is None else getattr(w, "shape", w))


def test_values_are_checked(K):
    c = calls(K)
    for x, bad in (("kda_paged_tree_attention", dict(scale=float("nan"))), ("kda_paged_tree_attention", dict(scale="x")),
                   ("kda_paged_fork", dict(page_size=0)), ("kda_paged_fork", dict(page_size=-4)), ("kda_recurrent_tree", dict(qk_eps=-1.0)),
                   ("kda_recurrent_tree", dict(qk_eps="x")), ("kda_recurrent_tree_commit", dict(qk_eps=float("nan"))),
                   ("kda_paged_tree_commit", dict(parents=None, tokens=0)), ("kda_paged_tree_commit", dict(parents=None, tokens=65))):
        with pytest.raises((TypeError, ValueError, K.KdaError)):
            getattr(K, x)(**{**c[x], **bad})
    for x in ("kda_paged_fork", "kda_paged_compact"):     # an output that is an input
        with pytest.raises(K.KdaError):
            getattr(K, x)(**{**c[x], "new_table": c[x]["block_table"]})
    big = {**c["kda_recurrent_tree"], "parents": None, "num_tokens": None}
    for x in ("q", "k", "v", "g", "beta", "out"):
        big[x] = z(2, 65, *big[x].shape[2:])
    with pytest.raises(K.KdaError):
        K.kda_recurrent_tree(**big)


def test_nothing_to_do(K):
    """No rows, no copies."""
    q = z(0, 5, 4, 64)
    cache = z(9, 4, 2, 64)
    out, lse = K.kda_paged_tree_attention(q, cache, cache, z(0, 6, dt=I32), z(0, dt=I32), None, 1.0)
    assert out.shape == q.shape and lse.shape == (0, 5, 4)
    assert K.kda_paged_tree_commit(cache, cache, z(0, 6, dt=I32), z(0, dt=I32), None, z(0, dt=I32)).shape == (0,)
    K.kda_paged_copy(cache, cache, z(0, 2, dt=I32))
    table, refs, copies = K.kda_paged_compact(z(0, 6, dt=I32), z(9, dt=I32))
    assert table.shape == (0, 6) and not refs.any() and bool((copies == -1).all())


def test_outputs_are_the_callers(K):
    c = calls(K)
    a = c["kda_paged_fork"]
    got = K.kda_paged_fork(**a)
    assert all(x is a[y] for x, y in zip(got, ("new_table", "new_lens", "new_refs", "copies", "short_of")))
    a = c["kda_paged_tree_attention"]
    assert all(x is a[y] for x, y in zip(K.kda_paged_tree_attention(**a), ("out", "lse")))
    a = c["kda_recurrent_tree"]
    assert K.kda_recurrent_tree(**a) is a["out"]
