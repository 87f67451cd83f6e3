"""KDA for a tree of drafted tokens on the GPU: outputs and committed states against the recurrence in fp64
(tests/tree_reference.py says where the bounds come from), against the calls for one token and for a line
of tokens, and what a call must leave alone."""
import random

import pytest
import torch

from tests import tree_reference as R

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def K(cuda_device):
    from linear_attention_fwd_gb300 import build, kda
    build.build()
    return kda


def make(seed, N, T, H, dk, dv, dt, slots=None, unit=True, lowest=-5.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    norm = (lambda x: x / x.norm(dim=-1, keepdim=True)) if unit else (lambda x: x)
    return dict(q=norm(rnd(N, T, H, dk)).to(dt), k=norm(rnd(N, T, H, dk)).to(dt), v=rnd(N, T, H, dv).to(dt),
                g=(lowest * torch.sigmoid(2 * rnd(N, T, H, dk) - 2)).to(dt), beta=torch.sigmoid(rnd(N, T, H)).to(dt),
                state=0.3 * rnd(slots or N, H, dk, dv))


def verify(K, c, rows, parents, idx=None, num=None, eps=None, **kw):
    before = c["state"].clone()
    out = K.kda_recurrent_tree(**c, parents=parents, state_indices=idx, num_tokens=num, qk_eps=eps, **kw)
    assert torch.equal(c["state"], before)
    _, ref, oabs = R.recurrent(**c, rows=rows, idx=idx, eps=eps)
    R.check_outputs(out, ref, oabs, rows, eps)
    for n, p in enumerate(rows):
        assert not out[n, len(p):].any()
        if idx is not None and not 0 <= int(idx[n]) < c["state"].shape[0]:
            assert not out[n].any()
    return out


def commit(K, c, rows, parents, accepted, idx=None, num=None, eps=None):
    a = {x: c[x] for x in ("k", "v", "g", "beta")}
    kept, _, _ = R.recurrent(q=None, **a, state=c["state"], rows=rows, idx=idx, eps=eps)
    before = c["state"].clone()
    K.kda_recurrent_tree_commit(**a, state=c["state"], parents=parents, accepted=torch.tensor(accepted, dtype=torch.int32, device="cuda"),
                                state_indices=idx, num_tokens=num, qk_eps=eps)
    named = set()
    for n, p in enumerate(rows):
        slot = n if idx is None else int(idx[n])
        if kept[n] is None or not 0 <= accepted[n] < len(p):
            continue
        named.add(slot)
        S, A = kept[n][accepted[n]]
        R.check_state(c["state"][slot], S, A, len(R.path(p, accepted[n])), S.shape[1], eps)
    for slot in set(range(before.shape[0])) - named:
        assert torch.equal(c["state"][slot], before[slot])


@pytest.mark.parametrize("T", [1, 2, 3, 7, 8, 9, 16, 17, 31, 32, 33, 63, 64])
@pytest.mark.parametrize("dt,dk,dv", [(F32, 64, 128), (BF16, 128, 128), (F32, 128, 64), (BF16, 64, 64)])
def test_widths(K, T, dt, dk, dv):
    c = make(T, 2, T, 3, dk, dv, dt)
    rows, parents = R.drafts(T, 2, T)
    verify(K, c, rows, parents)
    commit(K, c, rows, parents, [T - 1, T // 2])


@pytest.mark.parametrize("kind", ["chain", "star", "tree"])
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
def test_shapes_of_trees(K, kind, dt, dk, dv):
    c = make(5, 3, 21, 2, dk, dv, dt)
    rows, parents = R.drafts(5, 3, 21, kind)
    verify(K, c, rows, parents)
    commit(K, c, rows, parents, [20, 0, 11])


@pytest.mark.parametrize("dt", [F32, BF16])
def test_ragged_counts_and_slots(K, dt):
    """Counts outside [0, T], slots outside the pool, rows that accept nothing or past their count."""
    num = [5, 0, 12, 40, -3, 1, 7]
    idx = torch.tensor([3, 1, -1, 0, 2, 9, 6], dtype=torch.int32, device="cuda")
    c = make(6, 7, 12, 2, 128, 128, dt, slots=9)
    rows, parents = R.drafts(6, 7, 12, num=num)
    nt = torch.tensor(num, dtype=torch.int32, device="cuda")
    c["g"][0, 5:] = float("nan")     # behind row 0's count
    c["q"][5], c["v"][1] = float("inf"), float("nan")
    verify(K, {**c, "q": c["q"].clone()}, [r if n not in (1, 5) else [] for n, r in enumerate(rows)], parents, idx, nt)
    commit(K, c, rows, parents, [4, 0, 3, 11, 0, 0, 7], idx, nt)


def test_a_line_is_what_steps_compute(K):
    c = make(7, 2, 9, 2, 128, 128, F32)
    rows, _ = R.drafts(7, 2, 9, "chain")
    out = verify(K, c, rows, None)
    steps = K.kda_recurrent_steps(**c, update_state=False)
    assert float((out - steps).abs().max()) <= 1e-5
    commit(K, c, rows, None, [8, 3])


def test_parents_out_of_range_start_anew(K):
    """A parent that is no earlier token counts as -1."""
    c = make(8, 1, 6, 2, 64, 64, F32)
    bad = torch.tensor([[0, 0, 9, 1, -5, 5]], dtype=torch.int32, device="cuda")
    verify(K, c, [[-1, 0, -1, 1, -1, -1]], bad)
    commit(K, c, [[-1, 0, -1, 1, -1, -1]], bad, [3])


@pytest.mark.parametrize("dt", [F32, BF16])
def test_qknorm(K, dt):
    c = make(9, 2, 13, 2, 128, 128, dt, unit=False)
    c["k"][0, 2] = 0
    c["q"][1, 3] = 0
    rows, parents = R.drafts(9, 2, 13)
    verify(K, c, rows, parents, eps=1e-6)
    commit(K, c, rows, parents, [12, 6], eps=1e-6)
    verify(K, c, rows, parents, eps=0.0)


@pytest.mark.parametrize("lowest", [-1e-4, -40.0, -1e4])
def test_decays_of_any_size(K, lowest):
    c = make(10, 2, 40, 2, 128, 128, F32, lowest=lowest)
    c["g"][0, 3, :, ::2] = -float("inf")
    rows, parents = R.drafts(10, 2, 40, "chain")
    verify(K, c, rows, parents)
    commit(K, c, rows, parents, [39, 39])


@pytest.mark.parametrize("dt", [F32, BF16])
def test_nan_stays_on_its_branch(K, dt):
    c = make(11, 1, 5, 2, 128, 64, dt)
    rows = [[-1, 0, 0, 1, 2]]
    parents = torch.tensor(rows, dtype=torch.int32, device="cuda")
    clean = K.kda_recurrent_tree(**c, parents=parents)
    for x in ("q", "k", "v", "g", "beta"):
        d = {y: t.clone() for y, t in c.items()}
        d[x][0, 1] = float("nan")
        out = K.kda_recurrent_tree(**d, parents=parents)
        for i in (0, 2, 4):
            assert torch.equal(out[0, i], clean[0, i]), (x, i)
        assert bool(out[0, 1].isnan().all())


@pytest.mark.parametrize("T", [8, 14, 29, 47, 64])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_what_is_not_finite_stays_on_its_branch(K, T, dt):
    """NaN and infinities in a middle token of a tree of any number of tiles."""
    c = make(23, 2, T, 2, 128, 128, dt)
    rows, parents = R.drafts(23, 2, T)
    at = T // 3
    below = [{i for i in range(T) if at in R.path(p, i)} for p in rows]
    clean = K.kda_recurrent_tree(**c, parents=parents)
    for x, value in (("q", "nan"), ("k", "nan"), ("v", "nan"), ("v", "inf"), ("v", "-inf"), ("beta", "nan")):
        d = {y: t.clone() for y, t in c.items()}
        d[x][:, at] = float(value)
        out = K.kda_recurrent_tree(**d, parents=parents)
        for n in range(2):
            for i in range(T):
                if i not in (below[n] if x != "q" else {at}):
                    assert torch.equal(out[n, i], clean[n, i]), (x, n, i)
                else:
                    assert not out[n, i].isfinite().any(), (x, n, i)


def test_magnitudes(K):
    for scale in (2.0 ** -60, 2.0 ** 60):
        c = make(12, 1, 10, 2, 128, 128, BF16)
        c["state"] *= scale
        c["v"] = (c["v"].float() * scale).to(BF16)
        rows, parents = R.drafts(12, 1, 10)
        verify(K, c, rows, parents)
        commit(K, c, rows, parents, [9])


@pytest.mark.parametrize("dt", [F32, BF16])
def test_other_stream_and_repeated(K, dt):
    c = make(13, 4, 17, 4, 128, 128, dt)
    rows, parents = R.drafts(13, 4, 17)
    first = verify(K, c, rows, parents)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = K.kda_recurrent_tree(**c, parents=parents, stream=side)
    side.synchronize()
    assert torch.equal(out, first)


def test_captured(K):
    """Verify and commit in one graph, replayed on new inputs."""
    c = make(14, 3, 9, 2, 128, 128, BF16)
    rows, parents = R.drafts(14, 3, 9)
    accepted = torch.tensor([8, -1, 4], dtype=torch.int32, device="cuda")
    out = torch.empty_like(c["v"])
    a = {x: c[x] for x in ("k", "v", "g", "beta")}

    def both():
        K.kda_recurrent_tree(**c, parents=parents, out=out)
        K.kda_recurrent_tree_commit(**a, state=c["state"], parents=parents, accepted=accepted)
    both()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for seed in (15, 16):
        d = make(seed, 3, 9, 2, 128, 128, BF16)
        for x in c:
            c[x].copy_(d[x])
        kept, ref, oabs = R.recurrent(**c, rows=rows)
        graph.replay()
        torch.cuda.synchronize()
        R.check_outputs(out, ref, oabs, rows)
        for n, i in ((0, 8), (2, 4)):
            S, A = kept[n][i]
            R.check_state(c["state"][n], S, A, 9, 128)
        assert torch.equal(c["state"][1], d["state"][1])
    assert random.Random(0)
