"""Calls for branching decode at the edges of what they take: scales of any sign, states with a value that is not finite, states and
values of any magnitude."""
import pytest
import torch

from tests import tree_reference as R
from tests.test_tree_gpu import make, verify, commit
from tests.test_tree_paged_gpu import cache, run

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def K(cuda_device):
    from linear_attention_fwd_gb300 import build, kda
    build.build()
    return kda


@pytest.mark.parametrize("scale", [-0.3, -1e-3, 0.0, -0.0, 1e-30, 3.0])
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("lens,T,Hq,Hkv,ps", [([700, 3, 0, 130], 21, 8, 2, 16), ([200, 65], 9, 5, 1, 7), ([300], 64, 16, 1, 64)])
def test_scales(K, scale, dt, lens, T, Hq, Hkv, ps):
    c = cache(31, lens, T, Hq, Hkv, 128, ps, dt)
    c["scale"] = scale
    num = [T, max(1, T // 3), T, 1][: len(lens)]
    rows, parents = R.drafts(31, len(lens), T, num=num)
    c["block_table"][0, 1] = -1          # a tile with places that have no token
    run(K, c, rows, parents, torch.tensor(num, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("T", [5, 30, 64])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_what_is_not_finite_in_a_state_stays_in_its_channel(K, dt, T, bad):
    """Value channels of a state do not meet."""
    c = make(33, 2, T, 2, 128, 128, dt)
    rows, parents = R.drafts(33, 2, T)
    a = {x: c[x] for x in ("k", "v", "g", "beta")}
    clean = K.kda_recurrent_tree(**c, parents=parents)
    last = torch.tensor([T - 1, T // 2], dtype=torch.int32, device="cuda")
    after, dirty = c["state"].clone(), c["state"].clone()
    dirty[0, 1, 17, 42] = bad
    out = K.kda_recurrent_tree(c["q"], **a, state=dirty, parents=parents)
    K.kda_recurrent_tree_commit(**a, state=after, parents=parents, accepted=last)
    K.kda_recurrent_tree_commit(**a, state=dirty, parents=parents, accepted=last)
    assert not out[0, :, 1, 42].isfinite().any()
    out[0, :, 1, 42] = clean[0, :, 1, 42]
    assert torch.equal(out, clean)
    assert not dirty[0, 1, :, 42].isfinite().any()
    dirty[0, 1, :, 42] = after[0, 1, :, 42]
    assert torch.equal(dirty, after)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("power", [-90, -60, 60, 100, 120])
def test_magnitudes_of_states_and_values(K, dt, power):
    scale = 2.0 ** power
    for T, kind in ((3, "chain"), (10, "tree"), (40, "tree")):
        c = make(35, 1, T, 2, 128, 128, dt)
        c["state"] *= scale
        c["v"] = (c["v"].float() * scale).to(dt)
        rows, parents = R.drafts(35, 1, T, kind)
        out = verify(K, c, rows, parents)
        assert bool(out.isfinite().all())
        commit(K, c, rows, parents, [T - 1])
