"""How exact the KDA calls for a drafted tree are, as root mean squares over a call's outputs against the recurrence in 64 bits and
relative to the outputs' own (bounds on sums of absolute values, as in tests/tree_reference.py, say little where those sums
grow along a path: with hardly any decay, a line of 40 tokens has ones a hundred times its outputs).

Bounds.  Keys of unit length and beta <= 1 make every token's step (I - beta k k^T) Diag(e^g) a map that lengthens nothing, so that errors
add along a path of D tokens and do not compound.
 - fp32: an output is a product with the state, and one with W for each token on the path.  A sum on the tensor cores is over parts of at
   most 16 channels, in which at most three sums of products' leading parts are truncated (2^-24 each on average, all towards zero:
   3 * 2^-24), and rounded additions of those; parts of 11 bits leave 2^-23 of a product, signs at random.  Less than 2^-22 for each
   of D + 1 sums together.
 - bf16: the output is off by at most 2^-8, the operands of the products with the state by 2^-11 each, signs at random: 2^-8 + 2^-10.
 - A state: per token the decay (2^-23), one more sum of fp32 and four roundings: 2^-22 for each of D tokens.
"""
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


def make(seed, N, T, H, dk, dv, dt, lowest):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    return dict(q=unit(rnd(N, T, H, dk)).to(dt), k=unit(rnd(N, T, H, dk)).to(dt), v=rnd(N, T, H, dv).to(dt),
                g=(lowest * torch.sigmoid(2 * rnd(N, T, H, dk) - 2)).to(dt), beta=torch.sigmoid(rnd(N, T, H)).to(dt),
                state=0.3 * rnd(N, H, dk, dv))


def rms(x):
    return float(x.square().mean().sqrt())


def relative(got, ref):
    return rms(got.detach().cpu().double() - ref) / rms(ref)


def outputs(K, c, rows, parents):
    _, ref, _ = R.recurrent(**c, rows=rows)
    return relative(K.kda_recurrent_tree(**c, parents=parents), ref)


@pytest.mark.parametrize("T,kind", [(1, "star"), (3, "star"), (8, "star"), (16, "star"), (40, "star"), (64, "star"), (2, "chain"), (5, "chain"),
                                    (12, "tree"), (33, "tree"), (64, "tree")])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 128), (128, 64), (64, 64)])
def test_fp32(K, T, kind, dk, dv):
    c = make(T, 3, T, 4, dk, dv, F32, -5.0)
    rows, parents = R.drafts(T, 3, T, kind)
    assert outputs(K, c, rows, parents) <= (R.depth(rows) + 1) * 2.0 ** -22


@pytest.mark.parametrize("T", [20, 40, 64])
@pytest.mark.parametrize("dt,least", [(F32, -1e-4), (BF16, -1e-4), (F32, -1.0), (BF16, -1.0)])
def test_lines_that_hardly_decay(K, T, dt, least):
    c = make(T, 2, T, 3, 128, 128, dt, least)
    rows, _ = R.drafts(T, 2, T, "chain")
    assert outputs(K, c, rows, None) <= (2.0 ** -8 + 2.0 ** -10 if dt == BF16 else (T + 1) * 2.0 ** -22)
    a = {x: c[x] for x in ("k", "v", "g", "beta")}
    kept, _, _ = R.recurrent(q=None, **a, state=c["state"], rows=rows)
    K.kda_recurrent_tree_commit(**a, state=c["state"], parents=None, accepted=torch.tensor([T - 1, T // 2], dtype=torch.int32, device="cuda"))
    for n, last in enumerate((T - 1, T // 2)):
        assert relative(c["state"][n], kept[n][last][0]) <= (last + 1) * 2.0 ** -22
