"""Branching decode as a server runs it: rows with a KDA layer and two layers of paged attention are verified a drafted tree
at a time, the accepted paths kept, rows forked on shared pages and ended, the pool closed up -- and every
accepted token's outputs are those of the same tokens decoded one by one."""
import random

import pytest
import torch

from tests import tree_reference as R

pytestmark = pytest.mark.gpu
I32 = torch.int32
H, HKV, D, PS, LAYERS = 4, 2, 128, 8, 2


@pytest.fixture(scope="module")
def K(cuda_device):
    from linear_attention_fwd_gb300 import build, kda
    build.build()
    return kda


def i32(x):
    return torch.tensor(x, dtype=I32, device="cuda")


class Inputs:
    """Every token's projected inputs, found again by its name (so that a token is the same wherever it is computed)."""

    def __init__(self, dt):
        self.dt = dt

    def __call__(self, name):
        gen = torch.Generator(device="cuda").manual_seed(name)
        rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
        unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
        kda = [unit(rnd(H, D)), unit(rnd(H, D)), rnd(H, D), -5 * torch.sigmoid(rnd(H, D) - 3), torch.sigmoid(rnd(H))]
        att = [[1.5 * rnd(H, D), rnd(HKV, D), rnd(HKV, D)] for _ in range(LAYERS)]
        return [x.to(self.dt) for x in kda], [[x.to(self.dt) for x in layer] for layer in att]


def stack(rows):
    return [torch.stack(x).contiguous() for x in zip(*rows)]


def one_by_one(K, inputs, names):
    """Outputs of the last token of `names`, decoded token by token: (KDA's, each attention layer's)."""
    state = torch.zeros(1, H, D, D, device="cuda")
    pages = -(-len(names) // PS)
    table = torch.arange(pages, dtype=I32, device="cuda")[None]
    caches = [[torch.zeros(pages, PS, HKV, D, dtype=inputs.dt, device="cuda") for _ in range(2)] for _ in range(LAYERS)]
    for t, name in enumerate(names):
        kda, att = inputs(name)
        o = K.kda_recurrent_step(*(x[None].contiguous() for x in kda), state)
        outs = [o[0]]
        for (q, k, v), (kc, vc) in zip(att, caches):
            K.kda_paged_append(k[None].contiguous(), v[None].contiguous(), kc, vc, table, i32([t]))
            outs.append(K.kda_paged_attention(q[None].contiguous(), kc, vc, table, i32([t + 1]), D ** -0.5)[0][0])
    return outs


@pytest.mark.parametrize("dt,tol", [(torch.float32, 2e-4), (torch.bfloat16, 3e-2)])
def test_branching_decode(K, dt, tol):
    # tol, relative to the outputs' largest value: bf16 outputs are off by 2^-8 each on both sides, KDA's by 2^-10 of sums of
    # absolute values some times as large on the drafted side; fp32 by (D + 1)(64 + 8 D) 2^-24 for paths of some 20 tokens
    rng = random.Random(1)
    inputs = Inputs(dt)
    N, W, T = 6, 12, 7
    pages = 60
    table, refs, lens = torch.full((N, W), -1, dtype=I32, device="cuda"), torch.zeros(pages, dtype=I32, device="cuda"), torch.zeros(N, dtype=I32, device="cuda")
    caches = [[torch.zeros(pages, PS, HKV, D, dtype=dt, device="cuda") for _ in range(2)] for _ in range(LAYERS)]
    state = torch.zeros(N, H, D, D, device="cuda")
    names = [[] for _ in range(N)]                     # the tokens of each row
    fresh = iter(range(1, 1 << 20))
    for turn in range(9):
        # rows continue, fork, end, and get room for the draft
        sources = [n if turn < 2 else rng.choice([n, n, n, rng.randrange(N), -1]) for n in range(N)]
        # (a row that ends is empty; what starts in it gets its room by a call of its own)
        for src, room in ((i32(sources), None), (i32(list(range(N))), i32([T] * N))):
            table, lens, refs, copies, short = K.kda_paged_fork(table, lens, refs, src, room, page_size=PS)
            assert short.tolist() == [0]
            for kc, vc in caches:
                K.kda_paged_copy(kc, vc, copies)
        state = torch.where((i32(sources) >= 0)[:, None, None, None], state[i32(sources).clamp_min(0).long()], 0.0).contiguous()
        names = [list(names[s]) if s >= 0 else [] for s in sources]
        if turn % 3 == 2:
            table, refs, copies = K.kda_paged_compact(table, refs)
            for kc, vc in caches:
                K.kda_paged_copy(kc, vc, copies)
        assert lens.tolist() == [len(x) for x in names]
        # a draft for each row
        num = [rng.randint(1, T) for _ in range(N)]
        trees = [R.tree(rng, m) for m in num]
        ids = [[next(fresh) for _ in range(m)] for m in num]
        full = [[inputs(ids[n][min(i, num[n] - 1)]) for i in range(T)] for n in range(N)]
        kda = [x.view(N, T, *x.shape[1:]) for x in stack([full[n][i][0] for n in range(N) for i in range(T)])]
        parents = i32([p + [0] * (T - len(p)) for p in trees])
        count = i32(num)
        outs = [K.kda_recurrent_tree(*kda, state, parents, num_tokens=count)]
        for layer, (kc, vc) in enumerate(caches):
            q, k, v = (x.view(N, T, *x.shape[1:]) for x in stack([full[n][i][1][layer] for n in range(N) for i in range(T)]))
            cu = torch.tensor([0] + num, device="cuda").cumsum(0).to(I32)
            flat = lambda x: torch.cat([x[n, : num[n]] for n in range(N)]).contiguous()  # noqa: E731
            K.kda_paged_append(flat(k), flat(v), kc, vc, table, lens, cu)
            outs.append(K.kda_paged_tree_attention(q, kc, vc, table, lens, parents, D ** -0.5, count)[0])
        accepted = [rng.choice([-1] + list(range(m))) for m in num]
        for n in range(N):
            for i in {accepted[n], rng.randrange(num[n])} - {-1}:
                want = one_by_one(K, inputs, names[n] + [ids[n][j] for j in R.path(trees[n], i)])
                for got, ref in zip(outs, want):
                    err = (got[n, i].float() - ref.float()).abs().max() / ref.float().abs().max()
                    assert float(err) <= tol, (turn, n, i, float(err))
        # the accepted paths are kept
        K.kda_recurrent_tree_commit(*kda[1:], state, parents, i32(accepted), num_tokens=count)
        new = [K.kda_paged_tree_commit(kc, vc, table, lens, parents, i32(accepted), count) for kc, vc in caches]
        assert torch.equal(new[0], new[1])
        lens = new[0]
        for n in range(N):
            names[n] += [ids[n][j] for j in R.path(trees[n], accepted[n])]
        # the counts say what the table says
        flat = table[table >= 0].long()
        assert torch.equal(torch.bincount(flat, minlength=pages), refs.long())
