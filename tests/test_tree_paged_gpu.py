"""Attention of a draft's tokens over a paged cache, and the accepted path moved together, on the GPU, against their
definitions in fp64 (tests/tree_reference.py)."""
import math

import pytest
import torch

from tests import tree_reference as R
from tests.lin_reference import check_paged

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def K(cuda_device):
    from linear_attention_fwd_gb300 import build, kda
    build.build()
    return kda


def cache(seed, lens, T, Hq, Hkv, d, ps, dt, spare=2, extra=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    N = len(lens)
    width = -(-(max(lens) + T) // ps) + extra
    pages = N * width + spare
    table = torch.randperm(pages, generator=gen, device="cuda")[: N * width].view(N, width).to(torch.int32)
    return dict(q=(2 * rnd(N, T, Hq, d)).to(dt), k_cache=rnd(pages, ps, Hkv, d).to(dt), v_cache=rnd(pages, ps, Hkv, d).to(dt),
                block_table=table, seq_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), scale=d ** -0.5)


def reference(c, rows):
    return R.attention(c["q"], c["k_cache"], c["v_cache"], c["block_table"], c["seq_lens"], rows, c["scale"])


def widened(c):
    """The same call under a table for 9000 tokens more: rows that may be long take the shared-out form, with a workspace."""
    table = c["block_table"]
    return {**c, "block_table": torch.cat([table, torch.full((table.shape[0], -(-9000 // c["k_cache"].shape[1])), -1, dtype=torch.int32, device="cuda")], 1)}


def forms(c):
    return [c, widened(c)] if c["q"].dtype == BF16 else [c]


def run(K, c, rows, parents, num=None, **kw):
    ref = reference(c, rows)
    for form in reversed(forms(c)):
        out, lse = K.kda_paged_tree_attention(**form, parents=parents, num_tokens=num, **kw)
        check_paged(out, lse, ref)
        for n, p in enumerate(rows):
            assert not out[n, len(p):].any() and bool((lse[n, len(p):] == -math.inf).all())
    return out, lse


@pytest.mark.parametrize("length", [0, 1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 700])
@pytest.mark.parametrize("dt,d", [(F32, 64), (F32, 128), (BF16, 64), (BF16, 128)])
def test_lengths(K, length, dt, d):
    c = cache(length, [length, length // 3], 6, 4, 2, d, 16, dt)
    run(K, c, *R.drafts(length, 2, 6))


@pytest.mark.parametrize("T", [1, 2, 5, 16, 31, 32, 33, 63, 64])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_widths(K, T, dt):
    c = cache(T, [70, 0], T, 8, 2, 128, 16, dt)
    run(K, c, *R.drafts(T, 2, T))


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 1), (3, 3), (5, 1), (12, 4), (16, 1), (17, 1), (24, 2)])
@pytest.mark.parametrize("T", [3, 40])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_head_layouts(K, Hq, Hkv, T, dt):
    c = cache(3, [150, 33], T, Hq, Hkv, 64 if T > 8 else 128, 32, dt)
    run(K, c, *R.drafts(3, 2, T))


@pytest.mark.parametrize("ps", [1, 2, 7, 13, 64, 100, 128, 1000])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_page_sizes(K, ps, dt):
    c = cache(4, [200, 64, 1, 129], 9, 4, 2, 64, ps, dt)
    run(K, c, *R.drafts(4, 4, 9))


@pytest.mark.parametrize("kind", ["chain", "star"])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_lines_and_stars(K, kind, dt):
    c = cache(5, [130, 0, 31], 40, 2, 1, 128, 16, dt)
    rows, parents = R.drafts(5, 3, 40, kind)
    out, lse = run(K, c, rows, parents)
    if kind == "chain":
        again, _ = K.kda_paged_tree_attention(**c, parents=None)
        assert torch.equal(again, out)


@pytest.mark.parametrize("dt", [F32, BF16])
def test_one_token_is_what_the_row_attention_computes(K, dt):
    c = cache(6, [500, 3, 64], 1, 8, 2, 128, 16, dt)
    out, lse = run(K, c, [[-1]] * 3, None)
    one, lse1 = K.kda_paged_attention(c["q"][:, 0].contiguous(), c["k_cache"], c["v_cache"], c["block_table"], c["seq_lens"] + 1, c["scale"])
    assert float((lse[:, 0] - lse1).abs().max()) <= 1e-4
    assert float((out[:, 0].float() - one.float()).abs().max()) <= (1e-5 if dt == F32 else 2.0 ** -6)


@pytest.mark.parametrize("dt", [F32, BF16])
def test_ragged_counts(K, dt):
    num = [5, 0, 12, 40, -3, 1, 12, 7]
    c = cache(7, [40, 100, 0, 300, 7, 1000, 64, 0], 12, 4, 2, 128, 16, dt)
    rows, parents = R.drafts(7, 8, 12, num=num)
    run(K, c, rows, parents, torch.tensor(num, dtype=torch.int32, device="cuda"))
    out, lse = K.kda_paged_tree_attention(**c, parents=parents, num_tokens=torch.zeros(8, dtype=torch.int32, device="cuda"))
    assert not out.any() and bool((lse == -math.inf).all())


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("lens,T", [([9000], 10), ([5000, 3, 0, 2500], 64)])
def test_long_rows_are_split(K, dt, lens, T):
    c = cache(8, lens, T, 8, 2, 128, 64, dt)
    c["q"] *= 2
    run(K, c, *R.drafts(8, len(lens), T))


@pytest.mark.parametrize("dt", [F32, BF16])
def test_many_rows(K, dt):
    lens = [(i * i * 7919) % 400 for i in range(60)]
    num = [(i * 31) % 9 for i in range(60)]
    c = cache(9, lens, 8, 4, 4, 64, 16, dt)
    rows, parents = R.drafts(9, 60, 8, num=num)
    run(K, c, rows, parents, torch.tensor(num, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("dt", [F32, BF16])
def test_more_rows_than_a_cta_has_threads(K, dt):
    lens = [(i * i * 7919) % 40 for i in range(700)]
    num = [(i * 31) % 4 for i in range(700)]
    c = cache(23, lens, 3, 2, 1, 64, 16, dt)
    rows, parents = R.drafts(23, 700, 3, num=num)
    run(K, c, rows, parents, torch.tensor(num, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("dt", [F32, BF16])
def test_many_tiles(K, dt):
    """More than 2^20 tiles: rows that share all their pages give what one of them gives alone.  Both sides round values that agree
    to 2^-14 of sum p |v| <= max |v| (weights of 16 bits, parts joined in another order) to the type."""
    tile = 64 if dt == BF16 else 32
    N, width = 2048, 512 * tile // 64
    c = cache(24, [64 * width - 7], 1, 1, 1, 64, 64, dt)
    rows = torch.tensor([[-1]], dtype=torch.int32, device="cuda")
    args = lambda n: (c["q"].expand(n, 1, 1, 64).contiguous(), c["k_cache"], c["v_cache"],  # noqa: E731
                      c["block_table"].expand(n, -1).contiguous(), c["seq_lens"].expand(n).contiguous(), rows.expand(n, 1).contiguous(), c["scale"])
    one, lse1 = K.kda_paged_tree_attention(*args(1))
    assert N * (c["seq_lens"].item() // tile + 1) >= 1 << 20
    out, lse = K.kda_paged_tree_attention(*args(N))
    step = torch.finfo(dt).eps * one.float().abs()
    assert bool(((out.float() - one.float()).abs() <= step + 2 ** -14 * c["v_cache"].abs().max().float()).all())
    assert bool(((lse - lse1).abs() <= 1e-4).all())


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_places_that_a_token_does_not_see(K, dt, bad):
    """Other branches, tokens past the count, and whatever lies behind: nothing of them reaches a token's results."""
    c = cache(10, [77, 0], 9, 4, 2, 128, 16, dt, extra=3)
    rows = [[-1, 0, 0, 1, 2, -1], [-1, 0, -1, 2, 0, 1, 3]]
    parents = torch.full((2, 9), -1, dtype=torch.int32, device="cuda")
    for n, p in enumerate(rows):
        parents[n, : len(p)] = torch.tensor(p, dtype=torch.int32)
    num = torch.tensor([6, 7], dtype=torch.int32, device="cuda")
    run(K, c, rows, parents, num)
    for n, sick, c in [(n, sick, form) for form in forms(c) for n, sick in ((0, 2), (1, 0))]:
        out, lse = K.kda_paged_tree_attention(**c, parents=parents, num_tokens=num)
        d = {x: t.clone() if isinstance(t, torch.Tensor) else t for x, t in c.items()}
        at = lambda pos: (int(c["block_table"][n, pos // 16]), pos % 16)  # noqa: E731
        length = int(c["seq_lens"][n])
        behind = [pos for pos in range(length + len(rows[n]), c["block_table"].shape[1] * 16) if int(c["block_table"][n, pos // 16]) >= 0]
        for pos in [length + sick] + behind:
            d["k_cache"][at(pos)] = bad
            d["v_cache"][at(pos)] = bad
        got, got_lse = K.kda_paged_tree_attention(**d, parents=parents, num_tokens=num)
        for i, p in enumerate(rows[n]):
            if sick not in R.path(rows[n], i):
                assert torch.equal(got[n, i], out[n, i]) and torch.equal(got_lse[n, i], lse[n, i]), i
            elif math.isnan(bad):
                assert bool(got[n, i].isnan().all()), i
        assert torch.equal(got[1 - n], out[1 - n])


@pytest.mark.parametrize("dt", [F32, BF16])
def test_pages_outside_the_pool_are_left_out(K, dt):
    c = cache(11, [100, 40, 20], 5, 4, 2, 128, 16, dt)
    c["block_table"][0, 2] = -1
    c["block_table"][0, 5] = c["k_cache"].shape[0]
    c["block_table"][1, :] = 1 << 30          # nothing left
    c["block_table"][2, 1] = -7               # the draft's own page
    rows, parents = R.drafts(11, 3, 5)
    out, lse = run(K, c, rows, parents)
    assert not out[1].any() and bool((lse[1] == -math.inf).all())


@pytest.mark.parametrize("dt", [F32, BF16])
def test_lengths_past_the_table(K, dt):
    """A length past the table is cut to it, and the drafted tokens then lie past it."""
    c = cache(12, [50, 40, 20], 7, 4, 2, 64, 16, dt)
    width = c["block_table"].shape[1] * 16
    c["seq_lens"].copy_(torch.tensor([1 << 30, width - 3, -5]))
    rows, parents = R.drafts(12, 3, 7)
    check_paged(*K.kda_paged_tree_attention(**c, parents=parents), reference(c, rows))
    if dt == BF16:
        c = widened(c)     # (the lengths then end elsewhere)
        check_paged(*K.kda_paged_tree_attention(**c, parents=parents), reference(c, rows))


@pytest.mark.parametrize("dt", [F32, BF16])
def test_scores_of_minus_infinity(K, dt):
    """K of infinities against positive queries: such tokens weigh nothing; a token of nothing else is empty."""
    c = cache(13, [30, 0], 3, 2, 1, 64, 8, dt)
    c["q"] = c["q"].abs() + 0.1
    c["k_cache"][c["block_table"][0, 1].long()] = -float("inf")
    c["k_cache"][c["block_table"][1, 0].long(), 1] = -float("inf")
    out, lse = run(K, c, [[-1, -1, 1], [-1, -1, 1]], torch.tensor([[-1, -1, 1]] * 2, dtype=torch.int32, device="cuda"))
    assert not out[1, 1].any() and bool((lse[1, 1] == -math.inf).all())


def test_large_scores_and_equal_scores(K):
    for dt in (F32, BF16):
        c = cache(14, [300], 10, 4, 1, 128, 16, dt)
        c["q"] *= 30
        run(K, c, *R.drafts(14, 1, 10))
        c["q"].zero_()
        run(K, c, *R.drafts(14, 1, 10))


@pytest.mark.parametrize("dt", [F32, BF16])
def test_streams_workspaces_repeats(K, dt):
    """The same bits each time: with a workspace of the caller's full of NaN, on another stream, two calls at once."""
    c = widened(cache(15, [3000, 700], 11, 8, 2, 128, 16, dt))
    rows, parents = R.drafts(15, 2, 11)
    out, lse = run(K, c, rows, parents)
    need = K.kda_paged_tree_attention_workspace_bytes(c["q"], c["k_cache"], c["block_table"])
    assert need > 0
    ws = [torch.full((max(need, 16),), 255, dtype=torch.uint8, device="cuda") for _ in range(2)]
    side = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [K.kda_paged_tree_attention(**c, parents=parents, workspace=ws[i], stream=side[i]) for i in range(2) for _ in range(3)]
    torch.cuda.synchronize()
    for o, s in got:
        assert torch.equal(o, out) and torch.equal(s, lse)
    o, none = K.kda_paged_tree_attention(**c, parents=parents, output_lse=False)
    assert none is None and torch.equal(o, out)


def test_captured(K):
    c = cache(16, [900, 80], 7, 8, 2, 128, 16, BF16)
    rows, parents = R.drafts(16, 2, 7)
    accepted = torch.tensor([6, 2], dtype=torch.int32, device="cuda")
    out, lse = K.kda_paged_tree_attention(**c, parents=parents)
    lens = torch.empty_like(c["seq_lens"])
    a = {x: c[x] for x in ("k_cache", "v_cache", "block_table", "seq_lens")}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        K.kda_paged_tree_attention(**c, parents=parents, out=out, lse=lse)
        K.kda_paged_tree_commit(**a, parents=parents, accepted=accepted, new_lens=lens)
    for seed, ls in ((17, [900, 80]), (18, [5, 600])):
        d = cache(seed, [900, 80], 7, 8, 2, 128, 16, BF16)
        for x in ("q", "k_cache", "v_cache"):
            c[x].copy_(d[x])
        c["seq_lens"].copy_(torch.tensor(ls))
        ref = reference(c, rows)
        graph.replay()
        torch.cuda.synchronize()
        check_paged(out, lse, ref)
        assert lens.tolist() == [x + len(R.path(p, i)) for x, p, i in zip(ls, rows, (6, 2))]


@pytest.mark.parametrize("d", [64, 128])
def test_every_wait_giving_up(K, d):
    """wait_polls = 0: all results are NaN, the status says so, and the next call is right."""
    c = widened(cache(30, [600, 0, 3000], 9, 8, 2, d, 16, BF16))
    rows, parents = R.drafts(30, 3, 9)
    need = K.kda_paged_tree_attention_workspace_bytes(c["q"], c["k_cache"], c["block_table"])
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    out, lse = torch.zeros_like(c["q"]), torch.zeros(3, 9, 8, device="cuda")
    a = [c[x] for x in ("q", "k_cache", "v_cache", "block_table", "seq_lens")]
    assert K.kda_device_status() == K.KDA_OK
    K.kda_paged_tree_attention_bounded(*a, parents, c["scale"], None, out, lse, ws, 0)
    torch.cuda.synchronize()
    assert bool(out.isnan().all()) and bool(lse.isnan().all())
    assert K.kda_device_status() == K.KDA_ERR_TIMEOUT
    assert K.kda_device_status() == K.KDA_OK
    run(K, c, rows, parents, workspace=ws)
    assert K.kda_device_status() == K.KDA_OK


# ------------------------------------------------------------------ the accepted path
def committed(c, rows, accepted):
    """The caches and lengths after the call, by indexing."""
    kc, vc = c["k_cache"].cpu().clone(), c["v_cache"].cpu().clone()
    pages, ps = kc.shape[:2]
    table = c["block_table"].cpu()
    width, lens = table.shape[1] * ps, []
    for n, p in enumerate(rows):
        length = max(0, min(int(c["seq_lens"][n]), width))
        way = R.path(p, accepted[n]) if 0 <= accepted[n] < len(p) else []
        place = lambda pos: (int(table[n, pos // ps]), pos % ps) if pos < width and 0 <= int(table[n, pos // ps]) < pages else None  # noqa: E731
        moves = [(place(length + a), place(length + r)) for r, a in enumerate(way)]
        moves = [x for x in moves if x[0] and x[1]]
        for x in (kc, vc):
            rows_ = [x[s].clone() for s, _ in moves]
            for (_, t), row in zip(moves, rows_):
                x[t] = row
        lens.append(min(length + len(way), width))
    return kc, vc, lens


@pytest.mark.parametrize("ps", [1, 3, 16, 64])
@pytest.mark.parametrize("T,Hkv,d", [(1, 1, 64), (7, 2, 128), (64, 3, 64), (40, 8, 128)])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_commit(K, ps, T, Hkv, d, dt):
    num = [T, T // 2, 0, T, 70, T, 1]
    c = cache(20, [0, 5, 30, 63, 64, 100, 17], T, Hkv, Hkv, d, ps, dt)
    for kind in ("tree", "chain", "star"):
        rows, parents = R.drafts(20, 7, T, kind, num)
        accepted = [T - 1, T // 2 - 1, 0, T // 2, min(T, 70) - 1, -1, 0]
        kc, vc, lens = committed(c, rows, accepted)
        got = K.kda_paged_tree_commit(c["k_cache"], c["v_cache"], c["block_table"], c["seq_lens"], parents,
                                      torch.tensor(accepted, dtype=torch.int32, device="cuda"), torch.tensor(num, dtype=torch.int32, device="cuda"))
        assert got.tolist() == lens
        assert torch.equal(c["k_cache"].cpu(), kc) and torch.equal(c["v_cache"].cpu(), vc)


def test_commit_at_the_edges(K):
    """Places past the table or outside the pool, lengths outside it, a line without parents, lengths in place."""
    c = cache(21, [20, 20, 20, 20], 6, 2, 2, 64, 4, BF16)
    c["block_table"][1, 5] = -1
    c["block_table"][2, 6] = 1 << 30
    c["seq_lens"].copy_(torch.tensor([c["block_table"].shape[1] * 4 - 2, 20, 20, 1 << 30]))
    rows = [R.tree(None, 6, "chain")] * 4
    parents = torch.tensor([[-1, 0, -1, 2, 2, 4]] * 4, dtype=torch.int32, device="cuda")
    accepted = [5, 5, 5, 5]
    at = torch.tensor(accepted, dtype=torch.int32, device="cuda")
    for p, used in ((parents, [[-1, 0, -1, 2, 2, 4]] * 4), (None, rows)):
        kc, vc, lens = committed(c, used, accepted)
        got = K.kda_paged_tree_commit(c["k_cache"], c["v_cache"], c["block_table"], c["seq_lens"], p, at, tokens=6)
        assert got.tolist() == lens
        assert torch.equal(c["k_cache"].cpu(), kc) and torch.equal(c["v_cache"].cpu(), vc)
    lens = committed(c, rows, accepted)[2]
    got = K.kda_paged_tree_commit(c["k_cache"], c["v_cache"], c["block_table"], c["seq_lens"], None, at, tokens=6, new_lens=c["seq_lens"])
    assert got is c["seq_lens"] and got.tolist() == lens


def test_commit_with_lengths_in_place(K):
    """new_lens may be seq_lens: every token still goes by the old length."""
    T, N = 40, 300
    c = cache(22, [n % 70 for n in range(N)], T, 2, 2, 64, 16, BF16)
    rows, parents = R.drafts(22, N, T, "tree", None)
    accepted = [T - 1 - n % 5 for n in range(N)]
    kc, vc, lens = committed(c, rows, accepted)
    K.kda_paged_tree_commit(c["k_cache"], c["v_cache"], c["block_table"], c["seq_lens"], parents,
                            torch.tensor(accepted, dtype=torch.int32, device="cuda"), new_lens=c["seq_lens"])
    assert c["seq_lens"].tolist() == lens
    assert torch.equal(c["k_cache"].cpu(), kc) and torch.equal(c["v_cache"].cpu(), vc)
