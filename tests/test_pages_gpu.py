"""Rows of a block table forked, ended and extended, a pool closed up, pages copied: whole numbers and copies equal to
plain Python's (tests/tree_reference.py)."""
import random

import pytest
import torch

from tests import tree_reference as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K(cuda_device):
    from linear_attention_fwd_gb300 import build, kda
    build.build()
    return kda


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def pool(seed, N, W, ps, spare, share=0.5, reserve=0.3):
    """A consistent table: rows that share first pages with an earlier one, some with pages kept past their length."""
    rng = random.Random(seed)
    lens, table, nxt = [], [], 0
    order = list(range(N * W + spare))
    rng.shuffle(order)
    for n in range(N):
        row = [-1] * W
        length = rng.choice([0, 1, ps, W * ps, rng.randint(0, W * ps)])
        held = -(-length // ps)
        if rng.random() < reserve:
            held = rng.randint(held, W)
        same = 0
        if n and rng.random() < share:
            other = rng.randrange(n)
            same = min(held, lens[other] // ps, length // ps)
            row[:same] = table[other][:same]
        for e in range(same, held):
            row[e] = order[nxt]
            nxt += 1
        lens.append(length)
        table.append(row)
    pages = nxt + spare
    rename = {}
    names = list(range(max(1, pages)))
    rng.shuffle(names)
    for row in table:
        for e, p in enumerate(row):
            if p >= 0:
                if p not in rename:
                    rename[p] = names[len(rename)]
                row[e] = rename[p]
    refs = [0] * max(1, pages)
    for row in table:
        for p in row:
            if p >= 0:
                refs[p] += 1
    return table, lens, refs


def check_fork(K, table, lens, refs, sources, new, ps):
    want = R.fork(table, lens, refs, sources, new, ps)
    args = [i32(table), i32(lens), i32(refs), i32(sources), None if new is None else i32(new)]
    before = [None if x is None else x.clone() for x in args]
    got = K.kda_paged_fork(*args, page_size=ps)
    for x, y in zip(args, before):
        assert x is None or torch.equal(x, y)
    assert got[4].tolist() == [want[4]]
    assert got[1].tolist() == want[1]
    assert got[0].tolist() == want[0]
    assert got[2].tolist() == want[2]
    assert [tuple(x) for x in got[3].tolist()] == want[3]
    return want


def sources(rng, N):
    return [rng.choice([n, n, rng.randrange(N), -1, rng.randrange(N)]) for n in range(N)]


@pytest.mark.parametrize("N,W", [(1, 1), (2, 3), (8, 40), (33, 130), (70, 513), (300, 17), (5, 3000)])
@pytest.mark.parametrize("ps", [1, 5, 16])
def test_fork(K, N, W, ps):
    rng = random.Random(N * W)
    for seed, spare in ((1, 2 * N + N * W // 4), (2, N), (3, 0)):
        table, lens, refs = pool(seed, N, W, ps, spare)
        want = check_fork(K, table, lens, refs, sources(rng, N), [rng.choice([0, 0, 1, ps, -4, 3 * ps]) for _ in range(N)], ps)
        if want[4] == 0:   # what the counts say after the call is what the table says
            count = [0] * len(refs)
            for row in want[0]:
                for p in row:
                    if p >= 0:
                        count[p] += 1
            assert count == want[2]
        check_fork(K, table, lens, refs, list(range(N)), None, ps)
        check_fork(K, table, lens, refs, [-1] * N, None, ps)


def test_fork_of_shared_last_pages_and_bad_entries(K):
    """A partly filled page that two rows name is copied by both; entries and sources out of range; lengths past the table."""
    table = [[3, 1, -1, -1], [3, 1, -1, -1], [5, 99, -9, -1], [0, 2, 4, 7]]
    refs = [0] * 20
    for row in table:
        for p in row:
            if 0 <= p < 20:
                refs[p] += 1
    for src in ([0, 1, 2, 3], [1, 1, 0, 0], [3, 3, 3, 3], [7, -2, 2, 2], [2, 0, 1, 0]):
        for lens in ([6, 6, 4, 13], [6, 5, 9, 1 << 30], [-3, 0, 8, 16]):
            check_fork(K, table, lens, refs, src, [0, 1, 4, 1 << 30], 4)


def test_fork_of_large_pools(K):
    for N, W, pages in ((4, 7, 300000), (600, 5, 40000), (20000, 2, 50001)):
        rng = random.Random(pages)
        refs, table = [0] * pages, []
        names = rng.sample(range(pages), N * W)
        for n in range(N):
            table.append(names[n * W: (n + 1) * W - 1] + [-1])
            for p in table[n][:-1]:
                refs[p] = 1
        lens = [rng.randint((W - 1) * 16 - 15, (W - 1) * 16) for _ in range(N)]
        check_fork(K, table, lens, refs, sources(rng, N), [17] * N, 16)


@pytest.mark.parametrize("N,W,spare", [(1, 1, 0), (1, 1, 3), (2, 3, 1), (8, 40, 100), (33, 130, 3000), (70, 513, 1), (300, 17, 5000), (3, 9, 100000)])
def test_compact(K, N, W, spare):
    for seed in (1, 2):
        table, _, refs = pool(seed, N, W, 4, spare)
        table[0][-1] = -5 if table[0][-1] < 0 else table[0][-1]
        want = R.compact(table, refs)
        got = K.kda_paged_compact(i32(table), i32(refs))
        assert got[0].tolist() == want[0]
        assert got[1].tolist() == want[1]
        assert [tuple(x) for x in got[2].tolist()] == want[2]
        again = K.kda_paged_compact(got[0], got[1])        # nothing left to move
        assert torch.equal(again[0], got[0]) and torch.equal(again[1], got[1]) and bool((again[2] == -1).all())


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("ps,Hkv,d,M", [(1, 1, 64, 1), (3, 2, 64, 5), (16, 8, 128, 30), (100, 1, 128, 7), (7, 3, 128, 0), (256, 16, 128, 3)])
def test_copy(K, dt, ps, Hkv, d, M):
    gen = torch.Generator(device="cuda").manual_seed(M)
    pages = 2 * M + 3
    kc, vc = (torch.randn(pages, ps, Hkv, d, generator=gen, device="cuda").to(dt) for _ in range(2))
    order = torch.randperm(pages, generator=gen, device="cuda")[: 2 * M].view(M, 2).to(torch.int32)
    order[1::3, 0] = -1
    order[2::5, 1] = pages
    want = [x.clone() for x in (kc, vc)]
    for a, b in order.tolist():
        if 0 <= a < pages and 0 <= b < pages:
            for x in want:
                x[b] = x[a]
    K.kda_paged_copy(kc, vc, order.contiguous())
    assert torch.equal(kc, want[0]) and torch.equal(vc, want[1])


def test_captured_with_buffers_of_the_callers(K):
    """Fork, copies and compaction in one graph, replayed on other tables."""
    N, W, ps = 12, 9, 4
    table, lens, refs = pool(5, N, W, ps, 40)
    pages = len(refs)
    st = dict(table=i32(table), lens=i32(lens), refs=i32(refs), src=i32(list(range(N))))
    kc, vc = (torch.randn(pages, ps, 2, 64, device="cuda") for _ in range(2))
    out = dict(new_table=torch.empty_like(st["table"]), new_lens=torch.empty_like(st["lens"]), new_refs=torch.empty_like(st["refs"]),
               copies=torch.empty(N, 2, dtype=torch.int32, device="cuda"), short_of=torch.empty(1, dtype=torch.int32, device="cuda"))
    com = dict(new_table=torch.empty_like(st["table"]), new_refs=torch.empty_like(st["refs"]), copies=torch.empty(pages // 2, 2, dtype=torch.int32, device="cuda"))

    def both():
        K.kda_paged_fork(st["table"], st["lens"], st["refs"], st["src"], page_size=ps, **out)
        K.kda_paged_copy(kc, vc, out["copies"])
        K.kda_paged_compact(out["new_table"], out["new_refs"], **com)
        K.kda_paged_copy(kc, vc, com["copies"])
    both()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    rng = random.Random(1)
    for _ in range(3):
        src = sources(rng, N)
        st["src"].copy_(i32(src))
        rows = lambda t, c, ls: [[c[t[n][x // ps], x % ps] for x in range(ls[n])] for n in range(N)]  # noqa: E731
        was = rows(table, kc.cpu().clone(), lens)
        graph.replay()
        torch.cuda.synchronize()
        now = rows(com["new_table"].tolist(), kc.cpu(), out["new_lens"].tolist())
        for n in range(N):
            want = was[src[n]] if src[n] >= 0 else []
            assert len(now[n]) == len(want) and all(torch.equal(x, y) for x, y in zip(now[n], want))
        kc.copy_(torch.randn_like(kc))
