"""Rows that were set back below pages which other rows name too (a sample that is rewound and generated anew): a fork gives such a
row no page to write to that another row reads."""
import random

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K(cuda_device):
    from linear_attention_fwd_gb300 import build, kda
    build.build()
    return kda


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def counts(table, pages):
    c = [0] * pages
    for row in table:
        for p in row:
            if p >= 0:
                c[p] += 1
    return c


def cached(caches, table, lens, ps):
    """Keys and values of each row's tokens."""
    return [[x[table[n, : -(-length // ps)].long()].flatten(0, 1)[:length].clone() for x in caches] for n, length in enumerate(lens)]


def test_a_row_set_back_leaves_the_others_tokens(K):
    """Two rows share four pages of 16; one goes back to 40 tokens, is extended and appended to."""
    ps, pages = 16, 12
    table, lens = [[7, 2, 9, 4, -1], [7, 2, 9, 4, 5]], [40, 70]
    caches = [torch.randn(pages, ps, 2, 64, device="cuda") for _ in range(2)]
    before = cached(caches, i32(table), lens, ps)
    new, length, refs, copies, short = K.kda_paged_fork(i32(table), i32(lens), i32(counts(table, pages)), i32([0, 1]), i32([40, 8]), page_size=ps)
    assert short.tolist() == [0] and length.tolist() == lens
    K.kda_paged_copy(*caches, copies)
    add = [torch.randn(48, 2, 64, device="cuda") for _ in range(2)]
    K.kda_paged_append(*add, *caches, new, length, i32([0, 40, 48]))
    after = cached(caches, new, [80, 78], ps)
    for n, (first, more) in enumerate(((0, 40), (40, 8))):
        for x in range(2):
            assert torch.equal(after[n][x][: lens[n]], before[n][x]), n
            assert torch.equal(after[n][x][lens[n]:], add[x][first: first + more]), n
    # the lowest free pages, entry by entry; the shared ones are the other row's alone (0 was copied into, 1, 3 are room)
    assert new.tolist() == [[7, 2, 0, 1, 3], [7, 2, 9, 4, 5]]
    assert copies.tolist() == [[9, 0], [-1, -1]]
    assert refs.tolist() == counts(new.tolist(), pages)


def test_a_page_past_two_ends_is_nobodys(K):
    """Both holders have gone back: the page is given up by both and free for the next call."""
    table, lens = [[3, 1], [3, 1], [0, -1]], [4, 0, 2]
    args = [i32(table), i32(lens), i32(counts(table, 5))]
    new, _, refs, copies, short = K.kda_paged_fork(*args, i32([0, 1, 2]), i32([0, 4, 0]), page_size=4)
    assert short.tolist() == [0]
    assert new.tolist() == [[3, -1], [2, -1], [0, -1]]      # (page 1 still had its two references when the call began)
    assert refs.tolist() == [1, 0, 1, 1, 0]
    assert (copies == -1).all()


def test_pages_of_its_own_past_the_length_stay(K):
    table, lens = [[2, 0, 4, -1], [2, -1, -1, -1]], [3, 3]
    new, _, refs, copies, short = K.kda_paged_fork(i32(table), i32(lens), i32(counts(table, 6)), i32([0, 1]), i32([9, 0]), page_size=4)
    assert short.tolist() == [0]
    assert new.tolist() == [[1, 0, 4, -1], [3, -1, -1, -1]]
    assert copies.tolist() == [[2, 1], [2, 3]]
    assert refs.tolist() == [1, 1, 0, 1, 1, 0]


def grown(seed, N, W, ps, spare):
    """A consistent table of rows that share first pages with an earlier one and were set back afterwards, any number of them."""
    rng = random.Random(seed)
    table, lens, nxt = [], [], 0
    for n in range(N):
        full = rng.randint(0, W)
        same = rng.randint(0, min(full, sum(p >= 0 for p in table[-1]))) if n and rng.random() < 0.7 else 0
        row = (table[-1][:same] if same else []) + list(range(nxt, nxt + full - same))
        nxt += full - same
        table.append(row + [-1] * (W - full))
        lens.append(rng.randint(0, full * ps))
    names = list(range(max(1, nxt + spare)))
    rng.shuffle(names)
    return [[names[p] if p >= 0 else -1 for p in row] for row in table], lens, len(names)


# (narrow tables, a row a warp, several segments a row, more rows than a batch, more than are kept in shared memory)
@pytest.mark.parametrize("N,W", [(1, 3), (2, 3), (8, 40), (33, 130), (70, 513), (300, 17), (5, 3000), (1500, 6), (9000, 2)])
@pytest.mark.parametrize("ps", [1, 5, 16])
def test_no_row_may_write_where_another_reads(K, N, W, ps):
    rng = random.Random(N + ps)
    for seed, spare in ((1, 4 * N + N * W), (2, N)):
        table, lens, pages = grown(seed, N, W, ps, spare)
        refs = counts(table, pages)
        src = [rng.choice([n, n, rng.randrange(N), -1]) for n in range(N)]
        more = [rng.choice([0, 0, 1, ps, 3 * ps]) for _ in range(N)]
        new, length, after, copies, short = (x.tolist() for x in K.kda_paged_fork(i32(table), i32(lens), i32(refs), i32(src), i32(more), page_size=ps))
        if short[0]:
            assert new == table and length == lens and after == refs and all(c == [-1, -1] for c in copies)
            continue
        assert after == counts(new, pages)
        heirs, lowest = {}, iter(p for p in range(pages) if refs[p] == 0)
        for n, s in enumerate(src):
            x = lens[s] if s >= 0 else 0
            full, held, room = x // ps, -(-x // ps), min(W, -(-(x + more[n]) // ps)) if s >= 0 else 0
            heir = s >= 0 and heirs.setdefault(s, n) == n
            assert length[n] == x
            for e in range(W):
                was, now = table[s][e] if s >= 0 else -1, new[n][e]
                if e < full:
                    assert now == was
                    continue
                # what the row may write to is its own
                assert now < 0 or after[now] == 1, (n, e)
                own = heir and was >= 0 and refs[was] == 1
                if own:
                    assert now == was
                elif e < held or e < room:
                    assert now == next(lowest)
                else:
                    assert now == -1
                if e == full and full < held:
                    assert copies[n] == ([-1, -1] if own else [was, now])
            if full == held:
                assert copies[n] == [-1, -1]


def test_copies_follow_their_list(K):
    """A list that a fork writes anew right behind a copy that has read the old one, many times in one graph: every copy goes by
    the list as its own fork leaves it."""
    N, W, ps, Hkv, d, rounds = 24, 3, 4, 2, 64, 60
    pages = 3 * N
    rng = random.Random(3)
    table = [[n, -1, -1] for n in range(N)]
    lens = [rng.randint(1, ps - 1) for _ in range(N)]
    tables, lengths, refs = i32(table), i32(lens), i32(counts(table, pages))
    src = [[rng.randrange(N) for _ in range(N)] for _ in range(rounds)]
    srcs = [i32(x) for x in src]
    copies = torch.full((N, 2), -1, dtype=torch.int32, device="cuda")
    outs = [[torch.empty_like(x) for x in (tables, lengths, refs)] for _ in range(rounds)]
    short = torch.zeros(1, dtype=torch.int32, device="cuda")
    caches = [torch.randn(pages, ps, Hkv, d, device="cuda") for _ in range(2)]
    first = [x.clone() for x in caches]

    def run():
        t, x, r = tables, lengths, refs
        for i in range(rounds):
            new = outs[i]
            K.kda_paged_fork(t, x, r, srcs[i], page_size=ps, new_table=new[0], new_lens=new[1], new_refs=new[2], copies=copies, short_of=short)
            K.kda_paged_copy(*caches, copies)
            t, x, r = new
    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    row = list(range(N))                                 # the row of the first table whose tokens each one has
    for s in src:
        row = [row[n] for n in s]
    for _ in range(3):
        for x, y in zip(caches, first):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        assert short.tolist() == [0]
        last = outs[-1][0].tolist()
        for n in range(N):
            for x, y in zip(caches, first):
                assert torch.equal(x[last[n][0], : lens[row[n]]], y[row[n], : lens[row[n]]]), n
