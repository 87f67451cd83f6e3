"""Paged key-value cache on the GPU: append against indexing, attention against its fp64 definition
(tests/lin_reference.py says where the bounds come from)."""
import math

import pytest
import torch

from tests import lin_reference as R

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def K(cuda_device):
    from linear_attention_fwd_gb300 import build, kda
    build.build()
    return kda


def cache(seed, lens, Hq, Hkv, d, ps, dt, spare=2, extra=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    N = len(lens)
    width = max(1, -(-max(lens) // ps)) + extra
    pages = N * width + spare
    table = torch.randperm(pages, generator=gen, device="cuda")[: N * width].view(N, width).to(torch.int32)
    return dict(q=(2 * rnd(N, Hq, d)).to(dt), k_cache=rnd(pages, ps, Hkv, d).to(dt), v_cache=rnd(pages, ps, Hkv, d).to(dt),
                block_table=table, seq_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), scale=d ** -0.5)


def reference(c):
    return R.paged_forward(c["q"], c["k_cache"], c["v_cache"], c["block_table"], c["seq_lens"], c["scale"])


@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 31, 63, 64, 65, 100, 257, 1000])
@pytest.mark.parametrize("dt,d", [(F32, 64), (F32, 128), (BF16, 64), (BF16, 128)])
def test_lengths(K, length, dt, d):
    c = cache(length, [length, max(1, length // 3)], 8, 2, d, 16, dt)
    R.check_paged(*K.kda_paged_attention(**c), reference(c))


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 1), (5, 1), (7, 7), (12, 4), (16, 1), (24, 2), (17, 1), (40, 1), (64, 1), (66, 2)])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_head_layouts(K, Hq, Hkv, dt):
    c = cache(3, [150, 33, 1], Hq, Hkv, 128, 32, dt)
    R.check_paged(*K.kda_paged_attention(**c), reference(c))


@pytest.mark.parametrize("ps", [1, 2, 7, 13, 64, 100, 128, 1000])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_page_sizes(K, ps, dt):
    c = cache(4, [200, 64, 1, 129], 8, 2, 64, ps, dt)
    R.check_paged(*K.kda_paged_attention(**c), reference(c))


@pytest.mark.parametrize("dt", [F32, BF16])
def test_empty_rows(K, dt):
    c = cache(5, [0, 40, 0, 0, 300, 0], 8, 2, 128, 16, dt)
    out, lse = K.kda_paged_attention(**c)
    R.check_paged(out, lse, reference(c))
    assert not out[0].any() and bool((lse[3] == -math.inf).all())
    c["seq_lens"].zero_()
    out, lse = K.kda_paged_attention(**c)
    assert not out.any() and bool((lse == -math.inf).all())


@pytest.mark.parametrize("dt", [F32, BF16])
def test_ragged_batch(K, dt):
    lens = [(i * i * 7919) % 1500 for i in range(40)]
    c = cache(6, lens, 8, 2, 128, 16, dt)
    R.check_paged(*K.kda_paged_attention(**c), reference(c))


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("lens", [[9000], [6000, 3, 0, 2500]])
def test_long_rows_are_split(K, dt, lens):
    c = cache(7, lens, 8, 2, 128, 64, dt)
    c["q"] *= 2
    R.check_paged(*K.kda_paged_attention(**c), reference(c))


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_what_lies_past_a_row_never_reaches_it(K, dt, bad):
    lens = [100, 1, 64, 0, 37]
    c = cache(8, lens, 8, 2, 128, 16, dt, extra=2)
    ref = reference(c)
    used = torch.zeros(c["k_cache"].shape[:2], dtype=torch.bool, device="cuda")
    for n, length in enumerate(lens):
        t = torch.arange(length, device="cuda")
        used[c["block_table"][n].long()[t // 16], t % 16] = True
    for x in ("k_cache", "v_cache"):
        c[x][~used] = bad
    R.check_paged(*K.kda_paged_attention(**c), ref)


@pytest.mark.parametrize("dt", [F32, BF16])
def test_pages_outside_the_pool_are_left_out(K, dt):
    c = cache(9, [200, 90, 33], 4, 2, 128, 16, dt)
    pages = c["k_cache"].shape[0]
    c["block_table"][0, 3] = -1
    c["block_table"][0, 11] = pages
    c["block_table"][1, :] = 1 << 30          # a row whose every page is bad
    c["block_table"][2, 0] = -(1 << 31)
    R.check_paged(*K.kda_paged_attention(**c), reference(c))


@pytest.mark.parametrize("dt", [F32, BF16])
def test_lengths_are_clamped(K, dt):
    c = cache(10, [64, 48], 4, 2, 64, 16, dt)
    c["seq_lens"] = torch.tensor([1 << 30, -5], dtype=torch.int32, device="cuda")
    R.check_paged(*K.kda_paged_attention(**c), reference(c))


@pytest.mark.parametrize("dt", [F32, BF16])
def test_scores_of_lowest_value(K, dt):
    """Keys that make scores the lowest finite value or -infinity weigh nothing; a row of nothing else is empty."""
    c = cache(11, [70, 20], 2, 1, 64, 16, dt)
    c["q"] = c["q"].abs() + 0.5
    t = torch.arange(0, 70, 3, device="cuda")
    c["k_cache"][c["block_table"][0].long()[t // 16], t % 16] = -math.inf
    t = t + 1
    t = t[t < 70]
    c["k_cache"][c["block_table"][0].long()[t // 16], t % 16] = torch.finfo(dt).min / 1024
    t = torch.arange(20, device="cuda")
    c["k_cache"][c["block_table"][1].long()[t // 16], t % 16] = -math.inf
    out, lse = K.kda_paged_attention(**c)
    R.check_paged(out, lse, reference(c))
    assert not out[1].any() and bool((lse[1] == -math.inf).all())


@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
def test_scales(K, scale):
    c = cache(12, [100, 7], 8, 2, 128, 16, BF16)
    c["scale"] = scale
    R.check_paged(*K.kda_paged_attention(**c), reference(c))


def test_no_lse_and_given_buffers(K):
    c = cache(13, [500, 20], 8, 2, 128, 16, BF16)
    ws = torch.full((max(1, K.kda_paged_attention_workspace_bytes(c["q"], c["k_cache"], c["block_table"])),), 255, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(c["q"])
    got, lse = K.kda_paged_attention(**c, out=out, output_lse=False, workspace=ws)
    assert got is out and lse is None
    R.check_paged(out, None, reference(c))


def test_offsets_past_32_bits(K):
    """A cache of more than 2^31 elements: the last pages are read and written where they are."""
    ps, Hkv, d = 64, 8, 128
    pages = (1 << 31) // (ps * Hkv * d) + 40
    kc, vc = (torch.zeros(pages, ps, Hkv, d, dtype=BF16, device="cuda") for _ in range(2))
    table = torch.tensor([[pages - 1, 3, pages - 2]], dtype=torch.int32, device="cuda")
    k, v = (torch.randn(150, Hkv, d, device="cuda").to(BF16) for _ in range(2))
    cu, pos = torch.tensor([0, 150], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    K.kda_paged_append(k, v, kc, vc, table, pos, cu)
    assert torch.equal(kc[pages - 1], k[:64]) and torch.equal(vc[pages - 2, :22], v[128:])
    c = dict(q=torch.randn(1, 16, d, device="cuda").to(BF16), seq_lens=torch.tensor([150], dtype=torch.int32, device="cuda"), scale=0.1)
    out, lse = K.kda_paged_attention(k_cache=kc, v_cache=vc, block_table=table, **c)
    small = torch.tensor([[0, 1, 2]])
    pick = table[0].long()
    R.check_paged(out, lse, R.paged_forward(c["q"], kc[pick], vc[pick], small, c["seq_lens"], 0.1))


def plain_append(c, k, v, positions, cu):
    ps = c["k_cache"].shape[1]
    kc, vc = c["k_cache"].clone(), c["v_cache"].clone()
    for n in range(positions.numel()):
        b, e = (n, n + 1) if cu is None else (int(cu[n]), int(cu[n + 1]))
        for u in range(b, e):
            p = int(positions[n]) + u - b
            if 0 <= p < c["block_table"].shape[1] * ps and 0 <= int(c["block_table"][n, p // ps]) < kc.shape[0]:
                kc[c["block_table"][n, p // ps], p % ps] = k[u]
                vc[c["block_table"][n, p // ps], p % ps] = v[u]
    return kc, vc


@pytest.mark.parametrize("dt,Hkv,d", [(F32, 1, 64), (BF16, 3, 64), (BF16, 8, 128), (F32, 2, 128)])
@pytest.mark.parametrize("ps", [1, 13, 16])
@pytest.mark.parametrize("lens", [None, [5, 0, 33, 1, 0, 70]])
def test_append(K, dt, Hkv, d, ps, lens):
    c = cache(30, [150] * 6, 1, Hkv, d, ps, dt)
    positions = torch.tensor([0, 3, 64, 149, 148, 77], dtype=torch.int32, device="cuda")   # some run past the table
    cu = None if lens is None else torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
    tokens = 6 if lens is None else sum(lens)
    k, v = (torch.randn(tokens, Hkv, d, device="cuda").to(dt) for _ in range(2))
    want = plain_append(c, k, v, positions, cu)
    K.kda_paged_append(k, v, c["k_cache"], c["v_cache"], c["block_table"], positions, cu)
    assert torch.equal(c["k_cache"], want[0]) and torch.equal(c["v_cache"], want[1])


def test_append_skips_bad_places(K):
    c = cache(31, [64] * 4, 1, 2, 64, 16, BF16)
    c["block_table"][1, :] = -1
    c["block_table"][2, 1] = c["k_cache"].shape[0]
    positions = torch.tensor([-3, 0, 10, 1 << 30], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 9, 20, 40, 45], dtype=torch.int32, device="cuda")
    k, v = (torch.randn(45, 2, 64, device="cuda").to(BF16) for _ in range(2))
    want = plain_append(c, k, v, positions, cu)
    K.kda_paged_append(k, v, c["k_cache"], c["v_cache"], c["block_table"], positions, cu)
    assert torch.equal(c["k_cache"], want[0]) and torch.equal(c["v_cache"], want[1])


def test_append_then_attend_on_another_stream_and_in_a_graph(K):
    """Decode steps: a token appended and attended over, captured once and replayed."""
    c = cache(32, [300, 40, 0], 8, 2, 128, 16, BF16, extra=1)
    k, v = (torch.randn(3, 2, 128, device="cuda").to(BF16) for _ in range(2))
    pos, lens = c["seq_lens"].clone(), c["seq_lens"] + 1
    kc, vc = c["k_cache"].clone(), c["v_cache"].clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    K.kda_paged_append(k, v, kc, vc, c["block_table"], pos, stream=s)
    want, wl = K.kda_paged_attention(c["q"], kc, vc, c["block_table"], lens, c["scale"], stream=s)
    s.synchronize()
    R.check_paged(want, wl, R.paged_forward(c["q"], kc, vc, c["block_table"], lens, c["scale"]))
    out, lse = torch.empty_like(want), torch.empty_like(wl)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        K.kda_paged_append(k, v, c["k_cache"], c["v_cache"], c["block_table"], pos)
        K.kda_paged_attention(c["q"], c["k_cache"], c["v_cache"], c["block_table"], lens, c["scale"], out=out, lse=lse)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("dt,d", [(BF16, 128), (BF16, 64), (F32, 64)])
@pytest.mark.parametrize("lens,Hq,Hkv", [([20011], 4, 1), ([1, 14533], 24, 2), ([0, 0, 9999, 0], 2, 2), ([1], 3, 1), ([0], 2, 1), ([64, 65, 1, 0], 8, 4),
                                         ([(i * 7919) % 400 for i in range(39)] + [12000], 8, 4), ([0] * 63 + [9000] + [5] * 30, 6, 3),
                                         ([8000] + [1] * 400, 1, 1)])
def test_shares_of_all_kinds(K, dt, d, lens, Hq, Hkv):
    """Tables wide enough for the shared-out form whatever the lengths: few units with many parts, more units than
    shares, shares that hold a unit's start only."""
    c = cache(8, lens, Hq, Hkv, d, 16, dt)
    wide = torch.full((len(lens), 600 * 16), -1, dtype=torch.int32, device="cuda")
    wide[:, : c["block_table"].shape[1]] = c["block_table"]
    c["block_table"] = wide
    R.check_paged(*K.kda_paged_attention(**c), reference(c))


# The shared-out form of attention (tables wider than a cluster's 8 x 1024 tokens) on everything that the one-launch
# form is tested on above.  What the table holds past a row's pages is never looked up.
def widen(K, c):
    ps = c["k_cache"].shape[1]
    rows, width = c["block_table"].shape
    wide = torch.full((rows, max(width, -(-8200 // ps))), 1 << 30, dtype=torch.int32, device="cuda")
    wide[:, :width] = c["block_table"]
    c["block_table"] = wide
    assert K.kda_paged_attention_workspace_bytes(c["q"], c["k_cache"], wide) > 0
    return c


def test_narrow_tables_take_one_launch(K):
    for c in (cache(40, [64] * 3, 8, 2, 128, 16, BF16), cache(40, [8192], 8, 2, 64, 64, F32)):
        assert K.kda_paged_attention_workspace_bytes(c["q"], c["k_cache"], c["block_table"]) == 0


@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 31, 63, 64, 65, 100, 257, 1000])
@pytest.mark.parametrize("dt,d", [(F32, 64), (F32, 128), (BF16, 64), (BF16, 128)])
def test_lengths_shared_out(K, length, dt, d):
    c = widen(K, cache(length, [length, max(1, length // 3)], 8, 2, d, 16, dt))
    R.check_paged(*K.kda_paged_attention(**c), reference(c))


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 1), (5, 1), (7, 7), (12, 4), (16, 1), (24, 2), (17, 1), (40, 1), (64, 1), (66, 2)])
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("lens", [[150, 33, 1], [2000], [300] * 60])
def test_head_layouts_shared_out(K, Hq, Hkv, dt, lens):
    """Few rows (a join per unit) and many (a join per boundary), heads in one block and in several."""
    c = widen(K, cache(3, lens, Hq, Hkv, 128, 32, dt))
    R.check_paged(*K.kda_paged_attention(**c), reference(c))


@pytest.mark.parametrize("ps", [1, 2, 7, 13, 64, 100, 128, 1000])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_page_sizes_shared_out(K, ps, dt):
    c = widen(K, cache(4, [200, 64, 1, 129], 8, 2, 64, ps, dt))
    R.check_paged(*K.kda_paged_attention(**c), reference(c))


@pytest.mark.parametrize("dt", [F32, BF16])
def test_empty_rows_shared_out(K, dt):
    c = widen(K, cache(5, [0, 40, 0, 0, 300, 0], 8, 2, 128, 16, dt))
    out, lse = K.kda_paged_attention(**c)
    R.check_paged(out, lse, reference(c))
    assert not out[0].any() and bool((lse[3] == -math.inf).all())
    c["seq_lens"].zero_()
    out, lse = K.kda_paged_attention(**c)
    assert not out.any() and bool((lse == -math.inf).all())


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("ps", [16, 13])
def test_what_lies_past_a_row_never_reaches_it_shared_out(K, dt, bad, ps):
    lens = [100, 1, 64, 0, 37, 1500]
    c = widen(K, cache(8, lens, 8, 2, 128, ps, dt, extra=2))
    ref = reference(c)
    used = torch.zeros(c["k_cache"].shape[:2], dtype=torch.bool, device="cuda")
    for n, length in enumerate(lens):
        t = torch.arange(length, device="cuda")
        used[c["block_table"][n].long()[t // ps], t % ps] = True
    for x in ("k_cache", "v_cache"):
        c[x][~used] = bad
    R.check_paged(*K.kda_paged_attention(**c), ref)


@pytest.mark.parametrize("dt", [F32, BF16])
def test_pages_outside_the_pool_are_left_out_shared_out(K, dt):
    c = widen(K, cache(9, [200, 90, 33, 1000], 4, 2, 128, 16, dt))
    pages = c["k_cache"].shape[0]
    c["block_table"][0, 3] = -1
    c["block_table"][0, 11] = pages
    c["block_table"][1, :] = 1 << 30          # a row whose every page is bad
    c["block_table"][2, 0] = -(1 << 31)
    c["block_table"][3, 8:40] = -1            # whole tiles, and more than a CTA's share
    R.check_paged(*K.kda_paged_attention(**c), reference(c))


@pytest.mark.parametrize("dt", [F32, BF16])
def test_lengths_are_clamped_shared_out(K, dt):
    c = widen(K, cache(10, [64, 48], 4, 2, 64, 16, dt))
    c["seq_lens"] = torch.tensor([1 << 30, -5], dtype=torch.int32, device="cuda")
    R.check_paged(*K.kda_paged_attention(**c), reference(c))


@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
def test_scales_shared_out(K, scale):
    c = widen(K, cache(12, [700, 7], 8, 2, 128, 16, BF16))
    c["scale"] = scale
    R.check_paged(*K.kda_paged_attention(**c), reference(c))


def test_no_lse_and_a_used_workspace(K):
    c = widen(K, cache(13, [3000, 20], 8, 2, 128, 16, BF16))
    ws = torch.full((K.kda_paged_attention_workspace_bytes(c["q"], c["k_cache"], c["block_table"]),), 255, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(c["q"])
    got, lse = K.kda_paged_attention(**c, out=out, output_lse=False, workspace=ws)
    assert got is out and lse is None
    R.check_paged(out, None, reference(c))


@pytest.mark.parametrize("dt", [F32, BF16])
def test_calls_share_a_workspace(K, dt):
    """Calls back to back on one stream with one workspace (its contents on entry all ones), splits and joins of
    each kind, and the same in a replayed graph: bit for bit what each gives alone, and right."""
    cases = [widen(K, cache(41 + i, lens, 24, 2, 128, 16, dt)) for i, lens in
             enumerate([[5000], [(i * 7919) % 900 for i in range(50)], [0, 3, 2500], [64] * 200])]
    alone = [K.kda_paged_attention(**c) for c in cases]
    for c, (out, lse) in zip(cases, alone):
        R.check_paged(out, lse, reference(c))
    need = max(K.kda_paged_attention_workspace_bytes(c["q"], c["k_cache"], c["block_table"]) for c in cases)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    got = [K.kda_paged_attention(**cases[i % 4], workspace=ws) for i in range(24)]
    torch.cuda.synchronize()
    for i, (out, lse) in enumerate(got):
        assert torch.equal(out, alone[i % 4][0]) and torch.equal(lse, alone[i % 4][1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            got = [K.kda_paged_attention(**c, workspace=ws) for c in cases]
    torch.cuda.synchronize()
    for _ in range(4):
        for out, lse in got:
            out.zero_(), lse.zero_()
        ws.fill_(255)
        torch.cuda.synchronize()
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        for (out, lse), (want, wl) in zip(got, alone):
            assert torch.equal(out, want) and torch.equal(lse, wl)
