"""Linear attention with a decay per head on the GPU against its fp64 definition (tests/lin_reference.py
says where the bounds come from)."""
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


def make(seed, B, T, H, Hk, dk, dv, dt, decay="token", init=0, scale=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    d = dict(q=unit(rnd(B, T, Hk, dk)).to(dt), k=unit(rnd(B, T, Hk, dk)).to(dt), v=(scale * rnd(B, T, H, dv)).to(dt))
    d["g"] = d["head_g"] = None
    if decay in ("token", "both"):
        d["g"] = -torch.nn.functional.softplus(rnd(B, T, H) - 1.0)
    if decay in ("head", "both"):
        d["head_g"] = -torch.exp2(-torch.linspace(1, 8, H, device="cuda"))
    if decay == "resets":      # tokens that forget everything among tokens that forget little or nothing
        g = -0.02 * rnd(B, T, H).abs()
        g[torch.rand(B, T, H, generator=gen, device="cuda") < 0.08] = -math.inf
        g[torch.rand(B, T, H, generator=gen, device="cuda") < 0.05] = -3000.0
        g[torch.rand(B, T, H, generator=gen, device="cuda") < 0.2] = 0.0
        d["g"] = g
    d["initial_state"] = scale * rnd(init, H, dk, dv) if init else None
    return d


def reference(d, cu=None):
    return R.lin_forward(d["q"], d["k"], d["v"], d["g"], d["head_g"], d["initial_state"], cu)


LENGTHS = [1, 2, 31, 32, 33, 63, 64, 65, 127, 129, 200, 321]


@pytest.mark.parametrize("T", LENGTHS)
@pytest.mark.parametrize("dt,dk,dv", [(F32, 64, 64), (F32, 128, 128), (BF16, 128, 128), (BF16, 64, 128), (BF16, 128, 64), (BF16, 64, 64)])
def test_dense_lengths(K, T, dt, dk, dv):
    d = make(T, 2, T, 2, 2, dk, dv, dt, init=2 if T % 2 else 0)
    out, fin = K.kda_lin_chunk_fwd(**d)
    R.check_lin(out, fin, reference(d))


@pytest.mark.parametrize("decay", ["none", "token", "head", "both", "resets"])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_decays_and_shared_heads(K, decay, dt):
    d = make(7, 1, 190, 6, 2, 128, 128, dt, decay=decay, init=1)
    out, fin = K.kda_lin_chunk_fwd(**d)
    R.check_lin(out, fin, reference(d))


@pytest.mark.parametrize("dt", [F32, BF16])
def test_strong_decays(K, dt):
    d = make(8, 1, 150, 2, 2, 128, 128, dt, init=1)
    d["g"] = d["g"] * 40.0
    out, fin = K.kda_lin_chunk_fwd(**d)
    R.check_lin(out, fin, reference(d))


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("scale", [2.0 ** -60, 2.0 ** 60])
def test_magnitudes_of_v_and_state(K, dt, scale):
    d = make(9, 1, 140, 2, 1, 128, 128, dt, init=1, scale=scale)
    out, fin = K.kda_lin_chunk_fwd(**d)
    R.check_lin(out, fin, reference(d))


@pytest.mark.parametrize("dt,dk", [(F32, 128), (F32, 64), (BF16, 128), (BF16, 64)])
def test_packed_with_empty_members(K, dt, dk):
    lens = [1, 64, 0, 130, 17, 1, 65, 0, 300]
    cu = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
    d = make(11, 1, sum(lens), 4, 2, dk, 128, dt, init=len(lens))
    out, fin = K.kda_lin_chunk_fwd(**d, cu_seqlens=cu)
    R.check_lin(out, fin, reference(d, cu))


@pytest.mark.parametrize("dt,dk,dv", [(F32, 128, 128), (BF16, 128, 128), (BF16, 64, 128), (BF16, 128, 64), (BF16, 64, 64), (F32, 64, 64)])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_neighbours_never_leak(K, dt, dk, dv, bad):
    """NaN and infinities of one sequence stay in it, whatever shares its tiles."""
    lens = [70, 5, 129, 64]
    cu = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
    d = make(12, 1, sum(lens), 2, 1, dk, dv, dt, init=4)
    clean = reference(d, cu)
    for x in ("q", "k", "v", "g"):
        for b, e in ((70, 75), (204, 268)):
            d[x][:, b:e] = bad if x != "g" else math.nan
    out, fin = K.kda_lin_chunk_fwd(**d, cu_seqlens=cu)
    for b, e in ((0, 70), (75, 204)):
        R.check_lin(out[:, b:e], None, tuple(x[:, b:e] for x in clean[:1]) + (None,) + (clean[2][:, b:e], None))
    for n in (0, 2):
        R.check_lin(out[:, :0], fin[n], (clean[0][:, :0], clean[1][n], clean[2][:, :0], clean[3][n]))


@pytest.mark.parametrize("dt,dk,dv", [(F32, 128, 128), (BF16, 128, 128), (BF16, 64, 128), (BF16, 64, 64)])
@pytest.mark.parametrize("B,T,H", [(1, 1500, 2), (1, 4200, 1), (2, 2100, 3)])
def test_long_few_heads(K, dt, dk, dv, B, T, H):
    """Fewer (sequence, head) pairs than SMs: sequences may be cut into parts."""
    d = make(13, B, T, H, 1, dk, dv, dt, decay="both", init=B)
    d["g"] *= 0.02      # slow enough that every part sees the ones before it
    out, fin = K.kda_lin_chunk_fwd(**d)
    R.check_lin(out, fin, reference(d))


@pytest.mark.parametrize("dt", [F32, BF16])
def test_long_packed_few_heads(K, dt):
    lens = [0, 1, 2000, 63, 700, 64, 1]
    cu = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
    d = make(14, 1, sum(lens), 1, 1, 128, 128, dt, init=len(lens))
    d["g"] *= 0.02
    out, fin = K.kda_lin_chunk_fwd(**d, cu_seqlens=cu)
    R.check_lin(out, fin, reference(d, cu))


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("n,long,H", [(7, 2600, 3), (300, 2100, 1), (300, 2100, 5)])
def test_one_long_among_short(K, dt, n, long, H):
    """Packed: the long sequence is cut, the others are not; few sequences and more than are ranked."""
    lens = [(5 * i) % 9 for i in range(n)]
    lens[n // 2] = long
    cu = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
    d = make(27, 1, sum(lens), H, 1, 64, 64, dt, decay="both", init=n)
    d["g"] *= 0.02
    out, fin = K.kda_lin_chunk_fwd(**d, cu_seqlens=cu)
    R.check_lin(out, fin, reference(d, cu))


@pytest.mark.parametrize("n", [4, 300])
def test_offsets_that_overlap_stay_in_bounds(K, n):
    """Offsets that are not as documented (every other member is the whole): more parts than there are slots, and
    nothing outside the tensors is touched.  The members that the first slots hold are right."""
    T = 1500
    d = make(28, 1, T, 1, 1, 64, 64, BF16, decay="head")
    cu = torch.tensor([0, T] * (n // 2) + [0], dtype=torch.int32, device="cuda")
    out, fin = K.kda_lin_chunk_fwd(**d, cu_seqlens=cu)
    ref = reference(d)
    R.check_lin(out, fin[:1], ref)
    assert not fin[1].any()
    torch.cuda.synchronize()


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("T", [130, 2500])
def test_resume_in_place_equals_one_call(K, dt, T):
    d = make(15, 1, T, 2, 2, 128, 128, dt, init=1)
    ref = reference(d)
    half = 65
    st = d["initial_state"].clone()
    cut = lambda lo, hi: {x: (d[x][:, lo:hi].contiguous() if d[x] is not None and x not in ("head_g", "initial_state") else d[x]) for x in d}  # noqa: E731
    a, b = cut(0, half), cut(half, T)
    a["initial_state"] = b["initial_state"] = st
    o1, f1 = K.kda_lin_chunk_fwd(**a, final_state=st)
    o2, f2 = K.kda_lin_chunk_fwd(**b, final_state=st)
    assert f1 is st and f2 is st
    R.check_lin(torch.cat([o1, o2], 1), st, ref)


def test_malformed_offsets_stay_in_bounds(K):
    """Offsets are clamped on the device: nothing outside the packed tensors is touched."""
    d = make(16, 1, 100, 2, 2, 128, 128, BF16, init=3)
    cu = torch.tensor([0, 50, 40, 100000], dtype=torch.int32, device="cuda")
    out, fin = K.kda_lin_chunk_fwd(**d, cu_seqlens=cu)
    # members: [0, 50), [50, 50), [40, 100)
    ref = R.lin_forward(d["q"][:, :50], d["k"][:, :50], d["v"][:, :50], d["g"][:, :50], None, d["initial_state"][:1])
    R.check_lin(out[:, :40], fin[:1], (ref[0][:, :40], ref[1], ref[2][:, :40], ref[3]))
    assert torch.equal(fin[1], d["initial_state"][1])


def test_no_tokens(K):
    d = make(17, 2, 0, 2, 2, 128, 128, BF16, init=2)
    out, fin = K.kda_lin_chunk_fwd(**d)
    assert out.shape == (2, 0, 2, 128) and torch.equal(fin, d["initial_state"])
    d["initial_state"] = None
    assert not K.kda_lin_chunk_fwd(**d)[1].any()


@pytest.mark.parametrize("dt", [F32, BF16])
def test_outputs_only_and_canaries(K, dt):
    d = make(18, 1, 77, 3, 3, 128, 128, dt)
    big = torch.full((79, 3, 128), 7.0, dtype=dt, device="cuda")
    out, fin = K.kda_lin_chunk_fwd(**d, out=big[1:78][None], output_final_state=False)
    assert fin is None and bool((big[0] == 7).all()) and bool((big[78] == 7).all())
    R.check_lin(out, None, reference(d))


@pytest.mark.parametrize("rows,H,Hk,dk,dv", [(1, 1, 1, 64, 64), (1, 32, 32, 128, 128), (3, 4, 2, 128, 64), (5, 6, 2, 64, 128), (70, 8, 8, 128, 128), (3, 120, 8, 128, 128)])
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("decay", ["token", "head", "both", "none"])
def test_step(K, rows, H, Hk, dk, dv, dt, decay):
    d = make(21, 1, rows, H, Hk, dk, dv, dt, decay=decay)
    pool = torch.randn(rows + 2, H, dk, dv, device="cuda")
    before = pool.clone()
    idx = torch.randperm(rows + 2, device="cuda")[:rows].to(torch.int32)
    cu = torch.arange(rows + 1)
    ref = R.lin_forward(d["q"], d["k"], d["v"], d["g"], d["head_g"], before[idx.long()], cu)
    out = K.kda_lin_recurrent_step(d["q"][0], d["k"][0], d["v"][0], None if d["g"] is None else d["g"][0], d["head_g"], pool, idx)
    R.check_lin(out[None], pool[idx.long()], ref)
    other = torch.ones(rows + 2, dtype=torch.bool, device="cuda")
    other[idx.long()] = False
    assert torch.equal(pool[other], before[other])


def test_step_skips_rows_outside_the_pool(K):
    d = make(22, 1, 4, 2, 2, 128, 128, BF16)
    pool = torch.randn(3, 2, 128, 128, device="cuda")
    before = pool.clone()
    idx = torch.tensor([-1, 3, 1, 1 << 30], dtype=torch.int32, device="cuda")
    out = torch.full((4, 2, 128), 5.0, dtype=BF16, device="cuda")
    K.kda_lin_recurrent_step(d["q"][0], d["k"][0], d["v"][0], d["g"][0], None, pool, idx, out=out)
    assert torch.equal(pool[0], before[0]) and torch.equal(pool[2], before[2]) and not torch.equal(pool[1], before[1])
    assert bool((out[[0, 1, 3]] == 5).all()) and not bool((out[2] == 5).any())


def test_step_forgets_everything(K):
    d = make(23, 1, 2, 2, 2, 128, 128, F32)
    d["g"][:] = -math.inf
    pool = torch.randn(2, 2, 128, 128, device="cuda")
    K.kda_lin_recurrent_step(d["q"][0], d["k"][0], d["v"][0], d["g"][0], None, pool)
    assert torch.equal(pool, d["k"][0][..., None] * d["v"][0][..., None, :])


def test_steps_equal_a_prompt(K):
    """The recurrent form carried over 70 tokens gives the chunked form's outputs and state."""
    d = make(24, 1, 70, 3, 3, 128, 128, BF16)
    pool = torch.zeros(1, 3, 128, 128, device="cuda")
    outs = [K.kda_lin_recurrent_step(d["q"][:, t].contiguous(), d["k"][:, t].contiguous(), d["v"][:, t].contiguous(),
                                     d["g"][:, t].contiguous(), None, pool) for t in range(70)]
    R.check_lin(torch.stack(outs, 1), pool, reference(d))


def test_another_stream_and_graph(K):
    d = make(25, 1, 3000, 2, 2, 128, 128, BF16, init=1)
    want, wfin = K.kda_lin_chunk_fwd(**d)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out, fin = K.kda_lin_chunk_fwd(**d, stream=s)
    s.synchronize()
    assert torch.equal(out, want) and torch.equal(fin, wfin)
    ws = torch.empty(max(1, K.kda_lin_chunk_fwd_workspace_bytes(d["q"], d["v"])), dtype=torch.uint8, device="cuda")
    out.zero_(), fin.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        K.kda_lin_chunk_fwd(**d, out=out, final_state=fin, workspace=ws)
    for _ in range(2):
        ws.fill_(255)      # what the workspace holds on entry does not matter
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(fin, wfin)


def test_many_units(K):
    """More (sequence, head) pairs than SMs, lengths of every kind."""
    lens = [(37 * i) % 211 for i in range(90)]
    cu = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
    d = make(26, 1, sum(lens), 4, 4, 128, 128, BF16)
    out, fin = K.kda_lin_chunk_fwd(**d, cu_seqlens=cu)
    R.check_lin(out, fin, reference(d, cu))


@pytest.mark.parametrize("T,H,dk", [(150, 2, 128), (2500, 2, 64)])
def test_waits_that_give_up(K, T, H, dk):
    """With a bound of zero every wait gives up at once: outputs and states are NaN, the status says so, and the
    next call on the same context is right."""
    d = make(29, 1, T, H, H, dk, 128, BF16, init=1)
    ref = reference(d)
    out = torch.zeros(1, T, H, 128, dtype=BF16, device="cuda")
    fin = torch.zeros(1, H, dk, 128, device="cuda")
    ws = torch.empty(max(1, K.kda_lin_chunk_fwd_workspace_bytes(d["q"], d["v"])), dtype=torch.uint8, device="cuda")
    assert K.kda_device_status() == K.KDA_OK
    args = (d["q"], d["k"], d["v"], d["g"], None, d["initial_state"], None, out, fin, ws)
    K.kda_lin_chunk_fwd_bounded(*args, 0)
    assert K.kda_device_status() == K.KDA_ERR_TIMEOUT
    assert bool(out.isnan().all()) and bool(fin.isnan().all())
    assert K.kda_device_status() == K.KDA_OK
    K.kda_lin_chunk_fwd_bounded(*args, 1 << 20)
    R.check_lin(out, fin, ref)
    assert K.kda_device_status() == K.KDA_OK


@pytest.mark.parametrize("B,H,T", [(5, 32, 1100), (1, 160, 2100), (4, 40, 2085), (9, 24, 3077), (3, 57, 1536), (1, 304, 1100), (16, 19, 1090), (20, 19, 640)])
def test_more_heads_than_one_round(K, B, H, T):
    """(sequence, head) pairs just above a round of one CTA per SM: the ones left over are cut, from the middle of a
    sequence's heads on."""
    d = make(31, B, T, H, H, 64, 64, BF16, decay="head", init=B)
    out, fin = K.kda_lin_chunk_fwd(**d)
    R.check_lin(out, fin, reference(d))


@pytest.mark.parametrize("lens,H", [([2500], 8), ([1000], 3), ([64], 160), ([2200, 1], 8), ([513, 0, 1900], 12), ([30000], 1), ([100, 5000, 7, 90], 5), ([3000, 64], 40), ([40, 9000], 1)])
def test_few_packed_sequences(K, lens, H):
    """One packed sequence is cut like a dense batch's, few by their share."""
    d = make(33, 1, sum(lens), H, H, 128, 64, BF16, decay="head", init=len(lens))
    d["cu_seqlens"] = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
    out, fin = K.kda_lin_chunk_fwd(**d)
    R.check_lin(out, fin, reference({k: x for k, x in d.items() if k != "cu_seqlens"}, d["cu_seqlens"]))


def test_overlapping_launches_share_a_workspace(K):
    """Calls back to back on one stream with one workspace, whose cut and uncut sequences start at different times,
    and the same in a replayed graph: bit for bit what each gives alone."""
    H, mixes = 12, [[4000, 900, 100, 0], [300, 2500, 1200, 1000], [5000, 0, 0, 0]]
    cases = []
    for i, lens in enumerate(mixes):
        d = make(40 + i, 1, 5000, H, H, 128, 128, BF16, decay="head", init=4)
        d["cu_seqlens"] = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
        cases.append((d, *K.kda_lin_chunk_fwd(**d)))
    torch.cuda.synchronize()
    ws = torch.empty(K.kda_lin_chunk_fwd_workspace_bytes(d["q"], d["v"], d["cu_seqlens"]), dtype=torch.uint8, device="cuda")
    got = [K.kda_lin_chunk_fwd(**cases[i % 3][0], workspace=ws) for i in range(24)]
    torch.cuda.synchronize()
    for i, (out, fin) in enumerate(got):
        assert torch.equal(out, cases[i % 3][1]) and torch.equal(fin, cases[i % 3][2])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            got = [K.kda_lin_chunk_fwd(**cases[i][0], workspace=ws) for i in range(3)]
    torch.cuda.synchronize()
    for _ in range(5):
        for out, fin in got:
            out.zero_()
            fin.zero_()
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        for i, (out, fin) in enumerate(got):
            assert torch.equal(out, cases[i][1]) and torch.equal(fin, cases[i][2])


@pytest.mark.parametrize("dt,dk,dv", [(F32, 128, 128), (BF16, 128, 128), (BF16, 64, 128), (BF16, 128, 64)])
@pytest.mark.parametrize("T", [1, 150, 2500])
def test_states_up_to_the_largest_float(K, dt, dk, dv, T):
    """States within 2^-6 of the largest finite value, most of them past what rounds to a finite bf16; q small enough
    that every sum stays finite (sum |q_i| <= sqrt(dk) / 16)."""
    d = make(51, 1, T, 2, 2, dk, dv, dt, decay="none", init=1)
    gen = torch.Generator(device="cuda").manual_seed(52)
    rnd = lambda: torch.rand(d["initial_state"].shape, generator=gen, device="cuda")  # noqa: E731
    d["initial_state"] = torch.finfo(F32).max * (1 - 2.0 ** -6 * rnd()) * torch.where(rnd() < 0.5, -1.0, 1.0)
    d["initial_state"][0, :, 0, :] = torch.finfo(F32).max
    d["q"] = d["q"] / 16
    out, fin = K.kda_lin_chunk_fwd(**d)
    R.check_lin(out, fin, reference(d))
