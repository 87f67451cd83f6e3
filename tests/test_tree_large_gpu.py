"""The calls for branching decode where offsets pass 32 bits: caches and pools of states of more than 2^32 values, a row's outputs of
more than 2^31 vectors of 16 bytes.  In a large pool a call gives the bits that it gives on the same pages in a small one."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K(cuda_device):
    from linear_attention_fwd_gb300 import build, kda
    build.build()
    return kda


@pytest.fixture(autouse=True)
def give_back():
    yield
    torch.cuda.empty_cache()


def test_outputs_past_the_count_are_cleared(K):
    """61 of 64 drafted tokens of (2^21 + 2^18) heads lie past the row's count: 2.3e9 vectors of zeros."""
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("78 GB of queries and outputs")
    T, H, D, m = 64, (1 << 21) + (1 << 18), 128, 3
    gen = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda").bfloat16()  # noqa: E731
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    q = torch.empty(1, T, H, D, dtype=torch.bfloat16, device="cuda")
    q[0, :m] = rnd(m, H, D)
    kc, vc = rnd(2, 8, 1, D), rnd(2, 8, 1, D)
    out, lse = torch.full_like(q, 7.0), torch.full((1, T, H), 7.0, device="cuda")
    K.kda_paged_tree_attention(q, kc, vc, i32([[1, 0]]), i32([9]), i32([[-1, 0, -1] + [0] * (T - 3)]), D ** -0.5, i32([m]), out=out, lse=lse)
    for i in range(m, T):
        assert not out[0, i].any() and bool((lse[0, i] == -float("inf")).all()), i
    k, v = (torch.cat([x[1, :, 0], x[0, :, 0]]).double() for x in (kc, vc))
    for i, path in enumerate(([0], [0, 1], [2])):
        at = list(range(9)) + [9 + j for j in path]
        for heads in (slice(0, 200), slice(H // 2, H // 2 + 200), slice(H - 200, H)):
            p = torch.softmax(q[0, i, heads].double() @ k[at].T * D ** -0.5, 1)
            want = p @ v[at]
            err = (out[0, i, heads].double() - want).abs()
            # half a step of bf16, the weights' 16 bits (as tests/tree_reference.py)
            assert bool((err <= 2.0 ** -8 * want.abs() + 2.0 ** -14 * (p @ v[at].abs())).all()), (i, heads)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def pools(dt, ps, lens, T, Hkv, D, least):
    """(small caches, large caches, small table, large table): the same pages, the large pool's at its end."""
    gen = torch.Generator(device="cuda").manual_seed(ps)
    N, W = len(lens), -(-(max(lens) + T) // ps)
    small = [torch.randn(N * W, ps, Hkv, D, generator=gen, device="cuda").to(dt) for _ in range(2)]
    order = torch.randperm(N * W, generator=gen, device="cuda")
    pages = -(-least // (ps * Hkv * D)) + N * W
    large = [torch.empty(pages, ps, Hkv, D, dtype=dt, device="cuda") for _ in range(2)]
    for x, y in zip(small, large):
        y[pages - N * W:] = x
    return small, large, order.view(N, W).to(torch.int32), (order.view(N, W) + (pages - N * W)).to(torch.int32)


@pytest.mark.parametrize("dt,ps", [(torch.bfloat16, 16), (torch.bfloat16, 7), (torch.float32, 16)])
def test_caches(K, dt, ps):
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("41 GB of caches")
    lens, T, Hkv, D = [700, 33, 0], 20, 8, 128
    small, large, t0, t1 = pools(dt, ps, lens, T, Hkv, D, (1 << 32) + (1 << 28))
    gen = torch.Generator(device="cuda").manual_seed(7)
    q = torch.randn(3, T, 16, D, generator=gen, device="cuda").to(dt)
    parents, num = i32([[-1, 0, 0, 1, 2] + list(range(4, T - 1))] * 3), i32([T, 5, 11])
    for wide in (0, 9000 // ps):      # (in one launch, and shared out)
        got = []
        for caches, table in ((small, t0), (large, t1)):
            table = torch.cat([table, torch.full((3, wide), -1, dtype=torch.int32, device="cuda")], 1)
            got.append(K.kda_paged_tree_attention(q, *caches, table, i32(lens), parents, D ** -0.5, num))
        assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
        assert bool(got[0][0].isfinite().all()) and got[0][0].any()
    was = [x.clone() for x in small]
    new = [K.kda_paged_tree_commit(*caches, table, i32(lens), parents, i32([T - 1, 4, 2]), num) for caches, table in ((small, t0), (large, t1))]
    assert new[0].tolist() == new[1].tolist() and not torch.equal(small[0], was[0])
    end = small[0].shape[0]
    for x, y in zip(small, large):
        assert torch.equal(x, y[-end:])
    first = large[0].shape[0] - end
    K.kda_paged_copy(*small, i32([[0, 1], [end - 1, 2]]))
    K.kda_paged_copy(*large, i32([[first, first + 1], [first + end - 1, first + 2], [-1, 0]]))
    for x, y in zip(small, large):
        assert torch.equal(x, y[-end:])


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_states(K, dt):
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("18 GB of states")
    N, T, H, D, slots = 3, 9, 64, 128, 4200
    gen = torch.Generator(device="cuda").manual_seed(9)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    a = dict(k=unit(rnd(N, T, H, D)).to(dt), v=rnd(N, T, H, D).to(dt), g=-rnd(N, T, H, D).abs().to(dt), beta=torch.sigmoid(rnd(N, T, H)).to(dt))
    q = unit(rnd(N, T, H, D)).to(dt)
    small = rnd(N, H, D, D)
    large = torch.empty(slots, H, D, D, device="cuda")
    assert large.numel() > 1 << 32
    at = i32([slots - 1, 4100, slots - 2])
    large[at.long()] = small
    parents, accepted = i32([[-1, 0, 0, 1, 2, 4, 4, 5, 7]] * N), i32([8, 3, -1])
    one = K.kda_recurrent_tree(q, **a, state=small, parents=parents)
    two = K.kda_recurrent_tree(q, **a, state=large, parents=parents, state_indices=at)
    assert torch.equal(one, two) and bool(one.isfinite().all())
    K.kda_recurrent_tree_commit(**a, state=small, parents=parents, accepted=accepted)
    K.kda_recurrent_tree_commit(**a, state=large, parents=parents, accepted=accepted, state_indices=at)
    assert torch.equal(large[at.long()], small)
