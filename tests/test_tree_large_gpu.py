"""Attention of a draft where a row's outputs are more than 2^31 vectors of 16 bytes."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K(cuda_device):
    from linear_attention_fwd_gb300 import build, kda
    build.build()
    return kda


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
