"""The calls for branching decode side by side on several streams, many at once: every result is, bit for bit, that of the call by
itself."""
import pytest
import torch

from tests import tree_reference as R

pytestmark = pytest.mark.gpu
F32, BF16, I32 = torch.float32, torch.bfloat16, torch.int32


@pytest.fixture(scope="module")
def K(cuda_device):
    from linear_attention_fwd_gb300 import build, kda
    build.build()
    return kda


def i32(x):
    return torch.tensor(x, dtype=I32, device="cuda")


def attention(K, seed, lens, T, Hq, Hkv, d, ps, dt):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda").to(dt)  # noqa: E731
    N, width = len(lens), -(-(max(lens) + T) // ps)
    kc, vc, q = rnd(N * width, ps, Hkv, d), rnd(N * width, ps, Hkv, d), rnd(N, T, Hq, d)
    table = torch.randperm(N * width, generator=gen, device="cuda").view(N, width).to(I32)
    num = [1 + (n * 7 + seed) % T for n in range(N)]
    _, parents = R.drafts(seed, N, T, num=num)
    lens, num = i32(lens), i32(num)
    return lambda: K.kda_paged_tree_attention(q, kc, vc, table, lens, parents, d ** -0.5, num)


def states(K, seed, N, T, H, dt):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    a = dict(k=unit(rnd(N, T, H, 128)).to(dt), v=rnd(N, T, H, 128).to(dt), g=-torch.rand(N, T, H, 128, generator=gen, device="cuda").to(dt),
             beta=torch.sigmoid(rnd(N, T, H)).to(dt))
    q, state = unit(rnd(N, T, H, 128)).to(dt), rnd(N, H, 128, 128)
    rows, parents = R.drafts(seed, N, T)
    accepted = i32([(n * 5) % T for n in range(N)])

    def both():
        new = state.clone()
        out = K.kda_recurrent_tree(q, **a, state=new, parents=parents)
        K.kda_recurrent_tree_commit(**a, state=new, parents=parents, accepted=accepted)
        return out, new
    return both


def pages(K, N, W, ps):
    table = torch.arange(N * W, dtype=I32, device="cuda").view(N, W).clone()
    table[1::2, : W // 2] = table[::2, : W // 2][: N // 2]
    refs = torch.bincount(table.flatten().long(), minlength=2 * N * W).to(I32)
    lens = i32([(n * 37) % (W * ps) for n in range(N)])
    src = i32([n if n % 3 else (n * 5) % N for n in range(N)])
    more = torch.full((N,), 2 * ps, dtype=I32, device="cuda")
    first = torch.arange(2 * N * W * ps * 64, device="cuda").float().view(2 * N * W, ps, 1, 64)

    def run():
        kc, vc = first.clone(), first.flip(0).clone()
        t, x, r, copies, short = K.kda_paged_fork(table, lens, refs, src, more, page_size=ps)
        K.kda_paged_copy(kc, vc, copies)
        t2, r2, c2 = K.kda_paged_compact(t, r)
        K.kda_paged_copy(kc, vc, c2)
        return t, x, r, copies, short, t2, r2, c2, kc, vc
    return run


def test_side_by_side(K):
    works = [attention(K, 1, [3000, 17, 900, 0, 5000], 16, 16, 4, 128, 16, BF16), attention(K, 2, [3000, 17, 900, 0, 5000], 16, 16, 4, 128, 7, BF16),
             attention(K, 3, [300, 5], 8, 8, 2, 128, 16, BF16), attention(K, 4, [700, 40, 0], 5, 8, 2, 64, 16, F32),
             states(K, 5, 8, 12, 16, BF16), states(K, 6, 4, 40, 8, F32), pages(K, 40, 12, 4), pages(K, 3, 300, 2)]
    alone = [w() for w in works]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in works]
    for turn in range(12):
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
        got = []
        for n in range(len(works)):
            at = (n + turn) % len(works)
            with torch.cuda.stream(streams[n]):
                got.append((at, [works[at]() for _ in range(3)]))
        torch.cuda.synchronize()
        for at, results in got:
            for r in results:
                for x, y in zip(r, alone[at]):
                    assert torch.equal(x, y), (turn, at)
