"""The debug build's input checks of the calls for a drafted tree through KDA states: log decays at most 0, of any size, of the
tokens that a call uses and no others."""
import pytest
import torch

pytestmark = pytest.mark.gpu
F32, BF16, I32 = torch.float32, torch.bfloat16, torch.int32
PARENTS = [[-1, 0, 0, 1, 2], [-1, -1, 1, 2, 2], [-1, 0, 1, 2, 3], [-1, 0, 1, 2, 3]]
ACCEPTED, PATHS = [4, 2, -1, 3], [{0, 2, 4}, {1, 2}, set(), {0, 1, 2, 3}]


@pytest.fixture(scope="module")
def K(cuda_device):
    from linear_attention_fwd_gb300 import build, kda
    release = build.build()
    kda.use_library(build.build(debug=True))
    assert kda.kda_debug_checks() & 1
    yield kda
    kda.use_library(release)


def i32(x):
    return torch.tensor(x, dtype=I32, device="cuda")


def status(K, call, g, num, idx):
    gen = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    N, T, H = g.shape[:3]
    dt = g.dtype
    a = dict(k=rnd(N, T, H, 64).to(dt), v=rnd(N, T, H, 128).to(dt), g=g, beta=torch.sigmoid(rnd(N, T, H)).to(dt), state=rnd(7, H, 64, 128))
    kw = dict(parents=i32(PARENTS), state_indices=i32(idx), num_tokens=None if num is None else i32(num))
    if call == "verify":
        K.kda_recurrent_tree(rnd(N, T, H, 64).to(dt), **a, **kw)
    else:
        K.kda_recurrent_tree_commit(**a, accepted=i32(ACCEPTED), **kw)
    return K.kda_device_status()


def decays(dt):
    g = torch.full((4, 5, 3, 64), -0.5, device="cuda").to(dt)
    g[0, 0, 1, ::2] = -40.0
    g[0, 2, 2] = -float("inf")
    g[1, 1, 0, 63] = -1e30
    g[1, 2, 0, 5] = 0.0
    return g


@pytest.mark.parametrize("call", ["verify", "commit"])
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("num", [None, [5, 3, 5, 9]])
def test_decays_of_any_size_pass(K, call, dt, num):
    assert status(K, call, decays(dt), num, [3, 0, 6, 1]) == K.KDA_OK


@pytest.mark.parametrize("call", ["verify", "commit"])
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("num", [None, [5, 3, 5, 4]])
@pytest.mark.parametrize("bad", [0.25, float("nan"), float("inf")])
def test_only_what_is_used_is_checked(K, call, dt, num, bad):
    """Row 2 accepts nothing, row 3's slot lies outside the pool."""
    idx = [3, 0, 6, 7]
    for n in range(4):
        for i in range(5):
            count = 5 if num is None else num[n]
            used = idx[n] < 7 and (i < count if call == "verify" else i in PATHS[n] and ACCEPTED[n] < count)
            g = decays(dt)
            g[n, i, 2, 63] = bad
            assert status(K, call, g, num, idx) == (K.KDA_ERR_INPUT if used else K.KDA_OK), (n, i)
            assert K.kda_device_status() == K.KDA_OK
