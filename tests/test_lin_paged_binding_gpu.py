"""What the binding of the linear-attention and paged-cache calls refuses, and that a refused call leaves
everything as it was."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def K(cuda_device):
    from linear_attention_fwd_gb300 import build, kda
    build.build()
    return kda


def z(*s, dt=BF16):
    return torch.zeros(*s, dtype=dt, device="cuda")


def chunk_args():
    return dict(q=z(1, 8, 2, 64), k=z(1, 8, 2, 64), v=z(1, 8, 4, 128), g=z(1, 8, 4, dt=torch.float32), head_g=z(4, dt=torch.float32),
                initial_state=z(1, 4, 64, 128, dt=torch.float32), out=z(1, 8, 4, 128), final_state=z(1, 4, 64, 128, dt=torch.float32))


@pytest.mark.parametrize("name,value,error", [
    ("q", lambda t: t.float(), TypeError), ("k", lambda t: t.float(), TypeError), ("v", lambda t: t[..., :64], ValueError),
    ("k", lambda t: t[:, :7], ValueError), ("k", lambda t: t.cpu(), ValueError), ("g", lambda t: t.to(BF16), TypeError),
    ("g", lambda t: t[:, :, :2], ValueError), ("head_g", lambda t: t[:3], ValueError), ("initial_state", lambda t: t.transpose(2, 3), ValueError),
    ("initial_state", lambda t: t.transpose(2, 3).contiguous(), ValueError), ("out", lambda t: t.float(), TypeError),
    ("final_state", lambda t: t[:, :2], ValueError), ("q", lambda t: t[0], ValueError), ("q", lambda t: None, ValueError), ("q", lambda t: 3, TypeError),
    ("q", lambda t: t.transpose(1, 2), ValueError), ("q", lambda t: t.to(torch.float16), TypeError),
])
def test_chunk_refusals(K, name, value, error):
    a = chunk_args()
    a["out"] += 5
    out = a["out"]
    a[name] = value(a[name])
    # (q sets the type, device and sizes that the others are held to, so that they may be named for it)
    with pytest.raises(error, match=None if name == "q" else name):
        K.kda_lin_chunk_fwd(**a)
    assert bool((out == 5).all())


def test_status_errors_come_through(K):
    a = chunk_args()
    a["q"], a["k"] = z(1, 8, 3, 64), z(1, 8, 3, 64)      # heads not a multiple of q and k's
    with pytest.raises(K.KdaError) as e:
        K.kda_lin_chunk_fwd(**a)
    assert e.value.status == K.KDA_ERR_SHAPE and "kda_lin_chunk_fwd" in str(e.value)
    with pytest.raises(K.KdaError) as e:                  # head size 32
        K.kda_lin_recurrent_step(z(1, 1, 32), z(1, 1, 32), z(1, 1, 64), None, None, z(1, 1, 32, 64, dt=torch.float32))
    assert e.value.status == K.KDA_ERR_UNSUPPORTED
    big = z(1, 2000, 1, 128)
    with pytest.raises(K.KdaError) as e:
        K.kda_lin_chunk_fwd(big, big, big, workspace=z(16, dt=torch.uint8))
    assert e.value.status == K.KDA_ERR_WORKSPACE


def test_step_and_paged_refusals(K):
    i32 = torch.int32
    st = z(3, 2, 64, 64, dt=torch.float32)
    x = z(2, 2, 64)
    with pytest.raises(ValueError, match="state_indices"):
        K.kda_lin_recurrent_step(x, x, x, None, None, st, z(3, dt=i32))
    with pytest.raises(TypeError, match="state_indices"):
        K.kda_lin_recurrent_step(x, x, x, None, None, st, z(2, dt=torch.int64))
    with pytest.raises(ValueError, match="state"):
        K.kda_lin_recurrent_step(x, x, x, None, None, st[:, :1].contiguous())
    kc, table, lens = z(4, 16, 2, 64), z(2, 3, dt=i32), z(2, dt=i32)
    with pytest.raises(ValueError, match="block_table"):
        K.kda_paged_attention(z(3, 4, 64), kc, kc, table, z(3, dt=i32), 1.0)
    with pytest.raises(ValueError, match="v_cache"):
        K.kda_paged_attention(z(2, 4, 64), kc, kc[:3], table, lens, 1.0)
    with pytest.raises(ValueError, match="q"):
        K.kda_paged_attention(z(2, 4, 128), kc, kc, table, lens, 1.0)
    with pytest.raises(TypeError):
        K.kda_paged_attention(z(2, 4, 64), kc, kc, table, lens, "one")
    with pytest.raises(K.KdaError):
        K.kda_paged_attention(z(2, 3, 64), kc, kc, table, lens, 1.0)        # 3 query heads on 2
    with pytest.raises(ValueError, match="cu_seqlens"):
        K.kda_paged_append(z(5, 2, 64), z(5, 2, 64), kc, kc, table, lens, z(2, dt=i32))
    with pytest.raises(K.KdaError):
        K.kda_paged_append(z(5, 2, 64), z(5, 2, 64), kc, kc, table, lens)   # one token per row: 5 tokens, 2 rows
    with pytest.raises(TypeError, match="k_cache"):
        K.kda_paged_append(z(2, 2, 64), z(2, 2, 64), kc.float(), kc, table, lens)


def test_every_form_of_stream_argument(K):
    x = torch.randn(2, 2, 64, device="cuda").to(BF16)
    st = torch.randn(2, 2, 64, 64, device="cuda")
    want = K.kda_lin_recurrent_step(x, x, x, None, None, st.clone())
    s = torch.cuda.Stream()
    for form in (s, s.cuda_stream, torch.cuda.ExternalStream(s.cuda_stream)):
        pool = st.clone()
        s.wait_stream(torch.cuda.current_stream())
        got = K.kda_lin_recurrent_step(x, x, x, None, None, pool, stream=form)
        s.synchronize()
        assert torch.equal(got, want)
    with torch.cuda.stream(s):
        s.wait_stream(torch.cuda.default_stream())
        got = K.kda_lin_recurrent_step(x, x, x, None, None, st.clone())
    s.synchronize()
    assert torch.equal(got, want)


def test_the_library_can_be_switched(K):
    """use_library rebinds the calls to another build of the library (and back)."""
    x = torch.randn(1, 3, 2, 64, device="cuda").to(BF16)
    want, _ = K.kda_lin_chunk_fwd(x, x, x)
    path = K.LIB_PATH
    from linear_attention_fwd_gb300 import build
    debug = build.build(debug=True)
    try:
        K.use_library(debug)
        assert K.kda_debug_checks() != 0
        got, _ = K.kda_lin_chunk_fwd(x, x, x)
    finally:
        K.use_library(path)
    assert torch.equal(got, want) and K.kda_debug_checks() == 0


def test_flags_without_a_truth_value_are_refused(K):
    """A flag whose truth cannot be asked raises what asking raises, and nothing is written."""
    both = torch.ones(2)
    a = chunk_args()
    a["out"] += 5
    a["final_state"] = None
    with pytest.raises(RuntimeError, match="ambiguous"):
        K.kda_lin_chunk_fwd(**a, output_final_state=both)
    kc, table, lens = z(4, 16, 2, 64), z(2, 3, dt=torch.int32), z(2, dt=torch.int32)
    out = z(2, 4, 64) + 5
    with pytest.raises(RuntimeError, match="ambiguous"):
        K.kda_paged_attention(z(2, 4, 64), kc, kc, table, lens, 1.0, out=out, output_lse=both)
    torch.cuda.synchronize()
    assert bool((a["out"] == 5).all()) and bool((out == 5).all())
