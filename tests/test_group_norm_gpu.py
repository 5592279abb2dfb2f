"""qsa_group_norm on the GPU against its 64-bit definition."""
import pytest

torch = pytest.importorskip("torch")
import linear_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qsa():
    from sparse_selected_cell_gb300 import qsa as q
    if not torch.cuda.is_available():
        pytest.fail("CUDA GPU required")
    q.lib()
    return q


def rand(shape, dtype, seed, scale=1.0, shift=0.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale + shift).to(dtype).cuda()


SIZES = [8, 16, 24, 32, 64, 72, 128, 136, 256, 264, 504, 512, 1000, 1024, 1032, 2048, 4096, 4104, 8192]


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_sizes(qsa, size, dtype):
    for n_tok, n_groups, centred, gated, silu, per_group, w_type in (
            (1, 1, False, True, True, False, dtype), (5, 3, True, True, True, True, torch.float32),
            (67, 2, True, False, True, False, dtype), (3, 32, False, False, False, True, dtype),
            (9, 5, False, True, False, False, torch.float32)):
        x = rand((n_tok, n_groups, size), dtype, size + n_tok, 0.5, 0.3)
        gate = rand(x.shape, dtype, 7, 2.0) if gated else None
        shape = (n_groups, size) if per_group else (size,)
        w, b = rand(shape, w_type, 8, 0.2, 1.0), rand(shape, w_type, 9, 0.2)
        want, mag = ref.group_norm(x, w, b, gate, 1e-5, centred, silu)
        got = qsa.group_norm(x, w, b, gate=gate, eps=1e-5, centred=centred, activation="silu" if silu else "none")
        ref.check_norm(got, want, mag, dtype)


def test_defaults_and_missing_weights(qsa):
    x, gate = rand((33, 4, 128), torch.bfloat16, 1), rand((33, 4, 128), torch.bfloat16, 2)
    w, b = rand((128,), torch.bfloat16, 3), rand((128,), torch.bfloat16, 4)
    for args, kw, ref_args in (((), {}, (None, None, None, 1e-6, False, False)),
                               ((w,), dict(gate=gate), (w, None, gate, 1e-6, False, True)),
                               ((None, b), dict(centred=True), (None, b, None, 1e-6, True, False))):
        want, mag = ref.group_norm(x, *ref_args)
        ref.check_norm(qsa.group_norm(x, *args, **kw), want, mag, x.dtype)


def test_strides_and_in_place(qsa):
    """Slices of wider rows; written over x, and over the gate; neighbours untouched."""
    wide = rand((50, 3 * 256 + 64), torch.bfloat16, 1)
    x, gate = wide[:, 64:64 + 256].view(50, 2, 128), wide[:, 320:576].view(50, 2, 128)
    w = rand((128,), torch.bfloat16, 3)
    want, mag = ref.group_norm(x, w, None, gate, 1e-6, False, True)
    got = qsa.group_norm(x, w, gate=gate)
    ref.check_norm(got, want, mag, x.dtype)
    for target in (x, gate):
        copy = wide.clone()
        cx, cg = copy[:, 64:320].view(50, 2, 128), copy[:, 320:576].view(50, 2, 128)
        out = cx if target is x else cg
        assert qsa.group_norm(cx, w, gate=cg, out=out) is out and torch.equal(out, got)
        out.copy_(target)
        assert torch.equal(copy, wide)


def test_small_large_and_odd_values(qsa):
    """Zeros (eps alone), magnitudes at both ends of FP16, gates far out; an infinity stays in its group."""
    x = rand((6, 4, 64), torch.float16, 1)
    x[0] = 0
    x[1] *= 2.0 ** -14
    x[2] = x[2].sign() * 60000
    gate = rand(x.shape, torch.float16, 2)
    gate[3], gate[4] = 60000, -60000
    want, mag = ref.group_norm(x, None, None, gate, 1e-6, False, True)
    fine = want.abs() < 65000
    got = qsa.group_norm(x, gate=gate)
    ref.check_norm(torch.where(fine, got, 0), torch.where(fine, want, 0), mag, x.dtype)
    assert bool((got[0] == 0).all())
    x[5, 1, 3] = float("inf")
    again = qsa.group_norm(x, gate=gate)
    assert torch.equal(again[:5], got[:5]) and torch.equal(again[5, 2:], got[5, 2:]) and torch.equal(again[5, 0], got[5, 0])


def test_large_mean(qsa):
    """Centred: the squares are of what is left after the mean, so a mean of 2^8 times the spread costs no bits."""
    x = (rand((40, 2, 128), torch.float32, 1) + 256).to(torch.float16)
    want, mag = ref.group_norm(x, None, None, None, 1e-6, True, False)
    ref.check_norm(qsa.group_norm(x, centred=True), want, mag, x.dtype)


def test_offsets_past_32_bits(qsa):
    n_tok = 300
    x = torch.zeros((n_tok, 8_000_000), dtype=torch.bfloat16, device="cuda")[:, :256].view(n_tok, 2, 128)
    x.copy_(rand((n_tok, 2, 128), torch.float32, 1))
    want, mag = ref.group_norm(x, None, None, None, 1e-6, False, False)
    ref.check_norm(qsa.group_norm(x), want, mag, x.dtype)


def test_refusals(qsa):
    x = rand((4, 2, 128), torch.bfloat16, 1)
    w = rand((128,), torch.bfloat16, 1)
    for args, kw in (((x.float(),), {}), ((x.cpu(),), {}), ((x[0],), {}), ((x.transpose(1, 2),), {}), ((x[..., :100],), {}),
                     ((x, w.half()), {}), ((x, w[:64]), {}), ((x, w, w.float()), {}), ((x, w.repeat(2).view(2, 128), w), {}),
                     ((x,), dict(gate=x.half())), ((x,), dict(gate=x[:2])), ((x,), dict(out=x[:2])), ((x,), dict(eps=-1.0)),
                     ((x,), dict(activation="relu")), ((rand((2, 1, 8200), torch.bfloat16, 1),), {})):
        with pytest.raises((TypeError, ValueError, RuntimeError)):
            qsa.group_norm(*args, **kw)
    assert qsa.group_norm(x[:0]).shape == (0, 2, 128)
