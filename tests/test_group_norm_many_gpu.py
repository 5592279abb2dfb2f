"""qsa_group_norm on the GPU where groups are so many that a thread has two of them, and at the ends of its range, against its
64-bit definition."""
import pytest

torch = pytest.importorskip("torch")
import linear_ref as ref  # noqa: E402
from test_group_norm_gpu import qsa, rand  # noqa: E402,F401

pytestmark = pytest.mark.gpu
LANES = {8: 1, 16: 2, 24: 4, 32: 4, 64: 8, 72: 16, 128: 16, 136: 32, 256: 32}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("size", list(LANES))
def test_two_groups_to_a_thread(qsa, size, dtype):  # noqa: F811
    for n_groups, centred, gated, silu, per_group, w_type in (
            (5, False, True, True, False, dtype), (3, True, True, True, True, torch.float32), (17, True, False, True, True, dtype),
            (1, False, False, False, False, torch.float32), (32, False, True, False, True, dtype)):
        n_tok = 4 * 256 * 2 * 160 // (LANES[size] * n_groups) + 3
        x = rand((n_tok, n_groups, size), dtype, size + n_groups, 0.5, 0.3)
        gate = rand(x.shape, dtype, 7, 2.0) if gated else None
        shape = (n_groups, size) if per_group else (size,)
        w, b = rand(shape, w_type, 8, 0.2, 1.0), rand(shape, w_type, 9, 0.2)
        want, mag = ref.group_norm(x, w, b, gate, 1e-5, centred, silu)
        got = qsa.group_norm(x, w, b, gate=gate, eps=1e-5, centred=centred, activation="silu" if silu else "none")
        ref.check_norm(got, want, mag, dtype)


def test_border_of_the_two(qsa):  # noqa: F811
    """A token less than what two groups to a thread are taken for, as many, one more: each token's results are the same."""
    n = 4 * 256 * 2 * 152 // (16 * 8)
    x, w = rand((n + 1, 8, 128), torch.bfloat16, 1), rand((128,), torch.bfloat16, 2)
    whole = qsa.group_norm(x, w, gate=x)
    for m in (n - 1, n, 1000):
        assert torch.equal(qsa.group_norm(x[:m], w, gate=x[:m]), whole[:m])


@pytest.mark.parametrize("size", [64, 1000, 8192])
def test_range(qsa, size):  # noqa: F811
    for scale in (2.0 ** 55, 2.0 ** -60):            # (normal deviates: 4 standard deviations are 2^57)
        x = rand((50, 2, size), torch.float32, size).clamp(-4, 4).mul(scale).bfloat16()
        for centred in (False, True):
            want, mag = ref.group_norm(x, None, None, None, 0.0, centred, False)
            ref.check_norm(qsa.group_norm(x, eps=0.0, centred=centred), want, mag, x.dtype)
