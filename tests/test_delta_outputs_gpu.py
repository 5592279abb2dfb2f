"""qsa_delta_prompt's and qsa_delta_step's outputs against the rule in 64 bits by 2-norms: what enters them has the bits of
32-bit sums, whichever way a sequence goes (token by token, by chunks, in segments) and whatever the type."""
import pytest

torch = pytest.importorskip("torch")
import delta_norms as norms  # noqa: E402
from test_delta_gpu import CASES, SCALE, batch, cu_of, gated, qsa  # noqa: E402,F401

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16]


def check(qsa, inputs, state, slots, old, cu, dtype, what="", eps=1e-6):  # noqa: F811
    want, size = norms.delta(*inputs, state, slots, old, cu, eps, SCALE)
    got = qsa.delta_prompt(*inputs, state, slots, old, cu, eps=eps)
    # each sequence by itself: a short one's errors are not to be lost among a long one's
    for lo, hi in zip(cu[:-1].tolist(), cu[1:].tolist()):
        if hi > lo:
            norms.check(got[lo:hi], want[lo:hi], size[lo:hi], dtype, (what, lo, hi))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lens,n_k,n_v", [([61], 2, 4), ([300, 64, 129], 1, 3), ([700], 1, 2), ([32, 20], 1, 2), ([1100], 1, 1),
                                          ([2200], 1, 2), ([4200, 300], 1, 2), ([2047, 33], 2, 4)])
def test_ways(qsa, lens, n_k, n_v, dtype):  # noqa: F811
    check(qsa, *batch(lens, n_k, n_v, dtype, seed=len(lens) + n_v), dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("name", ["no decay", "strong decay", "full write", "one key no decay", "opposite keys", "uneven values", "values that jump"])
def test_gates_and_values(qsa, name, dtype):  # noqa: F811
    for lens in ([140, 20], [2180]):
        inputs, state, slots, _, cu = batch(lens, 1, 2, dtype, seed=4)
        check(qsa, gated(inputs, **CASES[name]), state, slots, None, cu, dtype, name)


@pytest.mark.parametrize("dtype", TYPES)
def test_single_tokens(qsa, dtype):  # noqa: F811
    inputs, state, slots, old, cu = batch([1] * 60, 2, 4, dtype, seed=2)
    want, size = norms.delta(*inputs, state, slots, old, cu, 1e-6, SCALE)
    norms.check(qsa.delta_step(*inputs, state, slots, old), want, size, dtype)
    assert cu_of([1] * 60).equal(cu)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lens", [[150], [2200]], ids=["chunks", "segments"])
def test_outputs_small_beside_their_state(qsa, lens, dtype):  # noqa: F811
    """Queries nearly orthogonal to everything that has been written: the sums cancel, what remains has its own bits."""
    inputs, state, slots, _, cu = batch(lens, 1, 2, dtype, seed=9)
    q, k, v, *rest = inputs
    far = torch.zeros(128, device="cuda")
    far[:64] = 1
    k, q = k * far.to(dtype), (q * (1 - far) + q * far * 2.0 ** -6).to(dtype)
    state = state * far
    check(qsa, (q, k, v, *rest), state, slots, None, cu, dtype)
