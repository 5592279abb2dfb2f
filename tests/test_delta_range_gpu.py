"""The ranges that qsa_delta_prompt and qsa_delta_step are documented for: values and states, keys and queries far out, tiny
rows against eps, and what is no number where it may not spread."""
import pytest

torch = pytest.importorskip("torch")
import linear_ref as ref  # noqa: E402
from test_delta_gpu import SCALE, batch, gated, qsa  # noqa: E402,F401

pytestmark = pytest.mark.gpu


def scaled_back(want, got, state, size):
    out, pool, big, off, end = want
    return got.double() / size, state.double() / size, (out / size, pool / size, big / size, off / size, end / size)


@pytest.mark.parametrize("size", [2.0 ** 112, 2.0 ** 60, 2.0 ** -60, 2.0 ** -70, 2.0 ** -84])
@pytest.mark.parametrize("lens", [[200, 9, 90], [2200]], ids=["three", "segments"])
def test_values_and_states(qsa, size, lens):  # noqa: F811
    """Of 3 to 5 standard deviations at most, times size: within 2^-90 and 2^120 but for a few small ones."""
    inputs, state, slots, old, cu = batch(lens, 1, 2, torch.bfloat16, seed=8)
    inputs = (*inputs[:2], inputs[2] * size, *inputs[3:])
    state = state * size
    want = ref.delta(*inputs, state, slots, old, cu, 1e-6, SCALE, ref.CHUNK)
    got = qsa.delta_prompt(*inputs, state, slots, old, cu)
    out, pool, scaled = scaled_back(want, got, state, size)
    ref.check_delta(out, pool, scaled, SCALE, torch.bfloat16, True, slots)


@pytest.mark.parametrize("size", [2.0 ** 56, 2.0 ** -60])
def test_keys_and_queries(qsa, size):  # noqa: F811
    inputs, state, slots, old, cu = batch([130, 9, 40], 1, 2, torch.bfloat16, seed=2)
    inputs = (inputs[0] * size, inputs[1] * size, *inputs[2:])
    want = ref.delta(*inputs, state, slots, old, cu, 0.0, SCALE, ref.CHUNK)
    got = qsa.delta_prompt(*inputs, state, slots, old, cu, eps=0.0)
    ref.check_delta(got, state, want, SCALE, torch.bfloat16, True, slots)


def test_rows_that_eps_outweighs(qsa):  # noqa: F811
    """Keys and queries ever further below sqrt(eps), down to zeros: nothing but finite, small outputs, and the formula's."""
    inputs, state, slots, old, cu = batch([150, 20], 1, 2, torch.bfloat16, seed=5)
    fall = torch.exp2(-torch.arange(170, device="cuda", dtype=torch.float32) * 0.75)[:, None, None]
    q, k = ((x.float() * fall).bfloat16() for x in inputs[:2])
    q[140:150], k[145:150], k[10] = 0, 0, 0
    inputs = gated((q, k, *inputs[2:]), a_log=float("-inf"))
    want = ref.delta(*inputs, state, slots, old, cu, 1e-6, SCALE, ref.CHUNK)
    got = qsa.delta_prompt(*inputs, state, slots, old, cu)
    assert bool(torch.isfinite(got).all())
    ref.check_delta(got, state, want, SCALE, torch.bfloat16, True, slots)


def test_numbers_stay_in_their_value_dim_and_head(qsa):  # noqa: F811
    """One value that is no number, one that is infinite: other value dims, the other head and the tokens before keep their bits."""
    for lens in ([300], [20], [2300]):
        inputs, state, slots, old, cu = batch(lens, 1, 2, torch.bfloat16, seed=6)
        clean = state.clone()
        want = qsa.delta_prompt(*inputs, clean, slots, old, cu)
        v = inputs[2].clone()
        v[lens[0] // 2, 0, 5], v[lens[0] // 2 + 1, 0, 77] = float("nan"), float("inf")
        got = qsa.delta_prompt(*inputs[:2], v, *inputs[3:], state, slots, old, cu)
        keep = torch.ones(128, dtype=torch.bool, device="cuda")
        keep[5] = keep[77] = False
        assert torch.equal(got[:, 1], want[:, 1]) and torch.equal(got[:, 0][:, keep], want[:, 0][:, keep])
        s = int(slots[0])
        assert torch.equal(state[s, 1], clean[s, 1]) and torch.equal(state[s, 0][keep], clean[s, 0][keep])
        first = lens[0] // 2 // 64 * 64 if lens[0] > 32 else lens[0] // 2
        assert torch.equal(got[:first], want[:first])
        assert bool(torch.isnan(state[s, 0, 5]).all()) and not bool(torch.isfinite(state[s, 0, 77]).any())


def test_no_gate_leaves_nothing(qsa):  # noqa: F811
    """beta of zero and no decay: the state stays bit for bit, but where segments are put together by products of pairs of FP16
    (2^-22 of an element each, of 128 products one that is not zero)."""
    for lens in ([64, 20, 150], [1, 1, 1], [2200]):
        inputs, state, slots, _, cu = batch(lens, 1, 2, torch.bfloat16, seed=1)
        inputs = gated(inputs, b=float("-inf"), a_log=float("-inf"))
        given = state.clone()
        qsa.delta_prompt(*inputs, state, slots, None, cu)
        assert torch.equal(state, given) if lens != [2200] else torch.allclose(state, given, rtol=2 ** -20, atol=2 ** -24)
        first = [x[:len(lens)] for x in inputs[:5]] + list(inputs[5:])
        state = given.clone()
        qsa.delta_step(*first, state, slots)
        assert torch.equal(state, given)
