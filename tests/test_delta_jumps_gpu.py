"""qsa_delta_prompt where gates forget values far larger than the ones behind them: within a chunk of 64 tokens, at its borders, and
where the sequence ends."""
import pytest

torch = pytest.importorskip("torch")
import delta_norms as norms  # noqa: E402
import linear_ref as ref  # noqa: E402
from test_delta_gpu import SCALE, batch, gated, qsa  # noqa: E402,F401

pytestmark = pytest.mark.gpu
FINE = 2.0 ** -17       # of a state's 2-norm, as linear_ref.check_delta has it


def jump(lens, dtype, size, large, gate, silent=(0, 0), seed=3, base=1.0):
    """Values times base, tokens in `large` of each sequence times size, token `gate` forgets what was before it, tokens in `silent`
    have values of 0."""
    inputs, state, slots, _, cu = batch(lens, 1, 2, dtype, seed=seed)
    q, k, v, a, b, a_log, dt = gated(inputs, a_log=3.0)
    v *= base
    a.fill_(-6.0)                                   # exp(-20 softplus(-6 + dt_bias)): mild elsewhere
    for lo in cu[:-1].tolist():
        v[lo + large[0]:lo + large[1]] *= size
        v[lo + silent[0]:lo + silent[1]] = 0
        a[lo + gate] = 80.0
    return (q, k, v, a, b, a_log, dt), state, slots, cu


def outputs(qsa, inputs, state, slots, cu, dtype, chunks_from):  # noqa: F811
    """Outputs of all tokens from the given chunk of each sequence on, as if nothing had been forgotten; the state's error and norm."""
    want, size = norms.delta(*inputs, state, slots, None, cu, 1e-6, SCALE)
    end = ref.delta(*inputs, state, slots, None, cu, 1e-6, SCALE, ref.CHUNK)[1]
    got = qsa.delta_prompt(*inputs, state, slots, None, cu)
    for lo, hi in zip(cu[:-1].tolist(), cu[1:].tolist()):
        lo += 64 * chunks_from
        if hi > lo:
            norms.check(got[lo:hi], want[lo:hi], size[lo:hi], dtype, (lo, hi))
    used = slots.long()
    return (state[used].double() - end[used]).square().sum((-1, -2)).sqrt(), end[used].square().sum((-1, -2)).sqrt(), got, want


BIG = [(torch.bfloat16, 2.0 ** 20), (torch.bfloat16, 2.0 ** 50), (torch.bfloat16, 2.0 ** 100), (torch.float16, 2.0 ** 12)]


@pytest.mark.parametrize("dtype,size", BIG)
@pytest.mark.parametrize("lens", [[64 * 3 + 20], [150, 90, 200], [64 * 40]], ids=["one", "three", "segments"])
def test_forgotten_at_a_chunk_s_border(qsa, lens, dtype, size):  # noqa: F811
    """By its first token, or by the one before with nothing behind it in its own chunk: the next one knows nothing of it."""
    for gate, silent in ((64, (0, 0)), (63, (63, 64)), (40, (40, 64))):
        inputs, state, slots, cu = jump(lens, dtype, size, (0, gate), gate, silent)
        err, norm, _, _ = outputs(qsa, inputs, state, slots, cu, dtype, 1)
        assert bool((err <= FINE * norm).all()), (gate, (err / norm).max().item())


@pytest.mark.parametrize("dtype,size", BIG)
def test_a_state_forgotten_by_the_first_token(qsa, dtype, size):  # noqa: F811
    for lens in ([40], [200, 70], [64 * 34]):
        inputs, state, slots, cu = jump(lens, dtype, 1.0, (0, 0), 0)
        state = state * size
        err, norm, _, _ = outputs(qsa, inputs, state, slots, cu, dtype, 0)
        assert bool((err <= FINE * norm).all()), (lens, (err / norm).max().item())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("lens", [[64], [61], [128 + 50, 64]], ids=["64", "61", "two"])
@pytest.mark.parametrize("size", [2.0 ** 8, 2.0 ** 12, 2.0 ** 16])
def test_forgotten_within_a_chunk(qsa, lens, dtype, size):  # noqa: F811
    """30 large values, a gate, ordinary ones: the state at the sequence's end, and the outputs behind the gate."""
    base = 1.0 if dtype is torch.bfloat16 else 2.0 ** -4               # (FP16 ends at 2^16)
    inputs, state, slots, cu = jump(lens, dtype, size, (0, 30), 30, base=base)
    err, norm, got, want = outputs(qsa, inputs, state, slots, cu, dtype, 9)
    assert bool((err <= FINE * norm).all()), (err / norm).max().item()
    for lo in cu[:-1].tolist():
        d = (got[lo + 30:lo + 61].double() - want[lo + 30:lo + 61]).square().sum((0, 2)).sqrt()
        size_of = want[lo + 30:lo + 61].square().sum((0, 2)).sqrt()
        # the output's own rounding, and 2^-30 of the large ones
        assert bool((d <= (torch.finfo(dtype).eps / 2 + size * 2.0 ** -30 * 64) * size_of).all()), (d / size_of).max().item()


@pytest.mark.parametrize("size", [2.0 ** 24, 2.0 ** 30, 2.0 ** 40])
def test_what_forgotten_values_leave(qsa, size):  # noqa: F811
    """Far larger ones: errors of no more than 2^-30 of them in the outputs of their chunk, of 2^-34 in the state."""
    inputs, state, slots, cu = jump([64, 50], torch.bfloat16, size, (0, 30), 30)
    end = ref.delta(*inputs, state, slots, None, cu, 1e-6, SCALE, ref.CHUNK)[1]
    want, _ = norms.delta(*inputs, state, slots, None, cu, 1e-6, SCALE)
    got = qsa.delta_prompt(*inputs, state, slots, None, cu)
    for s, lo in zip(slots.long().tolist(), cu[:-1].tolist()):
        top = inputs[2][lo:lo + 30].double().abs().amax(0)                        # of each value dim
        row = (state[s].double() - end[s]).square().sum(-1).sqrt()
        assert bool((row <= FINE * end[s].square().sum(-1).sqrt() + 2.0 ** -34 * top).all())
        off = (got[lo + 30:lo + 50].double() - want[lo + 30:lo + 50]).abs()
        assert bool((off <= want[lo + 30:lo + 50].abs() * 2.0 ** -8 + 2.0 ** -30 * top).all())


@pytest.mark.parametrize("size", [2.0 ** 12, 2.0 ** 24])
def test_what_comes_later(qsa, size):  # noqa: F811
    """Large values at a chunk's end: the outputs before them, within the same errors; the chunk before is as it was."""
    inputs, state, slots, _, cu = batch([128], 1, 2, torch.bfloat16, seed=6)
    v = inputs[2].clone()
    v[120:] *= size
    inputs = (*inputs[:2], v, *inputs[3:])
    want, size_of = norms.delta(*inputs, state, slots, None, cu, 1e-6, SCALE)
    got = qsa.delta_prompt(*inputs, state, slots, None, cu)
    norms.check(got[:64], want[:64], size_of[:64], torch.bfloat16)
    top = v[64:].double().abs().amax(0)
    off = (got[64:120].double() - want[64:120]).abs()
    assert bool((off <= want[64:120].abs() * 2.0 ** -8 * 1.01 + 2.0 ** -17 * size_of[64:120] + 2.0 ** -30 * top).all())


@pytest.mark.parametrize("size", [2.0 ** 30, 2.0 ** 50, 2.0 ** 100])
@pytest.mark.parametrize("lens", [[250], [64 * 42]], ids=["chunks", "segments"])
def test_forgotten_within_a_chunk_then_everything(qsa, lens, size):  # noqa: F811
    """What is far below a chunk's largest is rounded, to zero at worst, never to more than twice itself: all stays finite and of its
    size, and from where the gates forget that, too, all is right again."""
    inputs, state, slots, cu = jump(lens, torch.bfloat16, size, (0, 30), 30)
    inputs[3][128] = 80.0
    want, size_of = norms.delta(*inputs, state, slots, None, cu, 1e-6, SCALE)
    end = ref.delta(*inputs, state, slots, None, cu, 1e-6, SCALE, ref.CHUNK)[1]
    got = qsa.delta_prompt(*inputs, state, slots, None, cu)
    assert bool(torch.isfinite(got).all()) and bool(torch.isfinite(state).all())
    assert bool((got[30:128].double().abs().amax(0) <= 4 * want[30:128].abs().amax(0) + SCALE * 2.0 ** -7).all())
    norms.check(got[128:], want[128:], size_of[128:], torch.bfloat16)
    s = slots.long()
    assert float((state[s] - end[s]).square().sum().sqrt()) <= FINE * float(end[s].square().sum().sqrt())
