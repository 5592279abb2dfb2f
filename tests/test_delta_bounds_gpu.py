"""qsa_delta_prompt with bounds that fall: reported, and nothing that an earlier call left in the workspace comes through."""
import pytest

torch = pytest.importorskip("torch")
import linear_ref as ref  # noqa: E402
from test_delta_gpu import BAD_LEN, SCALE, batch, i32, qsa  # noqa: E402,F401

pytestmark = pytest.mark.gpu
FALLING = [[300, 0, 300, 300], [0, 250, 10, 300], [0, 2 ** 31 - 1, -2 ** 31, 60], [300, 200, 100, 0], [0, 300, 0, 300], [0, 100, 99, 300],
           [200, 0, 200, 300], [0, 299, 298, 64]]


def call(qsa, cu, fill, n_tok=300, n_seq=3):  # noqa: F811
    inputs, state, slots, old, _ = batch([n_tok] + [0] * (n_seq - 1), 1, 2, torch.bfloat16, seed=1)
    ws = torch.full((qsa.delta_prompt_workspace_bytes(n_tok, n_seq, 1, 2),), fill, dtype=torch.uint8, device="cuda")
    out, status = torch.full((n_tok, 2, 128), 9.0, dtype=torch.bfloat16, device="cuda"), i32([0])
    qsa.delta_prompt(*inputs, state, slots, old, i32(cu), out=out, workspace=ws, dev_status=status)
    return out, state, int(status)


@pytest.mark.parametrize("cu", FALLING, ids=str)
def test_three(qsa, cu):  # noqa: F811
    want, state, status = call(qsa, cu, 0)
    assert status & BAD_LEN and bool(torch.isfinite(want).all()) and bool(torch.isfinite(state).all())
    for fill in (255, 0x3C):
        got, st, _ = call(qsa, cu, fill)
        assert torch.equal(got, want) and torch.equal(st, state)


@pytest.mark.parametrize("n_seq", [40, 300])
def test_many(qsa, n_seq):  # noqa: F811
    """On both sides of the number of sequences that go by length: ordinary bounds but for one in the middle."""
    each = 40
    cu = [each * i for i in range(n_seq + 1)]
    for value in (0, each * n_seq, cu[n_seq // 2 + 3]):
        cu[n_seq // 2] = value
        want, state, status = call(qsa, cu, 0, each * n_seq, n_seq)
        got, st, _ = call(qsa, cu, 255, each * n_seq, n_seq)
        assert status & BAD_LEN and torch.equal(got, want) and torch.equal(st, state) and bool(torch.isfinite(st).all())


def test_segments(qsa):  # noqa: F811
    for cu in ([2300, 0, 2300], [0, 2300, 0], [0, 2290, 100]):
        want, state, status = call(qsa, cu, 0, 2300, 2)
        got, st, _ = call(qsa, cu, 255, 2300, 2)
        assert status & BAD_LEN and torch.equal(got, want) and torch.equal(st, state) and bool(torch.isfinite(st).all())


def test_ordinary_bounds_in_many_sequences(qsa):  # noqa: F811
    """Nothing is left out where bounds do not fall: sequences of no token, and of chunks, beyond the number that go by length."""
    lens = [0, 64, 0, 33, 65, 1] * 50
    inputs, state, slots, old, cu = batch(lens, 1, 1, torch.bfloat16, seed=5)
    want = ref.delta(*inputs, state, slots, old, cu, 1e-6, SCALE, ref.CHUNK)
    got = qsa.delta_prompt(*inputs, state, slots, old, cu)
    ref.check_delta(got, state, want, SCALE, torch.bfloat16, True, slots)
