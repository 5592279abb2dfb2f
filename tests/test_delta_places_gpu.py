"""qsa_delta_prompt's places in its workspace where sequences are many and most of them short: each chunk has its own, whatever
stands between, and nothing is written behind the workspace."""
import pytest

torch = pytest.importorskip("torch")
import delta_norms as norms  # noqa: E402
import linear_ref as ref  # noqa: E402
from test_delta_gpu import SCALE, batch, qsa  # noqa: E402,F401

pytestmark = pytest.mark.gpu
STEPS = {
    "one prompt among single tokens": [1] * 40 + [700] + [1] * 40,
    "prompts of 33 and 65 side by side": [33, 65] * 8,
    "33 at every offset": [x for i in range(32) for x in (i, 33)],
    "65 at every offset": [x for i in range(0, 32, 3) for x in (i, 65, 0)],
    "empty ones between": [0, 64, 0, 0, 34, 0, 129, 0, 1, 33],
    "short ones alone": [3, 32, 1, 32, 17],
    "many": [1] * 300 + [200] + [2] * 30 + [90],
}


@pytest.mark.parametrize("name", list(STEPS))
def test_steps(qsa, name):  # noqa: F811
    lens = STEPS[name]
    inputs, state, slots, old, cu = batch(lens, 1, 2, torch.bfloat16, seed=len(lens))
    n = qsa.delta_prompt_workspace_bytes(sum(lens), len(lens), 1, 2)
    ws = torch.full((n + 4096,), 255, dtype=torch.uint8, device="cuda")
    want = ref.delta(*inputs, state, slots, old, cu, 1e-6, SCALE, ref.CHUNK)
    fine, size = norms.delta(*inputs, state, slots, old, cu, 1e-6, SCALE)
    got = qsa.delta_prompt(*inputs, state, slots, old, cu, workspace=ws[:n])
    ref.check_delta(got, state, want, SCALE, torch.bfloat16, True, slots)
    norms.check(got, fine, size, torch.bfloat16)
    assert bool((ws[n:] == 255).all())


def test_as_many_alone(qsa):  # noqa: F811
    """A prompt's results do not depend on the places that its neighbours' number gives it."""
    inputs, state, slots, old, cu = batch([1] * 30 + [300] + [1] * 30, 1, 2, torch.bfloat16, seed=3)
    whole = state.clone()
    got = qsa.delta_prompt(*inputs, whole, slots, old, cu)
    cut = [x[30:330] for x in inputs[:5]] + list(inputs[5:])
    alone = qsa.delta_prompt(*cut, state, slots[30:31], old[30:31], torch.tensor([0, 300], dtype=torch.int32, device="cuda"))
    assert torch.equal(got[30:330], alone) and torch.equal(whole[slots[30].long()], state[slots[30].long()])
