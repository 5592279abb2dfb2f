"""qsa_delta_prompt on both sides of the length from which a single long sequence is cut into segments: the documented ranges, what
is no number, late writers, captured calls; against the rule in 64 bits."""
import pytest

torch = pytest.importorskip("torch")
import delta_norms as norms  # noqa: E402
import linear_ref as ref  # noqa: E402
from test_delta_gpu import CASES, SCALE, batch, gated, i32, qsa  # noqa: E402,F401
from test_delta_range_gpu import scaled_back  # noqa: E402
from test_serve_order_gpu import check as check_late, late  # noqa: E402,F401

pytestmark = pytest.mark.gpu
LENS = [2559, 2560, 2561, 2700]


def test_the_border_is_here(qsa):  # noqa: F811
    """The workspace tells: segments need a state's room twice for each of eight."""
    sizes = [qsa.delta_prompt_workspace_bytes(n, 1, 1, 2) for n in (2559, 2560)]
    assert sizes[1] - sizes[0] > 2 << 20


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n", LENS)
def test_lengths(qsa, n, dtype):  # noqa: F811
    inputs, state, slots, old, cu = batch([n], 1, 3, dtype, seed=n)
    want = ref.delta(*inputs, state, slots, old, cu, 1e-6, SCALE, ref.CHUNK)
    fine, size = norms.delta(*inputs, state, slots, old, cu, 1e-6, SCALE)
    got = qsa.delta_prompt(*inputs, state, slots, old, cu)
    ref.check_delta(got, state, want, SCALE, dtype, True, slots)
    norms.check(got, fine, size, dtype)


@pytest.mark.parametrize("name", ["no decay", "strong decay", "no write", "full write", "one key no decay", "opposite keys", "zero keys",
                                  "uneven values", "values that jump"])
def test_gates_and_values(qsa, name):  # noqa: F811
    eps = 1e-3 if name == "zero keys" else 1e-6
    inputs, state, slots, _, cu = batch([2700], 1, 2, torch.bfloat16, seed=4)
    inputs = gated(inputs, **CASES[name])
    want = ref.delta(*inputs, state, slots, None, cu, eps, SCALE, ref.CHUNK)
    fine, size = norms.delta(*inputs, state, slots, None, cu, eps, SCALE)
    got = qsa.delta_prompt(*inputs, state, slots, None, cu, eps=eps)
    ref.check_delta(got, state, want, SCALE, torch.bfloat16, True, slots)
    norms.check(got, fine, size, torch.bfloat16)


@pytest.mark.parametrize("scale", [2.0 ** 112, 2.0 ** 60, 2.0 ** -60, 2.0 ** -84])
def test_values_and_states(qsa, scale):  # noqa: F811
    inputs, state, slots, old, cu = batch([2700], 1, 2, torch.bfloat16, seed=8)
    inputs = (*inputs[:2], inputs[2] * scale, *inputs[3:])
    state = state * scale
    want = ref.delta(*inputs, state, slots, old, cu, 1e-6, SCALE, ref.CHUNK)
    got = qsa.delta_prompt(*inputs, state, slots, old, cu)
    out, pool, scaled = scaled_back(want, got, state, scale)
    ref.check_delta(out, pool, scaled, SCALE, torch.bfloat16, True, slots)


def test_numbers_stay_in_their_value_dim_and_head(qsa):  # noqa: F811
    inputs, state, slots, old, cu = batch([2700], 1, 2, torch.bfloat16, seed=6)
    clean = state.clone()
    want = qsa.delta_prompt(*inputs, clean, slots, old, cu)
    v = inputs[2].clone()
    v[1350, 0, 5], v[1351, 0, 77] = float("nan"), float("inf")
    got = qsa.delta_prompt(*inputs[:2], v, *inputs[3:], state, slots, old, cu)
    keep = torch.ones(128, dtype=torch.bool, device="cuda")
    keep[5] = keep[77] = False
    s = int(slots[0])
    assert torch.equal(got[:, 1], want[:, 1]) and torch.equal(got[:, 0][:, keep], want[:, 0][:, keep])
    assert torch.equal(state[s, 1], clean[s, 1]) and torch.equal(state[s, 0][keep], clean[s, 0][keep])
    assert torch.equal(got[:1344], want[:1344])


def test_captured_and_repeated(qsa):  # noqa: F811
    inputs, state, slots, _, cu = batch([2700], 1, 2, torch.bfloat16, seed=11)
    first = state.clone()
    want = qsa.delta_prompt(*inputs, first, slots, None, cu)
    ws = torch.full((qsa.delta_prompt_workspace_bytes(2700, 1, 1, 2),), 255, dtype=torch.uint8, device="cuda")
    live, out = state.clone(), torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qsa.delta_prompt(*inputs, live, slots, None, cu, out=out, workspace=ws)
    for _ in range(3):
        live.copy_(state)
        graph.replay()
        assert torch.equal(out, want) and torch.equal(live, first)


def test_late_writers(qsa, late):  # noqa: F811
    def step(seed):
        inputs, state, slots, old, cu = batch([2700], 1, 2, torch.bfloat16, seed=seed)
        return [*[t.contiguous() for t in inputs], state, slots, old, cu]

    check_late(late, step(1), step(0), lambda *t: (qsa.delta_prompt(*t[:7], t[7], t[8], t[9], t[10]), t[7]))


def test_what_gates_forget(qsa):  # noqa: F811
    """Values 2^50 larger, forgotten at the end of their chunk, in the middle of a segment and right before the next one."""
    for large in (640, 1280):
        inputs, state, slots, _, cu = batch([2700], 1, 2, torch.bfloat16, seed=3)
        q, k, v, a, b, a_log, dt = gated(inputs, a_log=3.0)
        a.fill_(-6.0)
        v[large:large + 64] *= 2.0 ** 50
        a[large + 64] = 80.0
        inputs = (q, k, v, a, b, a_log, dt)
        end = ref.delta(*inputs, state, slots, None, cu, 1e-6, SCALE, ref.CHUNK)[1]
        want, size = norms.delta(*inputs, state, slots, None, cu, 1e-6, SCALE)
        got = qsa.delta_prompt(*inputs, state, slots, None, cu)
        norms.check(got[large + 64:], want[large + 64:], size[large + 64:], torch.bfloat16)
        s = slots.long()
        assert float((state[s] - end[s]).square().sum().sqrt()) <= 2.0 ** -17 * float(end[s].square().sum().sqrt())
        assert cu.equal(i32([0, 2700]))
