"""qsa_delta_prompt's ways through a step: segments of long sequences, many value heads to a key head, sequences by length,
short ones token by token; against the rule's 64-bit definition."""
import itertools

import pytest

torch = pytest.importorskip("torch")
import linear_ref as ref  # noqa: E402
from test_delta_gpu import CASES, SCALE, batch, check_prompt, cu_of, gated, i32, qsa  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,n_k,n_v,dtype", [([1024], 1, 1, torch.bfloat16), ([1031], 2, 6, torch.float16),
                                                ([4200], 1, 2, torch.bfloat16), ([2049, 100, 0, 1500], 1, 1, torch.float16),
                                                ([1100, 17], 4, 8, torch.bfloat16), ([3000], 8, 16, torch.bfloat16),
                                                ([2047], 1, 1, torch.float16), ([2048], 1, 1, torch.bfloat16), ([3100], 2, 6, torch.float16),
                                                ([2200, 3400], 4, 8, torch.bfloat16), ([9000], 1, 2, torch.bfloat16)])
def test_segments(qsa, lens, n_k, n_v, dtype):  # noqa: F811
    check_prompt(qsa, *batch(lens, n_k, n_v, dtype, seed=len(lens) + n_v))


@pytest.mark.parametrize("name", ["no decay", "strong decay", "no write", "full write", "one key no decay", "opposite keys",
                                  "zero keys", "uneven values", "values that jump"])
def test_values_in_segments(qsa, name):  # noqa: F811
    inputs, state, slots, old, cu = batch([2180, 1040], 1, 2, torch.bfloat16, seed=4)
    check_prompt(qsa, gated(inputs, **CASES[name]), state, slots, None, cu, eps=1e-3 if name == "zero keys" else 1e-6)


def test_segments_left_out_and_behind(qsa):  # noqa: F811
    """A long sequence without a slot, tokens behind the last sequence: rows and states stay as they are."""
    lens = [2200, 2300, 600]
    inputs, state, slots, old, cu = batch(lens, 1, 2, torch.bfloat16, seed=9)
    tail = [torch.cat((x, torch.full((90, *x.shape[1:]), float("nan"), dtype=x.dtype, device="cuda"))) for x in inputs[:5]]
    slots[1] = -1
    want = ref.delta(*inputs, state, slots, old, cu, 1e-6, SCALE, ref.CHUNK)
    n = sum(lens)
    out, given = torch.full((n + 90, 2, 128), 9.0, dtype=torch.bfloat16, device="cuda"), state.clone()
    qsa.delta_prompt(*tail, *inputs[5:], state, slots, old, cu, out=out)
    ref.check_delta(out[:n], state, want, SCALE, torch.bfloat16, True, slots)
    assert bool((out[2200:4500] == 9.0).all()) and bool((out[n:] == 9.0).all())
    rest = sorted(set(range(5)) - {int(slots[0]), int(slots[2])})
    assert torch.equal(state[rest], given[rest])


@pytest.mark.parametrize("n_k,n_v", [(1, 3), (1, 4), (2, 10), (1, 7)])
def test_many_value_heads_to_a_key_head(qsa, n_k, n_v):  # noqa: F811
    check_prompt(qsa, *batch([130, 64, 20], n_k, n_v, torch.bfloat16, seed=n_v))


@pytest.mark.parametrize("n_seq,hi", [(40, 90), (256, 30), (257, 30), (300, 70)])
def test_many_sequences(qsa, n_seq, hi):  # noqa: F811
    """On both sides of the number that go by length; among them empty ones and ones of 16, 17 and 64 tokens."""
    g = torch.Generator().manual_seed(n_seq)
    lens = torch.randint(0, hi, (n_seq,), generator=g).tolist()
    lens[:6] = [0, 16, 17, 64, 65, 1]
    check_prompt(qsa, *batch(lens, 1, 1, torch.bfloat16, seed=n_seq))


@pytest.mark.parametrize("lens", [[16], [17], [15, 1], [1] * 16, [1] * 17, [16, 17, 15], [0, 0, 1], [0] * 20])
def test_short_sequences(qsa, lens):  # noqa: F811
    check_prompt(qsa, *batch(lens, 2, 4, torch.float16, seed=len(lens)))


@pytest.mark.parametrize("lens", [[61], [1100], [2100], [90, 2200]])
def test_repeated_captured_and_side_by_side(qsa, lens):  # noqa: F811
    """The same bits again; from a captured call; and from two calls at once, on two streams, with a workspace and states each."""
    inputs, state, slots, _, cu = batch(lens, 1, 2, torch.bfloat16, seed=11)
    first = state.clone()
    want = qsa.delta_prompt(*inputs, first, slots, None, cu)
    size = qsa.delta_prompt_workspace_bytes(sum(lens), len(lens), 1, 2)
    ws = [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in range(2)]
    live, out = state.clone(), torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qsa.delta_prompt(*inputs, live, slots, None, cu, out=out, workspace=ws[0])
    for _ in range(3):
        live.copy_(state)
        graph.replay()
        assert torch.equal(out, want) and torch.equal(live, first)
    streams, outs, states = [torch.cuda.Stream() for _ in range(2)], [torch.empty_like(want) for _ in range(2)], [state.clone(), state.clone()]
    torch.cuda.synchronize()
    for _ in range(4):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                states[i].copy_(state)
                qsa.delta_prompt(*inputs, states[i], slots, None, cu, out=outs[i], workspace=ws[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(outs[i], want) and torch.equal(states[i], first)


def test_a_step_of_everything(qsa):  # noqa: F811
    """Long, ordinary, short and empty sequences, fresh ones and ones that go on, over three steps."""
    lens = [2500, 1, 0, 300, 16, 64, 17, 2]
    inputs, state, slots, old, _ = batch(lens, 1, 2, torch.bfloat16, seed=21)
    for turn in range(3):
        order = lens[turn:] + lens[:turn]
        cu = i32([0] + list(itertools.accumulate(order)))
        check_prompt(qsa, inputs, state, slots, old if turn == 0 else None, cu)
    assert cu_of(lens).shape == cu.shape


@pytest.mark.parametrize("chunks", [9, 33])
@pytest.mark.parametrize("size", [2.0 ** 50, 2.0 ** -50])
def test_nothing_left_after_large_values(qsa, size, chunks):  # noqa: F811
    """Chunks of values far out, then decays that leave nothing of them and values of zero or of ordinary size: what was large
    neither lingers in the units nor turns zeros into something else."""
    inputs, state, slots, old, cu = batch([64 * chunks], 1, 2, torch.bfloat16, seed=3)
    q, k, v, a, b, a_log, dt = (x.clone() for x in inputs)
    v[:128] *= size
    v[128:320] = 0
    a[128:192] = 80.0
    a_log.fill_(3.0)
    check_prompt(qsa, (q, k, v, a, b, a_log, dt), state * size, slots, old, cu)
