"""qsa_delta_prompt and qsa_delta_step on the GPU against the rule's 64-bit definition."""
import itertools

import pytest

torch = pytest.importorskip("torch")
import linear_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu
BAD_LEN, BAD_STATE = 64, 1024
SCALE = 128 ** -0.5


@pytest.fixture(scope="module")
def qsa():
    from sparse_selected_cell_gb300 import qsa as q
    if not torch.cuda.is_available():
        pytest.fail("CUDA GPU required")
    q.lib()
    return q


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def cu_of(lens):
    return i32([0] + list(itertools.accumulate(lens)))


def batch(lens, n_k, n_v, dtype, seed, apart=0):
    n = len(lens)
    slots = torch.randperm(n + 2, generator=torch.Generator().manual_seed(seed))[:n].int().cuda()
    old = i32([0 if i % 3 == 1 else 5 for i in range(n)])
    return ref.heads(sum(lens), n_k, n_v, dtype, seed, apart=apart), ref.pool(n + 2, n_v, seed), slots, old, cu_of(lens)


def check_prompt(qsa, inputs, state, slots, old, cu, eps=1e-6, scale=SCALE):
    want = ref.delta(*inputs, state, slots, old, cu, eps, scale, ref.CHUNK)
    status, given = i32([0]), state.clone()
    got = qsa.delta_prompt(*inputs, state, slots, old, cu, eps=eps, scale=scale, dev_status=status)
    ref.check_delta(got, state, want, scale, inputs[0].dtype, True, slots)
    rest = sorted(set(range(state.shape[0])) - {int(s) for s in slots})
    assert torch.equal(state[rest], given[rest]) and int(status) == 0
    return got


LENS = [[1], [2], [63], [64], [65], [127, 1, 129], [0, 3, 0, 70, 0], [200, 1, 64, 63, 128, 2], [0], [16, 17, 33, 48, 49]]


@pytest.mark.parametrize("n_k,n_v,dtype", [(1, 1, torch.bfloat16), (2, 4, torch.float16), (1, 3, torch.bfloat16), (4, 4, torch.float16)])
@pytest.mark.parametrize("lens", LENS, ids=lambda n: "-".join(map(str, n)))
def test_prompt(qsa, lens, n_k, n_v, dtype):
    check_prompt(qsa, *batch(lens, n_k, n_v, dtype, seed=len(lens) + n_v, apart=(n_v % 2) * 8))


@pytest.mark.parametrize("lens", [[31], [32], [33], [32, 0, 1, 33, 31, 7, 34], [8] * 9 + [200]], ids=lambda n: "-".join(map(str, n)))
def test_where_chunks_begin(qsa, lens):
    check_prompt(qsa, *batch(lens, 2, 6, torch.bfloat16, seed=len(lens)))


def test_long_prompt(qsa):
    check_prompt(qsa, *batch([1500, 700], 1, 2, torch.bfloat16, seed=5))


@pytest.mark.parametrize("n_k,n_v,dtype", [(1, 1, torch.bfloat16), (2, 4, torch.float16), (1, 3, torch.bfloat16), (16, 32, torch.bfloat16)])
@pytest.mark.parametrize("n_seq", [1, 3, 40])
def test_steps(qsa, n_seq, n_k, n_v, dtype):
    """Several steps in a row; the first finds some sequences fresh."""
    for step in range(3):
        inputs, fresh_state, slots, old, cu = batch([1] * n_seq, n_k, n_v, dtype, seed=n_seq, apart=8 * (n_v % 2))
        if step == 0:
            state = fresh_state
        inputs = [x.roll(step, 0) if x.dim() > 1 else x for x in inputs] if n_seq > 1 else inputs
        want = ref.delta(*inputs, state, slots, old if step == 0 else None, cu, 1e-6, SCALE, ref.STEP)
        got = qsa.delta_step(*inputs, state, slots, old if step == 0 else None)
        ref.check_delta(got, state, want, SCALE, dtype, False, slots)


def test_prompt_then_steps(qsa):
    """A prompt cut into steps of any kind ends near where the whole one does, and single tokens go on from it."""
    inputs, state, slots, _, _ = batch([150], 2, 4, torch.bfloat16, seed=3)
    old = i32([0])
    want = ref.delta(*inputs, state, slots, old, i32([0, 150]), 1e-6, SCALE, ref.CHUNK)
    part, got, at = state.clone(), [], 0
    for n in (70, 1, 1, 0, 64, 13, 1):
        cut = [x[at:at + n] for x in inputs[:5]] + list(inputs[5:])
        if n == 1:
            got.append(qsa.delta_step(*cut, part, slots, i32([at])))
        else:
            got.append(qsa.delta_prompt(*cut, part, slots, i32([at]), i32([0, n])))
        at += n
    ref.check_delta(torch.cat(got), part, want, SCALE, torch.bfloat16, True, slots)


def test_left_out_and_behind(qsa):
    """Sequences without a slot, slots past the pool, tokens behind the last sequence: rows and states stay as they are."""
    lens = [70, 130, 5, 64]
    inputs, state, slots, old, cu = batch(lens, 1, 2, torch.bfloat16, seed=9)
    tail = [torch.cat((x, torch.full((30, *x.shape[1:]), float("nan"), dtype=x.dtype, device="cuda"))) for x in inputs[:5]]
    slots[1], slots[3] = -1, 6
    want = ref.delta(*inputs, state, slots, old, cu, 1e-6, SCALE, ref.CHUNK)
    out, status, given = torch.full((sum(lens) + 30, 2, 128), 9.0, dtype=torch.bfloat16, device="cuda"), i32([0]), state.clone()
    qsa.delta_prompt(*tail, *inputs[5:], state, slots, old, cu, out=out, dev_status=status)
    n = sum(lens)
    ref.check_delta(out[:n], state, want, SCALE, torch.bfloat16, True, slots)
    mine = ~torch.isnan(want[0][:, 0, 0])
    assert bool((out[:n][~mine] == 9.0).all()) and bool((out[n:] == 9.0).all()) and int(status) == BAD_STATE
    rest = sorted(set(range(6)) - {int(slots[0]), int(slots[2])})
    assert torch.equal(state[rest], given[rest])
    # the same for single tokens
    inputs, state, slots, old, cu = batch([1] * 5, 1, 2, torch.bfloat16, seed=2)
    slots[0], slots[4] = 7, -3
    want = ref.delta(*inputs, state, slots, old, cu, 1e-6, SCALE, ref.STEP)
    out, status, given = torch.full((5, 2, 128), 9.0, dtype=torch.bfloat16, device="cuda"), i32([0]), state.clone()
    qsa.delta_step(*inputs, state, slots, old, out=out, dev_status=status)
    ref.check_delta(out, state, want, SCALE, torch.bfloat16, False, slots)
    assert bool((out[0] == 9.0).all()) and bool((out[4] == 9.0).all()) and int(status) == BAD_STATE
    rest = sorted(set(range(7)) - {int(s) for s in slots[1:4]})
    assert torch.equal(state[rest], given[rest])


def test_bounds_out_of_order(qsa):
    inputs, state, slots, old, _ = batch([100, 100, 100], 1, 1, torch.bfloat16, seed=1)
    for cu in ([0, 250, 10, 300], [0, 20, 40, 999], [-7, 20, 40, 60], [5, 20, 40, 60], [0, 2 ** 31 - 1, -2 ** 31, 60]):
        status = i32([0])
        qsa.delta_prompt(*inputs, state, slots, old, i32(cu), dev_status=status)
        assert int(status) & BAD_LEN, cu


def gated(inputs, a=None, b=None, a_log=None, dt_bias=None, **rows):
    q, k, v, ga, gb, al, db = (x.clone() for x in inputs)
    for name, x in (("q", q), ("k", k), ("v", v)):
        if name in rows:
            x.copy_(rows[name](x))
    if a is not None:
        ga.fill_(a)
    if b is not None:
        gb.fill_(b)
    if a_log is not None:
        al.fill_(a_log)
    if dt_bias is not None:
        db.fill_(dt_bias)
    return q, k, v, ga, gb, al, db


CASES = {
    "no decay": dict(a_log=float("-inf")),
    "strong decay": dict(a=4.0, a_log=2.7),
    "decay to nothing": dict(a=60.0, a_log=6.0),
    "no write": dict(b=float("-inf")),
    "full write": dict(b=float("inf"), a_log=float("-inf")),
    "one key": dict(k=lambda x: x[:1].expand_as(x), b=float("inf")),
    "one key no decay": dict(k=lambda x: x[:1].expand_as(x), b=3.0, a_log=float("-inf")),
    "opposite keys": dict(k=lambda x: x[:1] * torch.tensor([1.0, -1.0], device="cuda", dtype=x.dtype).repeat(x.shape[0])[:x.shape[0], None, None],
                          b=float("inf"), a_log=float("-inf")),
    "zero keys": dict(k=lambda x: x * 0),
    "zero queries and values": dict(q=lambda x: x * 0, v=lambda x: x * 0),
    "tiny rows": dict(k=lambda x: x * 2 ** -10, q=lambda x: x * 2 ** -10, v=lambda x: x * 2 ** -10),
    "large rows": dict(k=lambda x: x * 2 ** 9, q=lambda x: x * 2 ** 9, v=lambda x: x * 2 ** 9),
    "uneven values": dict(v=lambda x: x * torch.exp2((torch.arange(128, device="cuda") % 17 - 8).to(x.dtype)).to(x.dtype)),
    "values that jump": dict(v=lambda x: x * torch.exp2((torch.arange(x.shape[0], device="cuda") % 40 / 4 - 5)).to(x.dtype)[:, None, None]),
    "one dim keys": dict(k=lambda x: x * (torch.arange(128, device="cuda") == 77).to(x.dtype)),
}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("name", list(CASES))
def test_values(qsa, name, dtype):
    lens = [140, 64, 7]
    inputs, state, slots, old, cu = batch(lens, 1, 2, dtype, seed=4)
    inputs = gated(inputs, **CASES[name])
    eps = 1e-6 if name != "tiny rows" else 1e-12
    if name == "zero keys":
        eps = 1e-3
    check_prompt(qsa, inputs, state.clone(), slots, old, cu, eps=eps)
    first = [x[:3].contiguous() for x in inputs[:5]] + list(inputs[5:])
    want = ref.delta(*first, state, slots, old, cu_of([1, 1, 1]), eps, SCALE, ref.STEP)
    got = qsa.delta_step(*first, state, slots, old, eps=eps)
    ref.check_delta(got, state, want, SCALE, dtype, False, slots)


def test_bfloat16_range(qsa):
    """Values, states and keys far outside FP16's range."""
    for size in (2.0 ** 40, 2.0 ** -40):
        inputs, state, slots, old, cu = batch([130, 20], 1, 2, torch.bfloat16, seed=8)
        q, k, v, *rest = inputs
        inputs = (q * size, k * size, v * size, *rest)
        want = ref.delta(*inputs, state * size, slots, old, cu, 0.0, SCALE, ref.CHUNK)
        st = state * size
        got = qsa.delta_prompt(*inputs, st, slots, old, cu, eps=0.0)
        out, pool, big, off, end = want
        # the checks' floors are absolute: brought back to 1 first
        scaled = (out / size, pool / size, big / size, off / size, end / size)
        ref.check_delta(got.double() / size, st.double() / size, scaled, SCALE, torch.bfloat16, True, slots)


def test_infinities_stay_in_their_sequence(qsa):
    inputs, state, slots, old, cu = batch([70, 70, 70], 1, 2, torch.bfloat16, seed=6)
    clean = [x.clone() for x in inputs]
    st_clean = state.clone()
    want = qsa.delta_prompt(*clean, st_clean, slots, old, cu)
    for x in inputs[:5]:
        x[70:140] = float("nan")
    inputs[2][75] = float("inf")
    got = qsa.delta_prompt(*inputs, state, slots, old, cu)
    keep = [int(slots[0]), int(slots[2])]
    assert torch.equal(got[:70], want[:70]) and torch.equal(got[140:], want[140:]) and torch.equal(state[keep], st_clean[keep])


def test_same_bits_and_other_order(qsa):
    """The same call gives the same bits, whatever the workspace held, and a sequence's results do not depend on its neighbours."""
    lens = [300, 64, 129]
    inputs, state, slots, old, cu = batch(lens, 2, 4, torch.bfloat16, seed=7)
    ws = torch.full((qsa.delta_prompt_workspace_bytes(sum(lens), 3, 2, 4),), 255, dtype=torch.uint8, device="cuda")
    first = state.clone()
    want = qsa.delta_prompt(*inputs, first, slots, old, cu, workspace=ws)
    for _ in range(3):
        again = state.clone()
        assert torch.equal(qsa.delta_prompt(*inputs, again, slots, old, cu), want) and torch.equal(again, first)
    alone = state.clone()
    cut = [x[300:364] for x in inputs[:5]] + list(inputs[5:])
    assert torch.equal(qsa.delta_prompt(*cut, alone, slots[1:2], old[1:2], i32([0, 64])), want[300:364])
    assert torch.equal(alone[slots[1].long()], first[slots[1].long()])


def test_graph_and_streams(qsa):
    """Captured and replayed while the state goes on; two captures with a workspace each; on a stream that is not the current one."""
    lens = [65, 3]
    inputs, state, slots, _, cu = batch(lens, 1, 2, torch.bfloat16, seed=11)
    ws = [torch.empty(qsa.delta_prompt_workspace_bytes(68, 2, 1, 2), dtype=torch.uint8, device="cuda") for _ in range(2)]
    want = state.clone()
    outs = [qsa.delta_prompt(*inputs, want, slots, None, cu).clone() for _ in range(4)]
    out, graphs = torch.empty_like(outs[0]), []
    live = state.clone()
    for w in ws:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            qsa.delta_prompt(*inputs, live, slots, None, cu, out=out, workspace=w)
        graphs.append(g)
    for i in range(4):
        graphs[i % 2].replay()
        assert torch.equal(out, outs[i])
    assert torch.equal(live, want)
    side, live = torch.cuda.Stream(), state.clone()
    torch.cuda.synchronize()
    for i in range(4):
        got = qsa.delta_prompt(*inputs, live, slots, None, cu, stream=side)
    side.synchronize()
    assert torch.equal(got, outs[3]) and torch.equal(live, want)


def test_offsets_past_32_bits(qsa):
    """States past 2^31 floats, rows past 2^31 elements."""
    n_slots = 2 ** 31 // (2 * 128 * 128) + 3
    state = torch.zeros((n_slots, 2, 128, 128), device="cuda")
    slots = i32([n_slots - 1, 1])
    small = ref.pool(2, 2, 3)
    state[slots.long()] = small
    inputs = ref.heads(140, 1, 2, torch.bfloat16, 3)
    far = torch.empty((140, 16_000_000), dtype=torch.bfloat16, device="cuda")
    v = far[:, :256].view(140, 2, 128)
    v.copy_(inputs[2])
    moved = (*inputs[:2], v, *inputs[3:])
    cu = i32([0, 70, 140])
    want = qsa.delta_prompt(*inputs, small, i32([0, 1]), None, cu)
    assert torch.equal(qsa.delta_prompt(*moved, state, slots, None, cu), want) and torch.equal(state[slots.long()], small)
    two = [x[:2] for x in moved[:5]] + list(moved[5:])
    want = qsa.delta_step(*two, small, i32([0, 1]))
    assert torch.equal(qsa.delta_step(*two, state, slots), want) and torch.equal(state[slots.long()], small)


def test_refusals(qsa):
    inputs, state, slots, old, cu = batch([4, 5], 2, 4, torch.bfloat16, seed=1)
    names = ("q", "k", "v", "a", "b", "a_log", "dt_bias")
    base = dict(zip(names, inputs), state=state, state_slots=slots, old_lens=old)
    q, k, v, a, b, a_log, dt = inputs
    bad = [dict(q=q.float()), dict(q=q.cpu()), dict(q=q[:3]), dict(q=q[..., :64]), dict(k=k.half()), dict(k=k[:, :1]),
           dict(v=v[:, :3]), dict(a=a[:, :2]), dict(b=b.float()), dict(a_log=a_log.half()), dict(dt_bias=dt[:2]),
           dict(state=state.half()), dict(state=state[:, :2]), dict(state_slots=slots.long()), dict(old_lens=old[:1]),
           dict(eps=-1.0), dict(eps=float("nan")), dict(scale=float("inf")), dict(out=torch.empty_like(v).half()), dict(out=v)]
    for kw in bad + [dict(cu_tokens=cu[:2]), dict(cu_tokens=None), dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
                     dict(workspace=torch.empty(1 << 22, dtype=torch.uint8))]:
        with pytest.raises((TypeError, ValueError, RuntimeError)):
            qsa.delta_prompt(**{**base, "cu_tokens": cu, **kw})
    two = {n: x[:2] if n in names[:5] else x for n, x in base.items()}
    for kw in bad + [dict(state_slots=slots[:1], old_lens=None)]:
        kw = {n: x[:2] if n in names[:5] and x.shape[0] > 3 else x for n, x in kw.items()}
        with pytest.raises((TypeError, ValueError, RuntimeError)):
            qsa.delta_step(**{**two, **kw})
    qsa.delta_step(**two)
    qsa.delta_prompt(**base, cu_tokens=cu)
