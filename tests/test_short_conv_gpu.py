"""qsa_short_conv on the GPU against its 64-bit definition."""
import itertools

import pytest

torch = pytest.importorskip("torch")
import linear_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu
BAD_LEN, BAD_STATE = 64, 1024


@pytest.fixture(scope="module")
def qsa():
    from sparse_selected_cell_gb300 import qsa as q
    if not torch.cuda.is_available():
        pytest.fail("CUDA GPU required")
    q.lib()
    return q


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def make(lens, n_ch, width, dtype, seed, wide=0, w_type=None):
    g = torch.Generator().manual_seed(seed)
    n_tok = sum(lens)
    x = torch.randn((n_tok, n_ch + wide), generator=g).to(dtype).cuda()[:, :n_ch]
    w = (torch.randn((n_ch, width), generator=g) * width ** -0.5).to(w_type or dtype).cuda()
    bias = (torch.randn(n_ch, generator=g) * 0.1).to(w_type or dtype).cuda()
    state = torch.randn((len(lens) + 2, width - 1, n_ch), generator=g).to(dtype).cuda()
    slots = torch.randperm(len(lens) + 2, generator=g)[:len(lens)].int().cuda()
    old = torch.tensor([0 if i % 3 == 1 else 5 for i in range(len(lens))], dtype=torch.int32).cuda()
    return x, w, bias, state, slots, old, i32([0] + list(itertools.accumulate(lens)))


LENS = [[1], [2], [3], [0], [0, 0, 3, 0], [1, 1, 1, 1, 1], [15, 1, 16, 17, 2, 0, 0, 33, 3, 1], [14, 2, 30, 1, 48, 64], [129],
        [0, 5, 0], [63, 3, 1], [47, 1, 100], [2] * 40, [0] * 70 + [40] + [0] * 70 + [3, 0]]


@pytest.mark.parametrize("width,dtype", [(4, torch.bfloat16), (3, torch.float16), (2, torch.bfloat16), (2, torch.float16)])
@pytest.mark.parametrize("lens", LENS, ids=lambda n: f"{len(n)}x{max(n)}")
def test_ragged(qsa, lens, width, dtype):
    for n_ch, silu, with_bias in ((8, True, True), (1032, True, False), (264, False, True)):
        x, w, bias, state, slots, old, cu = make(lens, n_ch, width, dtype, seed=len(lens) + n_ch)
        bias = bias if with_bias else None
        want, new_state, size = ref.short_conv(x, w, state, slots, old, cu, bias, silu)
        status = i32([0])
        got = qsa.short_conv(x, w, state, slots, old, cu, bias=bias, activation="silu" if silu else "none", dev_status=status)
        ref.check_conv(got, want, size, dtype, width, n_ch)
        assert torch.equal(state, new_state) and int(status) == 0


@pytest.mark.parametrize("n_seq", [1, 2, 33, 300])
def test_one_token_each(qsa, n_seq):
    """Without cu_tokens; the same as with it; over several steps the states carry on."""
    x, w, bias, state, slots, old, cu = make([1] * n_seq, 136, 4, torch.bfloat16, seed=n_seq, wide=72, w_type=torch.float32)
    other = state.clone()
    for step in range(5):
        want, new_state, size = ref.short_conv(x, w, state, slots, old, cu, bias, True)
        got = qsa.short_conv(x, w, state, slots, old, bias=bias)
        ref.check_conv(got, want, size, x.dtype, 4)
        assert torch.equal(state, new_state)
        assert torch.equal(got, qsa.short_conv(x, w, other, slots, old, cu, bias=bias)) and torch.equal(state, other)
        old = None
        x = x.roll(1, 0) * 0.5


def test_split_steps_are_one(qsa):
    """A prompt in one step, and the same cut at every kind of place: the same bits."""
    x, w, bias, state, slots, _, _ = make([100], 520, 4, torch.bfloat16, seed=3)
    whole, first = state.clone(), i32([0])
    want = qsa.short_conv(x, w, whole, slots, first, i32([0, 100]), bias=bias)
    got, at = [], 0
    for n in (1, 2, 1, 3, 30, 0, 16, 17, 30):
        got.append(qsa.short_conv(x[at:at + n], w, state, slots, i32([at]), i32([0, n]), bias=bias))
        at += n
    assert at == 100 and torch.equal(torch.cat(got), want) and torch.equal(state, whole)


def test_left_out_and_behind(qsa):
    """Sequences without a slot, slots past the pool, tokens behind the last sequence: their rows and states stay as they are."""
    for lens in ([5, 20, 1, 40, 3], [1, 2, 1, 1, 1]):
        n_tok = sum(lens) + 21
        x, w, bias, state, slots, old, cu = make(lens, 72, 4, torch.bfloat16, seed=9)
        x = torch.cat((x, torch.full((21, 72), float("nan"), device="cuda", dtype=x.dtype)))
        slots[1], slots[3] = -1, 7
        want, new_state, size = ref.short_conv(x, w, state, slots, old, cu, bias, True)
        out, status = torch.full((n_tok, 72), 9.0, dtype=x.dtype, device="cuda"), i32([0])
        qsa.short_conv(x, w, state, slots, old, cu, bias=bias, out=out, dev_status=status)
        mine = ~torch.isnan(want[:, 0])
        ref.check_conv(out[mine], want[mine], size[mine], x.dtype, 4)
        assert bool((out[~mine] == 9.0).all()) and int((~mine).sum()) == lens[1] + lens[3] + 21
        assert torch.equal(state, new_state) and int(status) == BAD_STATE


def test_bounds_out_of_order(qsa):
    """Bounds that fall, or lie outside the tokens, are reported; nothing outside the arrays is touched."""
    x, w, bias, state, slots, old, _ = make([20, 20, 20], 64, 4, torch.bfloat16, seed=1)
    for cu in ([0, 30, 10, 60], [0, 20, 40, 99], [-7, 20, 40, 60], [5, 20, 40, 60], [0, 2 ** 31 - 1, -2 ** 31, 60]):
        status = i32([0])
        qsa.short_conv(x, w, state, slots, old, i32(cu), bias=bias, dev_status=status)
        assert int(status) & BAD_LEN, cu


def test_infinities_stay_in_their_sequence(qsa):
    x, w, bias, state, slots, old, cu = make([10, 10, 10], 64, 4, torch.float16, seed=2)
    x = x.clone()
    x[10:20] = float("inf")
    state[slots[1].long()] = float("nan")
    want, new_state, size = ref.short_conv(x[:10], w, state, slots[:1], old[:1], cu[:2], bias, True)
    got = qsa.short_conv(x, w, state, slots, old, cu, bias=bias)
    ref.check_conv(got[:10], want, size, x.dtype, 4)
    assert bool(torch.isfinite(got[20:]).all())


def test_many_channels_and_tokens(qsa):
    """Offsets past 2^31 elements: rows far apart."""
    n_tok, apart = 300, 8_000_000
    x = torch.zeros((n_tok, apart), dtype=torch.bfloat16, device="cuda")[:, :16]
    x.copy_(torch.randn((n_tok, 16), generator=torch.Generator().manual_seed(1)).cuda())
    _, w, bias, state, slots, _, _ = make([n_tok], 16, 4, torch.bfloat16, seed=5)
    cu = i32([0, n_tok])
    want, new_state, size = ref.short_conv(x, w, state, slots, None, cu, bias, True)
    got = qsa.short_conv(x, w, state, slots, None, cu, bias=bias)
    ref.check_conv(got, want, size, x.dtype, 4)
    assert torch.equal(state, new_state)


def test_refusals(qsa):
    x, w, bias, state, slots, old, cu = make([4, 4], 64, 4, torch.bfloat16, seed=1)
    call = lambda **kw: qsa.short_conv(**{**dict(x=x, weight=w, state=state, state_slots=slots, old_lens=old, cu_tokens=cu, bias=bias), **kw})  # noqa: E731
    for bad in (dict(x=x.float()), dict(x=x.cpu()), dict(x=x[:, :60]), dict(x=x.t()), dict(weight=w[:60]), dict(weight=w.half()),
                dict(weight=w[:, :3]), dict(bias=bias.float()), dict(bias=bias[:8]), dict(state=state.float()),
                dict(state=state[:, :2]), dict(state_slots=slots.long()), dict(old_lens=old[:1]), dict(cu_tokens=cu[:2]),
                dict(cu_tokens=None), dict(activation="relu"), dict(out=torch.empty_like(x).half()), dict(out=x)):
        with pytest.raises((TypeError, ValueError, RuntimeError)):
            call(**bad)
    call()


@pytest.mark.parametrize("width,dtype", [(4, torch.bfloat16), (2, torch.float16)])
def test_many_tokens(qsa, width, dtype):
    """Steps of so many tokens and channels that runs of 32 tokens are taken: sequences of every length around them, and one alone."""
    ragged = [n for lens in LENS for n in lens]
    for lens in (ragged + [1900, 31, 32, 33, 0], [2600]):
        x, w, bias, state, slots, old, cu = make(lens, 16392, width, dtype, seed=len(lens))
        want, new_state, size = ref.short_conv(x, w, state, slots, old, cu, bias, True)
        got = qsa.short_conv(x, w, state, slots, old, cu, bias=bias)
        ref.check_conv(got, want, size, dtype, width, 16392)
        assert torch.equal(state, new_state)
