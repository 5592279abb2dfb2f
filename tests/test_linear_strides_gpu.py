"""The operators of layers with a state on slices of wider arrays: the results of contiguous ones, bit for bit, and nothing written
beside them."""
import pytest

torch = pytest.importorskip("torch")
import linear_ref as ref  # noqa: E402
from test_delta_gpu import batch, qsa  # noqa: E402,F401

pytestmark = pytest.mark.gpu


def inside(t, before=1, behind=2):
    """t's values in the middle of rows that are wider, everything else 9."""
    wide = torch.full((t.shape[0], t.shape[1] + before + behind, *t.shape[2:]), 9.0, dtype=t.dtype, device=t.device)
    part = wide[:, before:before + t.shape[1]]
    part.copy_(t)
    return wide, part


def only_inside(wide, width, before=1):
    return bool((wide[:, :before] == 9.0).all()) and bool((wide[:, before + width:] == 9.0).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("lens", [[20, 3], [300, 70, 1], [2200]], ids=["short", "chunks", "segments"])
def test_rule(qsa, lens, dtype):  # noqa: F811
    n_k, n_v = 2, 4
    inputs, state, slots, old, cu = batch(lens, n_k, n_v, dtype, seed=3)
    other = state.clone()
    want = qsa.delta_prompt(*(x.contiguous() for x in inputs), state, slots, old, cu)
    q, k, v, a, b = (inside(x)[1] for x in inputs[:5])
    wide, out = inside(torch.zeros_like(want))
    got = qsa.delta_prompt(q, k, v, a, b, *inputs[5:], other, slots, old, cu, out=out)
    assert got is out and torch.equal(out, want) and only_inside(wide, n_v) and torch.equal(state, other)
    # the same for single tokens
    n = len(lens)
    want = qsa.delta_step(*(x[:n].contiguous() for x in inputs[:5]), *inputs[5:], state, slots, old)
    wide, out = inside(torch.zeros_like(want))
    qsa.delta_step(q[:n], k[:n], v[:n], a[:n], b[:n], *inputs[5:], other, slots, old, out=out)
    assert torch.equal(out, want) and only_inside(wide, n_v) and torch.equal(state, other)


@pytest.mark.parametrize("lens", [[1] * 7, [40, 3, 0, 200]])
def test_convolution(qsa, lens):  # noqa: F811
    g = torch.Generator().manual_seed(2)
    n_tok, n_ch = sum(lens), 264
    x = torch.randn((n_tok, n_ch), generator=g).bfloat16().cuda()
    w, state = torch.randn((n_ch, 4), generator=g).bfloat16().cuda(), torch.randn((len(lens), 3, n_ch), generator=g).bfloat16().cuda()
    slots = torch.arange(len(lens), dtype=torch.int32, device="cuda")
    for cu in [torch.tensor([0, *lens], device="cuda").cumsum(0).int()] + ([None] if max(lens) == 1 else []):
        first, second = state.clone(), state.clone()
        want = qsa.short_conv(x, w, first, slots, None, cu)
        wide, out = inside(torch.zeros_like(x), 8, 16)
        qsa.short_conv(inside(x, 16, 8)[1], w, second, slots, None, cu, out=out)
        assert torch.equal(out, want) and only_inside(wide, n_ch, 8) and torch.equal(first, second)


@pytest.mark.parametrize("groups,size", [(3, 128), (1, 4096), (5, 8), (2, 520)])
def test_norm(qsa, groups, size):  # noqa: F811
    x, z = (torch.randn((50, groups, size), generator=torch.Generator().manual_seed(i)).bfloat16().cuda() for i in range(2))
    want = qsa.group_norm(x, gate=z)
    wide, out = inside(torch.zeros_like(x))
    qsa.group_norm(inside(x)[1], gate=inside(z, 2, 0)[1], out=out)
    assert torch.equal(out, want) and only_inside(wide, groups)
    assert ref.DIM == 128


def test_norm_of_many_tokens_in_place(qsa):  # noqa: F811
    """Enough groups for two to a thread; over its own input, and over its gate."""
    x, z = (torch.randn((3001, 16, 128), generator=torch.Generator().manual_seed(i)).bfloat16().cuda() for i in range(2))
    want = qsa.group_norm(x, gate=z, centred=True)
    a, b = x.clone(), z.clone()
    assert torch.equal(qsa.group_norm(a, gate=z, centred=True, out=a), want)
    assert torch.equal(qsa.group_norm(x, gate=b, centred=True, out=b), want)
