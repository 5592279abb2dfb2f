"""The check of the delta rule's outputs by 2-norms: what it lets pass and what not, on the CPU."""
import pytest

torch = pytest.importorskip("torch")
import delta_norms as norms  # noqa: E402
import linear_ref as ref  # noqa: E402


def rule(lens, dtype, no_decay, bits=None, out_bits=None):
    """(want, L) and outputs by FP32 steps; with `bits` the state as it enters the outputs is rounded to so many."""
    q, k, v, a, b, a_log, dt = ref.heads(sum(lens), 1, 2, dtype, 5, device="cpu")
    if no_decay:
        a_log = torch.full_like(a_log, float("-inf"))
    state, slots = ref.pool(len(lens), 2, 5, device="cpu"), torch.arange(len(lens), dtype=torch.int32)
    cu = torch.tensor([0, *lens]).cumsum(0).int()
    want, size = norms.delta(q, k, v, a, b, a_log, dt, state, slots, None, cu, 1e-6, ref.DIM ** -0.5)
    alpha, beta = (x.float() for x in ref.gates(a, b, a_log, dt))
    unit = lambda x: (x.float() / torch.sqrt(x.float().square().sum(-1, keepdim=True) + 1e-6)).repeat_interleave(2, 1)  # noqa: E731
    qn, kn, out = unit(q), unit(k), torch.zeros(v.shape)
    for s, (lo, hi) in enumerate(ref.spans(cu)):
        st = state[s].clone()
        for t in range(lo, hi):
            st = alpha[t][:, None, None] * st
            st = st + (beta[t][:, None] * (v[t].float() - torch.einsum("hvk,hk->hv", st, kn[t])))[..., None] * kn[t][:, None, :]
            seen = st
            if bits is not None:
                e = torch.exp2(torch.floor(torch.log2(st.abs().clamp(min=2.0 ** -100))) - (bits - 1))
                seen = torch.round(st / e) * e
            out[t] = torch.einsum("hvk,hk->hv", seen, qn[t]) * ref.DIM ** -0.5
    return want, size, out.to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("no_decay", [False, True])
def test_what_passes_and_what_does_not(dtype, no_decay):
    want, size, got = rule([70, 30], dtype, no_decay)
    norms.check(got, want, size, dtype)
    for wrong in (torch.zeros_like(got), got.float().mul(1 + torch.finfo(dtype).eps).to(dtype), rule([70, 30], dtype, no_decay, bits=10)[2]):
        with pytest.raises(AssertionError):
            norms.check(wrong, want, size, dtype)


def test_rows_of_nobody_are_left_alone():
    want, size, got = rule([20], torch.bfloat16, False)
    want, got = want.clone(), got.clone()
    want[5:9], got[5:9] = float("nan"), float("nan")
    norms.check(got, want, size, torch.bfloat16)
