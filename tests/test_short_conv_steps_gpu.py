"""qsa_short_conv on the GPU without cu_tokens (one token to every sequence): every type, width and activation, more sequences than
run at once, and sequences left out, against its 64-bit definition."""
import pytest

torch = pytest.importorskip("torch")
import linear_ref as ref  # noqa: E402
from test_short_conv_gpu import BAD_STATE, i32, make, qsa  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("width", [2, 3, 4])
@pytest.mark.parametrize("n_seq,n_ch", [(1, 8), (40, 264), (1700, 8), (150, 16392)])
def test_steps(qsa, n_seq, n_ch, width, dtype):  # noqa: F811
    for silu, with_bias, w_type in ((True, True, dtype), (False, False, torch.float32)):
        x, w, bias, state, slots, old, cu = make([1] * n_seq, n_ch, width, dtype, seed=n_seq + width, wide=8, w_type=w_type)
        bias = bias if with_bias else None
        for step in range(2):
            want, new_state, size = ref.short_conv(x, w, state, slots, old, cu, bias, silu)
            got = qsa.short_conv(x, w, state, slots, old, bias=bias, activation="silu" if silu else "none")
            ref.check_conv(got, want, size, dtype, width, n_ch)
            assert torch.equal(state, new_state)
            old = None


@pytest.mark.parametrize("n_seq", [5, 900])
def test_left_out(qsa, n_seq):  # noqa: F811
    x, w, bias, state, slots, old, cu = make([1] * n_seq, 8, 3, torch.float16, seed=4)
    slots[1], slots[n_seq - 2] = -1, n_seq + 2
    x[1] = float("nan")
    want, new_state, size = ref.short_conv(x, w, state, slots, old, cu, bias, True)
    out, status = torch.full((n_seq, 8), 9.0, dtype=x.dtype, device="cuda"), i32([0])
    qsa.short_conv(x, w, state, slots, old, bias=bias, out=out, dev_status=status)
    mine = ~torch.isnan(want[:, 0])
    ref.check_conv(out[mine], want[mine], size[mine], x.dtype, 3)
    assert bool((out[~mine] == 9.0).all()) and int((~mine).sum()) == 2 and torch.equal(state, new_state) and int(status) == BAD_STATE
