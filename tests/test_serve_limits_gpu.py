"""The serving calls at sizes on both sides of the rules that choose between their kernels: the same results."""
import pytest

torch = pytest.importorskip("torch")
from test_cache_rows_gpu import cuda, rotation, step  # noqa: E402
from test_paged_attn_gpu import qsa  # noqa: E402, F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n_tok", [303, 304, 305, 306, 380, 381])
def test_write_of_so_many_tokens_is_that_of_each_alone(qsa, n_tok):  # noqa: F811
    """Eight or four warps to a token: the rows are computed alike, bit for bit."""
    qkv, cache, slots = step(n_tok, 24, 2, seed=n_tok)
    pos, inv, axis = cuda(*rotation(n_tok, 64, 2, 50000, seed=n_tok))
    d, slots = qkv.cuda(), slots.cuda()

    def write(parts):
        pools = cuda(*cache)
        q = [qsa.rope_append(d[a:b, :24], d[a:b, 24:26], d[a:b, 26:], pos[:, a:b].contiguous(), inv, axis, *pools, slots[a:b])
             for a, b in parts]
        return [torch.cat(q), *pools]

    for got, want in zip(write([(0, n_tok)]), write([(k, min(k + 100, n_tok)) for k in range(0, n_tok, 100)])):
        assert torch.equal(got, want)
