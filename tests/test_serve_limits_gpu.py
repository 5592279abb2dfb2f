"""The serving calls at sizes on both sides of the rules that choose between their kernels: the same results."""
import pytest

torch = pytest.importorskip("torch")
import serve_ref as ref  # noqa: E402
from test_cache_rows_gpu import cuda, rotation, step  # noqa: E402
from test_paged_attn_gpu import SCALE, make, qsa, run  # noqa: E402, F401

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


@pytest.mark.parametrize("items", [1, 31, 32, 33, 35, 36, 37, 38, 39, 40, 64, 65])
def test_attention_with_so_many_items(qsa, items):  # noqa: F811
    """One KV head, so an item a sequence: clusters, runs with few items and with many."""
    q, cache, tables, n = make([(997 * k) % 700 for k in range(1, items + 1)], 1, 12, seed=items)
    out, lse = run(qsa, q, cache, tables, n)
    ref.check_attn(out, lse, ref.paged_attn(q, *cache, tables, n, SCALE))


@pytest.mark.parametrize("items", [32, 33, 36, 37])
def test_so_many_items_captured(qsa, items):  # noqa: F811
    """The choice is made while the stream is being captured."""
    q, cache, tables, n = make([(997 * k) % 700 for k in range(1, items + 1)], 1, 12, seed=items)
    d = [t.cuda() for t in (q, *cache, tables, n)]
    want = qsa.paged_attn(*d)
    out = torch.zeros_like(want)
    ws = torch.empty(qsa.paged_attn_workspace_bytes(1, 12), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qsa.paged_attn(*d, out=out, workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("width", [65, 66, 67, 128, 512])
def test_attention_under_tables_of_any_width(qsa, width):  # noqa: F811
    """Tables wider than the sequences: one item takes clusters up to 66 pages, and runs from there."""
    q, cache, tables, n = make([1021], 1, 12, seed=1, width=width)
    out, lse = run(qsa, q, cache, tables, n)
    ref.check_attn(out, lse, ref.paged_attn(q, *cache, tables, n, SCALE))


def test_part_of_a_wide_table(qsa):  # noqa: F811
    """n_lpages below the tables' width: the bits of tables cut to it; longer sequences are clamped to it and reported."""
    q, cache, tables, n = make([1021, 64, 700], 2, 12, seed=2, width=512)
    cut = tables[:, :16].contiguous()
    want = run(qsa, q, cache, cut, n)
    ref.check_attn(*want, ref.paged_attn(q, *cache, tables, n, SCALE))
    for got, w in zip(run(qsa, q, cache, tables, n, n_lpages=16), want):
        assert torch.equal(got, w)
    for got, w in zip(run(qsa, q, cache, tables, n, n_lpages=11, want_status=64),
                      run(qsa, q, cache, cut, torch.tensor([11 * 64, 64, 700], dtype=torch.int32))):
        assert torch.equal(got, w)
    for bad in (513, -1):
        with pytest.raises(qsa.QsaError):
            run(qsa, q, cache, tables, n, n_lpages=bad)
