"""qsa_paged_attn where the cells that take most of the weight have V scales of zero (rows of zeros, as the cache's write
leaves them): they add to the sum of the weights and to nothing else, and the other cells keep their bits wherever those lie."""
import pytest

torch = pytest.importorskip("torch")
import serve_ref as ref  # noqa: E402
from test_paged_attn_gpu import SCALE, make, qsa, run  # noqa: E402, F401

pytestmark = pytest.mark.gpu


def raised(lens, cells, nats, seed, wide, v_scale=0.0, n_kv=1, group=4):
    """A batch in which dim 0 of every query is 4 and of every key 0, but for the named cells of each sequence, whose
    scores are `nats` (the others' are about normal, deviation 1.5) and whose V scale is `v_scale`."""
    q, cache, tables, n = make(lens, n_kv, group, seed, width=400 if wide else None)
    q[..., 0] = 4
    cache[0][..., 0] = 0
    for s, own in enumerate(cells):
        for c in own:
            page = int(tables[s, c // 64])
            cache[0][page, :, c % 64] = 0
            cache[0][page, :, c % 64, 0] = 127
            cache[2][page, :, c % 64] = nats / (4 * 127 * SCALE)
            cache[3][page, :, c % 64] = v_scale
            v = cache[1][page, :, c % 64]
            v[v == 0] = 1
    return q, cache, tables, n


def check(qsa, q, cache, tables, n, window=0):  # noqa: F811
    out, lse = run(qsa, q, cache, tables, n, window=window)
    ref.check_attn(out, lse, ref.paged_attn(q, *cache, tables, n, SCALE, window))


NATS = [8, 16, 20, 30, 40]


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("nats", NATS)
def test_first_step_without_values(qsa, nats, wide):  # noqa: F811
    """The first 32 cells have no values and the largest scores: nothing to go by when the row's reference is set."""
    q, cache, tables, n = raised([2048, 33, 700], [range(32)] * 3, nats, 31, wide)
    check(qsa, q, cache, tables, n)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("nats", NATS + [46])
def test_later_steps_without_values(qsa, nats, wide):  # noqa: F811
    """Whole steps of such cells in the middle and at the end, up to 66 binary orders above what came before."""
    q, cache, tables, n = raised([2048, 640, 6000], [range(1024, 1056), range(608, 640), range(5000, 5100)], nats, 32, wide)
    check(qsa, q, cache, tables, n)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("nats", NATS)
def test_a_windows_first_cell_without_values(qsa, nats, wide):  # noqa: F811
    """The window begins with the last cell of a step, and that cell has no values."""
    window = 1000
    lens = [1031, 3047, 1063]
    cells = [[length - window] for length in lens]
    assert all(c[0] % 32 == 31 for c in cells)
    q, cache, tables, n = raised(lens, cells, nats, 33, wide)
    check(qsa, q, cache, tables, n, window)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("v_scale", [0.0, 2.0 ** -24, -2.0 ** -24])
@pytest.mark.parametrize("nats", NATS)
def test_single_cells_among_others(qsa, nats, v_scale, wide):  # noqa: F811
    """One such cell in a step of ordinary ones, first, in the middle and last; also with the smallest V scales there are."""
    q, cache, tables, n = raised([2048, 2048, 2048, 3], [[5], [1500], [2047], [1]], nats, 34, wide, v_scale, n_kv=2, group=12)
    check(qsa, q, cache, tables, n)


@pytest.mark.parametrize("wide", [False, True])
def test_no_values_at_all(qsa, wide):  # noqa: F811
    q, cache, tables, n = raised([2048, 33, 700], [range(32)] * 3, 20, 35, wide)
    cache[3][torch.isfinite(cache[3])] = 0
    out, lse = run(qsa, q, cache, tables, n)
    assert not out.any()
    ref.check_attn(out, lse, ref.paged_attn(q, *cache, tables, n, SCALE))
