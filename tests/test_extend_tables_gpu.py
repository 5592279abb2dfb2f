"""qsa_extend_tables on the GPU against a token-by-token reference, and the whole serving step run together."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import serve_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qsa():
    from sparse_selected_cell_gb300 import qsa as q
    if not torch.cuda.is_available():
        pytest.fail("CUDA GPU required")
    q.lib()
    return q


def setup(n_seq, old, lo, hi, seed, width=None):
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, old + 1, n_seq)
    new = rng.integers(lo, hi + 1, n_seq)
    width = -(-(old + hi) // 64) + 1 if width is None else width
    pool = n_seq * width + 3
    perm = rng.permutation(pool)
    tables, at = np.full((n_seq, width), -1), 0
    for s in range(n_seq):
        held = -(-int(lens[s]) // 64)
        tables[s, :held] = perm[at:at + held]
        at += held
    return lens, new, tables, perm, at, pool


def run(qsa, lens, new, tables, free, head, n_tok, n_ppages):
    i = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
    t = i(tables)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = [torch.full((n,), -77, dtype=torch.int32, device="cuda") for n in (n_tok, n_tok, n_tok, len(lens), len(lens) + 1, 1)]
    got = qsa.extend_tables(i(lens), i(new), t, i(free), n_tok, n_ppages, free_head=None if head is None else i([head]), out=out,
                            dev_status=status)
    torch.cuda.synchronize()
    return [t.cpu().numpy()] + [x.cpu().numpy() for x in got], int(status.item())


def check(qsa, lens, new, tables, free, head, n_tok, n_ppages):
    got, bits = run(qsa, lens, new, tables, free, head, n_tok, n_ppages)
    *want, want_head, want_bits = ref.extend_tables(lens, new, tables, free, n_tok, n_ppages, head or 0)
    for name, g, w in zip(("tables", "slots", "positions", "token_seq", "seq_lens", "cu_tokens"), got, want):
        assert np.array_equal(g, w), name
    assert got[6].tolist() == [want_head]
    assert bits == want_bits
    return bits


@pytest.mark.parametrize("n_seq,old,lo,hi,pad", [
    (1, 0, 1, 1, 0), (1, 100, 1, 1, 5), (1, 64, 0, 0, 3), (1, 63, 5000, 5000, 0), (7, 200, 0, 3, 9), (64, 1000, 1, 1, 0),
    (300, 500, 0, 200, 1000), (1023, 300, 1, 1, 1), (1024, 300, 1, 1, 0), (1025, 300, 0, 2, 77), (5000, 130, 0, 3, 10),
    (3, 5, 4000, 4100, 4096)])
def test_against_reference(qsa, n_seq, old, lo, hi, pad):
    lens, new, tables, perm, at, pool = setup(n_seq, old, lo, hi, seed=n_seq + hi)
    assert check(qsa, lens, new, tables, perm, at, int(new.sum()) + pad, pool) == 0


def test_lengths_at_page_borders(qsa):
    lens = np.array([0, 1, 63, 64, 65, 127, 128, 0, 64])
    new = np.array([64, 63, 1, 1, 63, 2, 0, 0, 65])
    _, _, _, perm, _, pool = setup(9, 200, 0, 0, seed=1)
    tables, at = np.full((9, 4), -1), 0
    for s in range(9):
        held = -(-lens[s] // 64)
        tables[s, :held] = perm[at:at + held]
        at += held
    assert check(qsa, lens, new, tables, perm, at, int(new.sum()), pool) == 0


def test_nothing_to_do(qsa):
    assert check(qsa, np.zeros(0, int), np.zeros(0, int), np.zeros((0, 4), int), np.arange(5), 2, 70, 5) == 0
    assert check(qsa, np.array([5, 0]), np.array([0, 0]), np.array([[1, -1], [-1, -1]]), np.arange(5), 2, 0, 5) == 0
    assert check(qsa, np.array([0, 0]), np.array([70, 1]), np.full((2, 2), -1), np.arange(5), None, 71, 5) == 0   # no head: 0


def test_what_is_reported(qsa):
    lens, new, tables, perm, at, pool = setup(20, 300, 1, 200, seed=3)
    n_tok = int(new.sum())
    assert check(qsa, lens, new, tables, perm, at, n_tok - 250, pool) == 256                   # the token arrays are too short
    assert check(qsa, lens, new, tables, perm[:at + 9], at, n_tok, pool) == 128                # the free list runs out
    assert check(qsa, lens, new, tables, perm, len(perm) + 1, n_tok, pool) == 128
    assert check(qsa, lens, new, tables, perm, -1, n_tok, pool) & 128 == 128
    bad = perm.copy()
    bad[at + 2], bad[at + 4] = -1, pool
    assert check(qsa, lens, new, tables, bad, at, n_tok, pool) == 8                            # entries that are no pages
    part = next(s for s in range(20) if lens[s] % 64 and new[s])
    gone = tables.copy()
    gone[part, lens[part] // 64] = -1
    assert check(qsa, lens, new, gone, perm, at, n_tok, pool) == 128                           # the page to go on is not resident
    gone[part, lens[part] // 64] = pool + 5
    assert check(qsa, lens, new, gone, perm, at, n_tok, pool) == 8
    wrong, more = lens.copy(), new.copy()
    wrong[3], more[5], more[7] = -4, -1, 10 ** 6
    assert check(qsa, wrong, more, tables, perm, at, n_tok + 70000, pool) & 64 == 64           # lengths outside the table


def test_lengths_near_the_top_of_int32(qsa):
    """Sums of new lengths past 2^31 stop at the token arrays."""
    lens, new, tables, perm, at, pool = setup(50, 100, 1, 3, seed=4, width=40)
    new[10:] = 2 ** 31 - 1
    assert check(qsa, lens, new, tables, perm, at, 9000, pool) & 256


def test_refusals(qsa):
    i = lambda *shape: torch.zeros(shape, dtype=torch.int32, device="cuda")  # noqa: E731
    good = dict(seq_lens=i(3), new_lens=i(3), page_tables=i(3, 4), free_pages=i(9), n_tok=5, n_ppages=20)
    out = [i(5), i(5), i(5), i(3), i(4), i(1)]
    assert qsa.extend_tables(**good, out=out).slots is out[0]
    for bad in (dict(seq_lens=i(3).cpu()), dict(seq_lens=i(3).long()), dict(new_lens=i(2)), dict(page_tables=i(4, 4)),
                dict(page_tables=i(12)), dict(page_tables=i(3, 8)[:, ::2]), dict(free_pages=None), dict(free_head=i(2)), dict(n_tok=-1),
                dict(n_ppages=1 << 31), dict(out=out[:3] + [i(4)] + out[4:]), dict(out=[i(4)] + out[1:])):
        with pytest.raises((TypeError, ValueError)):
            qsa.extend_tables(**{**good, **bad})
    head = i(1)
    with pytest.raises(qsa.QsaError):                          # the head's place cannot be read and written by one call
        qsa.extend_tables(**good, free_head=head, out=out[:5] + [head])
    with pytest.raises(qsa.QsaError):
        qsa.extend_tables(**good, out=out[:3] + [good["new_lens"]] + out[4:])


def test_captured_steps_follow_the_lengths(qsa):
    """One captured step replayed: lengths, tables and the list's head advance on the device alone."""
    n_seq, width, pool = 4, 6, 40
    i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    free = torch.randperm(pool, generator=torch.Generator().manual_seed(2)).int().cuda()
    lens, new, tables, head = i([0, 63, 64, 130]), i([1, 1, 1, 1]), torch.full((n_seq, width), -1, dtype=torch.int32, device="cuda"), i([6])
    held = [0, 1, 1, 3]
    at = 0
    for s, n in enumerate(held):
        tables[s, :n] = free[at:at + n]
        at += n
    out = [torch.zeros(n, dtype=torch.int32, device="cuda") for n in (8, 8, 8, n_seq, n_seq + 1, 1)]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    want_lens, want_tables, want_head = lens.cpu().numpy(), tables.cpu().numpy(), 6
    with torch.cuda.graph(graph, stream=stream):
        step = qsa.extend_tables(lens, new, tables, free, 8, pool, free_head=head, out=out)
        lens.copy_(step.seq_lens)
        head.copy_(step.free_head)
    for _ in range(70):
        graph.replay()
        torch.cuda.synchronize()
        want_tables, slots, pos, seq, want_lens, cu, want_head, bits = ref.extend_tables(
            want_lens, [1] * n_seq, want_tables, free.cpu().numpy(), 8, pool, want_head)
        assert bits == 0
        assert step.slots.tolist() == slots.tolist() and step.positions.tolist() == pos.tolist()
        assert lens.tolist() == want_lens.tolist() and head.tolist() == [want_head]
        assert tables.cpu().numpy().tolist() == want_tables.tolist()


def test_serving_steps_run_together(qsa):
    """A prompt step and three decode steps: tables extended, keys and values rotated and written, attention over the
    whole cache, all on one stream without the host reading anything; the output is checked against FP64 attention over
    the cache as it stands, and the cache against the rotated keys and values, within half a step of their rows' scales."""
    n_kv, group, n_seq = 2, 12, 5
    n_heads = n_kv * group
    g = torch.Generator().manual_seed(5)
    inv = (10000.0 ** (-torch.arange(64, dtype=torch.float64) / 64)).cuda()
    pool = 40
    cache = [t.cuda() for t in ref.make_cache(pool, n_kv, seed=6)]
    tables = torch.full((n_seq, 6), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(pool, generator=g).int().cuda()
    head = torch.zeros(1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(n_seq, dtype=torch.int32, device="cuda")
    held_k = [[] for _ in range(n_seq)]
    held_v = [[] for _ in range(n_seq)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for new in ([130, 64, 0, 200, 1], [1] * 5, [1] * 5, [1, 0, 1, 1, 1]):
        n_tok = sum(new) + 3
        qkv = torch.randn((n_tok, n_heads + 2 * n_kv, 128), generator=g).bfloat16().cuda()
        step = qsa.extend_tables(lens, torch.tensor(new, dtype=torch.int32, device="cuda"), tables, free, n_tok, pool,
                                 free_head=head, dev_status=status)
        q = qsa.rope_append(qkv[:, :n_heads], qkv[:, n_heads:n_heads + n_kv], qkv[:, n_heads + n_kv:], step.positions, inv,
                            None, *cache, step.slots, dev_status=status)
        lens, head = step.seq_lens, step.free_head
        last = (step.cu_tokens[1:] - 1).clamp(min=0).long()
        out = qsa.paged_attn(q[last], *cache, tables, lens, dev_status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == 0, qsa.decode_status(int(status.item()))
        ref.check_attn(out, None, ref.paged_attn(q[last].cpu(), *[t.cpu() for t in cache], tables.cpu(), lens.cpu(), 128 ** -0.5))
        k = ref.turned(qkv[:, n_heads:n_heads + n_kv], step.positions[None], inv, None, False)
        for t, s in enumerate(step.token_seq.tolist()):
            if s >= 0:
                held_k[s].append(k[t])
                held_v[s].append(qkv[t, n_heads + n_kv:].double().cpu())
        for s in range(n_seq):
            assert len(held_k[s]) == int(lens[s])
            if not held_k[s]:
                assert not out[s].any()
                continue
            c = torch.arange(len(held_k[s]))
            slots = tables[s].cpu().long()[c // 64] * 64 + c % 64
            kk, vv = qsa.cache_gather(*cache, slots.int().cuda(), dtype=torch.float32)
            for got, held in ((kk, held_k[s]), (vv, held_v[s])):
                want = torch.stack(held)
                # half a step of a scale that was rounded up by at most 2^-10, and FP32 rotation
                assert ((got.double().cpu() - want).abs() <= want.abs().amax(-1, keepdim=True) / 127 * 0.502 + 1e-5).all()


def test_a_step_on_another_stream(qsa):
    """The calls of a step given a stream that is not the current one, with everything they return allocated by them:
    the same bits as on the current stream, whatever the current stream allocates meanwhile."""
    n_kv, n_heads, pool, new = 2, 24, 30, [70, 1, 300, 0, 64]
    g = torch.Generator().manual_seed(7)
    inv = (10000.0 ** (-torch.arange(64, dtype=torch.float64) / 64)).cuda()
    i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    qkv = torch.randn((sum(new), n_heads + 2 * n_kv, 128), generator=g).bfloat16().cuda()
    free, lens, add = torch.randperm(pool, generator=g).int().cuda(), i([0] * 5), i(new)
    last = (torch.tensor(new).cumsum(0) - 1).clamp(min=0).cuda()

    def step(stream):
        cache = [t.cuda() for t in ref.make_cache(pool, n_kv, seed=8)]
        tables = torch.full((5, 8), -1, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        t = qsa.extend_tables(lens, add, tables, free, len(qkv), pool, stream=stream)
        torch.full((1 << 20,), 7, dtype=torch.int32, device="cuda")
        q = qsa.rope_append(qkv[:, :n_heads], qkv[:, n_heads:n_heads + n_kv], qkv[:, n_heads + n_kv:], t.positions, inv,
                            None, *cache, t.slots, stream=stream)
        x = qsa.rope(qkv[:, :n_heads], t.positions, inv, stream=stream)
        torch.full((1 << 20,), -1, dtype=torch.int32, device="cuda")
        k, v = qsa.cache_gather(*cache, t.slots, stream=stream)
        torch.cuda.synchronize()
        held = q[last]
        torch.cuda.synchronize()
        out = qsa.paged_attn(held, *cache, tables, t.seq_lens, stream=stream)
        torch.cuda.synchronize()
        return [*t, q, x, k, v, out, tables]

    want = step(None)
    for stream in (torch.cuda.Stream(), torch.cuda.Stream().cuda_stream, 0):
        for got, w in zip(step(stream), want):
            assert torch.equal(got, w)
    assert torch.equal(want[6], want[7])                       # queries are turned alike by both calls
