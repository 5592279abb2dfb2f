"""qsa_paged_attn on the GPU against the 64-bit definition."""
import math

import pytest

torch = pytest.importorskip("torch")
import serve_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5
NAN16, BAD_LEN, BAD_PAGE = float("nan"), 64, 8


@pytest.fixture(scope="module")
def qsa():
    from sparse_selected_cell_gb300 import qsa as q
    if not torch.cuda.is_available():
        pytest.fail("CUDA GPU required")
    q.lib()
    return q


def make(lens, n_kv, group, seed, width=None, missing=0.0, spare=2, q_type=torch.bfloat16):
    """A batch with shuffled pages; cells past each length, spare pages and (as the tables name none) the entries past
    a length's last page hold what must never show: NaN scales and page numbers far outside the pool."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // 64) for n in lens]
    width = max(need + [1]) + 1 if width is None else width
    cache = ref.make_cache(sum(need) + spare, n_kv, seed)
    order = torch.randperm(sum(need) + spare, generator=g).int()
    tables = torch.full((len(lens), width), 1 << 30, dtype=torch.int32)
    at = 0
    for s, n in enumerate(lens):
        tables[s, :need[s]] = order[at:at + need[s]]
        at += need[s]
        if n % 64:
            last = int(tables[s, need[s] - 1])
            cache[2][last, :, n % 64:] = NAN16
            cache[3][last, :, n % 64:] = NAN16
    for p in order[at:].tolist():
        cache[2][p] = NAN16
        cache[3][p] = NAN16
    if missing:
        off = torch.rand(tables.shape, generator=g) < missing
        off &= torch.arange(width)[None] < torch.tensor(need)[:, None]
        tables[off] = -1
    q = torch.randn((len(lens), n_kv * group, 128), generator=g).to(q_type)
    return q, cache, tables, torch.tensor(lens, dtype=torch.int32)


def run(qsa, q, cache, tables, lens, out_type=torch.float32, want_status=0, **kw):
    n_seq, n_heads = q.shape[:2]
    out = torch.full((n_seq, n_heads, 128), NAN16, dtype=out_type, device="cuda")
    lse = torch.full((n_seq, n_heads), NAN16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.full((qsa.paged_attn_workspace_bytes(cache[0].shape[1], n_heads),), 0xFF, dtype=torch.uint8, device="cuda")
    got = qsa.paged_attn(q.cuda(), *[t.cuda() for t in cache], tables.cuda(), lens.cuda(), out=out, lse=lse, workspace=ws,
                         dev_status=status, **kw)
    assert got is out
    torch.cuda.synchronize()
    assert int(status.item()) == want_status, qsa.decode_status(int(status.item()))
    return out, lse


CASES = [  # lengths, KV heads, group
    ([1], 1, 1), ([1], 4, 12), ([0], 1, 12), ([0, 0, 0], 2, 4), ([63], 1, 8), ([64], 1, 8), ([65], 2, 16), ([128], 1, 12),
    ([0, 1, 2, 63, 64, 65, 127, 128, 129, 0], 2, 12), ([1021], 4, 12), ([257, 0, 4097], 1, 7), ([700, 1, 64], 2, 17),
    ([500], 1, 40), ([5] * 300, 1, 12), ([64] * 70, 4, 2), ([20001], 1, 12), ([3000, 10, 9000, 1, 0, 700], 4, 12),
    ([130 * k % 1000 for k in range(200)], 2, 3), ([66000], 8, 5),
]


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("lens,n_kv,group", CASES)
def test_against_definition(qsa, lens, n_kv, group, wide):
    """wide: tables far longer than the sequences, which takes the kernel for long ones."""
    width = max(300, max(lens) // 64 + 2) if wide else None
    q, cache, tables, n = make(lens, n_kv, group, seed=len(lens) * 100 + group, width=width)
    out, lse = run(qsa, q, cache, tables, n)
    ref.check_attn(out, lse, ref.paged_attn(q, *cache, tables, n, SCALE))


@pytest.mark.parametrize("window", [1, 5, 63, 64, 65, 1000, 1 << 20])
def test_window(qsa, window):
    """Cells before the window may hold anything, and the table's entries of pages before it are not read."""
    lens = [0, 1, 64, 65, 300, 1000, 1001, 5000]
    q, cache, tables, n = make(lens, 2, 12, seed=window % 97)
    want = ref.paged_attn(q, *cache, tables, n, SCALE, window)
    for s, length in enumerate(lens):
        first = max(0, length - window)
        if first % 64:
            cache[2][tables[s, first // 64], :, :first % 64] = NAN16
            cache[3][tables[s, first // 64], :, :first % 64] = NAN16
        tables[s, :first // 64] = 1 << 30
    out, lse = run(qsa, q, cache, tables, n, window=window)
    ref.check_attn(out, lse, want)


@pytest.mark.parametrize("q_type", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("out_type", [torch.bfloat16, torch.float16, torch.float32])
def test_types(qsa, q_type, out_type):
    q, cache, tables, n = make([0, 70, 2222, 5], 2, 6, seed=5, q_type=q_type)
    out, lse = run(qsa, q, cache, tables, n, out_type=out_type)
    ref.check_attn(out, lse, ref.paged_attn(q, *cache, tables, n, SCALE))


@pytest.mark.parametrize("missing", [0.1, 0.6, 1.0])
def test_pages_not_resident(qsa, missing):
    q, cache, tables, n = make([0, 64, 65, 1000, 6000, 12345], 2, 12, seed=6, missing=missing)
    out, lse = run(qsa, q, cache, tables, n)
    ref.check_attn(out, lse, ref.paged_attn(q, *cache, tables, n, SCALE))
    if missing == 1.0:
        assert not out.any()


def test_bad_lengths_and_pages_are_reported(qsa):
    q, cache, tables, n = make([100, 200, 64], 1, 12, seed=7, width=4)
    tables[1, 1] = cache[0].shape[0]
    masked = tables.clone()
    masked[1, 1] = -1
    lens = n.clone()
    lens[2] = -3
    out, lse = run(qsa, q, cache, tables, lens, want_status=BAD_LEN | BAD_PAGE)
    lens[2] = 0
    ref.check_attn(out, lse, ref.paged_attn(q, *cache, masked, lens, SCALE))
    # a length past the table is clamped to it
    q, cache, tables, n = make([256], 1, 12, seed=8, width=4)
    out, lse = run(qsa, q, cache, tables, torch.tensor([257], dtype=torch.int32), want_status=BAD_LEN)
    ref.check_attn(out, lse, ref.paged_attn(q, *cache, tables, n, SCALE))


@pytest.mark.parametrize("sm_scale", [0.0, -0.07, 1.0])
def test_scales_of_the_scores(qsa, sm_scale):
    """0: the mean of the values; negative: the order of the scores turns round; 1: nearly one cell takes all."""
    q, cache, tables, n = make([1, 777, 4000], 2, 12, seed=9)
    out, lse = run(qsa, q, cache, tables, n, sm_scale=sm_scale)
    ref.check_attn(out, lse, ref.paged_attn(q, *cache, tables, n, sm_scale))


def test_rows_and_values_of_any_size(qsa):
    """Query rows far outside FP16, value scales from subnormal to the largest, of both signs, and zeros."""
    q, cache, tables, n = make([3000, 70], 1, 12, seed=10)
    for i, e in enumerate([-100, -60, -30, -15, 12, 14, 20, 40]):
        q[:, i] = (q[:, i].float() * 2.0 ** e).bfloat16()
        if e > 0:                       # rows with a large factor hold one element only
            keep = q[:, i, :1].clone()
            q[:, i] = 0
            q[:, i, :1] = keep
    q[:, 8] = 0
    g = torch.Generator().manual_seed(3)
    vs = cache[3]
    live = torch.isfinite(vs)
    big = torch.randint(-24, 13, vs.shape, generator=g)
    vs[live] = (torch.ldexp(torch.ones(()), big) * torch.where(torch.rand(vs.shape, generator=g) < 0.5, -1.0, 1.0))[live].half()
    vs[live & (torch.rand(vs.shape, generator=g) < 0.1)] = 0
    out, lse = run(qsa, q, cache, tables, n)
    ref.check_attn(out, lse, ref.paged_attn(q, *cache, tables, n, SCALE))


def test_a_score_far_above_the_others(qsa):
    """One cell 20 to 90 above the rest, early, late and in the middle: the running maximum jumps."""
    q, cache, tables, n = make([4000] * 6, 1, 4, seed=11)
    for s, c in enumerate([0, 3999, 2000, 63, 64, 3000]):
        page = int(tables[s, c // 64])
        sign = torch.sign(q[s, 0].float())
        cache[0][page, 0, c % 64] = (127 * sign).to(torch.int8)
        cache[2][page, 0, c % 64] = 0.03 * (s + 1)
    out, lse = run(qsa, q, cache, tables, n)
    ref.check_attn(out, lse, ref.paged_attn(q, *cache, tables, n, SCALE))


def test_many_small_weights_beside_a_large_one(qsa):
    """30,000 cells at e^-9 of the top weight (each), all with the same value: their sum outweighs it, and must not be
    lost to the weights' rounding."""
    n = 30000
    q, cache, tables, lens = make([n], 1, 4, seed=12)
    q[:] = 1.0
    cache[0][:] = 0
    cache[1][:] = 100
    page = int(tables[0, 100])
    cache[0][page, 0, 7] = 127
    cache[1][page, 0, 7] = -100
    cache[2][page, 0, 7] = 9.0 / (SCALE * 128 * 127)
    out, lse = run(qsa, q, cache, tables, lens)
    ref.check_attn(out, lse, ref.paged_attn(q, *cache, tables, lens, SCALE))


def test_keys_with_outliers(qsa):
    """Rows whose scale one large dim sets: all other integers are 0 to 3, as channels with outliers leave them; queries
    all positive, so that the biased sums are as large as they get."""
    q, cache, tables, n = make([700, 3000, 64], 2, 12, seed=20)
    q = q.abs()
    cache[0][:] = cache[0] % 4
    cache[0][..., 17] = 127
    out, lse = run(qsa, q, cache, tables, n)
    ref.check_attn(out, lse, ref.paged_attn(q, *cache, tables, n, SCALE, bias=256))


def test_nan_scale_shows_in_its_own_sequence_only(qsa):
    """A key scale that is NaN poisons the rows that read it and no others."""
    q, cache, tables, n = make([500, 500, 300], 2, 12, seed=13)
    clean = run(qsa, q, cache, tables, n)[0]
    cache[2][int(tables[1, 2]), 0, 5] = NAN16
    out, lse = run(qsa, q, cache, tables, n)
    assert torch.isnan(out[1, :12]).all() and torch.isnan(lse[1, :12]).all()
    assert torch.equal(out[0], clean[0]) and torch.equal(out[2], clean[2]) and torch.equal(out[1, 12:], clean[1, 12:])


def test_same_bits_again_and_shared_pages(qsa):
    """Sequences that share all their pages, run twice over a workspace that held something else: the same bits."""
    q, cache, tables, n = make([9000, 64, 2000], 4, 12, seed=14)
    tables = tables[:1].repeat(3, 1)
    a, la = run(qsa, q, cache, tables, n)
    b, lb = run(qsa, q, cache, tables, n)
    assert torch.equal(a, b) and torch.equal(la, lb)
    ref.check_attn(a, la, ref.paged_attn(q, *cache, tables, n, SCALE))


def test_one_table_for_all_through_the_c_entry(qsa):
    """pt_stride = 0: every sequence reads the same table."""
    q, cache, tables, n = make([900, 64, 2000], 2, 12, seed=15)
    one = tables[2]
    dev = [t.cuda() for t in (q, *cache, one, n)]
    out = torch.empty(q.shape, device="cuda")
    size = qsa.paged_attn_workspace_bytes(2, 24)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    rc = qsa.lib().qsa_paged_attn(dev[0].data_ptr(), 0, *[t.data_ptr() for t in dev[1:6]], 0, len(one), cache[0].shape[0], 2,
                                  24, dev[6].data_ptr(), 3, 0, SCALE, out.data_ptr(), 2, None, ws.data_ptr(), size, None,
                                  torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    ref.check_attn(out, None, ref.paged_attn(q, *cache, one[None].repeat(3, 1), n, SCALE))


def test_two_streams_and_a_captured_graph(qsa):
    """Two calls at once on two streams, each with its own workspace; then one call captured, replayed on new lengths
    in place."""
    sets = [make([5000, 3, 777], 4, 12, seed=16), make([64, 8000], 2, 8, seed=17)]
    dev = [[t.cuda() for t in (q, *cache, tables, n)] for q, cache, tables, n in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    outs = []
    for _ in range(3):
        outs = []
        for d, st in zip(dev, streams):
            with torch.cuda.stream(st):
                outs.append(qsa.paged_attn(*d))
    torch.cuda.synchronize()
    for out, (q, cache, tables, n) in zip(outs, sets):
        ref.check_attn(out, None, ref.paged_attn(q, *cache, tables, n, SCALE))
    q, cache, tables, n = sets[0]
    d = dev[0]
    ws = torch.empty(qsa.paged_attn_workspace_bytes(4, 48), dtype=torch.uint8, device="cuda")
    out = torch.empty(q.shape, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qsa.paged_attn(*d, out=out, workspace=ws)
    for lens in ([5000, 3, 777], [1, 0, 64], [4999, 2, 700]):
        d[-1].copy_(torch.tensor(lens, dtype=torch.int32))
        out.fill_(NAN16)
        graph.replay()
        torch.cuda.synchronize()
        ref.check_attn(out, None, ref.paged_attn(q, *cache, tables, lens, SCALE), str(lens))


def test_cold_caches_and_a_small_call_before(qsa):
    """A long sequence right after a short one, with the caches full of something else, so that copies land late and out
    of order: the same bits as warm, several times."""
    small = [t.cuda() for t in (lambda q, c, t, n: (q, *c, t, n))(*make([1021], 4, 12, seed=18))]
    q, cache, tables, n = make([100000], 4, 12, seed=19)
    d = [t.cuda() for t in (q, *cache, tables, n)]
    first = qsa.paged_attn(*d)
    ref.check_attn(first, None, ref.paged_attn(q, *cache, tables, n, SCALE))
    flush = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    for k in range(20):
        flush.fill_(k)
        qsa.paged_attn(*small)
        assert torch.equal(qsa.paged_attn(*d), first)


@pytest.mark.parametrize("lens", [[900, 64, 2000], [40000, 3, 9000]])
def test_another_stream_with_everything_allocated_here(qsa, lens):
    """A call on a stream that is not the current one: output and workspace come from that stream's memory, so work that
    the current stream still has, or starts meanwhile, cannot touch them."""
    q, cache, tables, n = make(lens, 4, 12, seed=21)
    d = [t.cuda() for t in (q, *cache, tables, n)]
    first = qsa.paged_attn(*d)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for k in range(10):
        junk = [torch.full((9 << 20,), k, dtype=torch.uint8, device="cuda") for _ in range(3)]   # the current stream is busy
        outs.append(qsa.paged_attn(*d, stream=side if k % 2 else side.cuda_stream))
        del junk
        torch.full((17 << 20,), 0xFF, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for out in outs:
        assert torch.equal(out, first)


def test_captured_with_copies_and_a_fork(qsa):
    """A capture in which the calls follow copies, a fork and a join of streams, not only kernels."""
    q, cache, tables, n = make([9000, 70, 300], 4, 12, seed=22)
    d = [t.cuda() for t in (q, *cache, tables, n)]
    want = qsa.paged_attn(*d)
    held, out = torch.zeros_like(d[0]), torch.zeros(q.shape, device="cuda")
    ws = torch.empty(qsa.paged_attn_workspace_bytes(4, 48), dtype=torch.uint8, device="cuda")
    slots = torch.arange(64 * 3, dtype=torch.int32, device="cuda")
    k, v = qsa.cache_gather(*d[1:5], slots)
    k2, v2, side = torch.zeros_like(k), torch.zeros_like(v), torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held.copy_(d[0])
        side.wait_stream(torch.cuda.current_stream())
        qsa.paged_attn(held, *d[1:], out=out, workspace=ws)
        with torch.cuda.stream(side):
            qsa.cache_gather(*d[1:5], slots, k_out=k2, v_out=v2)
        torch.cuda.current_stream().wait_stream(side)
        qsa.paged_attn(held, *d[1:], out=out, workspace=ws)
        held.zero_()
    for _ in range(3):
        out.fill_(NAN16)
        k2.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(k2, k) and torch.equal(v2, v) and not held.any()


@pytest.mark.parametrize("lens", [[128] * 16, [256] * 16, [0] * 15 + [256], [0] * 16, [64] * 200])
def test_the_next_call_waits_for_all_of_it(qsa, lens):
    """Calls whose items are not cut between blocks, so that there is nothing to join: the next call of the stream
    reads the finished output all the same, eagerly and captured."""
    q, cache, tables, n = make(lens, 4, 12, seed=23, width=80)
    d = [t.cuda() for t in (q, *cache, tables, n)]
    want = qsa.paged_attn(*d, out=torch.empty(q.shape, dtype=torch.bfloat16, device="cuda"))
    pos = torch.arange(len(lens), dtype=torch.int32, device="cuda") + 5
    freq = (10000.0 ** (-torch.arange(64, dtype=torch.float64) / 64)).cuda()
    turned = qsa.rope(want, pos, freq)
    outs = [torch.empty_like(want) for _ in range(8)]
    ys = [torch.empty_like(want) for _ in range(8)]
    ws = torch.empty(qsa.paged_attn_workspace_bytes(4, 48), dtype=torch.uint8, device="cuda")

    def steps():
        for out, y in zip(outs, ys):
            qsa.paged_attn(*d, out=out, workspace=ws)
            qsa.rope(out, pos, freq, out=y)

    steps()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        steps()
    for run_all in (steps, graph.replay, graph.replay):
        for t in outs + ys:
            t.fill_(NAN16)
        torch.cuda.synchronize()
        run_all()
        torch.cuda.synchronize()
        assert all(torch.equal(t, want) for t in outs) and all(torch.equal(t, turned) for t in ys)


def test_raw_streams(qsa):
    """Streams given as plain handles, the default stream's 0 among them."""
    q, cache, tables, n = make([300, 5000], 4, 12, seed=24)
    d = [t.cuda() for t in (q, *cache, tables, n)]
    want = qsa.paged_attn(*d)
    torch.cuda.synchronize()
    for stream in (0, torch.cuda.Stream().cuda_stream, torch.cuda.current_stream()):
        got = qsa.paged_attn(*d, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(got, want)


def test_refusals(qsa):
    q, cache, tables, n = make([100], 2, 12, seed=18)
    d = [t.cuda() for t in (q, *cache, tables, n)]
    with pytest.raises(TypeError):
        qsa.paged_attn(q, *d[1:])
    with pytest.raises(TypeError):
        qsa.paged_attn(d[0].float(), *d[1:])
    with pytest.raises(ValueError):
        qsa.paged_attn(d[0][:, :23].contiguous(), *d[1:])
    with pytest.raises(ValueError):
        qsa.paged_attn(d[0], *d[1:5], d[5][0], d[6])
    with pytest.raises(ValueError):
        qsa.paged_attn(d[0], *d[1:], out=torch.empty((1, 24, 64), device="cuda"))
    with pytest.raises(ValueError):
        qsa.paged_attn(d[0], *d[1:], lse=torch.empty((1, 12), device="cuda"))
    with pytest.raises(qsa.QsaError):
        qsa.paged_attn(*d, window=-1)
    with pytest.raises(qsa.QsaError):
        qsa.paged_attn(*d, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert math.isfinite(float(qsa.paged_attn(*d).sum()))
