"""qsa_rope, qsa_rope_append and qsa_cache_gather on the GPU against their 64-bit definitions."""
import pytest

torch = pytest.importorskip("torch")
import serve_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu
BAD_CELL, BAD_AXIS = 4, 512


@pytest.fixture(scope="module")
def qsa():
    from sparse_selected_cell_gb300 import qsa as q
    if not torch.cuda.is_available():
        pytest.fail("CUDA GPU required")
    q.lib()
    return q


def rotation(n_tok, pairs, axes, far, seed):
    g = torch.Generator().manual_seed(seed)
    pos = torch.randint(-far // 8, far, (axes, n_tok), dtype=torch.int32, generator=g)
    inv = 10000.0 ** (-torch.arange(pairs, dtype=torch.float64) / pairs)
    axis = (torch.arange(pairs) * axes // pairs).int() if axes > 1 else None
    return pos, inv, axis


def cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


ROTATIONS = [(64, 1, False), (64, 3, False), (64, 1, True), (32, 2, False), (32, 2, True), (16, 4, False), (8, 1, True),
             (40, 3, False), (56, 3, True)]


@pytest.mark.parametrize("pairs,axes,interleaved", ROTATIONS)
@pytest.mark.parametrize("n_tok,n_heads,dtype", [(1, 1, torch.bfloat16), (7, 12, torch.float16), (130, 5, torch.bfloat16)])
def test_rope(qsa, pairs, axes, interleaved, n_tok, n_heads, dtype):
    pos, inv, axis = rotation(n_tok, pairs, axes, 200000, seed=pairs + n_tok)
    x = torch.randn((n_tok, n_heads, 128), generator=torch.Generator().manual_seed(1)).to(dtype)
    want = ref.turned(x, pos, inv, axis, interleaved)
    d = cuda(x, pos, inv, axis)
    got = qsa.rope(*d, interleaved=interleaved)
    ref.check_turned(got, x, want)
    if 2 * pairs < 128:
        assert torch.equal(got[..., 2 * pairs:], d[0][..., 2 * pairs:])
    # in place, on a slice of a wider tensor: the same bits, and the neighbours untouched
    wide = torch.randn((n_tok, n_heads + 3, 128)).to(dtype).cuda()
    wide[:, 2:2 + n_heads] = d[0]
    before = wide.clone()
    view = wide[:, 2:2 + n_heads]
    assert qsa.rope(view, *d[1:], interleaved=interleaved, out=view) is view
    assert torch.equal(view, got) and torch.equal(wide[:, :2], before[:, :2]) and torch.equal(wide[:, -1], before[:, -1])


def test_rope_far_positions(qsa):
    """Positions over the whole of int32: the angle's fraction of a turn keeps its bits (the reference's own angle, in
    FP64, is off by up to position * 2^-53 turns: 2^-22)."""
    pos = torch.tensor([[0, 1, -1, 2 ** 20 + 3, 10 ** 9 + 7, 2 ** 31 - 1, -2 ** 31]], dtype=torch.int32)
    inv = 10000.0 ** (-torch.arange(64, dtype=torch.float64) / 64)
    x = torch.randn((7, 3, 128), generator=torch.Generator().manual_seed(2)).half()
    got = qsa.rope(*cuda(x, pos, inv))
    ref.check_turned(got, x, ref.turned(x, pos, inv, None, False))
    assert torch.equal(got[0].cpu(), x[0])                    # position 0 turns nothing


def test_rope_large_and_negative_frequencies(qsa):
    pos = torch.arange(50, dtype=torch.int32)
    inv = torch.tensor([100.0, -3.0, 6.283185307179586, 1e-12, -1e-9, 0.0, 2.5, -40.0], dtype=torch.float64)
    x = torch.randn((50, 2, 128), generator=torch.Generator().manual_seed(3)).bfloat16()
    got = qsa.rope(*cuda(x, pos, inv))
    ref.check_turned(got, x, ref.turned(x, pos[None], inv, None, False))


def test_bad_axis_is_reported(qsa):
    pos, inv, _ = rotation(9, 16, 2, 1000, seed=4)
    axis = torch.zeros(16, dtype=torch.int32)
    axis[3], axis[5] = 2, -1
    x = torch.randn((9, 2, 128)).bfloat16()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = qsa.rope(*cuda(x, pos, inv, axis), dev_status=status)
    assert int(status.item()) == BAD_AXIS
    ref.check_turned(got, x, ref.turned(x, pos, inv, torch.zeros(16), False))


def step(n_tok, n_heads, n_kv, seed, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn((n_tok, n_heads + 2 * n_kv, 128), generator=g).to(dtype)
    pages = -(-n_tok // 64) + 2
    slots = torch.randperm(pages * 64, generator=g)[:n_tok].int()
    return qkv, ref.make_cache(pages, n_kv, seed), slots


@pytest.mark.parametrize("n_tok,n_heads,n_kv", [(1, 12, 1), (1, 48, 4), (3, 1, 1), (66, 24, 2), (257, 7, 5), (40, 96, 8),
                                                 (2000, 3, 1), (1700, 33, 3)])
@pytest.mark.parametrize("pairs,axes,interleaved", [(64, 1, False), (64, 3, True), (32, 2, False)])
def test_append(qsa, n_tok, n_heads, n_kv, pairs, axes, interleaved):
    qkv, cache, slots = step(n_tok, n_heads, n_kv, seed=n_tok)
    if n_tok > 2:
        slots[1] = -1                                          # not written
    pos, inv, axis = rotation(n_tok, pairs, axes, 100000, seed=5)
    d, dc, ds = qkv.cuda(), cuda(*cache), slots.cuda()
    q, k, v = d[:, :n_heads], d[:, n_heads:n_heads + n_kv], d[:, n_heads + n_kv:]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = qsa.rope_append(q, k, v, *cuda(pos, inv, axis), *dc, ds, interleaved=interleaved, dev_status=status)
    assert int(status.item()) == 0
    ref.check_turned(got, q, ref.turned(q, pos, inv, axis, interleaved))
    on = slots >= 0
    page, cell = slots[on].long() // 64, slots[on].long() % 64
    out = [t.cpu() for t in dc]
    # FP32 rotation: sines, cosines and products within 2^-20 of the pair's size, at most sqrt(2) of the row's largest
    want = ref.turned(k, pos, inv, axis, interleaved)[on]
    size = k.double().cpu().abs().amax((1, 2))[on].amax() * 2 ** 0.5
    slack = float((size * 2.0 ** -20 / want.abs().amax(-1)).max())
    ref.check_cells(out[0][page, :, cell], out[2][page, :, cell], want, slack)
    ref.check_cells(out[1][page, :, cell], out[3][page, :, cell], v.double().cpu()[on], 2.0 ** -24)
    for t, before in zip(out, cache):                          # every other cell is as it was
        keep = torch.ones(t.shape[0], 64, dtype=torch.bool)
        keep[page, cell] = False
        assert torch.equal(t.transpose(1, 2)[keep], before.transpose(1, 2)[keep])


def quantised(x):
    """The definition in FP32, where no rotation comes before: scale = max |x| / 127 rounded up to FP16."""
    want = x.float().abs().amax(-1) / 127
    scale = want.half()
    up = (scale.view(torch.int16) + 1).view(torch.half)
    scale = torch.where(scale.float() < want, up, scale).clamp(max=65504)
    return torch.round(x.float() / torch.where(scale == 0, 1.0, scale.float())[..., None]).clamp(-127, 127).to(torch.int8), scale


def test_append_without_rotation_is_exact(qsa):
    """Rows of every size: zeros, subnormal scales, ordinary ones, ones past what an FP16 scale can hold."""
    qkv, cache, slots = step(64, 0, 2, seed=6)
    qkv[:, :] *= torch.ldexp(torch.ones(()), torch.arange(-40, 24))[:, None, None].bfloat16()
    qkv[5] = 0
    d, dc = qkv.cuda(), cuda(*cache)
    assert qsa.rope_append(None, d[:, :2], d[:, 2:], None, None, None, *dc, slots.cuda()) is None
    page, cell = slots.long() // 64, slots.long() % 64
    for pool, scale, x in ((dc[0], dc[2], qkv[:, :2]), (dc[1], dc[3], qkv[:, 2:])):
        ints, s = quantised(x)
        assert torch.equal(scale.cpu()[page, :, cell], s)
        assert torch.equal(pool.cpu()[page, :, cell], ints)


def test_append_rows_that_are_not_finite(qsa):
    qkv, cache, slots = step(4, 0, 1, seed=7)
    qkv[0, 0, 5] = float("inf")
    qkv[1, 0, 100] = float("nan")
    qkv[2, 1, 0] = -float("inf")
    d, dc = qkv.cuda(), cuda(*cache)
    qsa.rope_append(None, d[:, :1], d[:, 1:], None, None, None, *dc, slots.cuda())
    page, cell = slots.long() // 64, slots.long() % 64
    ks, vs = dc[2].cpu()[page, 0, cell], dc[3].cpu()[page, 0, cell]
    assert torch.isnan(ks).tolist() == [True, True, False, False] and torch.isnan(vs).tolist() == [False, False, True, False]


def test_append_bad_slot_is_reported(qsa):
    qkv, cache, slots = step(5, 12, 1, seed=8)
    slots[3] = cache[0].shape[0] * 64
    d, dc = qkv.cuda(), cuda(*cache)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pos, inv, axis = cuda(*rotation(5, 64, 1, 100, seed=9))
    got = qsa.rope_append(d[:, :12], d[:, 12:13], d[:, 13:], pos, inv, axis, *dc, slots.cuda(), dev_status=status)
    assert int(status.item()) == BAD_CELL
    ref.check_turned(got, d[:, :12], ref.turned(d[:, :12], pos, inv, axis, False))   # its query is rotated all the same


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("n_cell,n_kv", [(1, 1), (3, 8), (1000, 4), (77, 3)])
def test_gather(qsa, n_cell, n_kv, dtype):
    cache = ref.make_cache(n_cell // 64 + 2, n_kv, seed=n_cell)
    slots = torch.randint(0, cache[0].shape[0] * 64, (n_cell,), generator=torch.Generator().manual_seed(9)).int()
    slots[n_cell // 2] = slots[0]                              # a cell may be named twice
    if n_cell > 2:
        slots[1] = -1
    k, v = qsa.cache_gather(*cuda(*cache), slots.cuda(), dtype=dtype)
    page, cell = slots.long().clamp(min=0) // 64, slots.long().clamp(min=0) % 64
    for got, pool, scale in ((k, cache[0], cache[2]), (v, cache[1], cache[3])):
        want = pool[page, :, cell].float() * scale[page, :, cell].float()[..., None]
        want[slots < 0] = 0
        assert got.dtype == dtype and torch.equal(got.cpu(), want.to(dtype))


def test_append_to_an_empty_pool(qsa):
    """No page at all: nothing is written, every slot is reported, the queries are rotated."""
    qkv, _, _ = step(6, 20, 2, seed=10)
    d = qkv.cuda()
    none = [torch.empty((0, 2, 64, 128), dtype=torch.int8, device="cuda")] * 2 + [torch.empty((0, 2, 64), dtype=torch.float16, device="cuda")] * 2
    pos, inv, axis = cuda(*rotation(6, 64, 1, 100, seed=11))
    for slot, want in ((3, BAD_CELL), (-1, 0)):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = qsa.rope_append(d[:, :20], d[:, 20:22], d[:, 22:], pos, inv, axis, *none, torch.full((6,), slot, dtype=torch.int32, device="cuda"),
                              dev_status=status)
        assert int(status.item()) == want
        ref.check_turned(got, d[:, :20], ref.turned(d[:, :20], pos, inv, axis, False))


def test_gather_many_cells(qsa):
    """More cells than one block takes, an odd number of heads, the last block ragged."""
    cache = ref.make_cache(40, 3, seed=12)
    slots = torch.randint(-5, 40 * 64, (2311,), generator=torch.Generator().manual_seed(13)).int()
    k, v = qsa.cache_gather(*cuda(*cache), slots.cuda(), dtype=torch.float32)
    page, cell = slots.long().clamp(min=0) // 64, slots.long().clamp(min=0) % 64
    for got, pool, scale in ((k, cache[0], cache[2]), (v, cache[1], cache[3])):
        want = pool[page, :, cell].float() * scale[page, :, cell].float()[..., None]
        want[slots < 0] = 0
        assert torch.equal(got.cpu(), want)


def test_gather_bad_slot_is_reported(qsa):
    cache = ref.make_cache(2, 2, seed=1)
    slots = torch.tensor([5, 128, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    k, v = qsa.cache_gather(*cuda(*cache), slots.cuda(), dev_status=status)
    assert int(status.item()) == BAD_CELL and k[0].any() and not k[1:].any() and not v[1:].any()


def test_empty_calls_and_refusals(qsa):
    dc = cuda(*ref.make_cache(2, 2, seed=2))
    e = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    assert qsa.cache_gather(*dc, none)[0].shape == (0, 2, 128)
    assert qsa.rope_append(e(0, 4, 128), e(0, 2, 128), e(0, 2, 128), None, None, None, *dc, none).shape == (0, 4, 128)
    slots = torch.zeros(3, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        qsa.rope_append(None, e(3, 4, 128), e(3, 4, 128), None, None, None, *dc, slots)          # heads of another cache
    with pytest.raises(TypeError):
        qsa.rope_append(None, e(3, 2, 128), e(3, 2, 128).half(), None, None, None, *dc, slots)
    with pytest.raises(ValueError):
        qsa.rope_append(None, e(3, 2, 128).transpose(0, 1).contiguous().transpose(0, 1), e(3, 2, 128), None, None, None, *dc, slots)
    with pytest.raises(TypeError):
        qsa.rope(e(3, 2, 128).float(), slots, None)
    with pytest.raises(qsa.QsaError):
        qsa.rope(e(3, 2, 128), slots, torch.ones(12, dtype=torch.float64, device="cuda"))
    with pytest.raises(TypeError):
        qsa.rope(e(3, 2, 128), slots, torch.ones(8, device="cuda"))
    with pytest.raises(ValueError):
        qsa.cache_gather(*dc, slots, k_out=e(3, 2, 64))
