"""Forms of the serving calls beside the usual ones: FP16 rows written, pools past 2^31 bytes; and every argument that does
not fit refused with a message of its own."""
import pytest

torch = pytest.importorskip("torch")
import serve_ref as ref  # noqa: E402
from test_cache_rows_gpu import cuda, quantised, rotation, step  # noqa: E402
from test_paged_attn_gpu import SCALE, qsa  # noqa: E402, F401

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- FP16 rows written

@pytest.mark.parametrize("n_tok,n_heads,n_kv", [(1, 12, 1), (66, 24, 2), (700, 7, 3)])
@pytest.mark.parametrize("pairs,axes,interleaved", [(64, 1, False), (64, 3, True), (32, 2, False)])
def test_append_fp16(qsa, n_tok, n_heads, n_kv, pairs, axes, interleaved):  # noqa: F811
    qkv, cache, slots = step(n_tok, n_heads, n_kv, seed=n_tok, dtype=torch.float16)
    pos, inv, axis = rotation(n_tok, pairs, axes, 100000, seed=5)
    d, dc = qkv.cuda(), cuda(*cache)
    q, k, v = d[:, :n_heads], d[:, n_heads:n_heads + n_kv], d[:, n_heads + n_kv:]
    got = qsa.rope_append(q, k, v, *cuda(pos, inv, axis), *dc, slots.cuda(), interleaved=interleaved)
    assert got.dtype == torch.float16
    ref.check_turned(got, q, ref.turned(q, pos, inv, axis, interleaved))
    page, cell = slots.long() // 64, slots.long() % 64
    out = [t.cpu() for t in dc]
    want = ref.turned(k, pos, inv, axis, interleaved)
    # the FP32 rotation is within 2^-20 of sqrt(2) times the row's largest value
    size = k.double().cpu().abs().amax((1, 2)).amax() * 2 ** 0.5
    slack = float((size * 2.0 ** -20 / want.abs().amax(-1)).max())
    ref.check_cells(out[0][page, :, cell], out[2][page, :, cell], want, slack)
    ref.check_cells(out[1][page, :, cell], out[3][page, :, cell], v.double().cpu(), 2.0 ** -24)
    for t, before in zip(out, cache):
        keep = torch.ones(t.shape[0], 64, dtype=torch.bool)
        keep[page, cell] = False
        assert torch.equal(t.transpose(1, 2)[keep], before.transpose(1, 2)[keep])


def test_append_fp16_without_rotation_is_exact(qsa):  # noqa: F811
    """Rows of every size FP16 has: zeros, subnormals, the largest."""
    qkv, cache, slots = step(40, 0, 2, seed=6, dtype=torch.float16)
    qkv = (qkv.float() * torch.ldexp(torch.ones(()), torch.arange(-24, 16))[:, None, None]).clamp(-65504, 65504).half()
    qkv[5] = 0
    qkv[7, :, 3] = 65504
    d, dc = qkv.cuda(), cuda(*cache)
    qsa.rope_append(None, d[:, :2], d[:, 2:], None, None, None, *dc, slots.cuda())
    page, cell = slots.long() // 64, slots.long() % 64
    for pool, scale, x in ((dc[0], dc[2], qkv[:, :2]), (dc[1], dc[3], qkv[:, 2:])):
        ints, s = quantised(x)
        assert torch.equal(scale.cpu()[page, :, cell], s)
        assert torch.equal(pool.cpu()[page, :, cell], ints)


def test_append_fp16_rows_that_are_not_finite(qsa):  # noqa: F811
    qkv, cache, slots = step(4, 0, 1, seed=7, dtype=torch.float16)
    qkv[0, 0, 5] = float("inf")
    qkv[1, 0, 100] = float("nan")
    qkv[2, 1, 0] = -float("inf")
    d, dc = qkv.cuda(), cuda(*cache)
    qsa.rope_append(None, d[:, :1], d[:, 1:], None, None, None, *dc, slots.cuda())
    page, cell = slots.long() // 64, slots.long() % 64
    ks, vs = dc[2].cpu()[page, 0, cell], dc[3].cpu()[page, 0, cell]
    assert torch.isnan(ks).tolist() == [True, True, False, False] and torch.isnan(vs).tolist() == [False, False, True, False]


# ---------------------------------------------------------------- a pool past 2^31 bytes

def test_pool_past_2_31_bytes(qsa):  # noqa: F811
    """Keys and values of 2.6 GB each: cells on both sides of 2^31 bytes written, read back and attended to as in a small
    pool that holds the same cells."""
    n_kv, group, pages = 8, 4, 40000
    small_pages = 70                       # page p of the small pool is page far[p] of the large one
    g = torch.Generator().manual_seed(3)
    edge = (1 << 31) // (n_kv * 64 * 128)
    far = torch.cat((torch.tensor([0, edge - 1, edge, edge + 1, pages - 1]), torch.randperm(pages, generator=g)[:200]))
    far = torch.tensor(list(dict.fromkeys(far.tolist()))[:small_pages])
    small = cuda(*ref.make_cache(small_pages, n_kv, seed=4))
    shape = (pages, n_kv, 64, 128)
    large = [torch.empty(shape, dtype=torch.int8, device="cuda") for _ in range(2)]
    large += [torch.full(shape[:3], float("nan"), dtype=torch.float16, device="cuda") for _ in range(2)]
    assert large[0].nbytes > 1 << 31
    for big, t in zip(large, small):
        big[far.cuda()] = t
    n_tok, n_heads = 90, n_kv * group
    qkv = torch.randn((n_tok, n_heads + 2 * n_kv, 128), generator=g).bfloat16().cuda()
    slots = torch.randperm(small_pages * 64, generator=g)[:n_tok].int()
    slots[:5] = torch.arange(5).int() * 64 + 7
    slots = torch.tensor(list(dict.fromkeys(slots.tolist()))).int()
    there = (far[slots.long() // 64] * 64 + slots.long() % 64).int().cuda()
    n_tok, slots = len(slots), slots.cuda()
    qkv = qkv[:n_tok]
    pos, inv, axis = cuda(*rotation(n_tok, 64, 1, 30000, seed=5))
    tables = torch.randperm(small_pages, generator=g)[:60].view(2, 30)
    lens = torch.tensor([1900, 1111], dtype=torch.int32, device="cuda")
    results = []
    for pools, at, table in ((small, slots, tables), (large, there, far[tables])):
        q = qsa.rope_append(qkv[:, :n_heads], qkv[:, n_heads:n_heads + n_kv], qkv[:, n_heads + n_kv:], pos, inv, axis, *pools, at)
        results.append([q, *qsa.cache_gather(*pools, at, dtype=torch.float32),
                        qsa.paged_attn(q[:2], *pools, table.int().cuda(), lens)])
    for got, want in zip(results[1], results[0]):
        assert torch.equal(got, want)
    for big, t in zip(large, small):
        assert torch.equal(big[far.cuda()], t)
    ref.check_attn(results[0][-1], None, ref.paged_attn(results[0][0][:2].cpu(), *[t.cpu() for t in small], tables, lens.cpu(), SCALE))


# ---------------------------------------------------------------- arguments that do not fit

def spoiled(t):
    """What an argument that has to be the tensor t must not be."""
    yield "a list", t.tolist()
    yield "on the host", t.cpu()
    yield "complex", t.to(torch.complex64)
    yield "one dim more", t[None]
    yield "flat", t.reshape(-1) if t.dim() > 1 else t[:, None]
    yield "strided", torch.stack((t, t), -1)[..., 0]
    if t.shape[0] > 1:
        yield "shorter", t[:-1].contiguous()
    if t.dim() > 1:
        yield "narrower", t[..., :-1].contiguous()


def refused(call, args, names, skip=()):
    call(**args)                                               # as they are, they fit
    for name in names:
        for what, bad in spoiled(args[name]):
            if (name, what) in skip:
                continue
            with pytest.raises((TypeError, ValueError)) as e:
                call(**{**args, name: bad})
            assert "do not fit together" not in str(e.value), f"{name}: {what}"
            assert "must" in str(e.value) or "expected" in str(e.value) or "heads" in str(e.value), f"{name}: {what}: {e.value}"


def test_every_refusal_says_what_is_wrong(qsa):  # noqa: F811
    i = lambda *shape: torch.zeros(shape, dtype=torch.int32, device="cuda")  # noqa: E731
    b = lambda *shape: torch.zeros(shape, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    k, v, ks, vs = cuda(*ref.make_cache(4, 2, seed=1))
    pools = dict(k_pool=k, v_pool=v, k_scale=ks, v_scale=vs)
    attn = dict(q=b(3, 8, 128), **pools, page_tables=i(3, 4), seq_lens=i(3), out=b(3, 8, 128),
                lse=torch.zeros((3, 8), device="cuda"))
    refused(qsa.paged_attn, attn, list(attn), skip={("page_tables", "narrower")})
    freq = torch.ones(64, dtype=torch.float64, device="cuda")
    turn = dict(positions=i(2, 5), inv_freq=freq, pair_axis=i(64))
    write = dict(q=b(5, 8, 128), k=b(5, 2, 128), v=b(5, 2, 128), **turn, **pools, slots=i(5) - 1, q_out=b(5, 8, 128))
    refused(qsa.rope_append, write, list(write), skip={("positions", "shorter")})          # fewer axes
    refused(qsa.rope, dict(x=b(5, 8, 128), **turn, out=b(5, 8, 128)), ["x", "positions", "inv_freq", "pair_axis", "out"],
            skip={("positions", "shorter")})
    read = dict(**pools, slots=i(5), k_out=b(5, 2, 128), v_out=b(5, 2, 128))
    refused(qsa.cache_gather, read, list(read))
    tables = dict(seq_lens=i(3), new_lens=i(3), page_tables=i(3, 4) - 1, free_pages=i(9), n_tok=5, n_ppages=4, free_head=i(1))
    refused(qsa.extend_tables, tables, ["seq_lens", "new_lens", "page_tables", "free_pages", "free_head"],
            skip={("page_tables", "narrower"), ("free_pages", "shorter"), ("free_pages", "one dim more"), ("free_pages", "flat"),
                  ("free_head", "strided")})                   # (one element lies as it should whatever its stride)
