"""The serving operators over the paged INT8 cache, as cases that can be timed and compared.

Each case is one call of one operator on inputs made from a seed.  `run` computes
it in its plain form (elementary torch operations, 32 bits or more) or, with
`own` set, through the library's kernels (`sparse_selected_cell_gb300.qsa`).

The operators (see `include/qsa.h` for the layouts):

  attn    one new token per sequence against its whole paged cache, or against the
          last `window` cells of it: softmax(q . k * scale) v over the resident
          cells, query head h reading KV head h // group; zeros (and a log-sum-exp
          of -inf) where nothing is left to attend to
  append  rotary positions (one or several axes) on a step's queries and keys, then
          the keys and values quantised to INT8 rows with one FP16 scale each and
          written to their slots of the cache.  The cells are read back as the
          values they stand for
  gather  cells read back from the cache as BF16 keys and values
  tables  page tables extended and slots mapped for a step's new tokens
"""
import math

import torch

own = False

HEAD_DIM = 128
PAGE = 64
THETA = 10000.0


def _qsa():
    from sparse_selected_cell_gb300 import qsa
    return qsa


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # a single short conversation: a call whose latency is all that counts
        dict(name="attn-1x1021", op="attn", n_seq=1, n_kv=4, group=12, lo=1021, hi=1021, window=0, out="bf16", lse=False),
        # one user far into a long document: the cache's length has to be split
        dict(name="attn-1x262149", op="attn", n_seq=1, n_kv=8, group=12, lo=262149, hi=262149, window=0, out="bf16", lse=True),
        # a serving batch, ragged from a fresh prompt to a long chat
        dict(name="attn-64x1-8192", op="attn", n_seq=64, n_kv=4, group=12, lo=1, hi=8192, window=0, out="bf16", lse=True),
        # many sequences under a sliding window, fewer query heads to a KV head
        dict(name="attn-512x4096-w1000", op="attn", n_seq=512, n_kv=4, group=8, lo=64, hi=4096, window=1000, out="bf16", lse=False),
        # the largest: a full batch of long contexts
        dict(name="attn-96x20000", op="attn", n_seq=96, n_kv=4, group=12, lo=16000, hi=20000, window=0, out="bf16", lse=False),
        # one sequence's next token
        dict(name="append-1", op="append", n_tok=1, n_kv=4, group=12, axes=1, pairs=64, interleaved=False, far=131072),
        # a decode batch
        dict(name="append-256", op="append", n_tok=256, n_kv=4, group=12, axes=1, pairs=64, interleaved=False, far=32768),
        # a prompt chunk with image and video tokens (time, height, width)
        dict(name="append-8192-thw", op="append", n_tok=8192, n_kv=4, group=12, axes=3, pairs=64, interleaved=False, far=40960),
        # a shared prefix handed to another consumer of BF16 keys and values
        dict(name="gather-1999", op="gather", n_cell=1999, n_kv=4),
        # a long context read back whole
        dict(name="gather-40960", op="gather", n_cell=40960, n_kv=8),
        # a decode step of a large batch: one new token each
        dict(name="tables-1024x1", op="tables", n_seq=1024, old=32768, lo=1, hi=1),
        # a step that takes in prompts, some sequences with nothing new
        dict(name="tables-300x0-2000", op="tables", n_seq=300, old=4096, lo=0, hi=2000),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "append", "gather", "tables"])
    if op == "attn":
        n_kv, group = rng.choice([1, 4, 8]), rng.choice([4, 8, 12, 16])
        n_seq = _log(rng, 1, 512)
        most = max(64, min(262144, 6 * 10 ** 6 // (n_seq * n_kv)))      # cells x KV heads of the batch
        hi = _log(rng, 33, most)
        lo = rng.choice([0, 1, hi // 2, hi])
        window = rng.choice([0, 0, 0, rng.randint(1, hi)])
        return dict(op=op, n_seq=n_seq, n_kv=n_kv, group=group, lo=lo, hi=hi, window=window, out="bf16", lse=rng.random() < 0.5)
    if op == "append":
        axes = rng.choice([1, 1, 2, 3])
        return dict(op=op, n_tok=_log(rng, 1, 8192), n_kv=rng.choice([1, 4, 8]), group=rng.choice([4, 8, 12]), axes=axes,
                    pairs=rng.choice([16, 32, 64, 64]), interleaved=rng.random() < 0.3, far=_log(rng, 2048, 1000000))
    if op == "gather":
        return dict(op=op, n_cell=_log(rng, 1, 40960), n_kv=rng.choice([1, 4, 8]))
    n_seq = _log(rng, 1, 1024)
    hi = _log(rng, 1, 300000 // n_seq + 1)
    return dict(op=op, n_seq=n_seq, old=_log(rng, 64, 32768), lo=rng.choice([0, 0, 1, hi]), hi=hi)


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _pool(n_pages, n_kv, g):
    """INT8 pages uniform in [-127, 127], FP16 scales uniform in [0.01, 0.03]."""
    shape = (n_pages, n_kv, PAGE, HEAD_DIM)
    k = torch.randint(-127, 128, shape, dtype=torch.int8, device="cuda", generator=g)
    v = torch.randint(-127, 128, shape, dtype=torch.int8, device="cuda", generator=g)
    ks = (torch.rand(shape[:3], device="cuda", generator=g) * 0.02 + 0.01).half()
    vs = (torch.rand(shape[:3], device="cuda", generator=g) * 0.02 + 0.01).half()
    return k, v, ks, vs


def _lens(n, lo, hi, g):
    return torch.randint(lo, hi + 1, (n,), dtype=torch.int32, device="cuda", generator=g)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"] == "attn":
        n_seq, n_kv, heads = case["n_seq"], case["n_kv"], case["n_kv"] * case["group"]
        width = -(-case["hi"] // PAGE)
        lens = _lens(n_seq, case["lo"], case["hi"], g)
        s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"] = _pool(n_seq * width, n_kv, g)
        s["page_tables"] = torch.randperm(n_seq * width, device="cuda", generator=g).int().view(n_seq, width)
        s["seq_lens"] = lens
        s["q"] = torch.randn((n_seq, heads, HEAD_DIM), device="cuda", generator=g).bfloat16()
        s["out_t"] = torch.empty((n_seq, heads, HEAD_DIM), dtype=torch.bfloat16, device="cuda")
        s["lse_t"] = torch.empty((n_seq, heads), dtype=torch.float32, device="cuda") if case["lse"] else None
        s["workspace"] = torch.empty(16 << 20, dtype=torch.uint8, device="cuda")
    elif case["op"] == "append":
        n, n_kv, heads, pairs = case["n_tok"], case["n_kv"], case["n_kv"] * case["group"], case["pairs"]
        # queries, keys and values side by side, as one projection leaves them
        qkv = torch.randn((n, heads + 2 * n_kv, HEAD_DIM), device="cuda", generator=g).bfloat16()
        s["q"], s["k"], s["v"] = qkv[:, :heads], qkv[:, heads:heads + n_kv], qkv[:, heads + n_kv:]
        s["positions"] = torch.randint(0, case["far"], (case["axes"], n), dtype=torch.int32, device="cuda", generator=g)
        i = torch.arange(pairs, device="cuda", dtype=torch.float64)
        s["inv_freq"] = THETA ** (-i / pairs)
        s["pair_axis"] = (torch.arange(pairs, device="cuda") * case["axes"] // pairs).int()
        pages = -(-n // PAGE) + 3
        s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"] = _pool(pages, n_kv, g)
        s["slots"] = torch.randperm(pages * PAGE, device="cuda", generator=g)[:n].int()
        s["q_out"] = torch.empty((n, heads, HEAD_DIM), dtype=torch.bfloat16, device="cuda")
        s["k_back"] = torch.empty((n, n_kv, HEAD_DIM), dtype=torch.bfloat16, device="cuda")
        s["v_back"] = torch.empty((n, n_kv, HEAD_DIM), dtype=torch.bfloat16, device="cuda")
    elif case["op"] == "gather":
        n, n_kv = case["n_cell"], case["n_kv"]
        pages = -(-n // PAGE) + 5
        s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"] = _pool(pages, n_kv, g)
        # whole pages in the order of a shuffled table, as a sequence's cells lie
        order = torch.randperm(pages, device="cuda", generator=g)
        cells = torch.arange(n, device="cuda")
        s["slots"] = (order[cells // PAGE] * PAGE + cells % PAGE).int()
        s["k_out"] = torch.empty((n, n_kv, HEAD_DIM), dtype=torch.bfloat16, device="cuda")
        s["v_out"] = torch.empty((n, n_kv, HEAD_DIM), dtype=torch.bfloat16, device="cuda")
    else:
        n_seq, old, hi = case["n_seq"], case["old"], case["hi"]
        width = -(-(old + hi) // PAGE)
        s["seq_lens"] = _lens(n_seq, 0, old, g)
        s["new_lens"] = _lens(n_seq, case["lo"], hi, g)
        s["n_tok"] = n_seq * hi                      # what the program's buffers hold; the step may bring fewer
        s["n_ppages"] = n_seq * width
        perm = torch.randperm(s["n_ppages"], device="cuda", generator=g).int()
        held = (s["seq_lens"].long() + PAGE - 1) // PAGE
        first = held.cumsum(0) - held
        lp = torch.arange(width, device="cuda")
        at = (first[:, None] + lp).clamp(max=s["n_ppages"] - 1)
        s["page_tables"] = torch.where(lp < held[:, None], perm[at], -1).int().contiguous()
        s["free_pages"] = perm                        # the held pages lie at the front: the list's head is behind them
        s["free_head"] = held.sum().int().view(1)
        i32 = lambda *shape: torch.empty(shape, dtype=torch.int32, device="cuda")  # noqa: E731
        s["out_t"] = (i32(s["n_tok"]), i32(s["n_tok"]), i32(s["n_tok"]), i32(n_seq), i32(n_seq + 1), i32(1))
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    if s["op"] == "attn":
        return _attn_own(s) if own else _attn_plain(s)
    if s["op"] == "append":
        return _append_own(s) if own else _append_plain(s)
    if s["op"] == "gather":
        return _gather_own(s) if own else _gather_plain(s)
    return _tables_own(s) if own else _tables_plain(s)


def _attn_own(s):
    out = _qsa().paged_attn(s["q"], s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"], s["page_tables"], s["seq_lens"],
                            window=s["window"], out=s["out_t"], lse=s["lse_t"], workspace=s["workspace"])
    return [out, s["lse_t"]]


def _append_own(s):
    qsa = _qsa()
    q = qsa.rope_append(s["q"], s["k"], s["v"], s["positions"], s["inv_freq"], s["pair_axis"], s["k_pool"], s["v_pool"],
                        s["k_scale"], s["v_scale"], s["slots"], interleaved=s["interleaved"], q_out=s["q_out"])
    k, v = qsa.cache_gather(s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"], s["slots"], k_out=s["k_back"], v_out=s["v_back"])
    return [q, k, v]


def _gather_own(s):
    return list(_qsa().cache_gather(s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"], s["slots"], k_out=s["k_out"], v_out=s["v_out"]))


def _tables_own(s):
    t = _qsa().extend_tables(s["seq_lens"], s["new_lens"], s["page_tables"], s["free_pages"], s["n_tok"], s["n_ppages"],
                             free_head=s["free_head"], out=s["out_t"])
    return [s["page_tables"], *t]


def _attn_plain(s):
    n_seq, width = s["page_tables"].shape
    n_kv, group = s["n_kv"], s["group"]
    pages = s["page_tables"].long()
    held = pages.clamp(min=0)

    def rows(pool, scale):
        x = pool[held].float() * scale[held].float()[..., None]             # [seq, page, kv, cell, dim]
        return x.transpose(1, 2).reshape(n_seq, n_kv, width * PAGE, HEAD_DIM)

    cell = torch.arange(width * PAGE, device="cuda")
    lens = s["seq_lens"].long()[:, None]
    ok = (cell < lens) & (pages >= 0).repeat_interleave(PAGE, 1)
    if s["window"]:
        ok &= cell >= lens - s["window"]
    q = s["q"].float().view(n_seq, n_kv, group, HEAD_DIM) * HEAD_DIM ** -0.5
    score = torch.matmul(q, rows(s["k_pool"], s["k_scale"]).transpose(2, 3))
    score = score.masked_fill(~ok[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, rows(s["v_pool"], s["v_scale"])) / torch.where(total == 0, 1.0, total)
    lse = (torch.log(total) + top).view(n_seq, -1) if s["lse"] else None
    return [out.view(n_seq, -1, HEAD_DIM).bfloat16(), lse]


def _turn(x, cos, sin, pairs, interleaved):
    """The first 2 * pairs dims of every row turned by its token's angles, the others as they are."""
    x, rot, rest = x.float(), x[..., :2 * pairs].float(), x[..., 2 * pairs:].float()
    a, b = (rot[..., 0::2], rot[..., 1::2]) if interleaved else (rot[..., :pairs], rot[..., pairs:])
    u, w = a * cos - b * sin, b * cos + a * sin
    rot = torch.stack((u, w), -1).flatten(-2) if interleaved else torch.cat((u, w), -1)
    return torch.cat((rot, rest), -1)


def _quantise(x):
    """FP32 rows -> INT8 rows and FP16 scales: the scale is the row's largest value / 127, rounded up (so no value passes 127)."""
    want = x.abs().amax(-1) / 127
    scale = want.half()
    up = (scale.view(torch.int16) + 1).view(torch.half)
    scale = torch.where(scale.float() < want, up, scale)
    div = torch.where(scale == 0, 1.0, scale.float())
    return torch.round(x / div[..., None]).clamp(-127, 127).to(torch.int8), scale


def _append_plain(s):
    # angles in 64 bits: a far position times a frequency, then the turn that is left of it
    angle = s["positions"].double()[s["pair_axis"].long()].T * s["inv_freq"]            # [token, pair]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    q = _turn(s["q"], cos, sin, s["pairs"], s["interleaved"]).bfloat16()
    k, ks = _quantise(_turn(s["k"], cos, sin, s["pairs"], s["interleaved"]))
    v, vs = _quantise(s["v"].float())
    page, cell = s["slots"].long() // PAGE, s["slots"].long() % PAGE
    s["k_pool"][page, :, cell] = k
    s["v_pool"][page, :, cell] = v
    s["k_scale"][page, :, cell] = ks
    s["v_scale"][page, :, cell] = vs
    return [q, *_gather_plain(s)]


def _gather_plain(s):
    page, cell = s["slots"].long() // PAGE, s["slots"].long() % PAGE
    k = s["k_pool"][page, :, cell].float() * s["k_scale"][page, :, cell].float()[..., None]
    v = s["v_pool"][page, :, cell].float() * s["v_scale"][page, :, cell].float()[..., None]
    return [k.bfloat16(), v.bfloat16()]


def _tables_plain(s):
    old, new, n_tok = s["seq_lens"].long(), s["new_lens"].long(), s["n_tok"]
    tables, free = s["page_tables"], s["free_pages"]
    total = old + new
    cu = torch.cat((new.new_zeros(1), new.cumsum(0)))
    held, need = (old + PAGE - 1) // PAGE, (total + PAGE - 1) // PAGE
    taken = (need - held).cumsum(0)
    base = s["free_head"].long() + taken - (need - held) - held          # + logical page: place in the free list
    lp = torch.arange(tables.shape[1], device="cuda")
    fresh = (lp >= held[:, None]) & (lp < need[:, None])
    tables.copy_(torch.where(fresh, free[(base[:, None] + lp).clamp(0, free.numel() - 1)], tables))
    tok = torch.arange(n_tok, device="cuda")
    seq = torch.searchsorted(cu[1:], tok, right=True)
    live = tok < cu[-1]
    seq_c = seq.clamp(max=old.numel() - 1)
    pos = old[seq_c] + tok - cu[seq_c]
    page = tables[seq_c, (pos // PAGE).clamp(max=tables.shape[1] - 1)].long()
    slots = torch.where(live, page * PAGE + pos % PAGE, -1)
    return [tables, slots.int(), torch.where(live, pos, 0).int(), torch.where(live, seq, -1).int(), total.int(), cu.int(),
            (s["free_head"].long() + taken[-1]).int().view(1)]


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    if case["op"] == "attn":
        n_seq, n_kv, heads = case["n_seq"], case["n_kv"], case["n_kv"] * case["group"]
        lo, hi = case["lo"], case["hi"]
        w = case["window"] or hi
        # the mean of min(length, window) over lengths lo .. hi
        below = max(0, min(hi, w) - lo)
        cells = n_seq * ((below * (lo + min(hi, w)) / 2 + (hi - lo - below) * w) / (hi - lo) if hi > lo else min(lo, w))
        read = cells * n_kv * 2 * (HEAD_DIM + 2) + cells / PAGE * 4 + n_seq * heads * HEAD_DIM * 2 + n_seq * 4
        write = n_seq * heads * (HEAD_DIM * 2 + (4 if case["lse"] else 0))
        return {"bytes": read + write, "flops": cells * heads * HEAD_DIM * 4}
    if case["op"] == "append":
        n, n_kv, heads = case["n_tok"], case["n_kv"], case["n_kv"] * case["group"]
        move = n * heads * HEAD_DIM * 4 + n * n_kv * 2 * (HEAD_DIM * 2 + HEAD_DIM + 2) + n * 4 * (case["axes"] + 1)
        back = n * n_kv * 2 * HEAD_DIM * 2               # the written cells as BF16
        return {"bytes": move + back, "flops": n * (heads + n_kv) * case["pairs"] * 6}
    if case["op"] == "gather":
        n, n_kv = case["n_cell"], case["n_kv"]
        return {"bytes": n * n_kv * 2 * (HEAD_DIM + 2 + 2 * HEAD_DIM) + 4 * n, "flops": n * n_kv * 2 * HEAD_DIM}
    n_seq, mean = case["n_seq"], (case["lo"] + case["hi"]) / 2
    tok = n_seq * mean
    return {"bytes": n_seq * (4 * 4 + 4) + 12 * n_seq * case["hi"] + tok / PAGE * 8, "flops": 2 * n_seq + 4 * tok}


# ---------------------------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    if case["op"] == "tables":
        return None                                       # whole numbers
    s = prepare(case, seed)
    if case["op"] == "attn":
        return _attn_exact(s)
    page, cell = torch.div(s["slots"].long(), PAGE, rounding_mode="floor"), s["slots"].long().remainder(PAGE)
    if case["op"] == "gather":
        return [torch.einsum("nhd,nh->nhd", pool[page, :, cell].double(), scale[page, :, cell].double())
                for pool, scale in ((s["k_pool"], s["k_scale"]), (s["v_pool"], s["v_scale"]))]
    return _append_exact(s)


def _attn_exact(s):
    """Sequence by sequence over its own cells."""
    n_kv, group = s["n_kv"], s["group"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    for i, n in enumerate(s["seq_lens"].tolist()):
        first = max(0, n - s["window"]) if s["window"] else 0
        at = torch.arange(first, n, device="cuda")
        page = s["page_tables"][i].long()[at // PAGE]
        at, page = at[page >= 0], page[page >= 0]
        if not at.numel():
            continue
        k = s["k_pool"][page, :, at % PAGE].double() * s["k_scale"][page, :, at % PAGE].double().unsqueeze(-1)     # [cell, kv, dim]
        v = s["v_pool"][page, :, at % PAGE].double() * s["v_scale"][page, :, at % PAGE].double().unsqueeze(-1)
        q = s["q"][i].double().view(n_kv, group, HEAD_DIM)
        score = torch.einsum("kgd,ckd->kgc", q, k) / math.sqrt(HEAD_DIM)
        lse[i] = torch.logsumexp(score, -1).flatten()
        out[i] = torch.einsum("kgc,ckd->kgd", torch.softmax(score, -1), v).reshape(-1, HEAD_DIM)
    return [out, lse if s["lse"] else None]


def _append_exact(s):
    """Each pair of dims as a complex number, multiplied by e^(i * position * frequency)."""
    pairs, n = s["pairs"], s["n_tok"]
    axis = s["pair_axis"].tolist()
    angle = torch.stack([s["positions"][axis[j]].double() * s["inv_freq"][j] for j in range(pairs)], 1)
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]
    first = torch.arange(pairs, device="cuda") * (2 if s["interleaved"] else 1)
    second = first + (1 if s["interleaved"] else pairs)

    def turned(x):
        x = x.double().clone()
        z = torch.complex(x[..., first], x[..., second]) * turn
        x[..., first], x[..., second] = z.real, z.imag
        return x

    def held(x):
        want = x.abs().amax(-1, keepdim=True) / 127
        bits = torch.frexp(want)[1] - 11                                  # the step of FP16's 11-bit significand, 2^-24 at least
        step = torch.ldexp(torch.ones_like(want), bits.clamp(min=-24))
        scale = torch.ceil(want / step) * step
        whole = torch.round(x / torch.where(scale == 0, 1.0, scale))
        return whole.clamp(-127, 127) * scale

    assert n == s["q"].shape[0]
    return [turned(s["q"]), held(turned(s["k"])), held(s["v"].double())]
