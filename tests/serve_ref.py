"""Plain 64-bit references of the serving operators, written from their definitions (tests only)."""
import math

import numpy as np
import torch

PAGE, DIM = 64, 128


def make_cache(n_pages, n_kv, seed, lo=0.01, hi=0.03, device="cpu"):
    """INT8 pages uniform in [-127, 127], FP16 scales uniform in [lo, hi]."""
    g = torch.Generator().manual_seed(seed)
    shape = (n_pages, n_kv, PAGE, DIM)
    k = torch.randint(-127, 128, shape, dtype=torch.int8, generator=g)
    v = torch.randint(-127, 128, shape, dtype=torch.int8, generator=g)
    ks = (torch.rand(shape[:3], generator=g) * (hi - lo) + lo).half()
    vs = (torch.rand(shape[:3], generator=g) * (hi - lo) + lo).half()
    return [t.to(device) for t in (k, v, ks, vs)]


def paged_attn(q, k_pool, v_pool, k_scale, v_scale, page_tables, seq_lens, sm_scale, window=0, bias=0):
    """-> (out, lse, mean |v|, reach, lengths): out and lse in FP64; mean |v| = the softmax-weighted mean of |v| (what a
    relative error of the weights scales with); reach = the largest sum over d of |q_d k_d| * |sm_scale| of a row's cells
    (what the error of an FP32 score scales with); with `bias`, |k_d| is taken larger by that many of its row's scales
    (for rows of small integers: the kernel sums q (k + 128) from -128 sum(q), so its FP32 roundings are of magnitudes up
    to sum |q| (|k| + 128) + 128 |sum q|, that is of |k| larger by 256)."""
    n_seq, n_heads, _ = q.shape
    n_kv = k_pool.shape[1]
    group = n_heads // n_kv
    out = torch.zeros(q.shape, dtype=torch.float64)
    mean = torch.zeros(q.shape, dtype=torch.float64)
    lse = torch.full((n_seq, n_heads), -math.inf, dtype=torch.float64)
    reach = torch.zeros((n_seq, n_heads), dtype=torch.float64)
    for s in range(n_seq):
        n = int(seq_lens[s])
        c = torch.arange(max(0, n - window) if window else 0, n)
        page = page_tables[s].long()[c // PAGE]
        c, page = c[page >= 0], page[page >= 0]
        if len(c) == 0:
            continue
        for h in range(n_kv):
            k = k_pool[page, h, c % PAGE].double() * k_scale[page, h, c % PAGE].double()[:, None]
            v = v_pool[page, h, c % PAGE].double() * v_scale[page, h, c % PAGE].double()[:, None]
            rows = slice(h * group, (h + 1) * group)
            x = q[s, rows].double()
            score = x @ k.T * sm_scale
            p = torch.softmax(score, -1)
            out[s, rows] = p @ v
            mean[s, rows] = p @ v.abs()
            lse[s, rows] = torch.logsumexp(score, -1)
            size = k.abs() + bias * k_scale[page, h, c % PAGE].double()[:, None]
            reach[s, rows] = (x.abs() @ size.T).amax(-1) * abs(sm_scale)
    return out, lse, mean, reach, torch.tensor([int(n) for n in seq_lens], dtype=torch.float64)


def check_attn(out, lse, ref, what=""):
    """Weights are rounded to FP16 once (half a step: 2^-11 of the weight), scores are FP32 sums of 128 exact products
    (the matrix unit may cut its partial sums: 32 steps of 2^-23 of the sum of magnitudes) and enter through an
    exponential good to 2^-20; twice that, since numerator and denominator both carry it.  A sum of n positive FP32
    terms is good to its longest chain of additions times 2^-24 (the standard bound of recursive summation); chains here
    are at most 128 + n / 64 additions long, on the matrix unit with steps of 2^-23.  Then the output's own rounding,
    half a step of its type."""
    want, want_lse, mean, reach, n = ref
    score = 32 * 2.0 ** -23 * reach + 2.0 ** -20 + ((128 + n / 32) * 2.0 ** -24)[:, None]
    tol = (2.0 ** -11 + 2 * score)[..., None] * mean + 2.0 ** -30 * mean.amax(-1, keepdim=True)
    got = out.double().cpu()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    tol = tol + (want.abs() + tol) * torch.finfo(out.dtype).eps / 2 + torch.finfo(out.dtype).tiny
    err = (got - want).abs()
    assert (err <= tol).all(), f"{what}: error {err.max():.3e}, {(err / tol).max():.2f} of the tolerance"
    if lse is not None:
        got = lse.double().cpu()
        empty = want_lse == -math.inf
        assert (got[empty] == -math.inf).all(), f"{what}: lse of an empty row"
        err = (got - want_lse).abs()[~empty]
        tol = (score + 2.0 ** -22 * want_lse.abs())[~empty] + 2.0 ** -20
        assert (err <= tol).all(), f"{what}: lse error {err.max():.3e}, {(err / tol).max():.2f} of the tolerance"


def turned(x, positions, inv_freq, pair_axis, interleaved):
    """x [n_tok, n_heads, 128] with its pairs turned, in FP64."""
    x = x.double().cpu().clone()
    pairs = len(inv_freq)
    axis = pair_axis.cpu().long() if pair_axis is not None else torch.zeros(pairs, dtype=torch.long)
    angle = positions.cpu().double()[axis].T * inv_freq.cpu()
    j = torch.arange(pairs)
    a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + pairs)
    c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    u, w = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    x[..., a], x[..., b] = u, w
    return x


def check_turned(got, x, want):
    """Half a step of the type, over FP32 sines, cosines and products (their angle is good to 2^-23 of a half turn:
    together within 8 steps of 2^-23 of the pair's largest value, here bounded by the row's)."""
    size = x.double().cpu().abs().amax(-1, keepdim=True) * math.sqrt(2)
    tol = want.abs() * torch.finfo(got.dtype).eps / 2 + size * 2.0 ** -20
    err = (got.double().cpu() - want).abs()
    assert (err <= tol).all(), f"error {err.max():.3e}, {(err / tol).max():.2f} of the tolerance"


def check_cells(ints, scale, want, slack):
    """A row's scale is max |x| / 127 rounded up to FP16 and its integers x / scale rounded; `slack`: how far the
    kernel's FP32 x may be from `want` (FP64), relative to the row's largest value."""
    ints, scale = ints.double().cpu(), scale.double().cpu()
    top = want.abs().amax(-1)
    lo = top * (1 - slack) / 127
    hi = torch.maximum(top * (1 + slack) / 127 * (1 + 2.0 ** -10), top * (1 + slack) / 127 + 2.0 ** -24)
    assert ((scale >= lo) & (scale <= hi)).all(), "scale"
    assert (ints.abs() <= 127).all()
    err = (ints * scale[..., None] - want).abs()
    tol = scale[..., None] * (0.5 + 2.0 ** -16) + slack * top[..., None]
    assert (err <= tol).all(), f"cell off by {(err / tol).max():.3f} of the tolerance"


def extend_tables(seq_lens, new_lens, tables, free, n_tok, n_ppages, head=0):
    """Token by token -> (tables, slots, positions, token_seq, seq_lens, cu, head, bits)."""
    tables, free = np.array(tables), np.array(free)
    n_seq, width = tables.shape
    slots, pos, seq = np.full(n_tok, -1), np.zeros(n_tok, int), np.full(n_tok, -1)
    lens, cu, bits, t = np.zeros(n_seq, int), [0], 0, 0
    if head < 0 or head > len(free):
        bits |= 128
        head = min(max(head, 0), len(free))
    taken = head
    for s in range(n_seq):
        o = min(max(int(seq_lens[s]), 0), width * PAGE)
        n = min(max(int(new_lens[s]), 0), width * PAGE - o)
        if o != seq_lens[s] or n != new_lens[s]:
            bits |= 64
        if n > n_tok - t:
            bits |= 256
            n = n_tok - t
        held = -(-o // PAGE)
        for c in range(o, o + n):
            lp = c // PAGE
            if lp >= held and (c % PAGE == 0):
                page = -1
                if taken >= len(free):
                    bits |= 128
                elif not 0 <= free[taken] < n_ppages:
                    bits |= 8
                else:
                    page = free[taken]
                tables[s, lp] = page
                taken += 1
            page = tables[s, lp]
            if page < 0 and lp < held:
                bits |= 128
            if page >= n_ppages:
                bits |= 8
                page = -1
            slots[t] = page * PAGE + c % PAGE if page >= 0 else -1
            pos[t], seq[t] = c, s
            t += 1
        lens[s] = o + n
        cu.append(t)
    return tables, slots, pos, seq, lens, np.array(cu), min(taken, len(free)), bits
