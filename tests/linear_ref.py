"""Plain 64-bit references of the layers with a state, written from their definitions (tests only)."""
import math

import torch

DIM = 128


def spans(cu_tokens):
    cu = [int(c) for c in cu_tokens]
    return list(zip(cu[:-1], cu[1:]))


def short_conv(x, weight, state, slots, old_lens, cu_tokens, bias, silu):
    """-> (out, new state, sum of |products|): rows that belong to nobody are NaN in out; the state in x's type."""
    width = weight.shape[1]
    out = torch.full(x.shape, math.nan, dtype=torch.float64, device=x.device)
    size = torch.zeros_like(out)
    state = state.clone()
    for s, (lo, hi) in enumerate(spans(cu_tokens)):
        slot = int(slots[s])
        if slot < 0 or slot >= state.shape[0]:
            continue
        held = state[slot] if old_lens is None or old_lens[s] > 0 else torch.zeros_like(state[slot])
        rows = torch.cat((held, x[lo:hi]))
        for t in range(lo, hi):
            terms = rows[t - lo:t - lo + width].double().T * weight.double()
            y = terms.sum(1) + (0 if bias is None else bias.double())
            out[t] = y * torch.sigmoid(y) if silu else y
            size[t] = terms.abs().sum(1) + (0 if bias is None else bias.double().abs())
        state[slot] = rows[rows.shape[0] - (width - 1):]
    return out, state, size


def check_conv(got, want, size, dtype, width, what=""):
    """One rounding to the type (half a step; FP16's subnormals: 2^-25), an FP32 sum of width + 1 terms, SiLU's slope of at
    most 1.1 and its own 2^-20."""
    mine = ~torch.isnan(want)
    err = (got.double() - want).abs()
    tol = want.abs() * (torch.finfo(dtype).eps / 2 + 2 ** -19) + 1.1 * (width + 2) * 2 ** -24 * size + 2 ** -25
    assert bool((err <= tol)[mine].all()), (what, float((err / tol)[mine].max()))


def group_norm(x, weight, bias, gate, eps, centred, silu):
    """-> (out, magnitude that FP32 errors scale with)."""
    x = x.double()
    m = x.mean(-1, keepdim=True) if centred else torch.zeros_like(x[..., :1])
    r = 1 / torch.sqrt((x - m).square().mean(-1, keepdim=True) + eps)
    w = 1.0 if weight is None else weight.double()
    b = 0.0 if bias is None else bias.double()
    y = (x - m) * r * w + b
    size = (x.abs() + x.abs().mean(-1, keepdim=True)) * r * abs(w) + abs(b)
    act = (lambda z: z * torch.sigmoid(z)) if silu else (lambda z: z)
    if gate is not None:
        return y * act(gate.double()), size * act(gate.double()).abs()
    return act(y), size * 1.1


def check_norm(got, want, size, dtype):
    """One rounding to the type; sums of at most 32 terms in a thread, five and eight more between threads (45 x 2^-24 of
    the mean magnitude, once for the mean and once for the square root of the mean square), a handful of single
    operations, SiLU's 2^-20: 2^-17 of the magnitudes together; FP16's subnormals 2^-25."""
    err = (got.double() - want).abs()
    tol = want.abs() * torch.finfo(dtype).eps / 2 + 2 ** -17 * size + 2 ** -25
    assert bool((err <= tol).all()), float((err / tol).max())


def gates(a, b, a_log, dt_bias):
    u = a.double() + dt_bias.double()
    soft = torch.clamp(u, min=0) + torch.log1p(torch.exp(-u.abs()))
    return torch.exp(-torch.exp(a_log.double()) * soft), torch.sigmoid(b.double())


def delta(q, k, v, a, b, a_log, dt_bias, state, slots, old_lens, cu_tokens, eps, scale, step):
    """Token by token -> (out, state, R, E): rows that belong to nobody are NaN in out.  R[t] bounds the 2-norm of a
    state row after token t (R = alpha R + |new|, keys being of unit length), E what an error of `step` * R made in every
    token comes to (E = alpha E + step R: the rule itself, alpha (I - beta k k^T), lengthens nothing); both [n_tok, n_v, 128].
    Also E at each sequence's end, by slot."""
    n_tok, n_v = v.shape[:2]
    rep = n_v // q.shape[1]
    alpha, beta = gates(a, b, a_log, dt_bias)
    unit = lambda x: x.double() / torch.sqrt(x.double().square().sum(-1, keepdim=True) + eps)  # noqa: E731
    qn, kn = (unit(x).repeat_interleave(rep, 1) for x in (q, k))
    out = torch.full(v.shape, math.nan, dtype=torch.float64, device=v.device)
    big, off = torch.zeros_like(out), torch.zeros_like(out)
    pool = state.double()
    end = torch.zeros(pool.shape[:3], dtype=torch.float64, device=v.device)
    for s, (lo, hi) in enumerate(spans(cu_tokens)):
        slot = int(slots[s])
        if slot < 0 or slot >= pool.shape[0]:
            continue
        st = pool[slot].clone()
        if old_lens is not None and old_lens[s] <= 0:
            st.zero_()
        r = st.square().sum(-1).sqrt()
        e = torch.zeros_like(r)
        for t in range(lo, hi):
            st *= alpha[t][:, None, None]
            new = beta[t][:, None] * (v[t].double() - torch.einsum("hvk,hk->hv", st, kn[t]))
            st += new[..., None] * kn[t][:, None, :]
            out[t] = torch.einsum("hvk,hk->hv", st, qn[t]) * scale
            # what the sums of the token are made of: the row before it, the value and the new one
            r = alpha[t][:, None] * r + new.abs()
            e = alpha[t][:, None] * e + step * (r + v[t].double().abs())
            big[t], off[t] = r, e
        pool[slot] = st
        end[slot] = e
    return out, pool, big, off, end


STEP = 2 ** -18      # a token by FP32 sums: 128 products in chains of 19 (20 x 2^-24 of the row's length), twice for q and k,
#                      the keys' length (12 x 2^-24), the decay (10 x 2^-24, |g| alpha <= 1/e included): 64 x 2^-24
CHUNK = 2 ** -16     # a token of a chunk: two pairs of FP16 factors (2^-21), matrix sums cut at 32 x 2^-23 of the magnitudes,
#                      three such products in a row


def check_delta(got, got_state, want, scale, dtype, chunked, slots):
    """Outputs: half a step of the type, the state's error, and in chunks three FP16 factors (2^-11 each) of what a state row's
    length bounds.  States: E in each row's 2-norm; and altogether, since the single errors (2^-24, in chunks 2^-21) point
    anywhere, 2^-17 of the whole."""
    out, pool, big, off, end = want
    mine = ~torch.isnan(out)
    err = (got.double() - out).abs()
    tol = out.abs() * (torch.finfo(dtype).eps / 2 * 1.01) + abs(scale) * (off + (3 * 2 ** -11 * big if chunked else 0)) + 2 ** -25
    assert bool((err <= tol)[mine].all()), ("out", float((err / tol)[mine].max()))
    used = sorted({int(x) for x in slots if 0 <= int(x) < pool.shape[0]})
    d = (got_state.double() - pool)[used]
    rows = d.square().sum(-1).sqrt()
    assert bool((rows <= end[used] + 2 ** -24 * pool[used].square().sum(-1).sqrt() + 1e-30).all()), "state rows"
    total = float(pool[used].square().sum().sqrt())
    assert float(d.square().sum().sqrt()) <= 2 ** -17 * total + 1e-30, ("state", float(d.square().sum().sqrt()) / max(total, 1e-30))


def heads(n_tok, n_k, n_v, dtype, seed, device="cuda", apart=0):
    """Queries, keys, values and gate inputs as slices of wider rows, decays as such layers are initialised."""
    g = torch.Generator().manual_seed(seed)
    qkv = torch.nn.functional.silu(torch.randn((n_tok, 2 * n_k + n_v + apart, DIM), generator=g)).to(dtype).to(device)
    ab = torch.randn((n_tok, 2 * n_v + apart), generator=g).to(dtype).to(device)
    a_log = torch.log(torch.rand(n_v, generator=g) * 15 + 1).to(device)
    dt = torch.exp(torch.rand(n_v, generator=g) * math.log(100) + math.log(1e-3))
    dt_bias = (dt + torch.log(-torch.expm1(-dt))).to(device)
    return (qkv[:, :n_k], qkv[:, n_k:2 * n_k], qkv[:, 2 * n_k:2 * n_k + n_v], ab[:, :n_v], ab[:, n_v:2 * n_v], a_log, dt_bias)


def pool(n_slots, n_v, seed, device="cuda", scale=0.2):
    return (torch.randn((n_slots, n_v, DIM, DIM), generator=torch.Generator().manual_seed(seed)) * scale).to(device)
