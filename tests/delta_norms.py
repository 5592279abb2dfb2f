"""The gated delta rule's outputs in 64 bits with the lengths of the state's rows, and a check of outputs by 2-norms (tests only)."""
import torch

import linear_ref as ref

# Errors of 32-bit sums and of pairs of FP16 (22 bits), relative to the lengths of what is multiplied: a pair is off by 2^-22 at
# most, a product of two pairs without lo lo by 3 x 2^-22, a sum of products over 128 dims or 64 tokens, by Cauchy, by that of the
# lengths.  Three such products lie between a state and an output (S k, T X, P V'), FP32 sums cut at 2^-23 with each:
# 3 x (3 x 2^-22 + 2^-23) < 2^-18.5; single roundings of the factors the rest up to 2^-18.
FINE = 2.0 ** -18


def delta(q, k, v, a, b, a_log, dt_bias, state, slots, old_lens, cu_tokens, eps, scale):
    """-> (out, L) [n_tok, n_v, 128]: L[t] is scale times the length of the state row after token t plus that of the value, which
    is what the sums behind out[t] are made of; rows that belong to nobody are NaN."""
    rep = v.shape[1] // q.shape[1]
    alpha, beta = ref.gates(a, b, a_log, dt_bias)
    unit = lambda x: x.double() / torch.sqrt(x.double().square().sum(-1, keepdim=True) + eps)  # noqa: E731
    qn, kn = (unit(x).repeat_interleave(rep, 1) for x in (q, k))
    out = torch.full(v.shape, float("nan"), dtype=torch.float64, device=v.device)
    size, vd = torch.zeros_like(out), v.double()
    for s, (lo, hi) in enumerate(ref.spans(cu_tokens)):
        slot = int(slots[s])
        if slot < 0 or slot >= state.shape[0]:
            continue
        st = state[slot].double()
        if old_lens is not None and old_lens[s] <= 0:
            st = torch.zeros_like(st)
        for t in range(lo, hi):
            before = alpha[t][:, None, None] * st
            new = beta[t][:, None] * (vd[t] - torch.einsum("hvk,hk->hv", before, kn[t]))
            st = before + new[..., None] * kn[t][:, None, :]
            out[t] = torch.einsum("hvk,hk->hv", st, qn[t]) * scale
            size[t] = before.square().sum(-1).sqrt() + vd[t].abs()
    return out, size * abs(scale)


def excess(got, want, size, dtype):
    """How far the outputs are from the 64-bit ones rounded to the type, and how far they may be, as 2-norms of each head.
    An output whose error before rounding is e is rounded to another value than it should be with a probability of e / step, and
    is then a step off: the mean square is e times a step.  With |e| <= FINE L and steps of at most eps |out|, by Cauchy:
    FINE |L| eps |out|, and twice that for what chance adds; and (2^-25)^2 an element below FP16's normal numbers."""
    mine = ~torch.isnan(want[:, 0, 0])
    got, want, size = got[mine].double(), want[mine], size[mine]
    norm = lambda x: x.square().sum((0, 2)).sqrt()  # noqa: E731
    may = (2 * FINE * norm(size) * torch.finfo(dtype).eps * norm(want) + want.shape[0] * 128 * 2.0 ** -50).sqrt()
    return norm(got - want.to(dtype).double()), may


def check(got, want, size, dtype, what=""):
    off, may = excess(got, want, size, dtype)
    assert bool((off <= may).all()), (what, float((off / may).max()))
