"""The operators of linear-attention layers with the gated delta rule, as cases that can be timed and compared.

A model with such layers runs them beside its selected-cell attention layers: the
short convolution and the delta rule take the place of the cache and its
attention, and keep a state of fixed size per sequence.  Each case is one call of
one operator on inputs made from a seed.  `run` computes it in its plain form
(elementary torch operations, 32 bits) or, with `own` set, through the library's
kernels (`sparse_selected_cell_gb300.qsa`; `include/qsa.h` has the layouts).

  conv    a causal depthwise convolution over the last `width` inputs of a sequence,
          then SiLU, for the new tokens of several sequences laid end to end; the last
          width - 1 inputs of a sequence are its state
  prompt  the gated delta rule over the new tokens of several sequences laid end to end:
          S_t = exp(g_t) S_{t-1} + beta_t (v_t - exp(g_t) S_{t-1} k_t) k_t^T, o_t = S_t q_t, with q
          and k of unit length (q times 128^-1/2), g = -exp(a_log) softplus(a + dt_bias),
          beta = sigmoid(b)
  step    the same for one token of every sequence
  norm    each group of a token's channels normalised (by its root mean square, or centred
          and by its standard deviation), weighted, and multiplied by SiLU(gate)
"""
import itertools
import math
import random

import torch

own = False

DIM = 128           # of a key and of a value head
CHUNK = 64          # tokens of the plain form's chunks
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _qsa():
    from sparse_selected_cell_gb300 import qsa
    return qsa


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one token of one sequence: latency alone
        dict(name="conv-1", op="conv", n_seq=1, lo=1, hi=1, n_k=16, n_v=32, width=4, bias=False, fresh=0.0, type="bf16"),
        # a decode batch
        dict(name="conv-512x1", op="conv", n_seq=512, lo=1, hi=1, n_k=16, n_v=32, width=4, bias=False, fresh=0.0, type="bf16"),
        # a step that takes in prompts of very different lengths, some of them continued
        dict(name="conv-9x1-2000", op="conv", n_seq=9, lo=1, hi=2000, n_k=16, n_v=32, width=4, bias=True, fresh=0.5, type="bf16"),
        # a short message to one running conversation
        dict(name="prompt-1x61", op="prompt", n_seq=1, lo=61, hi=61, n_k=16, n_v=32, fresh=0.0, type="bf16"),
        # one prompt chunk of a long document: the sequence is one long chain
        dict(name="prompt-1x8192", op="prompt", n_seq=1, lo=8192, hi=8192, n_k=16, n_v=32, fresh=0.0, type="bf16"),
        # a ragged step of prompts
        dict(name="prompt-24x1-2000", op="prompt", n_seq=24, lo=1, hi=2000, n_k=8, n_v=16, fresh=0.5, type="fp16"),
        # the largest: a full batch of long prompts
        dict(name="prompt-12x4096", op="prompt", n_seq=12, lo=4096, hi=4096, n_k=16, n_v=32, fresh=1.0, type="bf16"),
        # one sequence's next token
        dict(name="step-1", op="step", n_seq=1, n_k=16, n_v=32, type="bf16"),
        # an ordinary decode batch
        dict(name="step-61", op="step", n_seq=61, n_k=16, n_v=32, type="bf16"),
        # a large decode batch: the states are read and written whole
        dict(name="step-768", op="step", n_seq=768, n_k=16, n_v=32, type="bf16"),
        # a decode batch's heads
        dict(name="norm-64", op="norm", n_tok=64, groups=32, size=128, gate=True, centred=False, type="bf16"),
        # a prompt chunk's
        dict(name="norm-8192", op="norm", n_tok=8192, groups=32, size=128, gate=True, centred=False, type="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv", "prompt", "prompt", "step", "norm"])
    kind = rng.choice(["bf16", "bf16", "fp16"])
    n_k = rng.choice([1, 4, 8, 16])
    n_v = n_k * rng.choice([1, 2, 2, 3])
    if op == "conv":
        n_seq = _log(rng, 1, 512)
        hi = _log(rng, 1, max(1, 12000 // n_seq))
        return dict(op=op, n_seq=n_seq, lo=rng.choice([0, 1, hi]), hi=hi, n_k=n_k, n_v=n_v, width=rng.choice([2, 3, 4, 4]),
                    bias=rng.random() < 0.5, fresh=rng.choice([0.0, 0.5, 1.0]), type=kind)
    if op == "prompt":
        n_seq = _log(rng, 1, 64)
        hi = _log(rng, 2, min(8192, max(2, 1200000 // (n_seq * n_v))))
        return dict(op=op, n_seq=n_seq, lo=rng.choice([0, 1, hi // 2, hi]), hi=hi, n_k=n_k, n_v=n_v,
                    fresh=rng.choice([0.0, 0.5, 1.0]), type=kind)
    if op == "step":
        return dict(op=op, n_seq=_log(rng, 1, 24000 // n_v), n_k=n_k, n_v=n_v, type=kind)
    size = rng.choice([64, 128, 128, 256, 1000])
    groups = rng.choice([1, 8, 32])
    return dict(op=op, n_tok=_log(rng, 1, 30000000 // (groups * size)), groups=groups, size=size, gate=rng.random() < 0.7,
                centred=rng.random() < 0.4, type=kind)


# ---------------------------------------------------------------- inputs

def _lens(case):
    """New tokens of each sequence, spread over the case's range: the case's own, so that outputs of all seeds are alike in shape."""
    if case["op"] == "step":
        return [1] * case["n_seq"]
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    lens = [rng.randint(case["lo"], case["hi"]) for _ in range(case["n_seq"])]
    lens[rng.randrange(len(lens))] = case["hi"]      # a step without a token is no step
    return lens


def _ragged(case, s, g):
    """Lengths, where the sequences begin, which go on from a state, and where in the pool the states lie."""
    n_seq, lens = case["n_seq"], _lens(case)
    s["cu_tokens"] = torch.tensor([0] + list(itertools.accumulate(lens)), dtype=torch.int32).cuda()
    s["n_tok"] = sum(lens)
    s["old_lens"] = torch.where(torch.rand(n_seq, device="cuda", generator=g) < case["fresh"], 0, 1000).int()
    s["state_slots"] = torch.randperm(n_seq + 2, device="cuda", generator=g)[:n_seq].int()


def _heads(case, s, n_tok, g):
    """Queries, keys and values side by side as the short convolution leaves them (past its SiLU), and the two gates'
    inputs side by side as a projection leaves them; decays and time steps as such layers are initialised."""
    n_k, n_v, dtype = case["n_k"], case["n_v"], TYPES[case["type"]]
    rand = lambda *shape: torch.randn(shape, device="cuda", generator=g)  # noqa: E731
    qkv = torch.nn.functional.silu(rand(n_tok, 2 * n_k + n_v, DIM)).to(dtype)
    s["q"], s["k"], s["v"] = qkv[:, :n_k], qkv[:, n_k:2 * n_k], qkv[:, 2 * n_k:]
    ab = rand(n_tok, 2 * n_v).to(dtype)
    s["a"], s["b"] = ab[:, :n_v], ab[:, n_v:]
    s["a_log"] = torch.log(torch.rand(n_v, device="cuda", generator=g) * 15 + 1)
    dt = torch.exp(torch.rand(n_v, device="cuda", generator=g) * math.log(100) + math.log(1e-3))
    s["dt_bias"] = dt + torch.log(-torch.expm1(-dt))
    s["out_t"] = torch.empty((n_tok, n_v, DIM), dtype=dtype, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s, dtype = dict(case), TYPES[case["type"]]
    rand = lambda *shape: torch.randn(shape, device="cuda", generator=g)  # noqa: E731
    if case["op"] == "norm":
        shape = (case["n_tok"], case["groups"], case["size"])
        s["x"] = (rand(*shape) * 0.3 + (0.1 if case["centred"] else 0.0)).to(dtype)
        s["gate_t"] = rand(*shape).to(dtype) if case["gate"] else None
        s["weight"] = (1 + 0.1 * rand(case["size"])).to(dtype)
        s["shift"] = (0.1 * rand(case["size"])).to(dtype) if case["centred"] else None
        s["out_t"] = torch.empty(shape, dtype=dtype, device="cuda")
        return s
    if case["op"] == "step":
        s["n_tok"] = case["n_seq"]
        s["state_slots"] = torch.randperm(case["n_seq"] + 2, device="cuda", generator=g)[:case["n_seq"]].int()
        s["old_lens"] = torch.full((case["n_seq"],), 1000, dtype=torch.int32, device="cuda")
    else:
        _ragged(case, s, g)
    if case["op"] == "conv":
        n_ch = (2 * case["n_k"] + case["n_v"]) * DIM
        # the projection's output: queries, keys and values, then the output gate, which the convolution leaves alone
        s["x"] = rand(s["n_tok"], n_ch + case["n_v"] * DIM).to(dtype)[:, :n_ch]
        s["weight"] = (rand(n_ch, case["width"]) * case["width"] ** -0.5).to(dtype)
        s["bias_t"] = (0.1 * rand(n_ch)).to(dtype) if case["bias"] else None
        s["state"] = rand(case["n_seq"] + 2, case["width"] - 1, n_ch).to(dtype)
        s["out_t"] = torch.empty((s["n_tok"], n_ch), dtype=dtype, device="cuda")
        return s
    _heads(case, s, s["n_tok"], g)
    s["state"] = rand(case["n_seq"] + 2, case["n_v"], DIM, DIM) * 0.2
    if own and case["op"] == "prompt":
        s["workspace"] = torch.empty(_qsa().delta_prompt_workspace_bytes(s["n_tok"], case["n_seq"], case["n_k"], case["n_v"]),
                                     dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    if s["op"] == "conv":
        return _conv_own(s) if own else _conv_plain(s)
    if s["op"] == "prompt":
        return _prompt_own(s) if own else _prompt_plain(s)
    if s["op"] == "step":
        return _step_own(s) if own else _step_plain(s)
    return _norm_own(s) if own else _norm_plain(s)


def _conv_own(s):
    # one token to every sequence needs no table of where they begin
    cu = None if s["lo"] == s["hi"] == 1 else s["cu_tokens"]
    out = _qsa().short_conv(s["x"], s["weight"], s["state"], s["state_slots"], s["old_lens"], cu, bias=s["bias_t"], out=s["out_t"])
    return [out, s["state"]]


def _prompt_own(s):
    out = _qsa().delta_prompt(s["q"], s["k"], s["v"], s["a"], s["b"], s["a_log"], s["dt_bias"], s["state"], s["state_slots"],
                              s["old_lens"], s["cu_tokens"], eps=EPS, out=s["out_t"], workspace=s["workspace"])
    return [out, s["state"]]


def _step_own(s):
    out = _qsa().delta_step(s["q"], s["k"], s["v"], s["a"], s["b"], s["a_log"], s["dt_bias"], s["state"], s["state_slots"],
                            s["old_lens"], eps=EPS, out=s["out_t"])
    return [out, s["state"]]


def _norm_own(s):
    return _qsa().group_norm(s["x"], s["weight"], s["shift"], gate=s["gate_t"], eps=EPS, centred=s["centred"], out=s["out_t"])


def _conv_plain(s):
    x, width, n_seq, n_tok = s["x"].float(), s["width"], s["n_seq"], s["n_tok"]
    cu, slots = s["cu_tokens"].long(), s["state_slots"].long()
    held = torch.where((s["old_lens"] > 0)[:, None, None], s["state"][slots].float(), 0.0)
    # every sequence's state before its tokens
    at = torch.arange(n_tok, device="cuda")
    seq = torch.searchsorted(cu[1:], at, right=True)
    full = x.new_zeros((n_tok + n_seq * (width - 1), x.shape[1]))
    place = at + (seq + 1) * (width - 1)
    full[place] = x
    begin = cu[:-1] + torch.arange(n_seq, device="cuda") * (width - 1)
    back = torch.arange(width - 1, device="cuda")
    full[begin[:, None] + back] = held
    taps = torch.arange(width, device="cuda") - (width - 1)
    w = s["weight"].float()
    y = sum(full[place + taps[j]] * w[:, j] for j in range(width))
    if s["bias_t"] is not None:
        y = y + s["bias_t"].float()
    s["state"][slots] = full[(cu[1:] + torch.arange(1, n_seq + 1, device="cuda") * (width - 1))[:, None] - (width - 1) + back].to(s["x"].dtype)
    return [(y / (1 + torch.exp(-y))).to(s["x"].dtype), s["state"]]


def _unit(x):
    x = x.float()
    return x * torch.rsqrt((x * x).sum(-1, keepdim=True) + EPS)


def _gates(s):
    """(g, beta) of every token and value head."""
    u = s["a"].float() + s["dt_bias"]
    soft = torch.clamp(u, min=0) + torch.log1p(torch.exp(-u.abs()))
    return -torch.exp(s["a_log"]) * soft, 1 / (1 + torch.exp(-s["b"].float()))


def _prompt_plain(s):
    """Chunk by chunk: with D_ij = exp(g_{j+1} + ... + g_i), V' = (I + strictly lower (beta K K^T D))^-1 beta (V - exp(G) K S),
    O = exp(G) Q S + lower (Q K^T D) V', S' = exp(G_C) S + K^T exp(G_C - G) V'."""
    n_seq, n_k, n_v, n_tok = s["n_seq"], s["n_k"], s["n_v"], s["n_tok"]
    cu = s["cu_tokens"].long()
    n_chunk = -(-s["hi"] // CHUNK)
    # the sequences side by side, padded with tokens that change nothing (beta = 0, g = 0)
    at = cu[:-1, None] + torch.arange(n_chunk * CHUNK, device="cuda")
    live = at < cu[1:, None]
    at = at.clamp(max=n_tok - 1)
    g, beta = _gates(s)
    rep = n_v // n_k

    def laid(x):                                     # [tok, head, ...] -> [seq, head, chunk, CHUNK, ...]
        x = torch.where(live[..., None, None], x[at], 0.0).transpose(1, 2)
        return x.reshape(n_seq, x.shape[1], n_chunk, CHUNK, x.shape[-1])

    q = laid(_unit(s["q"]) * DIM ** -0.5).repeat_interleave(rep, 1)
    k = laid(_unit(s["k"])).repeat_interleave(rep, 1)
    v, beta = laid(s["v"].float()), laid(beta[..., None])
    gc = laid(g[..., None])[..., 0].double().cumsum(-1)
    decay = torch.exp((gc[..., :, None] - gc[..., None, :]).clamp(max=0)).float()
    a = (beta * (k @ k.transpose(-1, -2)) * decay).tril(-1)
    p = ((q @ k.transpose(-1, -2)) * decay).tril()
    # the inverse of I + a, row by row: row i = e_i - a_i . (the rows before)
    t = torch.eye(CHUNK, device="cuda").expand(a.shape).contiguous()
    for i in range(1, CHUNK):
        t[..., i, :i] -= (a[..., i, None, :i] @ t[..., :i, :i])[..., 0, :]
    total, from_start, to_end = torch.exp(gc[..., -1]).float(), torch.exp(gc).float()[..., None], torch.exp(gc[..., -1:] - gc).float()[..., None]
    slots = s["state_slots"].long()
    state = torch.where((s["old_lens"] > 0)[:, None, None, None], s["state"][slots], 0.0).transpose(-1, -2)   # [seq, head, key dim, value dim]
    out = torch.empty_like(v)
    for c in range(n_chunk):
        kc, qc = k[:, :, c], q[:, :, c]
        vn = t[:, :, c] @ (beta[:, :, c] * (v[:, :, c] - from_start[:, :, c] * (kc @ state)))
        out[:, :, c] = from_start[:, :, c] * (qc @ state) + p[:, :, c] @ vn
        state = total[:, :, c, None, None] * state + (kc * to_end[:, :, c]).transpose(-1, -2) @ vn
    s["state"][slots] = state.transpose(-1, -2)
    out = out.reshape(n_seq, n_v, -1, DIM).transpose(1, 2)
    return [out[live].to(s["v"].dtype), s["state"]]


def _step_plain(s):
    rep, slots = s["n_v"] // s["n_k"], s["state_slots"].long()
    q = (_unit(s["q"]) * DIM ** -0.5).repeat_interleave(rep, 1)
    k, v = _unit(s["k"]).repeat_interleave(rep, 1), s["v"].float()
    g, beta = _gates(s)
    state = torch.where((s["old_lens"] > 0)[:, None, None, None], s["state"][slots], 0.0) * torch.exp(g)[..., None, None]
    vn = beta[..., None] * (v - (state @ k[..., None])[..., 0])
    state = state + vn[..., None] * k[..., None, :]
    s["state"][slots] = state
    return [(state @ q[..., None])[..., 0].to(s["v"].dtype), s["state"]]


def _norm_plain(s):
    x = s["x"].float()
    if s["centred"]:
        x = x - x.mean(-1, keepdim=True)
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * s["weight"].float()
    if s["shift"] is not None:
        y = y + s["shift"].float()
    if s["gate_t"] is not None:
        z = s["gate_t"].float()
        y = y * z / (1 + torch.exp(-z))
    return y.to(s["x"].dtype)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    if case["op"] == "norm":
        n = case["n_tok"] * case["groups"] * case["size"]
        return {"bytes": n * 2 * (3 if case["gate"] else 2) + case["size"] * 2, "flops": n * 8}
    n_seq, n_k, n_v = case["n_seq"], case["n_k"], case["n_v"]
    tok = sum(_lens(case))
    if case["op"] == "conv":
        n_ch, width = (2 * n_k + n_v) * DIM, case["width"]
        held = n_seq * (width - 1) * n_ch * 2
        return {"bytes": tok * n_ch * 4 + held * (2 - case["fresh"]) + n_ch * 2 * (width + case["bias"]), "flops": tok * n_ch * (2 * width + 4)}
    held = n_seq * n_v * DIM * DIM * 4
    move = tok * (2 * n_k + 2 * n_v) * DIM * 2 + tok * n_v * 4
    if case["op"] == "step":
        return {"bytes": move + 2 * held, "flops": tok * n_v * DIM * DIM * 7}
    # of a chunk and value head: Q K^T and K K^T (of a key head), the products with the inverse and with Q K^T, three with the state
    flops = tok * (n_k * 2 * CHUNK * DIM * 2 + n_v * (2 * CHUNK * DIM * 2 + 3 * DIM * DIM * 2))
    return {"bytes": move + held * (2 - case["fresh"]), "flops": flops}


# ---------------------------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _norm_exact(s)
    if case["op"] == "conv":
        return _conv_exact(s)
    return _delta_exact(s, _lens(case))


def _norm_exact(s):
    x = s["x"].double()
    if s["centred"]:
        y = (x - x.mean(-1, keepdim=True)) / torch.sqrt(x.var(-1, unbiased=False, keepdim=True) + EPS)
    else:
        y = x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS)
    y = y * s["weight"].double()
    if s["shift"] is not None:
        y = y + s["shift"].double()
    return y if s["gate_t"] is None else y * torch.nn.functional.silu(s["gate_t"].double())


def _conv_exact(s):
    """Sequence by sequence."""
    width, cu = s["width"], s["cu_tokens"].tolist()
    out = torch.empty(s["x"].shape, dtype=torch.float64, device="cuda")
    state = s["state"].double()
    for i, slot in enumerate(s["state_slots"].tolist()):
        held = state[slot] if s["old_lens"][i] > 0 else torch.zeros_like(state[slot])
        x = torch.cat((held, s["x"][cu[i]:cu[i + 1]].double()))
        if x.shape[0] >= width:
            y = torch.einsum("tcw,cw->tc", x.unfold(0, width, 1), s["weight"].double())
            out[cu[i]:cu[i + 1]] = torch.nn.functional.silu(y if s["bias_t"] is None else y + s["bias_t"].double())
        state[slot] = x[x.shape[0] - (width - 1):]
    return [out, state]


def _delta_exact(s, lens):
    """Token by token, the sequences that still have one together."""
    n_v, rep = s["n_v"], s["n_v"] // s["n_k"]
    u = s["a"].double() + s["dt_bias"].double()
    alpha = torch.exp(-torch.exp(s["a_log"].double()) * torch.nn.functional.softplus(u, threshold=100.0))
    beta = torch.sigmoid(s["b"].double())
    order = sorted(range(len(lens)), key=lambda i: -lens[i])              # the longest first: those with a token left are a prefix
    first = [0]
    for n in lens:
        first.append(first[-1] + n)
    begin = torch.tensor([first[i] for i in order], device="cuda")
    slots = s["state_slots"].long()[order]
    pool = s["state"].double()
    state = pool[slots] * (s["old_lens"][order] > 0)[:, None, None, None]
    out = torch.empty((s["n_tok"], n_v, DIM), dtype=torch.float64, device="cuda")
    some = len(lens)
    for t in range(max(lens)):
        while lens[order[some - 1]] <= t:
            some -= 1
        at = begin[:some] + t
        q, k = (x[at].double() / torch.sqrt(x[at].double().square().sum(-1, keepdim=True) + EPS) for x in (s["q"], s["k"]))
        q, k = q.repeat_interleave(rep, 1) / math.sqrt(DIM), k.repeat_interleave(rep, 1)
        state[:some] *= alpha[at][..., None, None]
        new = beta[at][..., None] * (s["v"][at].double() - torch.einsum("shvk,shk->shv", state[:some], k))
        state[:some] += torch.einsum("shv,shk->shvk", new, k)
        out[at] = torch.einsum("shvk,shk->shv", state[:some], q)
    pool[slots] = state
    return [out, pool]
