"""A linear-attention layer's operators run together, as a serving program runs them: table extension, short convolution, delta
rule, group norm; steps of prompts and of single tokens, captured, on other streams, and behind kernels that write late."""
import pytest

torch = pytest.importorskip("torch")
import linear_ref as ref  # noqa: E402
from test_delta_gpu import batch, i32, qsa  # noqa: E402,F401
from test_serve_order_gpu import check, late  # noqa: E402,F401

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5


class Layer:
    """Weights of one layer, and its states for some sequences."""

    def __init__(self, n_k, n_v, n_slots, dtype=torch.bfloat16, seed=1):
        g = torch.Generator().manual_seed(seed)
        self.n_k, self.n_v, self.n_ch = n_k, n_v, (2 * n_k + n_v) * 128
        self.conv = (torch.randn((self.n_ch, 4), generator=g) * 0.5).to(dtype).cuda()
        self.norm = (1 + 0.1 * torch.randn(128, generator=g)).to(dtype).cuda()
        self.a_log, self.dt_bias = (x.cuda() for x in ref.heads(1, n_k, n_v, dtype, seed)[5:])
        self.conv_state = torch.zeros((n_slots, 3, self.n_ch), dtype=dtype, device="cuda")
        self.state = torch.zeros((n_slots, n_v, 128, 128), device="cuda")

    def step(self, qsa, x, slots, old, cu, status=None, stream=None):  # noqa: F811
        """x [n_tok, channels | gate | a | b] -> (the convolution's output, the rule's, the norm's)."""
        n_tok, n_k, n_v = x.shape[0], self.n_k, self.n_v
        gate, ab = x[:, self.n_ch:self.n_ch + n_v * 128].view(n_tok, n_v, 128), x[:, self.n_ch + n_v * 128:]   # (a, b, then nothing)
        c = qsa.short_conv(x[:, :self.n_ch], self.conv, self.conv_state, slots, old, cu, dev_status=status, stream=stream)
        h = c.view(n_tok, 2 * n_k + n_v, 128)
        args = (h[:, :n_k], h[:, n_k:2 * n_k], h[:, 2 * n_k:], ab[:, :n_v], ab[:, n_v:2 * n_v], self.a_log, self.dt_bias, self.state, slots)
        if cu is None:
            y = qsa.delta_step(*args, old, dev_status=status, stream=stream)
        else:
            y = qsa.delta_prompt(*args, old, cu, dev_status=status, stream=stream)
        return c, y, qsa.group_norm(y, self.norm, gate=gate, stream=stream)

    def width(self):
        return -(-(self.n_ch + self.n_v * 128 + 2 * self.n_v) // 8) * 8      # tokens lie multiples of 8 elements apart


def test_layer_steps(qsa):  # noqa: F811
    """Prompts, single tokens, and both, by extend_tables' bounds and lengths; each operator against its 64-bit definition
    on what it was given."""
    n_seq, pool = 5, 60
    layer = Layer(2, 4, n_seq + 1)
    g = torch.Generator().manual_seed(3)
    slots = i32([3, 0, 5, 1, 2])
    tables = torch.full((n_seq, 8), -1, dtype=torch.int32, device="cuda")
    free, head = torch.randperm(pool, generator=g).int().cuda(), i32([0])
    lens, status = i32([0] * n_seq), i32([0])
    for new in ([130, 64, 7, 200, 1], [1] * 5, [1] * 5, [1, 0, 90, 1, 17], [1] * 5):
        single = new == [1] * 5
        n_tok = sum(new) if single else sum(new) + 11
        x = torch.randn((n_tok, layer.width()), generator=g).bfloat16().cuda()
        t = qsa.extend_tables(lens, i32(new), tables, free, n_tok, pool, free_head=head, dev_status=status)
        before = layer.conv_state.clone(), layer.state.clone()
        cu = None if single else t.cu_tokens
        c, y, z = layer.step(qsa, x, slots, lens, cu, status)
        n = sum(new)
        assert int(status) == 0, qsa.decode_status(int(status))
        want, conv_state, size = ref.short_conv(x[:n, :layer.n_ch], layer.conv, before[0], slots, lens, t.cu_tokens, None, True)
        ref.check_conv(c[:n], want, size, x.dtype, 4)
        assert torch.equal(layer.conv_state, conv_state)
        h, ab = c.view(n_tok, -1, 128)[:n], x[:n, layer.n_ch + 4 * 128:]
        want = ref.delta(h[:, :2], h[:, 2:4], h[:, 4:], ab[:, :4], ab[:, 4:], layer.a_log, layer.dt_bias, before[1], slots, lens,
                         t.cu_tokens, 1e-6, SCALE, ref.STEP if single else ref.CHUNK)
        ref.check_delta(y[:n], layer.state, want, SCALE, x.dtype, not single, slots)
        want, mag = ref.group_norm(y[:n], layer.norm, None, x[:n, layer.n_ch:layer.n_ch + 512].view(n, 4, 128), 1e-6, False, True)
        ref.check_norm(z[:n], want, mag, x.dtype)
        lens, head = t.seq_lens, t.free_head


def test_captured_decode_steps(qsa):  # noqa: F811
    """One captured decode step of the layer, replayed: states carry on as when it is called."""
    a, b = Layer(1, 2, 4, seed=2), Layer(1, 2, 4, seed=2)
    slots, x = i32([2, 0, 3]), torch.randn((3, a.width()), generator=torch.Generator().manual_seed(5)).bfloat16().cuda()
    old = i32([0, 0, 0])
    wants = [[t.clone() for t in a.step(qsa, x * (i + 1), slots, old if i == 0 else None, None)] for i in range(4)]
    b.step(qsa, x, slots, old, None)
    live = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = b.step(qsa, live, slots, None, None)
    for i in range(1, 4):
        live.copy_(x * (i + 1))
        graph.replay()
        for got, want in zip(outs, wants[i]):
            assert torch.equal(got, want)
    assert torch.equal(a.state, b.state) and torch.equal(a.conv_state, b.conv_state)


def test_a_step_on_another_stream(qsa):  # noqa: F811
    """The calls given a stream that is not the current one, with everything they return allocated by them."""
    x = torch.randn((300, Layer(1, 2, 3).width()), generator=torch.Generator().manual_seed(6)).bfloat16().cuda()
    slots, old, cu = i32([2, 0]), i32([0, 0]), i32([0, 90, 300])

    def step(stream):
        layer = Layer(1, 2, 3, seed=4)
        torch.cuda.synchronize()
        outs = []
        c = qsa.short_conv(x[:, :layer.n_ch], layer.conv, layer.conv_state, slots, old, cu, stream=stream)
        torch.full((1 << 20,), 7, dtype=torch.int32, device="cuda")
        h, ab = c.view(300, 4, 128), x[:, layer.n_ch + 256:]
        heads = h[:, :1], h[:, 1:2], h[:, 2:], ab[:, :2], ab[:, 2:4]
        y = qsa.delta_prompt(*heads, layer.a_log, layer.dt_bias, layer.state, slots, old, cu, stream=stream)
        torch.full((1 << 20,), -1, dtype=torch.int32, device="cuda")
        z = qsa.group_norm(y, layer.norm, gate=x[:, layer.n_ch:layer.n_ch + 256].view(300, 2, 128), stream=stream)
        two = [t[:2] for t in heads]
        w = qsa.delta_step(*two, layer.a_log, layer.dt_bias, layer.state, slots, stream=stream)
        torch.cuda.synchronize()
        outs += [c, y, z, w, layer.state, layer.conv_state]
        return outs

    want = step(None)
    for stream in (torch.cuda.Stream(), torch.cuda.Stream().cuda_stream, 0):
        for got, w in zip(step(stream), want):
            assert torch.equal(got, w)


# ---------------------------------------------------------------- inputs written late

@pytest.mark.parametrize("lens", [[61], [1, 1, 1], [9, 3], [400, 70, 1], [1100], [2300]])
def test_late_prompts(qsa, late, lens):  # noqa: F811
    def step(seed):
        inputs, state, slots, old, cu = batch(lens, 1, 2, torch.bfloat16, seed=seed)
        cut = cu.clone()
        if seed and len(lens) > 1:
            cut[1] = cut[1] // 2
        return [*[t.contiguous() for t in inputs], state, slots, old, cut]

    def call(*t):
        return qsa.delta_prompt(*t[:7], t[7], t[8], t[9], t[10]), t[7]

    check(late, step(1), step(0), call)


def test_late_steps(qsa, late):  # noqa: F811
    def step(seed):
        inputs, state, slots, old, _ = batch([1] * 9, 2, 4, torch.bfloat16, seed=seed)
        return [*[t.contiguous() for t in inputs], state, slots, old]

    check(late, step(1), step(0), lambda *t: (qsa.delta_step(*t), t[7]))


@pytest.mark.parametrize("lens", [None, [40, 1, 90, 3], [1] * 30])
def test_late_convolutions(qsa, late, lens):  # noqa: F811
    def step(seed):
        g = torch.Generator().manual_seed(seed)
        n_seq = len(lens) if lens else 20
        n_tok = sum(lens) if lens else n_seq
        rows = lambda *s: torch.randn(s, generator=g).bfloat16()  # noqa: E731
        t = [rows(n_tok, 256), rows(256, 4), rows(n_seq + 2, 3, 256), torch.randperm(n_seq + 2, generator=g)[:n_seq].int(),
             torch.randint(0, 2, (n_seq,), generator=g).int()]
        if lens:
            t.append(torch.tensor([0] + lens).cumsum(0).int())
            if seed:
                t[-1][1] //= 2
        return t

    check(late, step(1), step(0), lambda *t: (qsa.short_conv(*t), t[2]))


def test_late_norms(qsa, late):  # noqa: F811
    def step(seed):
        g = torch.Generator().manual_seed(seed)
        return [torch.randn(s, generator=g).bfloat16() for s in ((300, 4, 128), (300, 4, 128), (128,))]

    check(late, step(1), step(0), lambda x, z, w: (qsa.group_norm(x, w, gate=z),))
