"""The serving calls behind a kernel that releases its dependents first and writes their inputs afterwards: their blocks are
resident, and have run before on the inputs' old values, while lengths, tables, slots, positions, rows and pools change."""
import ctypes
import subprocess

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


@pytest.fixture(scope="module")
def late(tmp_path_factory):
    """late(pairs): each (from, to) copied by such a kernel on the current stream."""
    import os
    from sparse_selected_cell_gb300 import build
    out = str(tmp_path_factory.mktemp("early") / "early_release.so")
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "early_release.cu")
    subprocess.run([build._nvcc(), *build.ARCH, "-O2", "-shared", "-Xcompiler", "-fPIC", "-o", out, src], check=True)
    copy = ctypes.CDLL(out).early_release_copy
    copy.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_longlong, ctypes.c_int, ctypes.c_void_p]

    def call(source, target):
        assert source.nbytes == target.nbytes and target.nbytes % 16 == 0
        assert copy(source.data_ptr(), target.data_ptr(), target.nbytes // 16, 50, torch.cuda.current_stream().cuda_stream) == 0
    return call


class Arena:
    """Tensors laid one after the other in one buffer, so that one kernel writes them all."""

    def __init__(self, tensors):
        at, self.places = 0, []
        for t in tensors:
            self.places.append((at, t.dtype, t.shape))
            at += -(-t.nbytes // 256) * 256
        self.data = torch.zeros(at, dtype=torch.uint8, device="cuda")
        self.tensors = [self.data[a:a + torch.Size(s).numel() * d.itemsize].view(d).view(s) for a, d, s in self.places]
        for view, t in zip(self.tensors, tensors):
            view.copy_(t)


def check(late, old, new, call):
    """call(*inputs) right after they change from old to new, the change made late; `call` returns its outputs."""
    want = [t.clone() for t in call(*Arena(new).tensors)]
    source, live = Arena(new), Arena(old)
    first = live.data.clone()
    for _ in range(5):
        live.data.copy_(first)
        for t in call(*live.tensors):                           # caches hold the old values
            t.zero_()
        torch.cuda.synchronize()
        live.data.copy_(first)                                  # (the call may write to its inputs)
        late(source.data, live.data)
        got = call(*live.tensors)
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g, w)


@pytest.mark.parametrize("lens,n_kv", [([700, 64, 1000], 4), ([9000, 3, 20000], 4), ([300] * 100, 2)])
def test_attention(qsa, late, lens, n_kv):
    """The kernel for short sequences, the one for long ones with few items and its join, and with many."""
    def batch(seed):
        g = torch.Generator().manual_seed(seed)
        need = [-(-n // 64) for n in lens]
        cache = ref.make_cache(sum(need), n_kv, seed)
        tables = torch.zeros((len(lens), max(need)), dtype=torch.int32)
        order, at = torch.randperm(sum(need), generator=g).int(), 0
        for s, n in enumerate(need):
            tables[s, :n] = order[at:at + n]
            at += n
        cut = torch.tensor([max(1, n - 37 * seed) for n in lens], dtype=torch.int32)
        return [torch.randn((len(lens), n_kv * 12, 128), generator=g).bfloat16(), *cache, tables, cut]

    def call(*inputs):
        out = qsa.paged_attn(*inputs, lse=(lse := torch.empty(inputs[0].shape[:2], device="cuda")))
        return out, lse

    check(late, batch(1), batch(0), call)
    empty = batch(1)
    empty[-1].zero_()
    check(late, empty, batch(0), call)


@pytest.mark.parametrize("n_tok", [5, 700])
def test_write_and_read_back(qsa, late, n_tok):
    def step(seed):
        g = torch.Generator().manual_seed(seed)
        cache = ref.make_cache(n_tok // 64 + 3, 2, seed)
        slots = torch.randperm(cache[0].shape[0] * 64, generator=g)[:n_tok].int()
        qkv = torch.randn((n_tok, 28, 128), generator=g).bfloat16()
        pos = torch.randint(0, 9000, (2, n_tok), generator=g).int()
        inv = 10000.0 ** (-torch.arange(64, dtype=torch.float64) / (64 + seed))
        axis = ((torch.arange(64) + seed) % 2).int()
        return [qkv, pos, inv, axis, *cache, slots]

    def write(qkv, pos, inv, axis, k, v, ks, vs, slots):
        q = qsa.rope_append(qkv[:, :24], qkv[:, 24:26], qkv[:, 26:], pos, inv, axis, k, v, ks, vs, slots)
        return q, k, v, ks, vs

    def read(qkv, pos, inv, axis, k, v, ks, vs, slots):
        return (*qsa.cache_gather(k, v, ks, vs, slots), *qsa.cache_gather(k, v, ks, vs, slots, dtype=torch.float32))

    old = step(1)
    check(late, old, step(0), write)
    check(late, old, step(0), read)
    old[-1].fill_(-1)
    check(late, old, step(0), write)
    check(late, old, step(0), read)


def test_tables(qsa, late):
    def step(seed):
        g = torch.Generator().manual_seed(seed)
        i = lambda lo, hi, *shape: torch.randint(lo, hi, shape, dtype=torch.int32, generator=g)  # noqa: E731
        return [i(0, 400, 300), i(0, 20, 300), i(0, 10000, 300, 8), torch.randperm(10000, generator=g).int(), i(0, 9, 1)]

    def call(lens, new, tables, free, head):
        return (*qsa.extend_tables(lens, new, tables, free, 6500, 10000, free_head=head), tables)

    check(late, step(1), step(0), call)
