"""The serving operators' C entries refuse bad arguments on the host, before anything reaches a GPU."""
import ctypes

import pytest

OK, ARG, UNSUPPORTED, CAPACITY = 0, 1, 2, 3
FAKE, ODD = ctypes.c_void_p(0x100000), ctypes.c_void_p(0x100008)


@pytest.fixture(scope="module")
def lib():
    from sparse_selected_cell_gb300 import build as qbuild
    qbuild.build()
    from sparse_selected_cell_gb300 import qsa
    return qsa.lib()


def paged(lib, **kw):
    a = dict(q=FAKE, q_type=0, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, pt=FAKE, pt_stride=4, n_lpages=4, n_ppages=16, n_kv=2,
             n_heads=8, lens=FAKE, n_seq=3, window=0, scale=0.1, out=ctypes.c_void_p(0x200000), out_type=2, lse=None, ws=FAKE,
             ws_bytes=lib.qsa_paged_attn_workspace_bytes(2, 8), status=None, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.qsa_paged_attn(*a.values())


@pytest.mark.parametrize("bad", [dict(n_seq=-1), dict(n_lpages=-1), dict(n_ppages=-1), dict(n_kv=0), dict(n_heads=0),
                                 dict(n_heads=7), dict(window=-1), dict(q_type=2), dict(q_type=-1), dict(out_type=3),
                                 dict(pt_stride=-1), dict(pt_stride=3), dict(q=None), dict(out=None), dict(lens=None),
                                 dict(ws=None), dict(pt=None), dict(k=None), dict(vs=None), dict(q=ODD), dict(out=ODD),
                                 dict(k=ODD), dict(vs=ODD), dict(ws=ODD), dict(out=FAKE)])
def test_paged_attn_arguments(lib, bad):
    assert paged(lib, **bad) == ARG


def test_paged_attn_limits(lib):
    assert paged(lib, n_seq=0, q=None, out=None, ws=None) == OK
    assert paged(lib, ws_bytes=lib.qsa_paged_attn_workspace_bytes(2, 8) - 1) == CAPACITY
    assert paged(lib, n_seq=1 << 20, n_lpages=1 << 10, pt_stride=1 << 10) == UNSUPPORTED     # more than 2^30 pages
    assert paged(lib, n_ppages=1 << 25) == UNSUPPORTED                                       # pool rows past 2^31
    assert paged(lib, n_kv=2, n_heads=1 << 20) == UNSUPPORTED
    assert lib.qsa_paged_attn_workspace_bytes(0, 8) == 0
    assert lib.qsa_paged_attn_workspace_bytes(3, 8) == 0


def append(lib, **kw):
    a = dict(q=FAKE, qs=1024, k=FAKE, ks=256, v=FAKE, vs=256, type=0, pos=FAKE, n_axes=1, pos_stride=5, inv=FAKE,
             axis=None, n_pairs=64, inter=0, qo=FAKE, qos=1024, kp=FAKE, vp=FAKE, ksc=FAKE, vsc=FAKE, slots=FAKE,
             n_ppages=4, n_heads=8, n_kv=2, n_tok=5, status=None, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.qsa_rope_append(*a.values())


@pytest.mark.parametrize("bad", [dict(n_tok=-1), dict(n_kv=0), dict(n_heads=-1), dict(n_heads=0), dict(type=2),
                                 dict(n_pairs=12), dict(n_pairs=72), dict(n_pairs=-8), dict(n_axes=0), dict(n_axes=5),
                                 dict(pos_stride=4), dict(pos=None), dict(inv=None), dict(qs=1020), dict(qs=512),
                                 dict(qos=512), dict(qo=None), dict(k=None), dict(v=None), dict(k=ODD), dict(ks=255),
                                 dict(vs=128), dict(slots=None), dict(kp=None), dict(vsc=ODD), dict(qos=1032)])
def test_rope_append_arguments(lib, bad):
    assert append(lib, **bad) == ARG


def test_rope_append_limits(lib):
    assert append(lib, n_tok=0) == OK
    assert append(lib, n_ppages=1 << 25) == UNSUPPORTED
    assert append(lib, n_heads=1 << 17, qs=1 << 24, qos=1 << 24) == UNSUPPORTED


def rope(lib, **kw):
    a = dict(x=FAKE, xs=1024, type=0, pos=FAKE, n_axes=1, pos_stride=5, inv=FAKE, axis=None, n_pairs=64, inter=0,
             out=FAKE, os=1024, n_heads=8, n_tok=5, status=None, stream=None)
    a.update(kw)
    return lib.qsa_rope(*a.values())


@pytest.mark.parametrize("bad", [dict(x=None), dict(out=None), dict(xs=1020), dict(os=1023), dict(os=2048),
                                 dict(n_heads=0), dict(type=5), dict(n_pairs=4), dict(n_tok=-1)])
def test_rope_arguments(lib, bad):
    assert rope(lib, **bad) == ARG
    assert rope(lib, n_tok=0) == OK


def gather(lib, **kw):
    a = dict(k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, slots=FAKE, n=5, n_ppages=4, n_kv=2, ko=FAKE, vo=FAKE, type=0, status=None,
             stream=None)
    a.update(kw)
    return lib.qsa_cache_gather(*a.values())


@pytest.mark.parametrize("bad", [dict(n=-1), dict(n_kv=0), dict(type=3), dict(slots=None), dict(ko=None), dict(vo=ODD),
                                 dict(k=None), dict(ks=ODD), dict(n_ppages=-1)])
def test_gather_arguments(lib, bad):
    assert gather(lib, **bad) == ARG
    assert gather(lib, n=0) == OK
    assert gather(lib, n_ppages=1 << 25) == UNSUPPORTED


def tables(lib, **kw):
    a = dict(sl=FAKE, nl=FAKE, n_seq=3, pt=FAKE, pt_stride=4, n_lpages=4, n_ppages=16, free=FAKE, n_free=8, head=None,
             n_tok=10, slots=FAKE, pos=FAKE, seq=FAKE, lens=ctypes.c_void_p(0x200000), cu=FAKE, ho=FAKE, status=None,
             stream=None)
    a.update(kw)
    return lib.qsa_extend_tables(*a.values())


@pytest.mark.parametrize("bad", [dict(n_seq=-1), dict(n_tok=-1), dict(n_free=-1), dict(n_lpages=5), dict(sl=None),
                                 dict(nl=None), dict(pt=None), dict(free=None), dict(slots=None), dict(slots=ODD),
                                 dict(pos=None), dict(seq=ODD), dict(lens=None), dict(lens=FAKE), dict(cu=None),
                                 dict(ho=None), dict(head=FAKE)])
def test_extend_tables_arguments(lib, bad):
    assert tables(lib, **bad) == ARG


def test_extend_tables_limits(lib):
    assert tables(lib, n_ppages=1 << 25) == UNSUPPORTED
    assert tables(lib, n_tok=(1 << 30) + 1) == UNSUPPORTED
    assert tables(lib, n_lpages=1 << 25, pt_stride=1 << 25) == UNSUPPORTED


def test_packed_calls_refuse_alike(lib):
    """The calls with their arguments in one struct: every field arrives where the call's own parameter is."""
    from sparse_selected_cell_gb300 import qsa

    class Packed:                                              # the library with the packed calls behind the plain names
        qsa_paged_attn_workspace_bytes = staticmethod(lib.qsa_paged_attn_workspace_bytes)

    def through(name, pack):
        def call(*args):
            return getattr(lib, name)(pack(*[0 if x is None else getattr(x, "value", x) for x in args]))
        return call

    Packed.qsa_paged_attn = staticmethod(through("qsa_paged_attn_packed", qsa._PAGED_ARGS))
    Packed.qsa_rope_append = staticmethod(through("qsa_rope_append_packed", qsa._APPEND_ARGS))
    Packed.qsa_cache_gather = staticmethod(through("qsa_cache_gather_packed", qsa._GATHER_ARGS))
    Packed.qsa_extend_tables = staticmethod(through("qsa_extend_tables_packed", qsa._TABLES_ARGS))
    for test in (test_paged_attn_arguments, test_rope_append_arguments, test_gather_arguments, test_extend_tables_arguments):
        for bad in test.pytestmark[0].args[1]:
            test(Packed, bad)
    for test in (test_paged_attn_limits, test_rope_append_limits, test_extend_tables_limits):
        test(Packed)
    for name in ("qsa_paged_attn_packed", "qsa_rope_append_packed", "qsa_cache_gather_packed", "qsa_extend_tables_packed"):
        assert getattr(lib, name)(None) == ARG
