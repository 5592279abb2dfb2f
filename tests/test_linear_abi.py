"""The C entries of the layers with a state refuse bad arguments on the host, before anything reaches a GPU."""
import ctypes

import pytest

OK, ARG, UNSUPPORTED, CAPACITY = 0, 1, 2, 3
NAN, INF = float("nan"), float("inf")


def at(address):
    return ctypes.c_void_p(address)


@pytest.fixture(scope="module")
def lib():
    from sparse_selected_cell_gb300 import build as qbuild
    qbuild.build()
    from sparse_selected_cell_gb300 import qsa
    return qsa.lib()


def conv(lib, **kw):
    a = dict(x=at(0x100000), xs=64, type=0, w=at(0x200000), bias=at(0x210000), wt=0, width=4, act=1, state=at(0x300000),
             slots=at(0x400000), n_slots=3, old=at(0x410000), cu=at(0x420000), n_seq=3, n_tok=10, n_ch=64, out=at(0x500000),
             os=64, status=None, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.qsa_short_conv(*a.values())


@pytest.mark.parametrize("bad", [dict(n_seq=-1), dict(n_tok=-1), dict(n_slots=-1), dict(n_ch=0), dict(n_ch=60), dict(width=1),
                                 dict(width=5), dict(type=2), dict(type=-1), dict(wt=1), dict(wt=3), dict(act=2), dict(act=-1),
                                 dict(x=None), dict(x=at(0x100008)), dict(xs=56), dict(xs=65), dict(w=None),
                                 dict(w=at(0x200008)), dict(bias=at(0x210004)), dict(state=None), dict(state=at(0x300008)),
                                 dict(slots=None), dict(out=None), dict(out=at(0x500002)), dict(os=63), dict(os=56),
                                 dict(cu=None), dict(out=at(0x100000)), dict(out=at(0x100000 + 9 * 128)),
                                 dict(out=at(0x100000 - 9 * 128)), dict(out=at(0x100000 + 64), xs=128, os=128),
                                 dict(out=at(0x100000 + 128), xs=136, os=128)])
def test_conv_arguments(lib, bad):
    assert conv(lib, **bad) == ARG


def test_conv_limits(lib):
    assert conv(lib, n_seq=0, slots=None, state=None) == OK
    assert conv(lib, n_tok=(1 << 30) + 1) == UNSUPPORTED
    assert conv(lib, n_ch=(1 << 23) + 8, xs=1 << 24, os=1 << 24) == UNSUPPORTED


def prompt(lib, **kw):
    a = dict(q=at(0x1000000), qs=1024, k=at(0x1000200), ks=1024, v=at(0x1000400), vs=1024, type=0, a=at(0x2000000), as_=8,
             b=at(0x2000008), bs=8, a_log=at(0x3000000), dt=at(0x3000100), state=at(0x4000000), slots=at(0x5000000), n_slots=3,
             old=at(0x5000100), cu=at(0x5000200), n_seq=3, n_tok=10, n_k=2, n_v=4, eps=1e-6, scale=0.1, out=at(0x6000000),
             os=512, ws=at(0x7000000), ws_bytes=lib.qsa_delta_prompt_workspace_bytes(10, 3, 2, 4), status=None, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.qsa_delta_prompt(*a.values())


HEADS = [dict(n_seq=-1), dict(n_slots=-1), dict(n_k=0), dict(n_v=0), dict(n_k=3), dict(type=2), dict(eps=-1.0), dict(eps=NAN),
         dict(eps=INF), dict(scale=NAN), dict(scale=INF), dict(slots=None), dict(a_log=None), dict(dt=None), dict(state=None),
         dict(state=at(0x4000008)), dict(q=None), dict(k=None), dict(v=None), dict(a=None), dict(b=None), dict(a=at(0x2000001)),
         dict(out=None), dict(q=at(0x1000008)), dict(v=at(0x1000408)), dict(qs=1028), dict(ks=248), dict(vs=504), dict(as_=3),
         dict(bs=3), dict(os=504), dict(out=at(0x6000008)), dict(out=at(0x1000400), os=1024), dict(out=at(0x1000000), os=1024),
         dict(out=at(0x1000000 + 640), os=1024), dict(out=at(0x2000000))]


@pytest.mark.parametrize("bad", HEADS + [dict(n_tok=-1), dict(cu=None), dict(ws=None), dict(ws=at(0x7000080))])
def test_prompt_arguments(lib, bad):
    assert prompt(lib, **bad) == ARG


def test_prompt_limits(lib):
    assert prompt(lib, n_seq=0, slots=None, ws=None, cu=None) == OK
    assert prompt(lib, ws_bytes=lib.qsa_delta_prompt_workspace_bytes(10, 3, 2, 4) - 1) == CAPACITY
    assert prompt(lib, n_tok=(1 << 30) + 1) == UNSUPPORTED
    assert prompt(lib, n_k=1 << 17, n_v=1 << 17) == UNSUPPORTED
    for bad in ((-1, 1, 1, 1), (1, -1, 1, 1), (1, 1, 0, 1), (1, 1, 2, 3), (1, 1, 1, 0)):
        assert lib.qsa_delta_prompt_workspace_bytes(*bad) == 0
    assert lib.qsa_delta_prompt_workspace_bytes(0, 0, 1, 1) > 0


def step(lib, **kw):
    a = dict(q=at(0x1000000), qs=1024, k=at(0x1000200), ks=1024, v=at(0x1000400), vs=1024, type=0, a=at(0x2000000), as_=8,
             b=at(0x2000008), bs=8, a_log=at(0x3000000), dt=at(0x3000100), state=at(0x4000000), slots=at(0x5000000), n_slots=3,
             old=at(0x5000100), n_seq=3, n_k=2, n_v=4, eps=1e-6, scale=0.1, out=at(0x6000000), os=512, status=None, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.qsa_delta_step(*a.values())


@pytest.mark.parametrize("bad", HEADS)
def test_step_arguments(lib, bad):
    assert step(lib, **bad) == ARG


def test_step_limits(lib):
    assert step(lib, n_seq=0, q=None, state=None) == OK
    assert step(lib, n_seq=1 << 30) == UNSUPPORTED
    assert step(lib, n_k=1 << 17, n_v=1 << 17) == UNSUPPORTED


def norm(lib, **kw):
    a = dict(x=at(0x1000000), xs=512, gate=at(0x2000000), gs=512, type=0, w=at(0x3000000), bias=at(0x3100000), wt=0, per_group=0,
             n_tok=10, n_groups=4, size=128, eps=1e-6, centred=0, act=1, out=at(0x4000000), os=512, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.qsa_group_norm(*a.values())


@pytest.mark.parametrize("bad", [dict(n_tok=-1), dict(n_groups=0), dict(size=0), dict(size=12), dict(type=2), dict(wt=1),
                                 dict(act=2), dict(eps=-1.0), dict(eps=NAN), dict(eps=INF), dict(x=None), dict(out=None),
                                 dict(xs=504), dict(xs=516), dict(gs=504), dict(os=508), dict(x=at(0x1000008)),
                                 dict(gate=at(0x2000004)), dict(w=at(0x3000008)), dict(bias=at(0x3100008)),
                                 dict(out=at(0x1000000), os=520), dict(out=at(0x2000000), os=520), dict(out=at(0x1000010)),
                                 dict(out=at(0x2000000 + 9 * 1024))])
def test_norm_arguments(lib, bad):
    assert norm(lib, **bad) == ARG


def test_norm_limits(lib):
    assert norm(lib, n_tok=0, x=None, out=None) == OK
    assert norm(lib, size=8200, xs=1 << 16, gs=1 << 16, os=1 << 16) == UNSUPPORTED
    assert norm(lib, n_groups=(1 << 16) + 1, size=8, xs=1 << 20, gs=1 << 20, os=1 << 20) == UNSUPPORTED


def test_packed_calls_refuse_alike(lib):
    """The calls with their arguments in one struct: every field arrives where the call's own parameter is."""
    from sparse_selected_cell_gb300 import qsa

    class Packed:                                              # the library with the packed calls behind the plain names
        qsa_delta_prompt_workspace_bytes = staticmethod(lib.qsa_delta_prompt_workspace_bytes)

    def through(name, pack):
        def call(*args):
            return getattr(lib, name)(pack(*[0 if x is None else getattr(x, "value", x) for x in args]))
        return call

    Packed.qsa_short_conv = staticmethod(through("qsa_short_conv_packed", qsa._CONV_ARGS))
    Packed.qsa_delta_prompt = staticmethod(through("qsa_delta_prompt_packed", qsa._PROMPT_ARGS))
    Packed.qsa_delta_step = staticmethod(through("qsa_delta_step_packed", qsa._STEP_ARGS))
    Packed.qsa_group_norm = staticmethod(through("qsa_group_norm_packed", qsa._NORM_ARGS))
    for test in (test_conv_arguments, test_prompt_arguments, test_step_arguments, test_norm_arguments):
        for bad in test.pytestmark[0].args[1]:
            test(Packed, bad)
    for test in (test_conv_limits, test_prompt_limits, test_step_limits, test_norm_limits):
        test(Packed)
    for name in ("qsa_short_conv_packed", "qsa_delta_prompt_packed", "qsa_delta_step_packed", "qsa_group_norm_packed"):
        assert getattr(lib, name)(None) == ARG
