"""Calls of the layers with a state that are too large for one launch are refused as such, on the host."""
import pytest

from test_linear_abi import UNSUPPORTED, at, conv, lib, norm  # noqa: F401


def far(n):
    """Arrays that cannot meet, whatever n bytes they span."""
    return at(1 << 20), at((1 << 21) + 16 * n)


@pytest.mark.parametrize("n_ch,n_tok", [(1 << 20, 1 << 30), (1 << 23, 1 << 24), (65537 * 8, 1 << 30)])
def test_convolution(lib, n_ch, n_tok):  # noqa: F811
    x, out = far(n_tok * n_ch)
    assert conv(lib, x=x, xs=n_ch, out=out, os=n_ch, n_ch=n_ch, n_tok=n_tok) == UNSUPPORTED


@pytest.mark.parametrize("n_groups,size,n_tok", [(1 << 16, 256, 1 << 30), (1 << 16, 1024, 1 << 24), (1 << 16, 1032, 1 << 16)])
def test_norm(lib, n_groups, size, n_tok):  # noqa: F811
    row = n_groups * size
    x, out = far(n_tok * row)
    assert norm(lib, x=x, xs=row, gate=None, out=out, os=row, n_groups=n_groups, size=size, n_tok=n_tok) == UNSUPPORTED
