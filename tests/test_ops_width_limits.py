"""Widths within 1024 of 2^31, where counts of tiles and columns would pass 32 bits, are refused before the device is touched (CPU
only: the addresses are made up and never read)."""
import pytest

from tests.test_ops_refusals import _back, _egrad, _emb, _linear

TOP = 2 ** 31 - 16
LD = 2 ** 31


@pytest.mark.parametrize("kw", [dict(d_in=TOP, ld_x=LD), dict(d_out=TOP, ld_y=LD, ld_res=LD, ld_z=LD),
                                dict(d_in=TOP - 992, ld_x=LD)])
def test_linear(kw):
    q = [0x1000 * (i + 1) for i in range(6)]
    assert _linear(x=q[0], W=q[1], bias=q[2], res=q[3], y=q[4], zz=q[5], **kw) == 2


@pytest.mark.parametrize("kw", [dict(d_in=TOP, ld_x=LD, ld_dx=LD), dict(d_out=TOP, ld_dy=LD, ld_z=LD)])
def test_linear_backward(kw):
    assert _back(**kw) == 2


@pytest.mark.parametrize("d", [2 ** 31 - 1, 2 ** 31 - 1023])
def test_embedding(d):
    q = [0x1000 * (i + 1) for i in range(3)]
    assert _emb(ids=q[0], E=q[1], out=q[2], d=d, ld=LD, ld_out=LD) == 2
    assert _egrad(ids=q[0], g=q[1], G=q[2], d=d, ld=LD, ld_G=LD) == 2
