"""Frequency helper: arguments whose frequencies would not be numbers are refused (no GPU)."""
import math

import pytest

import bit_linear_moe_b200 as nv

INF, NAN = math.inf, math.nan
YARN = dict(rot_dim=64, scaling=nv.ROPE_SCALE_YARN, factor=2.0, original_len=4096.0)
NTK = dict(scaling=nv.ROPE_SCALE_NTK)


@pytest.fixture(scope="module", autouse=True)
def library():
    from bit_linear_moe_b200 import build
    build.build()


@pytest.mark.parametrize("kw", [
    dict(NTK, rot_dim=4, factor=1e200),                          # factor^2: an infinite base
    dict(NTK, rot_dim=128, theta=1e308, factor=100.0),
    dict(YARN, beta_slow=-INF), dict(YARN, beta_fast=INF), dict(YARN, beta_slow=NAN), dict(YARN, beta_fast=NAN),
    dict(YARN, original_len=INF), dict(YARN, original_len=NAN),
    dict(YARN, beta_fast=1e308, beta_slow=-1e308),               # their difference overflows
    dict(rot_dim=1024, theta=5e-324),                            # the fastest pairs would turn infinitely fast
    dict(rot_dim=64, theta=2.0 ** -1070, scaling=nv.ROPE_SCALE_LINEAR, factor=2.0),
])
def test_refused(kw):
    with pytest.raises(nv.NVFP4Error) as e:
        nv.nvfp4_rope_freqs(**kw)
    assert e.value.status == nv.ERR_SHAPE


@pytest.mark.parametrize("kw", [
    dict(NTK, rot_dim=128, theta=1e6, factor=1e6), dict(rot_dim=64, theta=1e-3), dict(rot_dim=64, theta=1e300),
    dict(YARN, beta_fast=1e300, beta_slow=0.0), dict(YARN, beta_slow=-5.0), dict(YARN, original_len=1e12),
    dict(YARN, factor=1e300), dict(YARN, original_len=1e308, theta=1e-6),
    dict(rot_dim=32, factor=INF, original_len=NAN, beta_fast=NAN, beta_slow=INF)])   # none of these is used
def test_finite(kw):
    f, m = nv.nvfp4_rope_freqs(**kw)
    assert f.isfinite().all() and (f >= 0).all() and math.isfinite(m) and f[0] <= 1 / (2 * math.pi)
