"""The gradients of bringing rows back, with scratch for the rows that no slot names,
without a GPU: argument checks (the handle is a fake pointer, never read)."""
import pytest

import fp32_sgemm_gb300 as sg
from fp32_sgemm_gb300 import _binding

S = _binding.Status
F = 0x10000


@pytest.fixture(scope="module")
def lib():
    sg.build()
    return sg.load_library()


def grad(lib, ty=2, T=4, D=8, k=2, dy=F, lddy=8, rows=F, ldr=8, slots=F, weights=F, drows=F, lddr=8, dw=F, owners=F, h=F):
    return lib.sgemmExpertCombineGradEx(h, ty, T, D, k, dy, lddy, rows, ldr, slots, weights, drows, lddr, dw, owners, None)


def test_refusals(lib):
    for bad in (dict(ty=4), dict(T=-1), dict(D=-1), dict(k=-1), dict(dy=None), dict(rows=None), dict(slots=None),
                dict(lddy=7), dict(ldr=7), dict(lddr=7), dict(h=None), dict(h=None, owners=None)):
        assert grad(lib, **bad) == S.INVALID_VALUE, bad
    for bad in (dict(dy=F + 1), dict(slots=F + 2), dict(weights=F + 2), dict(dw=F + 1), dict(owners=F + 2)):
        assert grad(lib, **bad) == S.MISALIGNED, bad
    assert grad(lib, T=2 ** 30) == S.NOT_SUPPORTED
    assert grad(lib, drows=None, dw=None, rows=None, owners=None, h=None) == S.SUCCESS
    assert grad(lib, T=0, dy=None, rows=None, slots=None, drows=None, dw=None, owners=None, h=None) == S.SUCCESS


def test_a_gradient_that_is_not_wanted_needs_no_pitch(lib):
    assert grad(lib, drows=None, lddr=0, dw=None, rows=None, ldr=0, h=None) == S.SUCCESS
    assert grad(lib, T=0, drows=None, lddr=0, dw=None, rows=None, ldr=0, h=None) == S.SUCCESS
    # The one that is wanted has to have its own.
    for bad in (dict(drows=None, lddr=0, ldr=7), dict(dw=None, rows=None, ldr=0, lddr=7), dict(drows=None, lddr=0, rows=None),
                dict(rows=None, ldr=0)):
        assert grad(lib, **bad) == S.INVALID_VALUE, bad
