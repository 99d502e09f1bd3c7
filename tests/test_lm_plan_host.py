"""Plan queries of the grouped products without a GPU: their checks answer as
the calls' do, and an empty product has no kernel."""
import ctypes

import pytest

import fp32_sgemm_gb300 as sg
from fp32_sgemm_gb300 import _binding

S = _binding.Status
F = 0x10000                     # a fake, aligned "device" address, never read
F32, BF16 = 0, 2


@pytest.fixture(scope="module")
def lib():
    sg.build()
    return sg.load_library()


def product(lib, ty=BF16, op=0, T=8, N=16, K=32, G=2, A=F, lda=32, B=F, ldb=16, sb=512, h=F, plan=True):
    p = _binding.GroupedPlan(kernel=9)
    st = lib.sgemmGroupedQueryPlan(h, ty, op, T, N, K, G, A, lda, B, ldb, sb, ctypes.byref(p) if plan else None)
    return st, p.as_dict()


def gradient(lib, ty=BF16, T=8, M=16, N=32, G=2, A=F, lda=16, B=F, ldb=32, h=F, plan=True):
    p = _binding.GroupedPlan(kernel=9)
    st = lib.sgemmGroupedWeightGradQueryPlan(h, ty, T, M, N, G, A, lda, B, ldb, ctypes.byref(p) if plan else None)
    return st, p.as_dict()


def test_refusals(lib):
    for args in (dict(plan=False), dict(ty=3), dict(op=2), dict(T=-1), dict(lda=31), dict(ldb=15), dict(sb=511),
                 dict(A=None), dict(h=None)):
        assert product(lib, **args)[0] == S.INVALID_VALUE, args
    for args in (dict(plan=False), dict(ty=3), dict(T=-1), dict(lda=15), dict(ldb=31), dict(B=None), dict(h=None)):
        assert gradient(lib, **args)[0] == S.INVALID_VALUE, args
    assert product(lib, G=1025)[0] == gradient(lib, G=1025)[0] == S.NOT_SUPPORTED
    assert product(lib, A=F + 1)[0] == gradient(lib, A=F + 1)[0] == S.MISALIGNED


def test_empty_products_have_no_kernel(lib):
    for st, p in (product(lib, T=0), product(lib, K=0, lda=1), gradient(lib, T=0), gradient(lib, M=0, lda=1)):
        assert st == S.SUCCESS and not any(p.values())
