"""The entry points of routing by expert without a GPU: their argument checks
answer before any CUDA call is made (the handle is a fake pointer, never read:
every call here is refused, or is empty)."""
import pytest

import fp32_sgemm_gb300 as sg
from fp32_sgemm_gb300 import _binding

S = _binding.Status
F = 0x10000                     # a fake, aligned "device" address
F32, F16, BF16 = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    sg.build()
    return sg.load_library()


def route(lib, ty=BF16, T=4, E=8, k=2, logits=F, ldl=8, weights=F, experts=F, h=F):
    return lib.sgemmRouteTopK(h, ty, T, E, k, 1, logits, ldl, weights, experts, None)


def route_grad(lib, ty=BF16, T=4, E=8, k=2, logits=F, ldl=8, weights=F, experts=F, d=F, ldd=8, h=F):
    return lib.sgemmRouteTopKGrad(h, ty, T, E, k, 1, logits, ldl, experts, weights, d, ldd, None)


@pytest.mark.parametrize("call", [route, route_grad])
def test_route(lib, call):
    for bad in (dict(ty=3), dict(T=-1), dict(E=0), dict(k=0), dict(k=9), dict(ldl=7), dict(logits=None),
                dict(weights=None), dict(experts=None), dict(h=None)):
        assert call(lib, **bad) == S.INVALID_VALUE, bad
    for bad in (dict(logits=F + 1), dict(weights=F + 2), dict(experts=F + 4)):
        assert call(lib, **bad) == S.MISALIGNED, bad
    for bad in (dict(E=1025, ldl=1025), dict(E=64, ldl=64, k=33), dict(T=2 ** 30)):
        assert call(lib, **bad) == S.NOT_SUPPORTED, bad
    assert call(lib, T=0, logits=None, weights=None, experts=None) == S.SUCCESS


def test_route_grad_output(lib):
    assert route_grad(lib, d=None) == S.INVALID_VALUE
    assert route_grad(lib, ldd=7) == S.INVALID_VALUE
    assert route_grad(lib, d=F + 1) == S.MISALIGNED


def dispatch(lib, ty=BF16, T=4, D=8, k=2, G=3, X=F, ldx=8, experts=F, rows=F, ldr=8, slots=F, ends=F, h=F):
    return lib.sgemmExpertDispatch(h, ty, T, D, k, G, X, ldx, experts, rows, ldr, slots, ends, None)


def test_dispatch(lib):
    for bad in (dict(ty=-1), dict(T=-1), dict(D=-1), dict(k=-1), dict(G=-1), dict(ldx=7), dict(ldr=7), dict(X=None),
                dict(experts=None), dict(rows=None), dict(slots=None), dict(ends=None), dict(h=None)):
        assert dispatch(lib, **bad) == S.INVALID_VALUE, bad
    for bad in (dict(X=F + 1), dict(ty=F32, rows=F + 2), dict(experts=F + 4), dict(slots=F + 2), dict(ends=F + 1)):
        assert dispatch(lib, **bad) == S.MISALIGNED, bad
    for bad in (dict(G=1025), dict(T=2 ** 30), dict(D=2 ** 31, ldx=2 ** 31, ldr=2 ** 31), dict(T=2 ** 40, k=2 ** 40)):
        assert dispatch(lib, **bad) == S.NOT_SUPPORTED, bad
    assert dispatch(lib, T=0, G=0, X=None, experts=None, rows=None, slots=None, ends=None, h=None) == S.SUCCESS


def combine(lib, ty=BF16, T=4, D=8, k=2, rows=F, ldr=8, slots=F, weights=F, Y=F, ldy=8, h=F):
    return lib.sgemmExpertCombine(h, ty, T, D, k, rows, ldr, slots, weights, Y, ldy, None)


def combine_grad(lib, ty=BF16, T=4, D=8, k=2, dy=F, lddy=8, rows=F, ldr=8, slots=F, weights=F, drows=F, lddr=8, dw=F,
                 h=F):
    return lib.sgemmExpertCombineGrad(h, ty, T, D, k, dy, lddy, rows, ldr, slots, weights, drows, lddr, dw, None)


def test_combine(lib):
    for bad in (dict(ty=4), dict(T=-1), dict(D=-1), dict(k=-1), dict(rows=None), dict(ldr=7), dict(slots=None),
                dict(h=None)):
        assert combine(lib, **bad) == S.INVALID_VALUE, bad
        assert combine_grad(lib, **bad) == S.INVALID_VALUE, bad
    for bad in (dict(rows=F + 1), dict(slots=F + 2), dict(weights=F + 2)):
        assert combine(lib, **bad) == S.MISALIGNED, bad
        assert combine_grad(lib, **bad) == S.MISALIGNED, bad
    assert combine(lib, Y=None) == S.INVALID_VALUE
    assert combine(lib, ldy=7) == S.INVALID_VALUE
    assert combine_grad(lib, dy=None) == S.INVALID_VALUE
    assert combine_grad(lib, lddr=7) == S.INVALID_VALUE
    assert combine_grad(lib, dw=F + 1) == S.MISALIGNED
    assert combine(lib, T=2 ** 30) == S.NOT_SUPPORTED
    assert combine(lib, T=0, rows=None, slots=None, weights=None, Y=None, h=None) == S.SUCCESS
    # Nothing asked for.
    assert combine_grad(lib, drows=None, dw=None, rows=None, h=None) == S.SUCCESS


S8 = 3


def quantize(lib, ty=BF16, T=4, K=32, X=F, ldx=32, Q=F, ldq=32, scales=F, h=F):
    return lib.sgemmInt8Quantize(h, ty, T, K, X, ldx, Q, ldq, scales, None)


def int8(lib, tx=BF16, tc=BF16, T=4, N=16, K=32, G=1, X=F, ldx=32, xs=None, B=F, ldb=32, sb=16 * 32, scales=F, ends=None,
         C=F, ldc=16, h=F):
    return lib.sgemmInt8(h, tx, tc, T, N, K, G, X, ldx, xs, B, ldb, sb, scales, ends, C, ldc, None)


def test_quantize(lib):
    for bad in (dict(ty=S8), dict(T=-1), dict(K=-1), dict(X=None), dict(ldx=31), dict(Q=None), dict(ldq=31),
                dict(scales=None), dict(h=None)):
        assert quantize(lib, **bad) == S.INVALID_VALUE, bad
    assert quantize(lib, X=F + 1) == S.MISALIGNED
    assert quantize(lib, scales=F + 2) == S.MISALIGNED
    assert quantize(lib, K=2 ** 31, ldx=2 ** 31, ldq=2 ** 31) == S.NOT_SUPPORTED
    assert quantize(lib, T=0, X=None, Q=None, scales=None, h=None) == S.SUCCESS


def test_int8(lib):
    for bad in (dict(tx=4), dict(tc=S8), dict(tc=-1), dict(T=-1), dict(N=-1), dict(K=-1), dict(G=-1), dict(X=None),
                dict(ldx=31), dict(B=None), dict(ldb=31), dict(scales=None), dict(C=None), dict(ldc=15), dict(h=None),
                dict(xs=F), dict(tx=S8), dict(G=2), dict(G=2, ends=F, sb=511), dict(sb=-1)):
        assert int8(lib, **bad) == S.INVALID_VALUE, bad
    for bad in (dict(X=F + 1), dict(scales=F + 2), dict(C=F + 1), dict(ends=F + 2), dict(tx=S8, xs=F + 1)):
        assert int8(lib, **bad) == S.MISALIGNED, bad
    for bad in (dict(K=131072, ldx=131072, ldb=131072, sb=16 * 131072), dict(G=1025, ends=F), dict(T=2 ** 31),
                dict(N=2 ** 31, ldc=2 ** 31)):
        assert int8(lib, **bad) == S.NOT_SUPPORTED, bad
    assert int8(lib, T=0, X=None, B=None, scales=None, C=None, h=None) == S.SUCCESS
    assert int8(lib, N=0, ldc=1, X=None, B=None, scales=None, C=None, h=None) == S.SUCCESS


def test_int8_workspace(lib):
    import ctypes
    n = ctypes.c_size_t(7)
    ask = lib.sgemmInt8WorkspaceSize
    assert ask(F, BF16, BF16, 0, 16, 32, 1, None, 32, None, 32, 512, ctypes.byref(n)) == S.SUCCESS and n.value == 0
    assert ask(None, BF16, BF16, 4, 16, 32, 1, F, 32, F, 32, 512, ctypes.byref(n)) == S.INVALID_VALUE
    assert ask(F, BF16, 7, 4, 16, 32, 1, F, 32, F, 32, 512, ctypes.byref(n)) == S.INVALID_VALUE
    assert ask(F, BF16, BF16, 4, 16, 32, 1, F, 32, F, 32, 512, None) == S.INVALID_VALUE
