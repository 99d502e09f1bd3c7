"""The language-model entry points without a GPU: their argument checks answer
before any CUDA call is made (the handle is a fake pointer, never read: every
call here is refused, or is empty)."""
import ctypes

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


def grouped(lib, ty=BF16, op=0, T=8, N=16, K=32, G=2, A=F, lda=None, B=F, ldb=None, sb=None, ends=F, C=F, ldc=None,
            h=F):
    ldb = (K if op else N) if ldb is None else ldb
    sb = N * K if sb is None else sb
    return lib.sgemmGrouped(h, ty, op, T, N, K, G, A, K if lda is None else lda, B, ldb, sb, ends, C,
                            N if ldc is None else ldc, None)


@pytest.mark.parametrize("args", [
    dict(ty=3), dict(ty=-1), dict(op=2), dict(T=-1), dict(N=-1), dict(K=-1), dict(G=-1), dict(lda=31), dict(ldb=15),
    dict(op=1, ldb=31), dict(ldc=15), dict(sb=16 * 32 - 1), dict(sb=-1), dict(A=None), dict(B=None), dict(C=None),
    dict(ends=None), dict(h=None),
])
def test_grouped_invalid(lib, args):
    assert grouped(lib, **args) == S.INVALID_VALUE


@pytest.mark.parametrize("args", [dict(A=F + 1), dict(B=F + 1), dict(C=F + 1), dict(ends=F + 2),
                                  dict(ty=F32, A=F + 2), dict(ty=F32, C=F + 2)])
def test_grouped_misaligned(lib, args):
    assert grouped(lib, **args) == S.MISALIGNED


@pytest.mark.parametrize("args", [dict(G=1025), dict(T=2 ** 31), dict(N=2 ** 31), dict(K=2 ** 31),
                                  dict(sb=2 ** 39)])
def test_grouped_not_supported(lib, args):
    assert grouped(lib, **args) == S.NOT_SUPPORTED


def test_grouped_empty_is_a_no_op(lib):
    assert grouped(lib, T=0, A=None, C=None, ends=None) == S.SUCCESS
    assert grouped(lib, N=0, B=None, C=None, ends=None, ldb=1, ldc=1) == S.SUCCESS


def weight_grad(lib, ty=BF16, T=8, M=16, N=32, G=2, A=F, lda=None, B=F, ldb=None, ends=F, C=F, ldc=None, sc=None,
                h=F):
    return lib.sgemmGroupedWeightGrad(h, ty, T, M, N, G, A, max(M, 1) if lda is None else lda, B,
                                      max(N, 1) if ldb is None else ldb, ends, C, max(N, 1) if ldc is None else ldc,
                                      M * N if sc is None else sc, None)


@pytest.mark.parametrize("args", [
    dict(ty=7), dict(T=-1), dict(M=-1), dict(N=-1), dict(G=-1), dict(lda=15), dict(ldb=31), dict(ldc=31),
    dict(sc=511), dict(sc=-1), dict(A=None), dict(B=None), dict(C=None), dict(ends=None), dict(h=None),
])
def test_weight_grad_invalid(lib, args):
    assert weight_grad(lib, **args) == S.INVALID_VALUE


def test_weight_grad_other_refusals(lib):
    assert weight_grad(lib, A=F + 1) == S.MISALIGNED
    assert weight_grad(lib, ends=F + 1) == S.MISALIGNED
    assert weight_grad(lib, G=1025) == S.NOT_SUPPORTED
    assert weight_grad(lib, M=0, C=None) == S.SUCCESS
    assert weight_grad(lib, G=0, C=None, ends=None) == S.SUCCESS


def loss(lib, ty=BF16, T=4, V=10, D=8, X=F, ldx=8, W=F, ldw=8, target=F, out=F, lse=F, h=F):
    return lib.sgemmCrossEntropy(h, ty, T, V, D, X, ldx, W, ldw, target, out, lse, None)


def loss_grad(lib, ty=BF16, T=4, V=10, D=8, X=F, ldx=8, W=F, ldw=8, target=F, lse=F, dloss=F, dX=F, lddx=8, dW=F,
              lddw=8, h=F):
    return lib.sgemmCrossEntropyGrad(h, ty, T, V, D, X, ldx, W, ldw, target, lse, dloss, dX, lddx, dW, lddw, None)


@pytest.mark.parametrize("args", [
    dict(ty=5), dict(T=-1), dict(V=0), dict(D=0), dict(ldx=7), dict(ldw=7), dict(X=None), dict(W=None),
    dict(target=None), dict(lse=None), dict(h=None),
])
def test_loss_invalid(lib, args):
    assert loss(lib, **args) == S.INVALID_VALUE
    assert loss_grad(lib, **args) == S.INVALID_VALUE


def test_loss_other_refusals(lib):
    assert loss(lib, out=None) == S.INVALID_VALUE
    assert loss(lib, target=F + 4) == S.MISALIGNED
    assert loss(lib, out=F + 2) == S.MISALIGNED
    assert loss(lib, T=0, X=None, W=None, target=None, out=None, lse=None) == S.SUCCESS
    assert loss(lib, V=2 ** 31, ldw=8) == S.NOT_SUPPORTED
    assert loss_grad(lib, dloss=None) == S.INVALID_VALUE
    assert loss_grad(lib, dX=None) == S.INVALID_VALUE
    assert loss_grad(lib, dW=None) == S.INVALID_VALUE
    assert loss_grad(lib, lddx=7) == S.INVALID_VALUE
    assert loss_grad(lib, lddw=7) == S.INVALID_VALUE
    assert loss_grad(lib, dW=F + 1) == S.MISALIGNED


def w4(lib, ty=BF16, M=2, N=16, K=128, group=32, X=F, ldx=128, Q=F, ldq=64, scales=F, lds=4, zeros=F, ldz=4, Y=F,
       ldy=16, h=F):
    return lib.sgemmW4(h, ty, M, N, K, group, X, ldx, Q, ldq, scales, lds, zeros, ldz, Y, ldy, None)


@pytest.mark.parametrize("args", [
    dict(ty=9), dict(M=-1), dict(N=-1), dict(K=-128), dict(group=16), dict(group=96), dict(group=0),
    dict(K=100, ldx=128), dict(group=128, K=192, ldx=192, ldq=96), dict(ldx=127), dict(ldq=63), dict(lds=3),
    dict(ldz=3), dict(ldy=15), dict(X=None), dict(Q=None), dict(scales=None), dict(Y=None), dict(h=None),
])
def test_w4_invalid(lib, args):
    assert w4(lib, **args) == S.INVALID_VALUE


def test_w4_other_refusals(lib):
    assert w4(lib, Q=F + 8) == S.MISALIGNED
    assert w4(lib, ldq=72) == S.MISALIGNED
    assert w4(lib, X=F + 1) == S.MISALIGNED
    assert w4(lib, scales=F + 1) == S.MISALIGNED
    assert w4(lib, N=2 ** 31) == S.NOT_SUPPORTED
    assert w4(lib, M=0, X=None, Y=None) == S.SUCCESS
    assert w4(lib, N=0, Q=None, scales=None, Y=None, ldy=1) == S.SUCCESS


def test_size_queries_need_a_place_for_the_answer(lib):
    assert lib.sgemmGroupedWorkspaceSize(F, BF16, 0, 8, 16, 32, 2, F, 32, F, 16, 512, None) == S.INVALID_VALUE
    assert lib.sgemmCrossEntropyWorkspaceSize(F, BF16, 4, 10, 8, F, 8, F, 8, None) == S.INVALID_VALUE
    assert lib.sgemmW4WorkspaceSize(F, BF16, 1, 16, 128, 32, None) == S.INVALID_VALUE


def test_grouped_workspace(lib):
    # 16-bit operands TMA can address need none; an odd pitch is copied to a
    # multiple of 8 elements; FP32 is held as three 16-bit planes.
    n = ctypes.c_size_t()

    def need(ty, lda, ldb, sb, A=F):
        assert lib.sgemmGroupedWorkspaceSize(F, ty, 0, 8, 16, 32, 2, A, lda, F, ldb, sb, ctypes.byref(n)) == S.SUCCESS
        return n.value
    assert need(BF16, 32, 16, 512) == 0
    assert need(BF16, 33, 16, 512) == 8 * 32 * 2
    assert need(BF16, 32, 16, 512, A=F + 2) == 8 * 32 * 2
    assert need(BF16, 32, 17, 17 * 32) == 2 * 32 * 16 * 2
    assert need(F32, 32, 16, 512) == 3 * (8 * 32 + 2 * 32 * 16) * 2


def test_python_refuses_cpu_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        sg.grouped_gemm(x, torch.zeros(2, 8, 8, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        sg.linear_cross_entropy(x, x, torch.zeros(4, dtype=torch.int64))
    with pytest.raises(TypeError):
        sg.w4_gemm("x", x, x)
