"""Every tile of the grouped products and their weight gradients against a
64-bit reference, on calls of which the plan query says that they take it; the
same for the bounded waits of the tiles of a pair and of the loss gradients.

Bounds as in test_gpu_grouped.py: one rounding to the type, and for the sum
K / 16 truncating steps of 2^-23 of sum |a b| (FP32: 2^-20).
"""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
TYPES = {"f32": 0, "f16": 1, "bf16": 2}


@pytest.fixture(scope="module")
def sg():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import fp32_sgemm_gb300 as m
    m.build()
    m.load_library()
    return m


def _sizes(T, G, seed):
    """G ragged sizes of T rows together, one group in five empty."""
    r = np.random.RandomState(seed)
    p = np.exp(0.5 * r.standard_normal(G))
    p[4::5] = 0
    return [int(v) for v in r.multinomial(T, p / p.sum())]


def _rand(shape, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(DTYPES[dtype])


def _ends(sizes):
    return torch.tensor(np.cumsum(sizes), dtype=torch.int32, device="cuda")


def _bound(ref, mag, dtype, K):
    steps = 2.0 ** -20 if dtype == "f32" else max(2.0 ** -16, K / 16 * 2.0 ** -23)
    return torch.finfo(DTYPES[dtype]).eps / 2 * ref.abs() + steps * mag + (2.0 ** -25 if dtype == "f16" else 0.0)


def _check_rows(y, x, w, sizes, trans, dtype):
    r = 0
    for g, n in enumerate(sizes):
        if n:
            a, b = x[r:r + n].double(), (w[g].t() if trans else w[g]).double()
            ref, mag = a @ b, a.abs() @ b.abs()
            assert ((y[r:r + n].double() - ref).abs() <= _bound(ref, mag, dtype, a.shape[1])).all(), f"group {g}"
        r += n
    assert (y[r:] == 0).all()


def _check_grads(dw, x, dy, sizes, trans, dtype):
    r = 0
    for g, n in enumerate(sizes):
        a, b = x[r:r + n].double(), dy[r:r + n].double()
        a, b = (b, a) if trans else (a, b)
        ref, mag = a.t() @ b, a.t().abs() @ b.abs()
        assert ((dw[g].double() - ref).abs() <= _bound(ref, mag, dtype, max(n, 1))).all(), f"group {g}"
        r += n


def _plan(sg, handle, dtype, x, w, trans):
    p = sg._binding.GroupedPlan()
    G, N = w.shape[0], w.shape[1 if trans else 2]
    st = sg.load_library().sgemmGroupedQueryPlan(handle.ptr, TYPES[dtype], int(trans), x.shape[0], N, x.shape[1], G,
                                                 x.data_ptr(), x.stride(0), w.data_ptr(), w.stride(1), w.stride(0),
                                                 ctypes.byref(p))
    assert st == 0
    return p.as_dict()


def _grad_plan(sg, handle, dtype, a, b, G):
    p = sg._binding.GroupedPlan()
    st = sg.load_library().sgemmGroupedWeightGradQueryPlan(handle.ptr, TYPES[dtype], a.shape[0], a.shape[1],
                                                           b.shape[1], G, a.data_ptr(), a.stride(0), b.data_ptr(),
                                                           b.stride(0), ctypes.byref(p))
    assert st == 0
    return p.as_dict()


# (type, rows, columns, groups) -> (kernel, rows of a tile).  On 152 SMs.
TILES = [
    ("16", 90, 640, 6, 2, 32),
    ("16", 1500, 512, 8, 2, 64),
    ("16", 3000, 512, 8, 2, 128),
    ("16", 20, 8192, 8, 3, 32),
    ("16", 500, 4096, 8, 3, 64),
    ("16", 70, 8192, 8, 3, 96),
    ("16", 800, 4096, 8, 3, 128),
    ("16", 150, 8200, 8, 3, 160),
    ("16", 215, 8192, 8, 3, 224),
    ("16", 5001, 1100, 8, 3, 256),
    ("16", 9000, 3001, 20, 3, 256),
    ("f32", 60, 8192, 6, 2, 32),
    ("f32", 180, 6000, 8, 2, 32),
    ("f32", 1500, 1100, 8, 2, 128),
    ("f32", 6000, 1100, 8, 3, 256),
    ("f32", 5003, 3001, 9, 3, 256),
]


@pytest.mark.parametrize("kind,T,N,G,kernel,rows", TILES, ids=[f"{t[0]}-{t[1]}-{t[2]}-{t[3]}" for t in TILES])
@pytest.mark.parametrize("trans", [False, True])
def test_forward_tiles(sg, kind, T, N, G, kernel, rows, trans):
    h = sg.Handle()
    for dtype in ("f32",) if kind == "f32" else ("bf16", "f16"):
        for K in (328, 521):
            sizes = _sizes(T - 3, G, T + K)
            x = _rand((T, K), dtype, 1)
            w = _rand((G, N, K) if trans else (G, K, N), dtype, 2)
            plan = _plan(sg, h, dtype, x, w, trans)
            assert (plan["kernel"], plan["tile_m"]) == (kernel, rows), plan
            _check_rows(sg.grouped_gemm(x, w, _ends(sizes), trans_w=trans, handle=h), x, w, sizes, trans, dtype)
    assert h.device_error() == 0
    h.close()


# (rows, groups, rows of a matrix, columns) -> kernel.
GRADS = [
    (700, 5, 100, 72, 2),
    (3001, 8, 512, 520, 2),
    (3001, 8, 520, 513, 3),
    (4100, 7, 1030, 777, 3),
    (5003, 300, 200, 136, 3),
    (3000, 1024, 72, 40, 2),
    (2500, 1024, 136, 264, 3),
]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("T,G,K,N,kernel", GRADS, ids=[f"{t[0]}-{t[1]}-{t[2]}-{t[3]}" for t in GRADS])
def test_weight_gradient_tiles(sg, dtype, trans, T, G, K, N, kernel):
    h = sg.Handle()
    sizes = _sizes(T - 5, G, T)
    x, dy = _rand((T, K), dtype, 3), _rand((T, N), dtype, 4)
    x[T - 5:], dy[T - 5:] = float("nan"), float("inf")
    plan = _grad_plan(sg, h, dtype, *((dy, x) if trans else (x, dy)), G)
    assert plan["kernel"] == kernel, plan
    dw = sg.grouped_gemm_weight_grad(x, dy, _ends(sizes), trans_w=trans, handle=h)
    _check_grads(dw, x, dy, sizes, trans, dtype)
    assert h.device_error() == 0
    h.close()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("trans", [False, True])
def test_long_contractions_of_many_rows(sg, dtype, trans):
    sizes, K, N = [700, 0, 333, 1], 12296, 520
    T = sum(sizes)
    x, w = _rand((T, K), dtype, 5), _rand((4, N, K) if trans else (4, K, N), dtype, 6)
    _check_rows(sg.grouped_gemm(x, w, _ends(sizes), trans_w=trans), x, w, sizes, trans, dtype)
    sizes = [30000, 7, 12345]
    x, dy = _rand((sum(sizes), 264), dtype, 7), _rand((sum(sizes), 200), dtype, 8)
    dw = sg.grouped_gemm_weight_grad(x, dy, _ends(sizes), trans_w=trans)
    r = 0
    for g, n in enumerate(sizes):
        a, b = (dy, x) if trans else (x, dy)
        a, b = a[r:r + n].double(), b[r:r + n].double()
        ref, mag = a.t() @ b, a.t().abs() @ b.abs()
        # (FP32: sums of 64-long pieces, added with rounding to nearest.)
        extra = n / 64 * 2.0 ** -24 if dtype == "f32" else 0.0
        assert ((dw[g].double() - ref).abs() <= _bound(ref, mag, dtype, n) + extra * mag).all()
        r += n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [[300, 100, 700], [-5, 10, 700], [100, 200, 9000], [800, -3, 2 ** 31 - 1]])
@pytest.mark.parametrize("K,N", [(96, 40), (520, 513)])
def test_weight_gradient_with_ends_out_of_order(sg, dtype, bad, K, N):
    # Pulled into range and reported; nothing outside the output is written.
    T, G = 700, 24
    ends = torch.tensor(bad + [T] * (G - 3), dtype=torch.int32, device="cuda")
    x, dy = _rand((T, K), dtype, 9), _rand((T, N), dtype, 10)
    h = sg.Handle()
    buf = torch.full((G + 2, K + 1, N + 3), 7.0, device="cuda").to(DTYPES[dtype])
    sg.grouped_gemm_weight_grad(x, dy, ends, out=buf[1:G + 1, :K, :N], handle=h)
    assert h.device_error() >> 24 == 6
    assert (buf[0] == 7).all() and (buf[G + 1] == 7).all() and (buf[:, K:] == 7).all() and (buf[:, :, N:] == 7).all()
    good = _sizes(T, G, 11)
    dw = sg.grouped_gemm_weight_grad(x, dy, _ends(good), handle=h)
    _check_grads(dw, x, dy, good, False, dtype)
    assert h.device_error() == 0
    h.close()


def _waiting_calls(sg, dtype, h):
    """name -> (call, kernel of the plan or None)."""
    def rand(*shape):
        return (_rand(shape, dtype, len(shape) + shape[0]) * 0.1).to(DTYPES[dtype])
    T, G = (5003, 8)
    x, wt, wn, dy = rand(T, 2056), rand(G, 1100, 2056), rand(G, 2056, 1100), rand(T, 1100)
    ends = _ends(_sizes(T, G, 12))
    head = rand(3000, 2056)
    target = torch.arange(T, device="cuda") % 3000
    dloss = torch.ones(T, device="cuda")
    few, many = x[:16].contiguous(), x[:400].contiguous()
    lse = {n: sg.linear_cross_entropy(v, head, target[:n].contiguous(), handle=h)[1] for n, v in ((16, few), (400, many))}

    def grads(v):
        n = v.shape[0]
        return lambda: sg.linear_cross_entropy_grad(v, head, target[:n].contiguous(), lse[n], dloss[:n].contiguous(),
                                                    handle=h)
    return {
        "pair": (lambda: [sg.grouped_gemm(x, wt, ends, trans_w=True, handle=h)],
                 _plan(sg, h, dtype, x, wt, True)["kernel"]),
        "pair_n": (lambda: [sg.grouped_gemm(x, wn, ends, handle=h)], _plan(sg, h, dtype, x, wn, False)["kernel"]),
        "weight_grad": (lambda: [sg.grouped_gemm_weight_grad(x, dy, ends, handle=h)],
                        _grad_plan(sg, h, dtype, x, dy, G)["kernel"]),
        "loss_grad_few": (grads(few), None),
        "loss_grad": (grads(many), None),
    }


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("name", ["pair", "pair_n", "weight_grad", "loss_grad_few", "loss_grad"])
@pytest.mark.parametrize("which,site", [(2, 1), (3, 2)])
def test_expiry_of_pairs_and_loss_gradients(sg, dtype, name, which, site):
    h = sg.Handle()
    call, kernel = _waiting_calls(sg, dtype, h)[name]
    assert kernel in (None, 3)
    want = call()
    assert h.device_error() == 0
    h.set_wait_timeout(20_000_000)
    h.set_test_withheld_signal(which)
    call()
    code = h.device_error()
    h.set_test_withheld_signal(0)
    h.set_wait_timeout(2_000_000_000)
    assert code >> 24 == site, f"site {code >> 24}"
    assert all(torch.equal(a, b) for a, b in zip(call(), want))
    assert h.device_error() == 0
    h.close()
