"""Long contractions of 16-bit operands with terms of one sign.  The tensor
core's running sum truncates: its loss, up to 1.7e-7 of the sum for every 16
terms, adds up, so that long sums are taken in runs of 8192 (4.4e-5 at the
most), added with rounding to nearest.

Criterion: the mean relative deviation of many outputs, whose final roundings
to f16 even out (columns of different size), stays below 2^-13, an eighth of a
unit in f16's last place.  One sum of 65536 terms is off by 3.9e-4.
"""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sg():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import fp32_sgemm_gb300 as m
    m.build()
    m.load_library()
    return m


def _positive(rows, cols, seed, scale):
    """Rows of random numbers in (0, 1], each times a factor of its own in
    [1, 2)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    v = torch.rand(rows, cols, generator=g, device="cuda") * scale
    return (v * (1 + torch.rand(rows, 1, generator=g, device="cuda"))).half()


def _unbiased(got, ref):
    assert (((got.double() - ref).abs() / ref) <= 2.0 ** -11 + 2.0 ** -13).all()
    assert abs(((got.double() - ref) / ref).mean().item()) <= 2.0 ** -13


@pytest.mark.parametrize("K,N,trans", [(264, 200, False), (264, 200, True), (100, 72, False), (777, 520, False)])
def test_weight_gradient_of_a_long_group(sg, K, N, trans):
    sizes = [65553, 100, 20001]
    T = sum(sizes)
    x, dy = _positive(K, T, 1, 1e-3).t().contiguous(), _positive(N, T, 2, 1.0).t().contiguous()
    ends = torch.tensor(sizes, device="cuda").cumsum(0).to(torch.int32)
    dw = sg.grouped_gemm_weight_grad(x, dy, ends, trans_w=trans)
    r = 0
    for g, n in enumerate(sizes):
        ref = x[r:r + n].double().t() @ dy[r:r + n].double()
        _unbiased(dw[g].t() if trans else dw[g], ref)
        r += n


@pytest.mark.parametrize("T,N,G,K", [(3000, 1100, 4, 40008), (3000, 512, 8, 40001), (90, 640, 6, 100000)])
@pytest.mark.parametrize("trans", [False, True])
def test_long_rows(sg, T, N, G, K, trans):
    x, w = _positive(T, K, 3, 1.0), _positive(N, K, 4, 1.0 / K).expand(1, N, K)
    # (All matrices alike, but for a factor of a power of two.)
    w = torch.cat([w * 2.0 ** -(g % 3) for g in range(G)])
    w = w if trans else w.transpose(1, 2).contiguous()
    ends = torch.arange(1, G + 1, device="cuda", dtype=torch.int32) * (T // G)
    y = sg.grouped_gemm(x, w, ends, trans_w=trans)
    for g in range(G):
        rows = slice(g * (T // G), (g + 1) * (T // G))
        _unbiased(y[rows], x[rows].double() @ (w[g].double().t() if trans else w[g].double()))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,V,D", [(20011, 300, 72), (40, 60001, 72), (300, 40001, 136)])
def test_loss_gradients(sg, dtype, T, V, D):
    # dW sums over the tokens, dX over the vocabulary; bounds of
    # test_gpu_loss.py.
    from test_gpu_loss import _check, _problem
    x, w, target, dloss = _problem(T, V, D, dtype, T)
    _check(sg, x, w, target, dloss, dtype)


def test_gradient_of_a_column_summed_over_many_tokens(sg):
    # Every token has the same target, whose row of d is p - 1 < 0 throughout:
    # terms of one sign in dW.
    T, V, D = 65553, 300, 264
    x, g = _positive(D, T, 5, 1.0).t().contiguous(), torch.Generator(device="cuda").manual_seed(6)
    w = (torch.randn(V, D, generator=g, device="cuda") * 0.01).half()
    target = torch.full((T,), 17, device="cuda")
    dloss = torch.full((T,), 1.0 / 64, device="cuda")
    _, lse = sg.linear_cross_entropy(x, w, target)
    _, dw = sg.linear_cross_entropy_grad(x, w, target, lse, dloss)
    p = (x.double() @ w.double().t() - lse.double()[:, None]).exp()
    ref = (1 - p[:, 17]) / 64 @ x.double()
    assert abs(((-dw[17].double() - ref) / ref).mean().item()) <= 2.0 ** -13
