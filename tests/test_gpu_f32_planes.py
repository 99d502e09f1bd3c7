"""FP32 products as six products of bf16 planes: what the planes left out may
cost, one product at a time and summed with equal signs.

One product (K = 1): the plane products left out are below 2^-23.9 of it; the
six others are added smallest first in a sum that keeps 24 bits at least and
truncates, so the last addition costs 2^-23 and the five before it, which are
2^-6 of the whole at most, 5 * 2^-29.  Together below 2^-22.

256 products of one sign: four pieces of 64, in each of which four additions of
the leading products truncate (4 * 2^-23) and the others cost 2^-25 in all;
three additions of the pieces (3 * 2^-24); the planes left out.  Together below
2^-20.
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


def _one_group(T):
    return torch.tensor([T], dtype=torch.int32, device="cuda")


def _worst(got, ref):
    return ((got.double() - ref).abs() / ref.abs()).max().item()


def _hard(n, sign):
    """FP32 values whose low bits are set in the places the planes cut at."""
    g = torch.Generator(device="cuda").manual_seed(n)
    v = 1.0 + torch.rand(n, generator=g, device="cuda")
    v[0] = 1 + 2.0 ** -7 - 2.0 ** -23                  # (both residuals as large as truncation leaves them)
    v[1] = 1 + 2.0 ** -7 + 2.0 ** -8 - 2.0 ** -23
    v[2] = 1 + 2.0 ** -8 + 2.0 ** -17
    v[3] = 2 - 2.0 ** -23
    v[4] = 1 + 2.0 ** -15 - 2.0 ** -23
    if sign:
        v[::2] *= -1
    return v


@pytest.mark.parametrize("sign", [False, True])
def test_single_products(sg, sign):
    x, w = _hard(300, sign)[:, None], _hard(260, sign)[None, None, :]
    got = sg.grouped_gemm(x.contiguous(), w.contiguous(), _one_group(300))
    assert _worst(got, x.double() @ w[0].double()) <= 2.0 ** -22


def test_single_products_over_the_range(sg):
    # Powers of two apart: the split is exact down to 2^-110 and the largest
    # numbers do not become infinite.
    v = _hard(64, False)
    for ex, ew in ((-100, 20), (60, -60), (126, -100), (-10, -80)):
        x, w = (v * 2.0 ** ex)[:, None].contiguous(), (v * 2.0 ** ew)[None, None, :].contiguous()
        got = sg.grouped_gemm(x, w, _one_group(64))
        assert _worst(got, x.double() @ w[0].double()) <= 2.0 ** -22
    top = torch.full((64, 1), torch.finfo(torch.float32).max, device="cuda")
    w = torch.full((1, 1, 16), 0.5, device="cuda")
    got = sg.grouped_gemm(top, w, _one_group(64))
    assert _worst(got, top.double() @ w[0].double()) <= 2.0 ** -21


def test_sums_of_one_sign(sg):
    g = torch.Generator(device="cuda").manual_seed(3)
    T, K, N = 300, 256, 200
    x = 1.0 + torch.rand(T, K, generator=g, device="cuda")
    w = 1.0 + torch.rand(1, K, N, generator=g, device="cuda")
    dy = 1.0 + torch.rand(T, N, generator=g, device="cuda")
    got = sg.grouped_gemm(x, w, _one_group(T))
    assert _worst(got, x.double() @ w[0].double()) <= 2.0 ** -20
    rows = 256
    dw = sg.grouped_gemm_weight_grad(x, dy, _one_group(rows))
    assert _worst(dw[0], x[:rows].double().t() @ dy[:rows].double()) <= 2.0 ** -20
