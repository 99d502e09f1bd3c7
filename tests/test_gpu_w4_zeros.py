"""Zero points of the 4-bit products over every value a byte has: formats that
store them less one decode to 1..16, signed ones to more.

q - zero is an integer in [-255, 15] and exact in the product.  With x a unit
vector and a scale of one the output is that integer, exact in every type; in
general the bound is that of test_gpu_w4.py: FP32 summation, 2^-20 of
sum |s (q - z) x|, and one rounding to the type.
"""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(scope="module")
def sg():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import fp32_sgemm_gb300 as m
    m.build()
    m.load_library()
    return m


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_every_zero_point_with_every_nibble(sg, dtype, group):
    # Row 16 z + q holds the nibble q in every column and the zero point z in
    # every group; x picks one column of each of the places of a word.
    groups = 3
    K = group * groups
    n = torch.arange(256 * 16, device="cuda")
    q = ((n % 16) * 17).to(torch.uint8)[:, None].repeat(1, K // 2)
    z = (n // 16).to(torch.uint8)[:, None].repeat(1, groups)
    s = torch.ones(len(n), groups, dtype=DTYPES[dtype], device="cuda")
    x = torch.zeros(9, K, dtype=DTYPES[dtype], device="cuda")
    for t in range(9):
        x[t, (t * (group + 1)) % K] = 1.0
    want = (n % 16 - n // 16).to(DTYPES[dtype])
    got = sg.w4_gemm(x, q, s, z)
    assert torch.equal(got, want.expand(9, len(n)))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M", [1, 7, 20, 33])
def test_random_zero_points(sg, dtype, group, M):
    g = torch.Generator(device="cuda").manual_seed(M + group)
    N, K = 97, 1152
    x = torch.randn(M, K, generator=g, device="cuda").to(DTYPES[dtype])
    q = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = (torch.randn(N, K // group, generator=g, device="cuda") * 0.02).to(DTYPES[dtype])
    z = torch.randint(0, 256, (N, K // group), generator=g, device="cuda", dtype=torch.uint8)
    v = torch.stack((q & 15, q >> 4), 2).view(N, K).double() - z.double().repeat_interleave(group, 1)
    w = v * s.double().repeat_interleave(group, 1)
    ref = x.double() @ w.t()
    eps = torch.finfo(DTYPES[dtype]).eps / 2
    bound = eps * ref.abs() + 2.0 ** -20 * (x.double().abs() @ w.abs().t()) * (1 + eps) + \
        (2.0 ** -25 if dtype == "f16" else 0.0)
    assert ((sg.w4_gemm(x, q, s, z).double() - ref).abs() <= bound).all()
