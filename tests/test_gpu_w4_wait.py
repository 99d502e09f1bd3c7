"""The bounded wait of the 4-bit kernel: weights that never come (left out by the
test hook) make it run out; the kernel stops issuing copies, lets those in
flight land, records the site and returns, and the next call is right."""
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


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32], ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("group,M,K", [(128, 1, 16384), (64, 7, 16384), (32, 20, 16384), (128, 32, 16384)])
def test_expiry_is_recorded_and_the_next_call_is_right(sg, dtype, group, M, K):
    g = torch.Generator(device="cuda").manual_seed(M)
    N = 2000
    x = torch.randn(M, K, generator=g, device="cuda").to(dtype)
    q = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.rand(N, K // group, generator=g, device="cuda").to(dtype)
    h = sg.Handle()
    want = sg.w4_gemm(x, q, scales, handle=h)
    assert h.device_error() == 0
    h.set_wait_timeout(20_000_000)
    h.set_test_withheld_signal(2)
    sg.w4_gemm(x, q, scales, handle=h)
    code = h.device_error()
    h.set_test_withheld_signal(0)
    h.set_wait_timeout(2_000_000_000)
    assert code >> 24 == 1, f"site {code >> 24}"
    assert torch.equal(sg.w4_gemm(x, q, scales, handle=h), want)
    assert h.device_error() == 0
    h.close()
