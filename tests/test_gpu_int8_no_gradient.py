"""The quantisation has no gradient, and says so where one is asked for."""
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


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16], ids=["f32", "f16", "bf16"])
def test_quantisation_says_that_it_has_no_gradient(sg, dtype):
    x = torch.randn(5, 48, device="cuda").to(dtype)
    q, s = sg.int8_quantize(x)
    assert not q.requires_grad and not s.requires_grad
    x.requires_grad_()
    q2, s2 = sg.int8_quantize(x)
    assert torch.equal(q2, q) and torch.equal(s2, s)
    assert not q2.requires_grad and s2.requires_grad
    with pytest.raises(NotImplementedError):
        s2.sum().backward()
    # The product in two calls, as in one.
    w, ws = sg.int8_quantize(torch.randn(16, 48, device="cuda"))
    y = sg.int8_gemm(q2, w, ws, x_scales=s2, dtype=dtype)
    assert torch.equal(y, sg.int8_gemm(x.detach(), w, ws))
    with pytest.raises(NotImplementedError):
        y.sum().backward()
    with pytest.raises(NotImplementedError):
        sg.int8_gemm(x, w, ws).sum().backward()
    assert x.grad is None
    with torch.no_grad():
        assert not sg.int8_quantize(x)[1].requires_grad
    assert not sg.int8_quantize(x.detach())[1].requires_grad
    # On a stream of its own.
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    q3, s3 = sg.int8_quantize(x, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(q3, q) and torch.equal(s3, s) and s3.requires_grad
