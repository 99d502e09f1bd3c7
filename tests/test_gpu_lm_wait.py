"""Bounded waits of the language-model kernels: a signal left out on purpose
makes a wait run out, the kernel records the site and returns, and the next
call is right again (the failure is made by the test hook; nothing faults)."""
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


def _calls(sg, dtype):
    g = torch.Generator(device="cuda").manual_seed(1)

    def rand(*shape):
        return (torch.randn(*shape, generator=g, device="cuda") * 0.1).to(dtype)
    few, some, many = rand(16, 2048), rand(400, 2048), rand(3000, 2048)
    w = rand(4, 512, 2048)

    def ends(*e):
        return torch.tensor(e, dtype=torch.int32, device="cuda")
    target = torch.randint(0, 3000, (400,), generator=g, device="cuda")
    dy = rand(3000, 512)
    return {
        "thin": lambda h: sg.grouped_gemm(some[:160], w, ends(30, 50, 90, 160), trans_w=True, handle=h),
        "middle": lambda h: sg.grouped_gemm(some, w, ends(100, 200, 300, 400), trans_w=True, handle=h),
        "pair": lambda h: sg.grouped_gemm(many, w, ends(700, 1500, 2100, 3000), trans_w=True, handle=h),
        "weight_grad": lambda h: sg.grouped_gemm_weight_grad(many, dy, ends(703, 1501, 2100, 3000), handle=h),
        "loss": lambda h: sg.linear_cross_entropy(some, many, target, handle=h)[0],
        "loss_few": lambda h: sg.linear_cross_entropy(few, many, target[:16].contiguous(), handle=h)[0],
    }


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("name", ["thin", "middle", "pair", "weight_grad", "loss", "loss_few"])
@pytest.mark.parametrize("which,site", [(2, 1), (3, 2)])
def test_expiry_is_recorded_and_the_next_call_is_right(sg, dtype, name, which, site):
    call = _calls(sg, dtype)[name]
    h = sg.Handle()
    want = call(h)
    assert h.device_error() == 0
    h.set_wait_timeout(20_000_000)
    h.set_test_withheld_signal(which)
    call(h)
    code = h.device_error()
    h.set_test_withheld_signal(0)
    h.set_wait_timeout(2_000_000_000)
    # (2: operands that never come, 1 or a stage that is never free, 2.)
    assert code >> 24 == site, f"site {code >> 24}"
    assert torch.equal(call(h), want)
    assert h.device_error() == 0
    h.close()
