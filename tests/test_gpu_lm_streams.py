"""Calls given a stream: what they read is not reused, and what they return is
not handed out, before that stream has passed."""
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


def _rand(*shape, dtype=torch.bfloat16, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_inputs_freed_right_after_the_call(sg, dtype):
    T, K, N = 2048, 1024, 1024
    ends = torch.tensor([700, 700, T], dtype=torch.int32, device="cuda")
    w = _rand(3, K, N, dtype=dtype, seed=1)
    want = sg.grouped_gemm(_rand(T, K, dtype=dtype, seed=2), w, ends)
    torch.cuda.synchronize()
    h, s = sg.Handle(), torch.cuda.Stream()
    for _ in range(3):
        x = _rand(T, K, dtype=dtype, seed=2)
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            torch.cuda._sleep(2_000_000)             # the product starts late
        y = sg.grouped_gemm(x, w, ends, handle=h, stream=s)
        del x
        junk = [torch.full((T, K), float("nan"), dtype=dtype, device="cuda") for _ in range(4)]
        torch.cuda.current_stream().wait_stream(s)
        assert torch.equal(y, want)
        del junk
    assert h.device_error() == 0
    h.close()


def test_every_operator_on_a_given_stream(sg):
    x, w = _rand(96, 256, seed=3), _rand(2, 256, 512, seed=4)
    dy, head = _rand(96, 512, seed=5), _rand(1000, 256, seed=6)
    ends = torch.tensor([40, 96], dtype=torch.int32, device="cuda")
    target = torch.arange(96, device="cuda") * 7
    dloss = torch.full((96,), 1 / 96, device="cuda")
    q = torch.arange(512 * 128, device="cuda").to(torch.uint8).view(512, 128)
    scales = _rand(512, 4, seed=7)

    def run(**kw):
        loss, lse = sg.linear_cross_entropy(x, head, target, **kw)
        return [sg.grouped_gemm(x, w, ends, **kw), sg.grouped_gemm_weight_grad(x, dy, ends, **kw), loss, lse,
                *sg.linear_cross_entropy_grad(x, head, target, lse, dloss, **kw),
                sg.w4_gemm(x[:5], q, scales, **kw)]
    want = run()
    torch.cuda.synchronize()
    h, s = sg.Handle(), torch.cuda.Stream()
    got = run(handle=h, stream=s)
    got_raw = run(handle=h, stream=s.cuda_stream)
    s.synchronize()
    for a, b, c in zip(want, got, got_raw):
        assert torch.equal(a, b) and torch.equal(a, c)
    h.close()


def test_a_handle_of_another_device_is_refused(sg):
    # One device here: a handle whose C handle is gone stands for a wrong one.
    h = sg.Handle()
    h.close()
    x, w = _rand(4, 16, seed=8), _rand(1, 16, 16, seed=9)
    with pytest.raises(sg.SgemmError):
        sg.grouped_gemm(x, w, torch.tensor([4], dtype=torch.int32, device="cuda"), handle=h)
