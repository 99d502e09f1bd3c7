"""The differentiable calls in torch's graph: gradients against torch's own on
the definition in 64 bits, and errors where there is no gradient."""
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


def _rand(*shape, seed, dtype=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * shape[-1] ** -0.5).to(dtype)


def _near(got, ref, dtype):
    # Two products and roundings to the type between one and the other.
    assert (got.double() - ref).norm() <= (2.0 ** -18 if dtype == torch.float32 else 2.0 ** -7) * ref.norm()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("need", ["xw", "x", "w"])
def test_grouped(sg, dtype, trans, need):
    sizes, K, N = [30, 0, 41], 136, 72
    ends = torch.tensor([30, 30, 71], dtype=torch.int32, device="cuda")
    x, w = _rand(71, K, seed=1, dtype=dtype), _rand(*((3, N, K) if trans else (3, K, N)), seed=2, dtype=dtype)
    x.requires_grad_("x" in need)
    w.requires_grad_("w" in need)
    # (A column sum: its gradient reaches the product as a broadcast.)
    y = sg.grouped_gemm(x, w, ends, trans_w=trans)
    scale = torch.arange(N, device="cuda", dtype=dtype) / N
    (x.sum() + (y * scale).sum()).backward() if "x" in need else (y * scale).sum().backward()
    xr, wr = x.detach().double().requires_grad_(), w.detach().double().requires_grad_()
    of = torch.tensor([0] * 30 + [2] * 41, device="cuda")
    yr = torch.einsum("tk,tnk->tn" if trans else "tk,tkn->tn", xr, wr[of])
    (xr.sum() + (yr * scale.double()).sum()).backward()
    for t, r, name in ((x, xr, "x"), (w, wr, "w")):
        if name in need:
            _near(t.grad, r.grad, dtype)
        else:
            assert t.grad is None


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("need", ["xw", "x", "w"])
def test_loss(sg, dtype, need):
    T, V, D = 50, 301, 72
    x, w = _rand(T, D, seed=3, dtype=dtype), _rand(V, D, seed=4, dtype=dtype) * 3
    w = w.detach()
    x.requires_grad_("x" in need)
    w.requires_grad_("w" in need)
    target = torch.arange(T, device="cuda") * 6
    target[::7] = -100
    loss, lse = sg.linear_cross_entropy(x, w, target)
    loss.mean().backward()
    xr, wr = x.detach().double().requires_grad_(), w.detach().double().requires_grad_()
    ref = torch.nn.functional.cross_entropy(xr @ wr.t(), target, ignore_index=-100, reduction="none")
    ref.mean().backward()
    assert ((loss.detach().double() - ref.detach()).abs() <= 2.0 ** -14).all()
    for t, r, name in ((x, xr, "x"), (w, wr, "w")):
        if name in need:
            _near(t.grad, r.grad, dtype)
        else:
            assert t.grad is None


def test_what_has_no_gradient_says_so(sg):
    x, w = _rand(9, 64, seed=5).requires_grad_(), _rand(30, 64, seed=6).requires_grad_()
    loss, lse = sg.linear_cross_entropy(x, w, torch.arange(9, device="cuda"))
    with pytest.raises(NotImplementedError):
        (loss.mean() + lse.square().mean()).backward()
    q = torch.zeros(8, 32, dtype=torch.uint8, device="cuda")
    y = sg.w4_gemm(x, q, torch.ones(8, 2, device="cuda"))
    assert y.shape == (9, 8) and (y.detach() == sg.w4_gemm(x.detach(), q, torch.ones(8, 2, device="cuda"))).all()
    with pytest.raises(NotImplementedError):
        y.sum().backward()
    # Twice differentiated: refused by torch, not wrong.
    ends = torch.tensor([9], dtype=torch.int32, device="cuda")
    wg = _rand(1, 64, 16, seed=7).requires_grad_()
    dx, = torch.autograd.grad(sg.grouped_gemm(x, wg, ends).square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        dx.sum().backward()


def test_no_graph_where_none_is_recorded(sg):
    x, w = _rand(9, 64, seed=8).requires_grad_(), _rand(1, 64, 16, seed=9).requires_grad_()
    ends = torch.tensor([9], dtype=torch.int32, device="cuda")
    with torch.no_grad():
        assert not sg.grouped_gemm(x, w, ends).requires_grad
        assert not sg.linear_cross_entropy(x, x, torch.arange(9, device="cuda"))[0].requires_grad
    assert not sg.grouped_gemm(x.detach(), w.detach(), ends).requires_grad
    out = torch.empty(9, 16, device="cuda")
    assert not sg.grouped_gemm(x, w, ends, out=out).requires_grad
    with pytest.raises(TypeError):
        sg.grouped_gemm(x, w, ends.long())


def test_forward_on_a_given_stream(sg):
    x, w = _rand(300, 264, seed=10).requires_grad_(), _rand(2, 264, 136, seed=11).requires_grad_()
    ends = torch.tensor([100, 300], dtype=torch.int32, device="cuda")
    sg.grouped_gemm(x, w, ends).square().sum().backward()
    want = x.grad.clone(), w.grad.clone()
    x.grad = w.grad = None
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = sg.grouped_gemm(x, w, ends, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    y.square().sum().backward()
    torch.cuda.synchronize()
    assert torch.equal(x.grad, want[0]) and torch.equal(w.grad, want[1])
