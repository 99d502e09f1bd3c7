"""Rows by expert and 8-bit products beyond 2^31 elements, and a training step of
an expert layer captured into a graph."""
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


def test_rows_beyond_2_31_elements(sg):
    T, k, D = 66000, 8, 4096                               # 2.16e9 elements of rows
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T, D, generator=g, device="cuda", dtype=torch.bfloat16)
    experts = torch.rand(T, 64, generator=g, device="cuda").topk(k, 1).indices
    rows, slots, ends = sg.expert_dispatch(x, experts, 64)
    assert rows.numel() > 2 ** 31 and int(ends[-1]) == T * k
    for t in range(0, T, 2999):
        assert torch.equal(rows[slots[t].long()], x[t].expand(k, D))
    weights = torch.full((T, k), 0.125, device="cuda")
    assert torch.equal(sg.expert_combine(rows, slots, weights), x)      # (eighths of eight equals: exact)
    drows, dweights = sg.expert_combine_grad(x, rows, slots, weights)
    for t in range(0, T, 2999):
        assert torch.equal(drows[slots[t].long()], (x[t] * 0.125).expand(k, D))
        dot = (x[t].double() ** 2).sum()
        assert ((dweights[t].double() - dot).abs() <= (D + 1) * 2.0 ** -24 * dot).all()


@pytest.mark.parametrize("T", [1, 3, 7, 40, 300])
def test_weights_beyond_2_31_bytes(sg, T):
    N, K = 70000, 32768
    g = torch.Generator(device="cuda").manual_seed(2)
    w = torch.empty(N, K, dtype=torch.int8, device="cuda")
    for a in range(0, N, 10000):
        w[a:a + 10000] = torch.randint(-128, 128, (min(10000, N - a), K), generator=g, device="cuda", dtype=torch.int8)
    assert w.numel() > 2 ** 31
    q = torch.randint(-128, 128, (T, K), generator=g, device="cuda", dtype=torch.int8)
    xs, ws = torch.rand(T, generator=g, device="cuda"), torch.rand(N, generator=g, device="cuda")
    y = sg.int8_gemm(q, w, ws, x_scales=xs, dtype=torch.float32)
    for a in (0, 65530, N - 40):                            # (around 2^31 bytes, and the last)
        total = (q.double() @ w[a:a + 40].double().t()).to(torch.int64)
        assert torch.equal(y[:, a:a + 40], total.float() * xs[:, None] * ws[a:a + 40])


def test_a_captured_training_step(sg):
    T, D, H, G, k = 200, 128, 96, 6, 2
    g = torch.Generator(device="cuda").manual_seed(3)

    def rand(*shape):
        return (torch.randn(*shape, generator=g, device="cuda") * shape[-1] ** -0.5).requires_grad_()
    router, up, down = rand(G, D), rand(G, H, D), rand(G, D, H)
    x = torch.randn(T, D, generator=g, device="cuda")
    c = torch.randn(T, D, generator=g, device="cuda")
    leaves = (router, up, down)

    def step():
        weights, experts = sg.route_topk(x @ router.t(), k)
        rows, slots, ends = sg.expert_dispatch(x, experts, G)
        h = torch.tanh(sg.grouped_gemm(rows, up, ends, trans_w=True))
        y = sg.expert_combine(sg.grouped_gemm(h, down, ends, trans_w=True), slots, weights)
        return torch.autograd.grad((y * c).sum(), leaves)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(2):
            step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        grads = step()
    for seed in (4, 5):
        x.copy_(torch.randn(T, D, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda"))
        want = [v.clone() for v in step()]
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(grads, want):
            assert torch.equal(a, b)
