"""Weights, scales and ends that a kernel right before the call has written (the
products read some of it before x is quantised, and none of it may be old), and
groups that are cut or alone."""
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


@pytest.mark.parametrize("T,N,K", [(1, 256, 512), (3, 500, 4096), (8, 512, 2048), (8, 300, 2050), (40, 512, 1024),
                                   (200, 300, 2047)])
def test_weights_written_right_before(sg, T, N, K):
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn(T, K, generator=g, device="cuda").bfloat16()
    q, s = sg.int8_quantize(x)
    kinds = [torch.randint(-128, 128, (N, K), generator=g, device="cuda", dtype=torch.int8) for _ in range(4)]
    ones = torch.ones(N, device="cuda")
    want = [((q.double() @ w.double().t()).float() * s[:, None] * ones).bfloat16() for w in kinds]
    w = torch.empty(N, K, dtype=torch.int8, device="cuda")
    torch.cuda.synchronize()
    got = []
    for i in range(200):
        w.copy_(kinds[i % 4])
        if i % 3 == 0:
            w[:1] += 0                                     # (a kernel of one CTA in between)
        got.append(sg.int8_gemm(x, w, ones))
    for i, y in enumerate(got):
        assert torch.equal(y, want[i % 4]), i


@pytest.mark.parametrize("T,N,K", [(6, 256, 512), (24, 200, 1030), (300, 256, 1024)])
def test_ends_written_right_before(sg, T, N, K):
    G = 5
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn(T, K, generator=g, device="cuda").half()
    q, s = sg.int8_quantize(x)
    w = torch.randint(-128, 128, (G, N, K), generator=g, device="cuda", dtype=torch.int8)
    ones = torch.ones(G, N, device="cuda")
    kinds = [torch.randint(0, T + 1, (G,), generator=g, device="cuda").sort().values.to(torch.int32) for _ in range(4)]
    want = []
    for e in kinds:
        y, a = torch.zeros(T, N, device="cuda", dtype=torch.float16), 0
        for i, b in enumerate(e.tolist()):
            y[a:b] = ((q[a:b].double() @ w[i].double().t()).float() * s[a:b, None] * ones[i]).half()
            a = b
        want.append(y)
    ends = torch.empty(G, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    got = []
    for i in range(200):
        ends.copy_(kinds[i % 4])
        got.append(sg.int8_grouped_gemm(x, w, ones, ends))
    for i, y in enumerate(got):
        assert torch.equal(y, want[i % 4]), i


@pytest.mark.parametrize("sizes,N,K,behind", [([2], 50, 300, 0), ([1], 70, 4096, 2), ([5], 33, 130, 4), ([40], 60, 700, 9),
                                              ([0], 20, 64, 3), ([3, 0, 2, 1], 40, 70001, 2), ([9, 1, 30], 40, 70001, 5),
                                              ([0, 60, 0, 0, 0, 0, 0, 0], 129, 513, 1)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_one_group_and_cut_groups(sg, sizes, N, K, behind, dtype):
    # One group with an end of its own, contractions in parts by group, all rows
    # in one of many groups.
    T, G = sum(sizes) + behind, len(sizes)
    g = torch.Generator(device="cuda").manual_seed(K)
    x = torch.randn(T, K, generator=g, device="cuda").to(dtype)
    w = torch.randint(-128, 128, (G, N, K), generator=g, device="cuda", dtype=torch.int8)
    ws = torch.rand(G, N, generator=g, device="cuda")
    ends = torch.tensor(sizes, device="cuda").cumsum(0).to(torch.int32)
    q, s = sg.int8_quantize(x)
    want, a = torch.zeros(T, N, dtype=dtype, device="cuda"), 0
    for i, n in enumerate(sizes):
        total = (q[a:a + n].double() @ w[i].double().t()).to(torch.int64)
        want[a:a + n] = (total.float() * s[a:a + n, None] * ws[i]).to(dtype)
        a += n
    assert torch.equal(sg.int8_grouped_gemm(x, w, ws, ends), want)
    assert torch.equal(sg.int8_grouped_gemm(q, w, ws, ends, x_scales=s, dtype=dtype), want)
