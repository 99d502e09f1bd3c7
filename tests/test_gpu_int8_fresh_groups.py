"""Ends of many groups that a kernel right before the call has written: they are read
before x is quantised, and none of them may be old."""
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


# Few rows a group in the mean, and more; tables of one piece of 32 ends and of many.
@pytest.mark.parametrize("T,N,K,G", [(40, 128, 256, 31), (40, 96, 160, 33), (64, 32, 256, 1024), (900, 64, 256, 40),
                                     (1100, 64, 272, 100)])
def test_ends_of_many_groups_written_right_before(sg, T, N, K, G):
    g = torch.Generator(device="cuda").manual_seed(T + G)
    x = torch.randn(T, K, generator=g, device="cuda").half()
    q, s = sg.int8_quantize(x)
    w = torch.randint(-128, 128, (G, N, K), generator=g, device="cuda", dtype=torch.int8)
    ones = torch.ones(G, N, device="cuda")
    kinds = [torch.randint(0, T + 1, (G,), generator=g, device="cuda").sort().values.to(torch.int32) for _ in range(3)]
    kinds.append(torch.zeros(G, dtype=torch.int32, device="cuda"))
    kinds[3][G // 2:] = T                                  # (all rows in one group)
    want = []
    for e in kinds:
        y, a = torch.zeros(T, N, device="cuda", dtype=torch.float16), 0
        for i, b in enumerate(e.tolist()):
            if a < b:
                y[a:b] = ((q[a:b].double() @ w[i].double().t()).float() * s[a:b, None]).half()
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
