"""Converted weights handed to the MMAs of an SM pair: products of many blocks, with
other weights each time, have the same bits as the exact sums whatever was in tensor
memory before."""
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


# Both kernels (tiles of up to 128 and 192 rows), whole contractions and parts,
# many tiles for each SM pair and one, groups.
@pytest.mark.parametrize("T,N,K,G", [(300, 2000, 4096, 1), (2500, 9000, 1024, 1), (8192, 4096, 1536, 1), (20, 4096, 4096, 1),
                                     (40, 500, 20000, 1), (4000, 1024, 1280, 7)])
def test_other_weights_each_time(sg, T, N, K, G):
    g = torch.Generator(device="cuda").manual_seed(T + K)
    x = torch.randn(T, K, generator=g, device="cuda").bfloat16()
    q, s = sg.int8_quantize(x)
    # (Large integers of one sign and the other: an old block stands out.)
    kinds = [torch.randint(-128, 128, (G, N, K), generator=g, device="cuda", dtype=torch.int8) for _ in range(2)]
    kinds.append(~kinds[0])
    ones = torch.ones(G, N, device="cuda")
    cuts = [T * i // G for i in range(G + 1)]
    ends = torch.tensor(cuts[1:], dtype=torch.int32, device="cuda")
    want = []
    for w in kinds:
        parts = [(q[a:b].double() @ w[i].double().t()).float() * s[a:b, None] for i, (a, b) in enumerate(zip(cuts, cuts[1:]))]
        want.append(torch.cat(parts))
    for i in range(30):
        w = kinds[i % 3]
        if G > 1:
            y = sg.int8_grouped_gemm(x, w, ones, ends, dtype=torch.float32)
        else:
            y = sg.int8_gemm(x, w[0], ones[0], dtype=torch.float32)
        assert torch.equal(y, want[i % 3]), i
