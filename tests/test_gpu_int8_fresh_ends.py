"""Weights that a kernel right before the call has written, in rows that end inside
a step of a warp: the last piece of an aligned row is read before x is quantised as
the pieces before it are, and none of it may be old."""
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


# Columns in whole steps of 256 and a rest of 16 to 240, a multiple of 16 or not;
# `pitch` a multiple of 16.  groups 0: one matrix.
CASES = [(4, 500, 2064, 0), (4, 300, 4100, 0), (8, 512, 1040, 0), (8, 300, 1920, 0), (8, 400, 2000, 0), (8, 200, 2031, 0),
         (6, 256, 160, 3), (12, 256, 896, 6), (12, 200, 960, 6), (40, 128, 1920, 8), (40, 128, 1007, 8), (9, 96, 4090, 9)]


@pytest.mark.parametrize("T,N,K,G", CASES)
def test_ends_of_rows_written_right_before(sg, T, N, K, G):
    g = torch.Generator(device="cuda").manual_seed(T + K)
    x = torch.randn(T, K, generator=g, device="cuda").bfloat16()
    q, s = sg.int8_quantize(x)
    groups, pitch = max(G, 1), (K + 15) // 16 * 16
    kinds = [torch.randint(-128, 128, (groups, N, K), generator=g, device="cuda", dtype=torch.int8) for _ in range(4)]
    ones = torch.ones(groups, N, device="cuda")
    sizes = torch.full((groups,), T // groups)
    sizes[0] += T % groups
    of = torch.arange(groups).repeat_interleave(sizes).cuda()
    ends = sizes.cumsum(0).to(torch.int32).cuda()
    want = [(torch.einsum("tk,tnk->tn", q.double(), w.double()[of]).float() * s[:, None]).bfloat16() for w in kinds]
    w = torch.zeros(groups, N, pitch, dtype=torch.int8, device="cuda")[:, :, :K]

    def product(integers):
        if G:
            kw = dict(x_scales=s, dtype=torch.bfloat16) if integers else {}
            return sg.int8_grouped_gemm(q if integers else x, w, ones, ends, **kw)
        return sg.int8_gemm(q, w[0], ones[0], x_scales=s, dtype=torch.bfloat16) if integers else sg.int8_gemm(x, w[0], ones[0])
    torch.cuda.synchronize()
    got = []
    for i in range(200):
        w.copy_(kinds[i % 4])
        if i % 3 == 0:
            w[:1, :1] += 0                                 # (a kernel of one CTA in between)
        got.append((i % 4, product(i % 5 == 4)))
    for i, (kind, y) in enumerate(got):
        assert torch.equal(y, want[kind]), i
