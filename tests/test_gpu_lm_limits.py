"""The shortest wait limit (1 ms) and calls that are correct but long: no wait
that only lasts as long as the work may run out."""
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


def _with_short_limit(sg, call):
    h = sg.Handle()
    want = call(h)
    assert h.device_error() == 0
    h.set_wait_timeout(1_000_000)
    got = call(h)
    assert h.device_error() == 0
    assert torch.equal(got, want)
    h.close()
    return got


def _close(got, a, b):
    # 16-bit sums of random signs: 2^-12 of sum |a b| is far above their
    # rounding, far below a block of 64 rows left out or counted twice.
    ref, mag = a.double().t() @ b.double(), a.double().abs().t() @ b.double().abs()
    assert ((got.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -12 * mag).all()


def test_one_long_contraction(sg):
    # One tile of a pair, 15626 blocks of 64 rows one after the other.
    T = 1_000_001
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T, 256, generator=g, device="cuda", dtype=torch.bfloat16)
    dy = torch.randn(T, 256, generator=g, device="cuda", dtype=torch.bfloat16)
    ends = torch.tensor([T], dtype=torch.int32, device="cuda")
    got = _with_short_limit(sg, lambda h: sg.grouped_gemm_weight_grad(x, dy, ends, handle=h))
    _close(got[0], x, dy)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_a_short_group_behind_long_ones(sg, dtype):
    # Only the smallest group, worked on last, ends inside 16 rows.
    sizes = [200_000, 200_000, 37] if dtype == torch.bfloat16 else [40_000, 40_000, 37]
    T, n = sum(sizes), 4096
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(T, n, generator=g, device="cuda", dtype=dtype)
    dy = torch.randn(T, n, generator=g, device="cuda", dtype=dtype)
    ends = torch.tensor([sizes[0], sizes[0] + sizes[1], T], dtype=torch.int32, device="cuda")
    got = _with_short_limit(sg, lambda h: sg.grouped_gemm_weight_grad(x, dy, ends, handle=h))
    _close(got[2], x[-37:], dy[-37:])
