"""Bounded waits of the 8-bit products on the tensor cores: a signal left out on
purpose makes a wait run out, the kernel records the site and returns, and the
next call is right again (the failure is made by the test hook; nothing faults).
And long calls at the shortest limit, in which no wait may run out."""
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


def _operands(T, N, K, G):
    g = torch.Generator(device="cuda").manual_seed(T + N)
    x = torch.randn(T, K, generator=g, device="cuda").bfloat16()
    w = torch.randint(-128, 128, (G, N, K), generator=g, device="cuda", dtype=torch.int8)
    return x, w, torch.rand(G, N, generator=g, device="cuda")


@pytest.mark.parametrize("name", ["dense", "cut", "cut_long", "groups", "groups_long"])
@pytest.mark.parametrize("which,site", [(2, 1), (3, 2)])
def test_expiry_is_recorded_and_the_next_call_is_right(sg, name, which, site):
    T, N, K, G = {"dense": (3000, 700, 2048, 1), "cut": (64, 700, 8192, 1), "cut_long": (64, 700, 65536, 1),
                  "groups": (900, 512, 2048, 4), "groups_long": (900, 512, 8192, 4)}[name]
    x, w, s = _operands(T, N, K, G)
    ends = torch.tensor([100, 400, 700, T], dtype=torch.int32, device="cuda")

    def call(h):
        return sg.int8_grouped_gemm(x, w, s, ends, handle=h) if G > 1 else sg.int8_gemm(x, w[0], s[0], handle=h)
    h = sg.Handle()
    want = call(h)
    assert h.device_error() == 0
    h.set_wait_timeout(20_000_000)
    h.set_test_withheld_signal(which)
    got = call(h)
    code = h.device_error()
    h.set_test_withheld_signal(0)
    h.set_wait_timeout(2_000_000_000)
    # (2: operands that never come, 1 or a stage that is never free, 2.)
    if name in ("cut", "groups"):
        # Parts of the contraction so short that a ring may hold one whole, and no
        # stage be filled or waited for again: then nothing runs out, and nothing
        # is missing.
        assert code >> 24 in (1, 2) or (code == 0 and torch.equal(got, want))
    else:
        assert code >> 24 == site, f"site {code >> 24}"
    assert torch.equal(call(h), want)
    assert h.device_error() == 0
    h.close()


def test_long_calls_at_the_shortest_limit(sg):
    h = sg.Handle()
    for T, N, K, G in ((16384, 4096, 8192, 1), (64, 300, 131071, 1), (20000, 256, 1024, 5)):
        x, w, s = _operands(T, N, K, G)
        ends = torch.tensor([0, 1, T - 300, T - 300, T], dtype=torch.int32, device="cuda")[-G:].contiguous()
        h.set_wait_timeout(2_000_000_000)
        want = sg.int8_grouped_gemm(x, w, s, ends, handle=h)
        h.set_wait_timeout(1_000_000)
        assert torch.equal(sg.int8_grouped_gemm(x, w, s, ends, handle=h), want)
        assert h.device_error() == 0
    h.close()
