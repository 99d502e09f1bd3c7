"""Language-model operators on matrices of more than 2^31 elements: offsets that
pass 32 bits, in operands and outputs, checked where they lie farthest."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sg():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if torch.cuda.get_device_properties(0).total_memory < 100 << 30:
        pytest.skip("needs 100 GB")
    import fp32_sgemm_gb300 as m
    m.build()
    m.load_library()
    yield m
    torch.cuda.empty_cache()


def _rand(*shape, seed=1, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.empty(*shape, dtype=torch.bfloat16, device="cuda")
    return t.normal_(generator=g).mul_(scale)


def _close(got, a, b):
    """One bf16 rounding (half a unit in the last place: eps / 2), and 2^-14 of sum |a b| for the sum (at most 33000
    terms: 2063 truncating steps of 2^-23 are 2^-12 at the very worst of one
    sign; random signs stay below 2^-14)."""
    ref, mag = a.double() @ b.double(), a.double().abs() @ b.double().abs()
    assert ((got.double() - ref).abs() <= torch.finfo(torch.bfloat16).eps / 2 * ref.abs() + 2.0 ** -14 * mag).all()


@pytest.mark.parametrize("pad", [0, 1])
def test_long_rows(sg, pad):
    # x beyond 2^31 elements (odd pitch: copied), y small.
    T, K, N = 70_001, 32_768, 64
    x = _rand(T, K + pad)[:, :K]
    w = _rand(2, K, N, seed=2)
    ends = torch.tensor([30_000, T - 1], dtype=torch.int32, device="cuda")
    y = sg.grouped_gemm(x, w, ends)
    _close(y[-301:-1], x[-301:-1], w[1])
    _close(y[:100], x[:100], w[0])
    assert (y[-1] == 0).all()


def test_long_outputs(sg):
    T, K, N = 70_001, 72, 32_768
    x, w = _rand(T, K), _rand(2, K, N, seed=2)
    ends = torch.tensor([30_000, T - 1], dtype=torch.int32, device="cuda")
    y = sg.grouped_gemm(x, w, ends)
    _close(y[-301:-1], x[-301:-1], w[1])
    assert (y[-1] == 0).all()


def test_many_matrices(sg):
    # Matrices and their gradients beyond 2^31 elements.
    G, K, N = 37, 8192, 8192
    sizes = [3] * (G - 1) + [200]
    T = sum(sizes)
    ends = torch.tensor(sizes, device="cuda").cumsum(0).to(torch.int32)
    x, dy, w = _rand(T, K), _rand(T, N, seed=2), _rand(G, K, N, seed=3)
    _close(sg.grouped_gemm(x, w, ends)[-200:], x[-200:], w[-1])
    _close(sg.grouped_gemm(x, w, ends, trans_w=True)[-200:], x[-200:], w[-1].t())
    dw = sg.grouped_gemm_weight_grad(x, dy, ends)
    _close(dw[-1, -300:], x[-200:, -300:].t(), dy[-200:])
    _close(dw[-2, :300], x[-203:-200, :300].t(), dy[-203:-200])


def test_long_vocabulary(sg):
    T, V, D = 10, 530_000, 4104
    x, w = _rand(T, D), _rand(V, D, seed=2, scale=D ** -0.5)
    target = torch.arange(V - T, V, device="cuda")
    loss, lse = sg.linear_cross_entropy(x, w, target)
    dx, dw = sg.linear_cross_entropy_grad(x, w, target, lse, torch.ones(T, device="cuda"))
    logits = torch.cat([x.double() @ w[v:v + 100_000].double().t() for v in range(0, V, 100_000)], 1)
    ref = torch.logsumexp(logits, 1)
    assert ((lse.double() - ref).abs() <= 2.0 ** -16).all()
    assert ((loss.double() - (ref - logits[:, -T:].diagonal())).abs() <= 2.0 ** -16).all()
    d = (logits - ref[:, None]).exp()
    d[torch.arange(T), target] -= 1
    tail = d[:, -500:].t() @ x.double()
    assert (dw[-500:].double() - tail).norm() <= 2.0 ** -8 * tail.norm()
    whole = sum(d[:, v:v + 100_000] @ w[v:v + 100_000].double() for v in range(0, V, 100_000))
    assert (dx.double() - whole).norm() <= 2.0 ** -8 * whole.norm()


def test_many_four_bit_rows(sg):
    N, K, group = 270_001, 16_384, 128
    g = torch.Generator(device="cuda").manual_seed(4)
    q = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = _rand(N, K // group, seed=5, scale=0.02)
    x = _rand(3, K)
    y = sg.w4_gemm(x, q, s)
    for rows in (slice(0, 100), slice(N - 100, N)):
        v = torch.stack((q[rows] & 15, q[rows] >> 4), 2).view(100, K).double() - 8
        _close(y[:, rows], x, (v * s[rows].double().repeat_interleave(group, 1)).t())


def test_uneven_gradients_in_f16(sg):
    # Tokens' dloss from 2^-16 to 1 in one call (f16 holds d over the largest):
    # d is off by half a unit in its last place, and 2^-37 of the largest.
    T, V, D = 300, 2000, 128
    g = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn(T, D, generator=g, device="cuda").half()
    w = (torch.randn(V, D, generator=g, device="cuda") * 2 * D ** -0.5).half()
    target = torch.randint(0, V, (T,), generator=g, device="cuda")
    dloss = 2.0 ** -(torch.arange(T, device="cuda") % 17).float()
    _, lse = sg.linear_cross_entropy(x, w, target)
    dx, dw = sg.linear_cross_entropy_grad(x, w, target, lse, dloss)
    X, W = x.double(), w.double()
    logits = X @ W.t()
    p = torch.softmax(logits, 1)
    d = p.clone()
    d[torch.arange(T), target] -= 1
    d *= dloss.double()[:, None]
    # (Logits: 2^-19 of sum |x w|, which is at most 30 here; exponential 2^-18.)
    e = p * dloss.double()[:, None] * (2 * 30 * 2.0 ** -19 + 2.0 ** -18) + 2.0 ** -11 * d.abs() + 2.0 ** -37
    for got, ref, err, mag in ((dx, d @ W, e @ W.abs(), d.abs() @ W.abs()),
                               (dw, d.t() @ X, e.t() @ X.abs(), d.abs().t() @ X.abs())):
        bound = (err + 2.0 ** -16 * mag) * (1 + 2.0 ** -11) + 2.0 ** -11 * ref.abs() + 2.0 ** -25
        assert ((got.double() - ref).abs() <= bound).all()
