"""Products grouped by expert and their gradients against a plain loop in 64
bits, at the group sizes, pitches and values where they can go wrong.

Tolerances.  16-bit results are sums in FP32 rounded once: half a unit in the
last place of the type (its eps / 2; plus half of f16's smallest step 2^-24),
and for the sum itself 2^-16 of sum |a b| (the
tensor core's running sum truncates: K / 16 steps of 2^-23 at the K used
here).  FP32 results: planes left out and FP32 sums, 2^-20 of sum |a b|.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
ROUND = {name: torch.finfo(t).eps / 2 for name, t in DTYPES.items()}
SUM = {"bf16": 2.0 ** -16, "f16": 2.0 ** -16, "f32": 2.0 ** -20}
STEP = {"bf16": 0.0, "f16": 2.0 ** -25, "f32": 0.0}


@pytest.fixture(scope="module")
def sg():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import fp32_sgemm_gb300 as m
    m.build()
    m.load_library()
    return m


def _rand(shape, dtype, seed, pitch_pad=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    t = torch.randn(*shape[:-1], shape[-1] + pitch_pad, generator=g) * scale
    return t.to(DTYPES[dtype]).cuda()[..., :shape[-1]]


def _ends(sizes):
    return torch.tensor(np.cumsum(sizes), dtype=torch.int32, device="cuda")


def _close(got, ref, mag, dtype):
    got, ref, mag = got.double().cpu(), ref.cpu(), mag.cpu()
    bound = ROUND[dtype] * ref.abs() + SUM[dtype] * mag + STEP[dtype]
    worst = ((got - ref).abs() - bound).max().item() if ref.numel() else 0.0
    assert worst <= 0.0, f"beyond the bound by {worst}"
    assert not torch.isnan(got).any()


def _forward_ref(x, w, sizes, trans):
    x, w = x.double(), w.double()
    if trans:
        w = w.transpose(1, 2)
    y = torch.zeros(x.shape[0], w.shape[2], dtype=torch.float64, device=x.device)
    mag = torch.zeros_like(y)
    r = 0
    for g, n in enumerate(sizes):
        y[r:r + n] = x[r:r + n] @ w[g]
        mag[r:r + n] = x[r:r + n].abs() @ w[g].abs()
        r += n
    return y, mag


def _grad_ref(x, dy, sizes, trans):
    x, dy = x.double(), dy.double()
    out, mag = [], []
    r = 0
    for n in sizes:
        a, b = x[r:r + n], dy[r:r + n]
        a, b = (b, a) if trans else (a, b)
        out.append(a.t() @ b)
        mag.append(a.t().abs() @ b.abs())
        r += n
    return torch.stack(out), torch.stack(mag)


# Group sizes: one row, none, sizes around the granules (16, 32), the blocks
# (64) and the tiles (128, 256), one group only, a long one beside short ones.
SIZES = [
    [1],
    [0, 1, 0],
    [3, 0, 5, 1, 0, 0, 7, 16],
    [15, 16, 17, 31, 32, 33],
    [63, 64, 65, 0, 127, 128, 129],
    [255, 256, 257, 1],
    [700, 2, 0, 41],
    [2] * 40,
]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("sizes", SIZES, ids=[str(i) for i in range(len(SIZES))])
def test_forward_and_gradients_by_group_sizes(sg, dtype, trans, sizes):
    T, G, K, N = sum(sizes), len(sizes), 200, 328
    x = _rand((T, K), dtype, 1)
    w = _rand((G, N, K) if trans else (G, K, N), dtype, 2)
    dy = _rand((T, N), dtype, 3)
    ends = _ends(sizes)
    y = sg.grouped_gemm(x, w, ends, trans_w=trans)
    _close(y, *_forward_ref(x, w, sizes, trans), dtype)
    dx = sg.grouped_gemm(dy, w, ends, trans_w=not trans)
    _close(dx, *_forward_ref(dy, w, sizes, not trans), dtype)
    dw = sg.grouped_gemm_weight_grad(x, dy, ends, trans_w=trans)
    _close(dw, *_grad_ref(x, dy, sizes, trans), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("K,N,pad", [(1, 1, 0), (7, 5, 0), (63, 65, 1), (64, 64, 0), (65, 129, 3), (256, 8, 8),
                                     (24, 1000, 0), (1001, 77, 0), (520, 513, 0)])
def test_odd_extents_and_pitches(sg, dtype, K, N, pad):
    sizes = [5, 0, 70, 130]
    T, G = sum(sizes), len(sizes)
    x = _rand((T, K), dtype, 4, pad)
    dy = _rand((T, N), dtype, 6, pad)
    ends = _ends(sizes)
    for trans in (False, True):
        w = _rand((G, N, K) if trans else (G, K, N), dtype, 5, pad)
        _close(sg.grouped_gemm(x, w, ends, trans_w=trans), *_forward_ref(x, w, sizes, trans), dtype)
        _close(sg.grouped_gemm_weight_grad(x, dy, ends, trans_w=trans), *_grad_ref(x, dy, sizes, trans), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_outside_every_group(sg, dtype):
    # Rows behind the last end: zero in y, no part in dw, even when they hold
    # infinities and NaN; the rows of the next group take no part either.
    sizes, T, K, N = [37, 0, 50], 300, 96, 136
    x, w, dy = _rand((T, K), dtype, 7), _rand((3, K, N), dtype, 8), _rand((T, N), dtype, 9)
    x[87:], dy[87:] = float("nan"), float("inf")
    ends = _ends(sizes)
    y = sg.grouped_gemm(x, w, ends)
    assert (y[87:] == 0).all()
    _close(y[:87], *_forward_ref(x[:87], w, sizes, False), dtype)
    dw = sg.grouped_gemm_weight_grad(x, dy, ends)
    _close(dw, *_grad_ref(x[:87], dy[:87], sizes, False), dtype)
    x[:87], dy[:87] = 1.0, 1.0
    x[37:87] = float("inf")
    dw = sg.grouped_gemm_weight_grad(x, dy, ends)
    assert (dw[0] == 37).all() and (dw[1] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_integers_are_exact(sg, dtype):
    # Integers up to 4: every product and sum is exact in FP32; sums up to 256
    # are exact in bf16.
    g = torch.Generator().manual_seed(5)
    sizes, K, N = [130, 1, 300, 60], 96, 200
    T = sum(sizes)
    x = torch.randint(-1, 2, (T, K), generator=g).to(DTYPES[dtype]).cuda()
    w = torch.randint(-1, 2, (4, K, N), generator=g).to(DTYPES[dtype]).cuda()
    y = sg.grouped_gemm(x, w, _ends(sizes))
    ref, _ = _forward_ref(x, w, sizes, False)
    assert torch.equal(y.double(), ref)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_long_rows_and_repeated_calls_give_the_same_bits(sg, dtype):
    sizes = [900, 0, 1500, 33]
    T, K, N = sum(sizes), 1024, 640
    x, w, dy = _rand((T, K), dtype, 10), _rand((4, K, N), dtype, 11), _rand((T, N), dtype, 12)
    ends = _ends(sizes)
    y, dw = sg.grouped_gemm(x, w, ends), sg.grouped_gemm_weight_grad(x, dy, ends)
    _close(y, *_forward_ref(x, w, sizes, False), dtype)
    _close(dw, *_grad_ref(x, dy, sizes, False), dtype)
    for _ in range(5):
        assert torch.equal(y, sg.grouped_gemm(x, w, ends))
        assert torch.equal(dw, sg.grouped_gemm_weight_grad(x, dy, ends))


def test_guard_bands_around_the_outputs(sg):
    sizes, K, N = [30, 100, 7], 130, 99
    T = sum(sizes)
    x, w, dy = _rand((T, K), "bf16", 13), _rand((3, K, N), "bf16", 14), _rand((T, N), "bf16", 15)
    ends = _ends(sizes)
    for pad in (5, 29):
        buf = torch.full((T + 4, N + pad), 77.0, dtype=torch.bfloat16, device="cuda")
        sg.grouped_gemm(x, w, ends, out=buf[2:T + 2, :N])
        _close(buf[2:T + 2, :N], *_forward_ref(x, w, sizes, False), "bf16")
        assert (buf[:2] == 77).all() and (buf[T + 2:] == 77).all() and (buf[:, N:] == 77).all()
        buf = torch.full((5, K + 3, N + pad), 77.0, dtype=torch.bfloat16, device="cuda")
        sg.grouped_gemm_weight_grad(x, dy, ends, out=buf[1:4, :K, :N])
        _close(buf[1:4, :K, :N], *_grad_ref(x, dy, sizes, False), "bf16")
        assert (buf[0] == 77).all() and (buf[4] == 77).all() and (buf[:, K:] == 77).all() and \
            (buf[:, :, N:] == 77).all()


def test_empty_problems(sg):
    ends = _ends([0, 0])
    x, w = _rand((0, 8), "bf16", 1), _rand((2, 8, 16), "bf16", 2)
    assert sg.grouped_gemm(x, w, ends).shape == (0, 16)
    assert (sg.grouped_gemm_weight_grad(x, _rand((0, 16), "bf16", 1), ends) == 0).all()
    x = _rand((4, 0), "bf16", 1)
    y = sg.grouped_gemm(x, torch.zeros(2, 0, 16, dtype=torch.bfloat16, device="cuda"), _ends([2, 2]))
    assert (y == 0).all()
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    y = sg.grouped_gemm(_rand((4, 8), "bf16", 1), torch.zeros(0, 8, 16, dtype=torch.bfloat16, device="cuda"), none)
    assert (y == 0).all()


def test_ends_out_of_order_are_reported_and_stay_in_bounds(sg):
    h = sg.Handle()
    x, w = _rand((64, 32), "bf16", 1), _rand((3, 32, 40), "bf16", 2)
    for bad in ([40, 20, 64], [-5, 10, 64], [10, 20, 900]):
        buf = torch.full((70, 40), 3.0, dtype=torch.bfloat16, device="cuda")
        sg.grouped_gemm(x, w, torch.tensor(bad, dtype=torch.int32, device="cuda"), out=buf[3:67], handle=h)
        assert h.device_error() >> 24 == 6
        assert (buf[:3] == 3).all() and (buf[67:] == 3).all()
    sg.grouped_gemm(x, w, _ends([10, 0, 54]), handle=h)
    assert h.device_error() == 0
    h.close()


def test_gradients_against_differences(sg):
    # <dy, y(x + s u) - y(x - s u)> / 2s = <dx, u>; the product is linear, so
    # the step only has to keep FP32's rounding small.
    sizes, K, N = [20, 0, 45], 64, 72
    T = sum(sizes)
    x, w, dy = _rand((T, K), "f32", 21), _rand((3, K, N), "f32", 22), _rand((T, N), "f32", 23)
    u, v = _rand((T, K), "f32", 24), _rand((3, K, N), "f32", 25)
    ends = _ends(sizes)
    dx = sg.grouped_gemm(dy, w, ends, trans_w=True)
    dw = sg.grouped_gemm_weight_grad(x, dy, ends)

    def along(xp, wp, xm, wm):
        d = sg.grouped_gemm(xp, wp, ends).double() - sg.grouped_gemm(xm, wm, ends).double()
        return (d * dy.double()).sum().item() / 2
    scale = T * N * K ** 0.5
    assert abs(along(x + u, w, x - u, w) - (dx.double() * u.double()).sum().item()) <= 1e-5 * scale
    assert abs(along(x, w + v, x, w - v) - (dw.double() * v.double()).sum().item()) <= 1e-5 * scale


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("K,N", [(4100, 72), (1537, 129), (8192, 256)])
@pytest.mark.parametrize("sizes", [[1], [0, 2, 0, 3, 0], [5, 40]], ids=["1", "2-3", "5-40"])
def test_few_rows_of_a_long_contraction(sg, dtype, trans, K, N, sizes):
    # (Cut along the contraction and joined.)  Two rows behind the last end.
    n = sum(sizes)
    x = _rand((n + 2, K), dtype, 40, pitch_pad=3)
    w = _rand((len(sizes), N, K) if trans else (len(sizes), K, N), dtype, 41)
    out = torch.full((n + 2, N + 5), 7.0, device="cuda").to(DTYPES[dtype])
    y = sg.grouped_gemm(x, w, _ends(sizes), trans_w=trans, out=out[:, :N])
    ref, mag = _forward_ref(x[:n], w, sizes, trans)
    _close(y[:n], ref, mag, dtype)
    assert (y[n:] == 0).all() and (out[:, N:] == 7.0).all()
    assert torch.equal(y, sg.grouped_gemm(x, w, _ends(sizes), trans_w=trans))


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("K", [256, 259, 2048, 2053])
@pytest.mark.parametrize("N", [1, 31, 100, 130])
def test_few_f32_rows(sg, trans, K, N):
    # Up to eight rows a group in the mean: groups around eight rows, NaN in
    # the rows behind the last end and in the matrices of empty groups.
    sizes = [8, 0, 1, 9, 17, 3, 0]
    n = sum(sizes)
    x = _rand((n + 3, K), "f32", 50)
    w = _rand((len(sizes), N, K) if trans else (len(sizes), K, N), "f32", 51)
    ref, mag = _forward_ref(x[:n], w, sizes, trans)
    x[n:], w[1], w[6] = float("nan"), float("nan"), float("nan")
    out = torch.full((n + 3, N + 2), 7.0, device="cuda")
    y = sg.grouped_gemm(x, w, _ends(sizes), trans_w=trans, out=out[:, :N])
    _close(y[:n], ref, mag, "f32")
    assert (y[n:] == 0).all() and (out[:, N:] == 7.0).all()
    ends = _ends(sizes)
    h = sg.Handle()
    ends[2] = 4                                      # runs backwards
    sg.grouped_gemm(x, w, ends, trans_w=trans, out=out[:, :N], handle=h)
    assert h.device_error() >> 24 == 6 and (out[:, N:] == 7.0).all()


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_matrices_without_rows_are_not_read(sg, dtype, trans):
    # Odd pitches, so that the matrices are copied first; those of groups
    # without a row hold NaN, and so does the workspace from an earlier call.
    g = torch.Generator(device="cuda").manual_seed(31)
    K, N, G = 77, 53, 9
    x = torch.randn(40, K, generator=g, device="cuda").to(DTYPES[dtype])
    w = torch.randn(*((G, N, K) if trans else (G, K, N)), generator=g, device="cuda").to(DTYPES[dtype])
    ends = torch.tensor([0, 13, 13, 13, 20, 20, 40, 40, 40], dtype=torch.int32, device="cuda")
    bad = w.clone()
    for i in (0, 2, 3, 5, 7, 8):
        bad[i] = float("nan")
    want = sg.grouped_gemm(x, w, ends, trans_w=trans)
    sg.grouped_gemm(x, torch.full_like(w, float("nan")), torch.arange(1, G + 1, dtype=torch.int32, device="cuda"),
                    trans_w=trans)
    got = sg.grouped_gemm(x, bad, ends, trans_w=trans)
    assert torch.isfinite(want).all() and torch.equal(want, got)


def test_other_stream(sg):
    sizes, K, N = [100, 28], 256, 512
    x, w = _rand((128, K), "bf16", 31), _rand((2, K, N), "bf16", 32)
    ends = _ends(sizes)
    h, s = sg.Handle(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y = sg.grouped_gemm(x, w, ends, handle=h)
    torch.cuda.current_stream().wait_stream(s)
    _close(y, *_forward_ref(x, w, sizes, False), "bf16")
    assert h.device_error() == 0
    h.close()


def test_graph_capture_with_new_groups(sg):
    K, N = 128, 256
    x, w = _rand((96, K), "bf16", 41), _rand((3, K, N), "bf16", 42)
    ends = _ends([32, 32, 32])
    out = torch.empty(96, N, dtype=torch.bfloat16, device="cuda")
    h = sg.Handle()
    sg.grouped_gemm(x, w, ends, out=out, handle=h)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sg.grouped_gemm(x, w, ends, out=out, handle=h)
    for sizes in ([32, 32, 32], [0, 96, 0], [1, 2, 93]):
        ends.copy_(_ends(sizes))
        graph.replay()
        torch.cuda.synchronize()
        _close(out, *_forward_ref(x, w, sizes, False), "bf16")
    h.close()


def test_refusals(sg):
    x, w, ends = _rand((8, 16), "bf16", 1), _rand((2, 16, 24), "bf16", 2), _ends([4, 4])
    with pytest.raises(TypeError):
        sg.grouped_gemm(x.double(), w, ends)
    with pytest.raises(TypeError):
        sg.grouped_gemm(x, w.half(), ends)
    with pytest.raises(TypeError):
        sg.grouped_gemm(x, w, ends.long())
    with pytest.raises(ValueError):
        sg.grouped_gemm(x, w, ends, trans_w=True)
    with pytest.raises(ValueError):
        sg.grouped_gemm(x, w, ends[:1])
    with pytest.raises(ValueError):
        sg.grouped_gemm(x.t(), w, ends)
    with pytest.raises(ValueError):
        sg.grouped_gemm(x, w[:1].expand(2, 16, 24), ends)
    with pytest.raises(ValueError):
        sg.grouped_gemm(x.cpu(), w, ends)
    with pytest.raises(ValueError):
        sg.grouped_gemm_weight_grad(x, _rand((9, 24), "bf16", 3), ends)
    with pytest.raises(sg.SgemmError):
        n = 1025
        sg.grouped_gemm(x, torch.zeros(n, 16, 8, dtype=torch.bfloat16, device="cuda"),
                        torch.full((n,), 8, dtype=torch.int32, device="cuda"))
