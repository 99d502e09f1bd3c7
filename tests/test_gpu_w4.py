"""Products with 4-bit weights against the definition in 64 bits.

Bound: q - zero and x are exact in the product, so what is left is FP32
summation (K / 16 steps of the tensor core, which truncates, then one scaled
addition per group): 2^-20 of sum |s (q - z) x| at these lengths, and one
rounding to the type (eps / 2, f16 at least 2^-25).
"""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
ROUND = {name: torch.finfo(t).eps / 2 for name, t in DTYPES.items()}
STEP = {"bf16": 0.0, "f16": 2.0 ** -25, "f32": 0.0}


@pytest.fixture(scope="module")
def sg():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import fp32_sgemm_gb300 as m
    m.build()
    m.load_library()
    return m


def _problem(M, N, K, group, dtype, zeros, seed=1, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(M, K + pad, generator=g, device="cuda").to(DTYPES[dtype])[:, :K]
    q = torch.randint(0, 256, (N, K // 2 + 16 * pad), generator=g, device="cuda", dtype=torch.uint8)[:, :K // 2]
    s = (torch.randn(N, K // group + pad, generator=g, device="cuda") * 0.02).to(DTYPES[dtype])[:, :K // group]
    z = torch.randint(0, 16, (N, K // group + pad), generator=g, device="cuda",
                      dtype=torch.uint8)[:, :K // group] if zeros else None
    return x, q, s, z


def _weights(q, s, z, group):
    N, half = q.shape
    v = torch.empty(N, 2 * half, dtype=torch.float64, device=q.device)
    v[:, 0::2] = (q % 16).double()
    v[:, 1::2] = (q // 16).double()
    v -= z.double().repeat_interleave(group, 1) if z is not None else 8.0
    return v * s.double().repeat_interleave(group, 1)


def _check(got, x, q, s, z, group, dtype):
    w = _weights(q, s, z, group)
    ref = x.double() @ w.t()
    bound = ROUND[dtype] * ref.abs() + 2.0 ** -20 * (x.double().abs() @ w.abs().t()) * (1 + ROUND[dtype]) + STEP[dtype]
    worst = ((got.double() - ref).abs() - bound).max().item()
    assert worst <= 0, f"beyond the bound by {worst}"


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M", [1, 2, 3, 7, 8, 9, 16, 17, 32, 33, 70])
def test_rows_and_groups(sg, dtype, group, M):
    for zeros in (False, True):
        x, q, s, z = _problem(M, 200, 1024, group, dtype, zeros)
        _check(sg.w4_gemm(x, q, s, z), x, q, s, z, group, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("N,K,group", [(1, 32, 32), (1, 128, 128), (15, 64, 32), (16, 96, 32), (17, 160, 32),
                                       (33, 64, 64), (100, 192, 64), (257, 1056, 32), (31, 1152, 128),
                                       (5000, 256, 128), (48, 20480, 64), (3, 65536, 128)])
def test_odd_extents(sg, dtype, N, K, group):
    for M in (1, 5):
        x, q, s, z = _problem(M, N, K, group, dtype, True, seed=N)
        _check(sg.w4_gemm(x, q, s, z), x, q, s, z, group, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_pitches_and_guard_bands(sg, dtype):
    x, q, s, z = _problem(4, 70, 288, 32, dtype, True, pad=3)
    buf = torch.full((6, 80), 5.0, dtype=DTYPES[dtype], device="cuda")
    sg.w4_gemm(x, q, s, z, out=buf[1:5, 2:72])
    _check(buf[1:5, 2:72], x, q, s, z, 32, dtype)
    assert (buf[0] == 5).all() and (buf[5] == 5).all() and (buf[:, :2] == 5).all() and (buf[:, 72:] == 5).all()


def test_every_nibble_in_every_place(sg):
    # Row n holds nibble n in one column at a time: the layout, exactly.
    K = 128
    q = torch.zeros(16, K // 2, dtype=torch.uint8, device="cuda")
    for n in range(16):
        q[n] = n * 17
    s = torch.ones(16, 1, dtype=torch.bfloat16, device="cuda")
    z = torch.zeros(16, 1, dtype=torch.uint8, device="cuda")
    x = torch.zeros(K, K, dtype=torch.bfloat16, device="cuda")
    x.fill_diagonal_(1.0)
    want = torch.arange(16, device="cuda").repeat(K, 1).to(torch.bfloat16)
    assert torch.equal(sg.w4_gemm(x, q, s, z), want)
    q[:, 0::2] &= 0x0F          # odd columns of every second byte to zero
    want[1::4] = 0
    assert torch.equal(sg.w4_gemm(x, q, s, z), want)
    assert torch.equal(sg.w4_gemm(x, q, s), want - 8)


def test_not_finite_values_stay_in_their_rows(sg):
    for dtype in ("bf16", "f16", "f32"):
        x, q, s, z = _problem(3, 40, 256, 64, dtype, False)
        y = sg.w4_gemm(x, q, s, z)
        x2 = x.clone()
        x2[1, 5] = float("nan")
        y2 = sg.w4_gemm(x2, q, s, z)
        assert torch.isnan(y2[1]).all()
        assert torch.equal(y2[0], y[0]) and torch.equal(y2[2], y[2])


def test_same_bits_and_graph(sg):
    x, q, s, z = _problem(6, 3000, 4096, 128, "bf16", True)
    h = sg.Handle()
    y = sg.w4_gemm(x, q, s, z, handle=h)
    out = torch.empty_like(y)
    sg.w4_gemm(x, q, s, z, out=out, handle=h)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sg.w4_gemm(x, q, s, z, out=out, handle=h)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, y)
    h.close()


def test_empty(sg):
    x, q, s, _ = _problem(4, 8, 64, 32, "bf16", False)
    assert sg.w4_gemm(x[:0], q, s).shape == (0, 8)
    assert sg.w4_gemm(x, q[:0], s[:0]).shape == (4, 0)
    assert (sg.w4_gemm(x[:, :0], q[:, :0], s[:, :0]) == 0).all()


def test_refusals(sg):
    x, q, s, z = _problem(4, 8, 64, 32, "bf16", True)
    with pytest.raises(TypeError):
        sg.w4_gemm(x, q.int(), s)
    with pytest.raises(TypeError):
        sg.w4_gemm(x, q, s.float())
    with pytest.raises(TypeError):
        sg.w4_gemm(x, q, s, z.int())
    with pytest.raises(ValueError):
        sg.w4_gemm(x, q[:, :16], s)
    with pytest.raises(ValueError):
        sg.w4_gemm(x, q, s[:4])
    with pytest.raises(ValueError):
        sg.w4_gemm(x, q, s, z[:, :1])
    with pytest.raises(sg.SgemmError):
        sg.w4_gemm(x, q, s.repeat(1, 2))             # groups of 16
    with pytest.raises(sg.SgemmError):
        buf = torch.zeros(8 * 32 + 1, dtype=torch.uint8, device="cuda")
        sg.w4_gemm(x, buf[1:].view(8, 32), s)        # not 16-byte aligned
