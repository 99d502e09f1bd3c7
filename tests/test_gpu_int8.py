"""Products in 8-bit integers with scales for each token and channel: bit for
bit against the definition (the sum of integers is exact, what follows are three
FP32 operations), at the sizes where it can go wrong."""
import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

F32, F16, BF16, S8 = torch.float32, torch.float16, torch.bfloat16, torch.int8
TYPES = pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=["f32", "f16", "bf16"])


@pytest.fixture(scope="module")
def sg():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import fp32_sgemm_gb300 as m
    m.build()
    m.load_library()
    return m


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(*shape, seed, dtype=F32):
    return torch.randn(*shape, generator=_gen(seed), device="cuda").to(dtype)


def _ints(*shape, seed, low=-128):
    return torch.randint(low, 128, shape, generator=_gen(seed), device="cuda", dtype=S8)


def _scales(*shape, seed):
    return torch.rand(*shape, generator=_gen(seed), device="cuda") * 0.01 + 0.001


def _quantized(x):
    """(q, s) from the definition: the scale rounded to FP32, the quotient's
    rounding in 64 bits, where it is on the right side of every tie."""
    x = x.double()
    most = x.abs().amax(1) if x.shape[1] else x.new_zeros(x.shape[0])
    good = most < math.inf
    s = (most / 127.0).float()
    s = torch.where(most > 0, s.clamp(min=2.0 ** -126), s)
    q = torch.where(good[:, None], x / torch.where(s > 0, s, 1.0).double()[:, None], 0.0).round().clamp(-127, 127)
    return q.to(S8), torch.where(good, s, math.nan)


def _product(q, xs, w, ws, dtype):
    """q [T, K] against w [N, K]: an exact sum (below 2^53 in 64 bits), then as
    the contract says."""
    total = (q.double() @ w.double().t()).to(torch.int64)
    return (total.float() * xs[:, None] * ws).to(dtype)


def _same(a, b):
    return a.dtype == b.dtype and a.shape == b.shape and torch.equal(torch.nan_to_num(a), torch.nan_to_num(b)) and \
        torch.equal(a.isnan(), b.isnan())


# ------------------------------------------------------------------ quantise

@TYPES
@pytest.mark.parametrize("T,K", [(1, 1), (3, 7), (1, 4096), (40, 255), (17, 1001), (5, 8192), (2, 16385), (3, 40000),
                                 (600, 64)])
def test_quantize(sg, dtype, T, K):
    x = _randn(T, K, seed=T + K, dtype=dtype)
    q, s = sg.int8_quantize(x)
    want, scales = _quantized(x)
    assert torch.equal(s, scales) and torch.equal(q, want)


@TYPES
def test_quantize_ties_and_extremes(sg, dtype):
    # Multiples of half a scale of 2^-k: ties that go to the even neighbour, and
    # the numbers beside them.
    info = torch.finfo(dtype)
    half = torch.arange(-254, 255, device="cuda", dtype=torch.float64) / 2
    rows = []
    for scale in (1.0, 2.0 ** -7, 0.25):
        v = (half * scale).to(dtype)
        v[0], v[-1] = -127 * scale, 127 * scale
        rows += [v, torch.nextafter(v.float(), torch.full_like(v.float(), math.inf)).to(dtype)]
        rows[-1][0] = -127 * scale
    rows.append(torch.zeros_like(rows[0]))
    tiny = torch.zeros_like(rows[0])
    tiny[3] = info.smallest_normal * info.eps          # the type's least number
    tiny[5] = -tiny[3]
    rows.append(tiny)
    huge = torch.full_like(rows[0], info.max)
    huge[::2] = info.min
    huge[7] = info.max / 3
    rows.append(huge)
    x = torch.stack(rows)
    q, s = sg.int8_quantize(x)
    want, scales = _quantized(x)
    assert torch.equal(s, scales) and torch.equal(q, want)
    assert (s[-3] == 0) and (q[-3] == 0).all()


def test_quantize_every_rounding(sg):
    # Scales whose quotients come close to ties: FP32 numbers at and around
    # every (n + 1/2) s.
    g = _gen(5)
    most = torch.rand(64, generator=g, device="cuda") + 0.5
    s = (most.double() / 127).float()
    n = torch.arange(-127, 127, device="cuda").double() + 0.5
    x = (s.double()[:, None] * n).float()
    x = torch.cat([x, torch.nextafter(x, torch.zeros_like(x)), torch.nextafter(x, x * 2), most[:, None]], 1)
    x = x.clamp(-most[:, None], most[:, None])
    q, got = sg.int8_quantize(x)
    want, scales = _quantized(x)
    assert torch.equal(got, scales) and torch.equal(q, want)


@TYPES
def test_quantize_rows_that_are_not_finite(sg, dtype):
    x = _randn(6, 333, seed=1, dtype=dtype)
    x[1, 17], x[3, 332], x[4, 0] = math.inf, math.nan, -math.inf
    q, s = sg.int8_quantize(x)
    want, scales = _quantized(x)
    assert s.isnan().tolist() == [False, True, False, True, True, False]
    assert _same(s, scales) and torch.equal(q, want)
    y = sg.int8_gemm(x, _ints(70, 333, seed=2), _scales(70, seed=3))
    assert y.isnan().all(1).tolist() == s.isnan().tolist() and y[0].isfinite().all()


@TYPES
def test_quantize_pitches(sg, dtype):
    wide = _randn(20, 400, seed=2, dtype=dtype)
    wide[:, 300:] = math.nan
    for a, n in ((0, 300), (1, 299), (8, 250), (3, 64)):
        x = wide[:, a:a + n]
        for u, v in zip(sg.int8_quantize(x), _quantized(x)):
            assert torch.equal(u, v)


# ------------------------------------------------------------------ products

SIZES = [(1, 1, 1), (1, 16, 64), (1, 4096, 512), (2, 33, 100), (5, 100, 1024), (8, 17, 4097), (9, 50, 300),
         (16, 1000, 256), (17, 40, 130), (16, 31, 20000), (1, 70, 70001), (40, 257, 129), (100, 513, 1025),
         (33, 1, 64), (200, 700, 2048), (700, 300, 3000), (193, 255, 127), (1000, 129, 16), (3, 3000, 1000)]


@TYPES
@pytest.mark.parametrize("T,N,K", SIZES)
def test_products(sg, dtype, T, N, K):
    x, w, ws = _randn(T, K, seed=T + N, dtype=dtype), _ints(N, K, seed=N + K), _scales(N, seed=K)
    q, s = _quantized(x)
    assert _same(sg.int8_gemm(x, w, ws), _product(q, s, w, ws, dtype))
    # Of integers, the lowest one among them.
    q = _ints(T, K, seed=T + K)
    xs = _scales(T, seed=T)
    assert _same(sg.int8_gemm(q, w, ws, x_scales=xs, dtype=dtype), _product(q, xs, w, ws, dtype))


@pytest.mark.parametrize("T", [1, 12, 100, 300])
@pytest.mark.parametrize("K", [1023, 1024, 1025, 8192, 16384, 131071])
def test_largest_sums(sg, T, K):
    # Every product as large as it can be and odd ones between: sums of one sign
    # that fill an accumulator to 2^24 and the 32-bit sum to 2^31 - 2^14.
    N = 70
    for fill in (-128, 127):
        q = torch.full((T, K), fill, dtype=S8, device="cuda")
        w = torch.full((N, K), fill, dtype=S8, device="cuda")
        q[:, ::7] = 127 if fill == 127 else -127
        w[::2, ::3] = -1
        w[::3] = fill
        one = torch.ones(T, device="cuda"), torch.ones(N, device="cuda")
        got = sg.int8_gemm(q, w, one[1], x_scales=one[0], dtype=F32)
        assert torch.equal(got, _product(q, one[0], w, one[1], F32))
    with pytest.raises(sg.SgemmError):
        sg.int8_gemm(torch.ones(T, 131072, device="cuda"), torch.ones(2, 131072, dtype=S8, device="cuda"), one[1][:2])


GROUPS = [([3, 0, 5], 64, 100), ([1, 1, 1, 1], 200, 512), ([0, 0, 7, 0], 33, 70), ([40, 1, 0, 90, 17], 130, 257),
          ([300, 200], 300, 1100), ([0, 0, 0], 20, 64), ([5, 700, 0, 3], 257, 515), ([16, 16, 16], 48, 6000),
          ([1] * 60 + [0] * 4, 96, 1024), ([2, 0] * 500, 17, 80)]


@TYPES
@pytest.mark.parametrize("sizes,N,K", GROUPS, ids=lambda v: None)
@pytest.mark.parametrize("behind", [0, 11])
def test_groups(sg, dtype, sizes, N, K, behind):
    T, G = sum(sizes) + behind, len(sizes)
    if T == 0:
        T = behind = 5
    ends = torch.tensor(sizes, device="cuda").cumsum(0).to(torch.int32)
    x, w, ws = _randn(T, K, seed=1, dtype=dtype), _ints(G, N, K, seed=2), _scales(G, N, seed=3)
    if behind:
        x[-behind:] = math.nan                        # (rows behind the last end take no part)
    q, s = _quantized(x)
    want = torch.zeros(T, N, dtype=dtype, device="cuda")
    a = 0
    for g, n in enumerate(sizes):
        want[a:a + n] = _product(q[a:a + n], s[a:a + n], w[g], ws[g], dtype)
        a += n
    assert _same(sg.int8_grouped_gemm(x, w, ws, ends), want)
    q, s = sg.int8_quantize(x)
    assert _same(sg.int8_grouped_gemm(q, w, ws, ends, x_scales=s, dtype=dtype), want)


@pytest.mark.parametrize("T", [2, 30, 300])
def test_pitches_and_odd_bases(sg, T):
    N, K, G = 90, 260, 3
    ends = torch.tensor([T // 2, T // 2, T], dtype=torch.int32, device="cuda")
    x, w, ws = _randn(T, K, seed=1, dtype=BF16), _ints(G, N, K, seed=2), _scales(G, N, seed=3)
    want = sg.int8_grouped_gemm(x, w, ws, ends)
    q, s = sg.int8_quantize(x)
    for a, pitch in ((0, 272), (1, 263), (4, 288), (16, 320), (3, 261 + 3)):
        xw = torch.full((T, pitch + 20), math.nan, dtype=BF16, device="cuda")[:, a:a + K]
        xw.copy_(x)
        ww = torch.full((G * N * pitch + 64,), 99, dtype=S8, device="cuda")[a:].as_strided((G, N, K), (N * pitch, pitch, 1))
        ww.copy_(w)
        qw = torch.full((T, pitch + 20), 99, dtype=S8, device="cuda")[:, a:a + K]
        qw.copy_(q)
        guard = torch.full((T + 2, N + 30), 7.0, dtype=BF16, device="cuda")
        out = guard[1:-1, a:a + N]
        assert _same(sg.int8_grouped_gemm(xw, ww, ws, ends, out=out), want)
        out.fill_(7.0)
        assert (guard == 7.0).all()
        assert _same(sg.int8_grouped_gemm(qw, ww, ws, ends, x_scales=s, dtype=BF16), want)
        # One matrix, of the last group.
        assert _same(sg.int8_gemm(xw, ww[2], ws[2]), sg.int8_gemm(x, w[2], ws[2]))


def test_ends_out_of_order_are_recorded(sg):
    h = sg.Handle()
    w, ws = _ints(3, 40, 128, seed=1), _scales(3, 40, seed=2)
    for T in (9, 400):
        x = _randn(T, 128, seed=3)
        guard = torch.full((T + 2, 40), 7.0, device="cuda")
        sg.int8_grouped_gemm(x, w, ws, torch.tensor([T, 2, T + 90], dtype=torch.int32, device="cuda"), out=guard[1:-1],
                             handle=h)
        assert h.device_error() >> 24 == 6
        assert (guard[0] == 7).all() and (guard[-1] == 7).all()
    h.close()


def test_sizes_of_zero(sg):
    def z(*shape, dtype=F32):
        return torch.zeros(*shape, dtype=dtype, device="cuda")
    assert sg.int8_gemm(z(0, 16), z(8, 16, dtype=S8), z(8)).shape == (0, 8)
    assert sg.int8_gemm(z(5, 16), z(0, 16, dtype=S8), z(0)).shape == (5, 0)
    out = torch.full((5, 8), 7.0, device="cuda")
    sg.int8_gemm(z(5, 0), z(8, 0, dtype=S8), z(8), out=out)
    assert (out == 0).all()
    out.fill_(7.0)
    sg.int8_grouped_gemm(z(5, 16), z(0, 8, 16, dtype=S8), z(0, 8), z(0, dtype=torch.int32), out=out)
    assert (out == 0).all()
    q, s = sg.int8_quantize(z(0, 16))
    assert q.shape == (0, 16) and s.shape == (0,)
    q, s = sg.int8_quantize(z(4, 0))
    assert q.shape == (4, 0) and s.tolist() == [0] * 4


# --------------------------------------------------------------- refusals

def test_refusals(sg):
    x, w, ws = torch.zeros(4, 64, device="cuda"), torch.zeros(8, 64, dtype=S8, device="cuda"), torch.ones(8, device="cuda")
    q, xs = w[:4], ws[:4]
    ends = torch.tensor([4], dtype=torch.int32, device="cuda")
    bad = [
        (TypeError, lambda: sg.int8_gemm(x.double(), w, ws)),
        (TypeError, lambda: sg.int8_gemm(q, w, ws)),                                  # integers without scales
        (TypeError, lambda: sg.int8_gemm(x, w, ws, x_scales=xs)),                     # scales without integers
        (TypeError, lambda: sg.int8_gemm(q, w, ws, x_scales=xs)),                     # without a type
        (TypeError, lambda: sg.int8_gemm(q, w, ws, x_scales=xs, dtype=torch.float64)),
        (TypeError, lambda: sg.int8_gemm(q, w, ws, x_scales=xs, dtype="bf16")),
        (ValueError, lambda: sg.int8_gemm(q, w, ws, x_scales=xs[:3], dtype=F32)),
        (TypeError, lambda: sg.int8_gemm(q, w, ws, x_scales=xs.half(), dtype=F32)),
        (TypeError, lambda: sg.int8_gemm(x, w.to(torch.uint8), ws)),
        (TypeError, lambda: sg.int8_gemm(x, w, ws.half())),
        (ValueError, lambda: sg.int8_gemm(x, w, ws[:7])),
        (ValueError, lambda: sg.int8_gemm(x, w[:, :63], ws)),
        (ValueError, lambda: sg.int8_gemm(x, w.t(), ws)),
        (ValueError, lambda: sg.int8_gemm(x, w[:1].expand(8, 64), ws)),
        (ValueError, lambda: sg.int8_gemm(x[:1].expand(4, 64), w, ws)),
        (ValueError, lambda: sg.int8_gemm(x, w, ws, out=torch.zeros(4, 9, device="cuda"))),
        (TypeError, lambda: sg.int8_gemm(x, w, ws, dtype=F16, out=torch.zeros(4, 8, device="cuda"))),
        (ValueError, lambda: sg.int8_gemm(x.cpu(), w, ws)),
        (ValueError, lambda: sg.int8_gemm(x, w.cpu(), ws)),
        (ValueError, lambda: sg.int8_grouped_gemm(x, w, ws, ends)),
        (ValueError, lambda: sg.int8_grouped_gemm(x, w[None], ws, ends)),
        (TypeError, lambda: sg.int8_grouped_gemm(x, w[None], ws[None], ends.long())),
        (TypeError, lambda: sg.int8_grouped_gemm(x, w[None], ws[None], None)),
        (TypeError, lambda: sg.int8_quantize(q)),
        (ValueError, lambda: sg.int8_quantize(x[0])),
    ]
    for i, (error, call) in enumerate(bad):
        with pytest.raises(error):
            call()
            pytest.fail(f"call {i} was taken")


def test_no_gradient(sg):
    x, w, ws = _randn(4, 64, seed=1), _ints(8, 64, seed=2), _scales(8, seed=3)
    want = sg.int8_gemm(x, w, ws)
    y = sg.int8_gemm(x.clone().requires_grad_(), w, ws)
    assert torch.equal(y.detach(), want)
    with pytest.raises(NotImplementedError):
        y.sum().backward()
    ends = torch.tensor([4], dtype=torch.int32, device="cuda")
    y = sg.int8_grouped_gemm(x, w[None], ws[None].clone().requires_grad_(), ends)
    with pytest.raises(NotImplementedError):
        y.sum().backward()


# ------------------------------------------------------- graphs and streams

def test_captured_and_on_other_streams(sg):
    def work(seed, T):
        x, w, ws = _randn(T, 1000, seed=seed, dtype=BF16), _ints(4, 300, 1000, seed=seed + 1), _scales(4, 300, seed=seed + 2)
        ends = torch.tensor([T // 4, T // 4, T // 2, T - 1], dtype=torch.int32, device="cuda")

        def run(**kw):
            q, s = sg.int8_quantize(x, **kw)
            return [q, s, sg.int8_grouped_gemm(x, w, ws, ends, **kw), sg.int8_gemm(x, w[0], ws[0], **kw),
                    sg.int8_gemm(q, w[1], ws[1], x_scales=s, dtype=F16, **kw)]
        return x, run
    jobs = [work(10 * i, T) for i, T in enumerate((4, 60, 500))]
    want = [run() for _, run in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    got = []
    for _ in range(5):
        for (_, run), s in zip(jobs, streams):
            with torch.cuda.stream(s):
                got.append(run())
        for (_, run), s in zip(jobs, streams):
            got.append(run(stream=s))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[i % 3]))
    for x, run in jobs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = run()
        for seed in (71, 72):
            x.copy_(_randn(*x.shape, seed=seed))
            fresh = run()
            graph.replay()
            assert all(torch.equal(a, b) for a, b in zip(out, fresh))


def test_served_experts(sg):
    """An expert layer in 8 bits as it is served: routing, dispatch, products,
    the way back, against the same steps in 64 bits on the quantised weights."""
    D, H, G, k = 96, 160, 8, 2
    up, down, router = _randn(G, H, D, seed=1) * 0.1, _randn(G, D, H, seed=2) * 0.1, _randn(G, D, seed=3)
    (uq, us), (dq, ds) = [sg.int8_quantize(m.view(-1, m.shape[2])) for m in (up, down)]
    uq, us, dq, ds = uq.view(G, H, D), us.view(G, H), dq.view(G, D, H), ds.view(G, D)
    for T in (1, 16, 900):
        x = _randn(T, D, seed=T)
        weights, experts = sg.route_topk(x @ router.t(), k)
        rows, slots, ends = sg.expert_dispatch(x, experts, G)
        h = torch.relu(sg.int8_grouped_gemm(rows, uq, us, ends))
        y = sg.expert_combine(sg.int8_grouped_gemm(h, dq, ds, ends), slots, weights)
        exact = torch.zeros(T, D, dtype=torch.float64, device="cuda")
        for j in range(k):
            e = experts[:, j]
            u = torch.einsum("td,thd->th", x.double(), (uq.double() * us.double()[:, :, None])[e]).relu()
            exact += weights[:, j:j + 1].double() * torch.einsum("th,tdh->td", u, (dq.double() * ds.double()[:, :, None])[e])
        # Each row in 8 bits twice: half a step of 1/127 of its largest entry
        # (below 5 of its root mean square), spread evenly: 5 / 254 / sqrt(3).
        assert (y.double() - exact).norm() <= 2 * 5 / 254 / math.sqrt(3) * exact.norm()
