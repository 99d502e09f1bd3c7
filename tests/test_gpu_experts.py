"""A router's choice, tokens sorted by expert and back, and their gradients:
against plain implementations in 64 bits, at the sizes and masks where they can
go wrong."""
import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
TYPES = pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=["f32", "f16", "bf16"])


@pytest.fixture(scope="module")
def sg():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import fp32_sgemm_gb300 as m
    m.build()
    m.load_library()
    return m


def _randn(*shape, seed, dtype=F32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def _half_step(v, dtype):
    """Half a unit in the last place of v in dtype, or of its smallest number."""
    info = torch.finfo(dtype)
    return v.abs() * (info.eps / 2) + info.smallest_normal * info.eps


# ------------------------------------------------------------------- router

def _route(logits, k, normalize):
    """(weights, experts, p over all experts as the weights see it, chosen) in 64 bits."""
    l = logits.double()
    order = torch.sort(l, dim=1, descending=True, stable=True)
    top, idx = order.values[:, :k], order.indices[:, :k]
    live = top > -math.inf
    experts = torch.where(live, idx, -1)
    taken = torch.zeros_like(l, dtype=torch.bool).scatter_(1, idx, live)
    most = l.amax(1, keepdim=True)
    power = (l - torch.where(most > -math.inf, most, 0.0)).exp()
    if normalize:
        power = power * taken
    total = power.sum(1, keepdim=True)
    p = power / torch.where(total > 0, total, 1.0)
    return torch.where(live, p.gather(1, idx), 0.0), experts, p, taken


def _check_route(sg, logits, k, normalize):
    """FP32 arithmetic of the weights: exp within 2 units and a rounded argument
    d = l - max (|d| units), the sum of E terms in at most 32 + 5 roundings and
    its arguments' sum_e p_e |d_e| <= log E <= 7 units, one division: below
    64 + |d| units of 2^-24 (twice for a weight and a sum)."""
    weights, experts = sg.route_topk(logits, k, normalize=normalize)
    want, want_experts, p, taken = _route(logits, k, normalize)
    assert weights.dtype == F32 and experts.dtype == torch.int64
    assert torch.equal(experts, want_experts)
    l = logits.double()
    most = l.amax(1, keepdim=True)
    d = torch.where(l > -math.inf, (l - most).abs(), 0.0)
    unit = (64.0 + d) * 2.0 ** -24
    at = experts.clamp(min=0)
    assert ((weights.double() - want).abs() <= want * unit.gather(1, at) + 2.0 ** -126).all()
    dweights = _randn(*weights.shape, seed=9)
    got = sg.route_topk_grad(logits, experts, dweights, normalize=normalize)
    assert got.dtype == logits.dtype and got.shape == logits.shape
    g = torch.zeros_like(l)
    g.scatter_add_(1, at, torch.where(experts >= 0, dweights.double(), 0.0))
    mean = (p * g).sum(1, keepdim=True)
    ref = p * (g - mean)
    # Weights twice in a product, k terms of the mean.
    terms = p * (g.abs() + (p * g.abs()).sum(1, keepdim=True))
    tol = (2 * unit + (k + 16) * 2.0 ** -24) * terms + 2.0 ** -120
    assert ((got.double() - ref).abs() <= tol + _half_step(ref.abs() + tol, logits.dtype)).all()
    assert (got[~taken] == 0).all() if normalize else (got[l == -math.inf] == 0).all()


@TYPES
@pytest.mark.parametrize("normalize", [True, False], ids=["normalized", "all"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 64, 2), (7, 3, 3), (300, 31, 4), (65, 32, 32), (9, 33, 5),
                                   (64, 60, 6), (33, 128, 8), (200, 200, 8), (17, 257, 9), (5, 512, 8),
                                   (3, 1000, 32), (2, 1024, 1)])
def test_route(sg, dtype, normalize, T, E, k):
    _check_route(sg, _randn(T, E, seed=T + E + k, dtype=dtype) * 3, k, normalize)


@TYPES
@pytest.mark.parametrize("normalize", [True, False], ids=["normalized", "all"])
def test_route_masks(sg, dtype, normalize):
    T, E, k = 40, 70, 6
    logits = _randn(T, E, seed=1, dtype=dtype) * 2
    logits[:, ::3] = -math.inf
    logits[3] = -math.inf                              # a token without an expert
    logits[4, 2:] = -math.inf                          # with one
    logits[5] = torch.finfo(dtype).min                 # the lowest value is a number
    logits[6] = torch.finfo(dtype).min
    logits[6, 69] = 0.0
    logits[7] = 0.0
    logits[8] = -0.0
    logits[8, 11] = 0.0                                # equal to -0
    logits[9, 1:] = 1.0                                # ties
    _check_route(sg, logits, k, normalize)
    weights, experts = sg.route_topk(logits, k, normalize=normalize)
    assert (experts[3] == -1).all() and (weights[3] == 0).all()
    assert experts[4].tolist() == [1] + [-1] * 5
    assert experts[7].tolist() == list(range(k)) and experts[8].tolist() == list(range(k))
    assert experts[9].tolist() == list(range(1, k + 1))


@TYPES
def test_route_strided_rows_and_neighbours(sg, dtype):
    wide = _randn(50, 101, seed=2, dtype=dtype)
    wide[:, :20] = math.inf
    wide[:, 81:] = math.nan
    _check_route(sg, wide[:, 20:81], 4, True)
    _check_route(sg, wide[:, 20:81], 4, False)


def test_route_nan_and_infinity_stay_in_their_row(sg):
    logits = _randn(6, 40, seed=3)
    clean = sg.route_topk(logits, 3)
    logits[2, 7] = math.nan
    logits[4, 5] = math.inf
    weights, experts = sg.route_topk(logits, 3)
    assert experts[2, 0] == 7 and experts[4, 0] == 5
    assert weights[2].isnan().all() and weights[4, 0].isnan()
    for t in (0, 1, 3, 5):
        assert torch.equal(weights[t], clean[0][t]) and torch.equal(experts[t], clean[1][t])


def test_route_gradient_against_differences(sg):
    # Central differences of the 64-bit formula around FP32 logits (step h: the
    # formula's third derivative is below 1, times h^2).
    logits = _randn(5, 12, seed=4)
    dweights = _randn(5, 3, seed=5)
    h = 1e-4
    for normalize in (True, False):
        _, experts = sg.route_topk(logits, 3, normalize=normalize)
        got = sg.route_topk_grad(logits, experts, dweights, normalize=normalize).double()
        for e in range(12):
            up, down = logits.double(), logits.double()
            up[:, e] += h
            down[:, e] -= h
            diff = ((_route(up, 3, normalize)[0] - _route(down, 3, normalize)[0]) * dweights.double()).sum(1) / (2 * h)
            assert ((got[:, e] - diff).abs() <= 1e-6 * dweights.double().abs().sum(1)).all()


def test_route_gradient_takes_any_choice(sg):
    # Experts that are not the k largest, the same one twice, none at all.
    logits = _randn(4, 9, seed=6)
    experts = torch.tensor([[8, 0], [3, 3], [-1, 5], [100, -7]], device="cuda")
    g = _randn(4, 2, seed=7)
    l = logits.double().requires_grad_()
    live = (experts >= 0) & (experts < 9)
    (torch.softmax(l, 1).gather(1, torch.where(live, experts, 0)) * torch.where(live, g.double(), 0.0)).sum().backward()
    got = sg.route_topk_grad(logits, experts, g, normalize=False).double()
    assert ((got - l.grad).abs() <= 2.0 ** -18).all()
    assert (got[3] == 0).all()


# ---------------------------------------------------------------- the sort

def _places(experts, G):
    """(slots, ends) choice by choice."""
    flat = experts.reshape(-1).tolist()
    key = [e if 0 <= e < G else G for e in flat]
    order = sorted(range(len(flat)), key=lambda a: key[a])      # stable
    slots = [0] * len(flat)
    for r, a in enumerate(order):
        slots[a] = r if key[a] < G else -1 - r
    ends, at = [], 0
    for g in range(G):
        at += key.count(g)
        ends.append(at)
    return slots, ends


def _experts(T, k, G, seed, bad=0.1):
    g = torch.Generator().manual_seed(seed)
    e = torch.randint(0, max(G, 1), (T, k), generator=g)
    e[torch.rand(T, k, generator=g) < bad] = -1
    e[torch.rand(T, k, generator=g) < bad / 4] = G
    return e


@pytest.mark.parametrize("T,k,G", [(1, 1, 1), (1, 8, 3), (16, 2, 64), (31, 1, 5), (33, 3, 7), (500, 2, 1024),
                                   (1000, 8, 256), (700, 3, 1), (2100, 2, 33), (9001, 2, 40), (64, 4, 0)])
def test_places(sg, T, k, G):
    experts = _experts(T, k, G, seed=T)
    slots, ends = _places(experts, G)
    x = _randn(T, 8, seed=1)
    rows, got, got_ends = sg.expert_dispatch(x, experts.cuda(), G)
    assert got.dtype == torch.int32 and got_ends.dtype == torch.int32
    assert got.reshape(-1).tolist() == slots and got_ends.tolist() == ends
    r = torch.tensor([s if s >= 0 else -1 - s for s in slots], device="cuda")
    want = torch.zeros_like(rows)
    want[r] = torch.where(torch.tensor(slots, device="cuda")[:, None] >= 0, x.repeat_interleave(k, 0), 0.0)
    assert torch.equal(rows, want)


def test_places_of_many(sg):
    # One expert for all, and a long skewed list, against a stable sort.
    for T, k, G, seed in ((60000, 8, 512, 1), (262145, 1, 1000, 2), (50000, 4, 3, 3)):
        experts = _experts(T, k, G, seed).cuda()
        if G == 3:
            experts.fill_(1)
        flat = experts.reshape(-1)
        key = torch.where((flat >= 0) & (flat < G), flat, G)
        order = torch.argsort(key, stable=True)
        want = torch.empty_like(order)
        want[order] = torch.arange(flat.numel(), device="cuda")
        want = torch.where(key < G, want, -1 - want).view(T, k)
        x = torch.arange(T, device="cuda", dtype=F32)[:, None]
        rows, slots, ends = sg.expert_dispatch(x, experts, G)
        assert torch.equal(slots.long(), want)
        assert torch.equal(ends.long(), torch.bincount(key, minlength=G + 1)[:G].cumsum(0))
        assert torch.equal(rows[:, 0], torch.where(key[order] < G, (order // k).float(), 0.0))


# ------------------------------------------------------------------- rows

SIZES = [(1, 1, 1, 1), (1, 2, 4, 1024), (5, 3, 7, 33), (40, 2, 8, 512), (33, 8, 5, 1001), (129, 1, 16, 2056),
         (7, 9, 30, 130), (12, 17, 20, 64), (200, 6, 3, 4096), (64, 2, 2, 8190)]


@TYPES
@pytest.mark.parametrize("T,k,G,D", SIZES)
def test_rows_there_and_back(sg, dtype, T, k, G, D):
    experts = _experts(T, k, G, seed=T + D).cuda()
    x = _randn(T, D, seed=1, dtype=dtype)
    rows, slots, ends = sg.expert_dispatch(x, experts, G)
    place = torch.where(slots >= 0, slots, -1 - slots).long()
    has = (slots >= 0)[:, :, None]
    assert torch.equal(rows[place], torch.where(has, x[:, None, :].expand(T, k, D), torch.zeros_like(x[:1, None])))
    n = int(ends[-1]) if G else 0
    assert n == int((slots >= 0).sum()) and (rows[n:] == 0).all()

    # k products and sums in FP32, one rounding to the type.
    rows = _randn(T * k, D, seed=2, dtype=dtype)
    rows[n:] = math.nan                               # (rows behind the last end take no part)
    weights = _randn(T, k, seed=3)
    got_rows = torch.where(has, rows.double()[place], 0.0)
    for w in (weights, None):
        y = sg.expert_combine(rows, slots, w)
        ww = (weights if w is not None else torch.ones_like(weights)).double()[:, :, None]
        want, terms = (got_rows * ww).sum(1), (got_rows * ww).abs().sum(1)
        tol = (k + 1) * 2.0 ** -24 * terms
        assert y.dtype == dtype
        assert ((y.double() - want).abs() <= tol + _half_step(want.abs() + tol, dtype)).all()

        dy = _randn(T, D, seed=4, dtype=dtype)
        drows, dweights = sg.expert_combine_grad(dy, rows, slots, w)
        want = torch.where(has, ww * dy.double()[:, None, :], 0.0)
        assert drows.dtype == dtype
        assert ((drows.double()[place] - want).abs() <= _half_step(want.abs() * (1 + 2.0 ** -23), dtype) +
                want.abs() * 2.0 ** -24).all()
        # D products and sums in FP32.
        products = got_rows * dy.double()[:, None, :]
        assert dweights.dtype == F32
        assert ((dweights.double() - products.sum(2)).abs() <= (D + 1) * 2.0 ** -24 * products.abs().sum(2) +
                2.0 ** -140).all()


@TYPES
def test_rows_with_pitches_and_odd_bases(sg, dtype):
    T, k, G, D = 37, 3, 6, 259
    experts = _experts(T, k, G, seed=1).cuda()
    wide = _randn(T, 300, seed=2, dtype=dtype)
    for a in (0, 1, 8):
        x = wide[:, a:a + D]
        rows, slots, _ = sg.expert_dispatch(x, experts, G)
        want = sg.expert_dispatch(x.contiguous(), experts, G)[0]
        assert torch.equal(rows, want)
        pitched = torch.full((T * k, 333), math.nan, dtype=dtype, device="cuda")[:, a:a + D]
        pitched.copy_(rows)
        weights = _randn(T, k, seed=3)
        # `out` with a guard on all sides.
        guard = torch.full((T + 2, D + 9), 7.0, dtype=dtype, device="cuda")
        out = guard[1:-1, a:a + D] if a < 8 else guard[1:-1, 8:8 + D]
        y = sg.expert_combine(pitched, slots, weights, out=out)
        assert y.data_ptr() == out.data_ptr()
        assert torch.equal(y, sg.expert_combine(rows, slots, weights))
        kept = guard.clone()
        out.fill_(7.0)
        assert (guard == 7.0).all() and not torch.equal(kept, guard)
        dy = _randn(T, 311, seed=4, dtype=dtype)[:, a:a + D]
        for u, v in zip(sg.expert_combine_grad(dy, pitched, slots, weights),
                        sg.expert_combine_grad(dy.contiguous(), rows, slots, weights)):
            assert torch.equal(u, v)


def test_sizes_of_zero(sg):
    x = torch.empty(0, 16, device="cuda")
    rows, slots, ends = sg.expert_dispatch(x, torch.empty(0, 2, dtype=torch.int64, device="cuda"), 4)
    assert rows.shape == (0, 16) and slots.shape == (0, 2) and ends.tolist() == [0, 0, 0, 0]
    assert sg.expert_combine(rows, slots).shape == (0, 16)
    none = torch.empty(5, 0, dtype=torch.int64, device="cuda")
    rows, slots, ends = sg.expert_dispatch(torch.ones(5, 16, device="cuda"), none, 4)
    assert rows.shape == (0, 16) and ends.tolist() == [0, 0, 0, 0]
    assert (sg.expert_combine(rows, slots) == 0).all()
    rows, slots, ends = sg.expert_dispatch(torch.empty(5, 0, device="cuda"), torch.ones(5, 2, dtype=torch.int64,
                                                                                        device="cuda"), 4)
    assert rows.shape == (10, 0) and ends.tolist() == [0, 10, 10, 10]
    drows, dweights = sg.expert_combine_grad(torch.empty(5, 0, device="cuda"), rows, slots)
    assert drows.shape == (10, 0) and (dweights == 0).all()
    weights, experts = sg.route_topk(torch.empty(0, 8, device="cuda"), 2)
    assert weights.shape == (0, 2) and experts.shape == (0, 2)
    assert sg.route_topk_grad(torch.empty(0, 8, device="cuda"), experts, weights).shape == (0, 8)


def test_slots_outside_the_rows_are_left_out(sg):
    # (Numbers no dispatch gives: nothing outside the tensors is read or written.)
    rows = torch.ones(4, 8, device="cuda")
    slots = torch.tensor([[0, 4], [2 ** 31 - 1, -2 ** 31]], dtype=torch.int32, device="cuda")
    assert torch.equal(sg.expert_combine(rows, slots), torch.tensor([[1.0], [0.0]], device="cuda").expand(2, 8))
    _, dweights = sg.expert_combine_grad(torch.ones(2, 8, device="cuda"), rows, slots)
    assert dweights.tolist() == [[8.0, 0.0], [0.0, 0.0]]


# --------------------------------------------------------------- refusals

def test_refusals(sg):
    l = torch.zeros(4, 8, device="cuda")
    for bad in (0, 9, -1):
        with pytest.raises(ValueError):
            sg.route_topk(l, bad)
    with pytest.raises(TypeError):
        sg.route_topk(l, 2.5)
    with pytest.raises(TypeError):
        sg.route_topk(l.double(), 2)
    with pytest.raises(ValueError):
        sg.route_topk(l.cpu(), 2)
    with pytest.raises(ValueError):
        sg.route_topk(l[0], 2)
    with pytest.raises(ValueError):
        sg.route_topk(l.t(), 2)
    with pytest.raises(ValueError):
        sg.route_topk(l[:1].expand(4, 8), 2)
    with pytest.raises(sg.SgemmError):
        sg.route_topk(torch.zeros(2, 1025, device="cuda"), 2)
    with pytest.raises(sg.SgemmError):
        sg.route_topk(torch.zeros(2, 64, device="cuda"), 33)
    w, e = sg.route_topk(l, 2)
    with pytest.raises(TypeError):
        sg.route_topk_grad(l, e.int(), w)
    with pytest.raises(TypeError):
        sg.route_topk_grad(l, e, w.half())
    with pytest.raises(ValueError):
        sg.route_topk_grad(l, e, w[:, :1].contiguous())
    with pytest.raises(ValueError):
        sg.route_topk_grad(l, e[:, :1], w[:, :1])
    x = torch.zeros(4, 16, device="cuda")
    with pytest.raises(ValueError):
        sg.expert_dispatch(x, e[:3], 8)
    with pytest.raises(ValueError):
        sg.expert_dispatch(x, e[:, 0], 8)
    with pytest.raises(TypeError):
        sg.expert_dispatch(x, e.int(), 8)
    with pytest.raises(TypeError):
        sg.expert_dispatch(x.long(), e, 8)
    with pytest.raises(ValueError):
        sg.expert_dispatch(x, e, -1)
    with pytest.raises(sg.SgemmError):
        sg.expert_dispatch(x, e, 1025)
    with pytest.raises(ValueError):
        sg.expert_dispatch(x[:1].expand(4, 16), e, 8)
    rows, slots, _ = sg.expert_dispatch(x, e, 8)
    with pytest.raises(ValueError):
        sg.expert_combine(rows[:7], slots)
    with pytest.raises(TypeError):
        sg.expert_combine(rows, slots.long())
    with pytest.raises(TypeError):
        sg.expert_combine(rows, slots, w.double())
    with pytest.raises(ValueError):
        sg.expert_combine(rows, slots, w[:3])
    with pytest.raises(ValueError):
        sg.expert_combine(rows, slots, w, out=torch.zeros(4, 17, device="cuda"))
    with pytest.raises(TypeError):
        sg.expert_combine(rows, slots, w, out=torch.zeros(4, 16, device="cuda", dtype=F16))
    with pytest.raises(ValueError):
        sg.expert_combine_grad(x[:3], rows, slots)
    with pytest.raises(TypeError):
        sg.expert_combine_grad(x.half(), rows, slots)


# ------------------------------------------------------------------ graphs

@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("normalize", [True, False], ids=["normalized", "all"])
def test_a_layer_and_its_gradients(sg, dtype, normalize):
    """Routing, dispatch, the experts' products and the way back, as a model
    uses them, in torch's graph."""
    T, D, H, G, k = 61, 72, 40, 5, 2
    x, router = _randn(T, D, seed=1, dtype=dtype) * 0.3, _randn(G, D, seed=2, dtype=dtype) * 0.3
    up, down = _randn(G, H, D, seed=3, dtype=dtype) * 0.1, _randn(G, D, H, seed=4, dtype=dtype) * 0.1
    leaves = [v.detach().requires_grad_() for v in (x, router, up, down)]
    x, router, up, down = leaves
    pad = torch.zeros(T, G, dtype=dtype, device="cuda")
    pad[::7] = -math.inf                              # padding goes to no expert
    weights, experts = sg.route_topk(x @ router.t() + pad, k, normalize=normalize)
    rows, slots, ends = sg.expert_dispatch(x, experts, G)
    h = torch.tanh(sg.grouped_gemm(rows, up, ends, trans_w=True))
    y = sg.expert_combine(sg.grouped_gemm(h, down, ends, trans_w=True), slots, weights)
    c = _randn(T, D, seed=5)
    (y.float() * c).sum().backward()
    assert (y[::7] == 0).all()

    xd, rd, ud, dd = [v.detach().double().requires_grad_() for v in leaves]
    p = torch.softmax(xd @ rd.t(), 1).gather(1, experts.clamp(min=0))
    w = p / p.sum(1, keepdim=True) if normalize else p
    w = torch.where(experts >= 0, w, 0.0)
    hd = torch.tanh(torch.einsum("td,tkhd->tkh", xd, ud[experts.clamp(min=0)]))
    yd = (torch.einsum("tkh,tkdh->tkd", hd, dd[experts.clamp(min=0)]) * w[:, :, None]).sum(1)
    (yd * c.double()).sum().backward()
    # Seven roundings to the type one behind another, each of its own values.
    tol = 2.0 ** -16 if dtype == F32 else 2.0 ** -5
    assert (y.double() - yd).norm() <= tol * yd.norm()
    for a, b in zip(leaves, (xd, rd, ud, dd)):
        assert (a.grad.double() - b.grad).norm() <= tol * b.grad.norm()


def test_gradients_that_are_not_asked_for(sg):
    experts = _experts(20, 2, 4, seed=1).cuda()
    rows, slots, _ = sg.expert_dispatch(_randn(20, 24, seed=2), experts, 4)
    weights, dy = _randn(20, 2, seed=3), _randn(20, 24, seed=4)
    both = sg.expert_combine_grad(dy, rows, slots, weights)
    for need in ("r", "w"):
        r, w = rows.clone().requires_grad_("r" in need), weights.clone().requires_grad_("w" in need)
        sg.expert_combine(r, slots, w).backward(dy)
        assert r.grad is None if "r" not in need else torch.equal(r.grad, both[0])
        assert w.grad is None if "w" not in need else torch.equal(w.grad, both[1])
    with torch.no_grad():
        assert not sg.expert_combine(rows.requires_grad_(), slots).requires_grad
    out = torch.empty(20, 24, device="cuda")
    assert not sg.expert_combine(rows, slots, out=out).requires_grad
    # A broadcast gradient (of a sum).
    r = rows.detach().clone().requires_grad_()
    sg.expert_combine(r, slots).sum().backward()
    assert torch.equal(r.grad, sg.expert_combine_grad(torch.ones(20, 24, device="cuda"), r.detach(), slots)[0])


def test_a_captured_layer_with_new_tokens(sg):
    T, D, G, k = 48, 256, 16, 2
    x, logits = _randn(T, D, seed=1, dtype=BF16), _randn(T, G, seed=2)
    w = _randn(G, D, D, seed=3, dtype=BF16) * 0.1

    def layer():
        weights, experts = sg.route_topk(logits, k)
        rows, slots, ends = sg.expert_dispatch(x, experts, G)
        return sg.expert_combine(sg.grouped_gemm(rows, w, ends), slots, weights)
    layer()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer()
    for seed in (11, 12, 13):
        x.copy_(_randn(T, D, seed=seed))
        logits.copy_(_randn(T, G, seed=seed + 10))
        want = layer()
        graph.replay()
        assert torch.equal(y, want)


def test_streams_side_by_side_and_given(sg):
    def work(seed):
        x, logits = _randn(700, 520, seed=seed, dtype=BF16), _randn(700, 37, seed=seed + 1)

        def run(**kw):
            weights, experts = sg.route_topk(logits, 3, **kw)
            rows, slots, ends = sg.expert_dispatch(x, experts, 37, **kw)
            y = sg.expert_combine(rows, slots, weights, **kw)
            return [weights, experts, rows, slots, ends, y, *sg.expert_combine_grad(y, rows, slots, weights, **kw),
                    sg.route_topk_grad(logits, experts, weights, **kw)]
        return run
    jobs = [work(10 * i) for i in range(3)]
    want = [j() for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    got = []
    for _ in range(5):
        for j, s in zip(jobs, streams):
            with torch.cuda.stream(s):
                got.append(j())
        for j, s in zip(jobs, streams):
            got.append(j(stream=s))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[i % 3]))
