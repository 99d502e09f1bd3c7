"""Choices that are dropped after the sort: a negative slot names no row, in the
gradients as in the sum, and rows that no slot names get gradient 0, whatever lay in
the memory before."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


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


def _slots(sg, T, k, G, seed, mark, share):
    """Slots of a sort with some choices dropped."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    experts = torch.randint(-1, G, (T, k), generator=g, device="cuda")
    _, slots, _ = sg.expert_dispatch(_randn(T, 1, seed=seed), experts, G)
    drop = torch.rand(T, k, generator=g, device="cuda") < share
    n = T * k
    if mark == "minus one":
        return torch.where(drop, torch.full_like(slots, -1), torch.where(slots < 0, torch.full_like(slots, -1), slots))
    if mark == "inverted":
        return torch.where(drop & (slots >= 0), -1 - slots, slots)
    if mark == "beyond":
        return torch.where(drop, torch.full_like(slots, n), slots)
    # All negatives name row 0 or the last row, as those of a sort would.
    wrong = torch.where(torch.rand(T, k, generator=g, device="cuda") < 0.5, -1, -n).to(torch.int32)
    return torch.where(drop | (slots < 0), wrong, slots)


def _gradients(dy, rows, slots, weights):
    """(drows, dweights' products) by the formula: drows as rounded, dweights in 64 bits."""
    n = rows.shape[0]
    has = (slots >= 0) & (slots < n)
    t, j = has.nonzero(as_tuple=True)
    r = slots[t, j].long()
    w = weights if weights is not None else torch.ones(slots.shape, device="cuda")
    drows = torch.zeros_like(rows)
    drows[r] = (w[t, j, None] * dy[t].float()).to(rows.dtype)
    terms = torch.zeros(*slots.shape, rows.shape[1], dtype=torch.float64, device="cuda")
    terms[t, j] = rows[r].double() * dy[t].double()
    return drows, terms


def _poison(T, k, D, dtype):
    """Blocks that the call's results and scratch are likely to lie in: NaN, and
    numbers that are choices."""
    bad = [torch.full((T * k, D), float("nan"), dtype=dtype, device="cuda"),
           torch.arange(T * k, dtype=torch.int32, device="cuda")]
    torch.cuda.synchronize()
    del bad


@pytest.mark.parametrize("mark", ["minus one", "inverted", "beyond", "any negative"])
@pytest.mark.parametrize("T,k,G,D,dtype", [(1, 1, 1, 8, F32), (40, 2, 8, 512, BF16), (33, 3, 5, 129, F16), (300, 1, 7, 64, BF16),
                                           (70, 9, 30, 33, F32), (500, 8, 16, 1024, F16), (5, 70, 100, 2056, BF16)])
@pytest.mark.parametrize("share", [0.3, 1.0])
def test_dropped_choices(sg, T, k, G, D, dtype, mark, share):
    slots = _slots(sg, T, k, G, seed=T + D, mark=mark, share=share)
    rows, dy = _randn(T * k, D, seed=1, dtype=dtype), _randn(T, D, seed=2, dtype=dtype)
    for weights in (_randn(T, k, seed=3), None):
        want, terms = _gradients(dy, rows, slots, weights)
        _poison(T, k, D, dtype)
        drows, dweights = sg.expert_combine_grad(dy, rows, slots, weights)
        assert torch.equal(drows, want)
        # D products and sums in FP32.
        tol = (D + 1) * 2.0 ** -24 * terms.abs().sum(2) + 2.0 ** -140
        assert ((dweights.double() - terms.sum(2)).abs() <= tol).all()
        # In torch's graph, each gradient with and without the other.
        for need in ("r", "w", "rw"):
            if weights is None and need != "r":
                continue
            r = rows.clone().requires_grad_("r" in need)
            w = weights.clone().requires_grad_("w" in need) if weights is not None else None
            y = sg.expert_combine(r, slots, w)
            _poison(T, k, D, dtype)
            y.backward(dy)
            assert r.grad is None if "r" not in need else torch.equal(r.grad, want)
            assert w is None or (w.grad is None if "w" not in need else torch.equal(w.grad, dweights))


def test_a_dropped_choice_against_differences(sg):
    # The sum is linear in rows: differences in FP32 are off by its roundings (k + 1
    # terms of size below 16, over a step of 1).
    T, k, D = 6, 3, 5
    rows, weights, c = _randn(T * k, D, seed=1), _randn(T, k, seed=2), _randn(T, D, seed=3)
    slots = torch.randperm(T * k, generator=torch.Generator().manual_seed(4)).to(torch.int32).view(T, k).cuda()
    slots[1, 0] = slots[4, 2] = slots[5, 1] = -1
    drows, _ = sg.expert_combine_grad(c, rows, slots, weights)
    for r in range(T * k):
        for d in range(D):
            up = rows.clone()
            up[r, d] += 1.0
            diff = ((sg.expert_combine(up, slots, weights).double() - sg.expert_combine(rows, slots, weights).double())
                    * c.double()).sum()
            assert abs(drows[r, d].double() - diff) <= (k + 3) * 2.0 ** -24 * 16 * c.abs().sum().double()


def test_a_layer_with_a_capacity_captured(sg):
    # Dropped after the sort, forward and backward in one graph, with new inputs.
    T, D, G, k = 64, 128, 8, 2
    x, logits, c = _randn(T, D, seed=1, dtype=BF16), _randn(T, G, seed=2), _randn(T, D, seed=3, dtype=BF16)

    def step():
        weights, experts = sg.route_topk(logits, k)
        rows, slots, ends = sg.expert_dispatch(x, experts, G)
        first = torch.cat((ends.new_zeros(1), ends[:-1]))[experts.clamp(min=0)]
        kept = torch.where(slots - first < 12, slots, torch.full_like(slots, -1))
        return [kept, sg.expert_combine(rows, kept, weights), *sg.expert_combine_grad(c, rows, kept, weights)]
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in (11, 12, 13):
        x.copy_(_randn(T, D, seed=seed))
        logits.copy_(_randn(T, G, seed=seed + 10))
        want = step()
        graph.replay()
        assert (want[0] < 0).any()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert torch.equal(want[2], _gradients(c, torch.empty_like(want[2]), want[0], sg.route_topk(logits, k)[0])[0])


def test_without_owners_rows_of_a_sort_are_written_once(sg):
    # The C entry that has no scratch: the slots of a sort name all rows.
    T, k, G, D = 50, 2, 5, 40
    slots = _slots(sg, T, k, G, seed=5, mark="inverted", share=0.2)
    rows, dy, weights = _randn(T * k, D, seed=1), _randn(T, D, seed=2), _randn(T, k, seed=3)
    want = sg.expert_combine_grad(dy, rows, slots, weights)
    drows, dweights = torch.full_like(rows, float("nan")), torch.full_like(weights, float("nan"))
    lib, h = sg.load_library(), sg.Handle()
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert lib.sgemmExpertCombineGrad(h.ptr, 0, T, D, k, dy.data_ptr(), D, rows.data_ptr(), D, slots.data_ptr(),
                                      weights.data_ptr(), drows.data_ptr(), D, dweights.data_ptr(), stream) == 0
    assert torch.equal(drows, want[0]) and torch.equal(dweights, want[1])
    h.close()
