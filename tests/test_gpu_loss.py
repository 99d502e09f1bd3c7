"""Vocabulary cross entropy and its gradients against the definition in 64
bits, at the sizes, targets and values where they can go wrong.

Bounds, element by element.  A logit is a sum in FP32: off by at most
D = SUM * max sum |x w| (SUM = 2^-16 for the tensor core's running sum at
these lengths, 2^-20 for FP32 operands).  The loss is then off by 2 D and
2^-20 of itself and of its parts.  d = g (p - 1[target]) is off by
|g p| (2 D + 2^-18) from its exponential, eps / 2 of itself where it is held
in 16 bits, by bf16's smallest step 2^-133 (FP32 holds it in bf16 planes), and
for f16, which holds it times a power of two, by 2^-37 of the largest g.  The products carry that through |W| or |X|, add SUM of their
own sum of magnitudes, and round once (eps / 2, f16: 2^-25 at least).
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


def _problem(T, V, D, dtype, seed, scale=2.0, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, D + pad, generator=g, device="cuda").to(DTYPES[dtype])[:, :D]
    w = (torch.randn(V, D + pad, generator=g, device="cuda") * scale * D ** -0.5).to(DTYPES[dtype])[:, :D]
    target = torch.randint(0, V, (T,), generator=g, device="cuda")
    dloss = torch.randn(T, generator=g, device="cuda") / T
    return x, w, target, dloss


def _check(sg, x, w, target, dloss, dtype, handle=None):
    V = w.shape[0]
    loss, lse = sg.linear_cross_entropy(x, w, target, handle=handle)
    dx, dw = sg.linear_cross_entropy_grad(x, w, target, lse, dloss, handle=handle)
    X, W = x.double(), w.double()
    logits = X @ W.t()
    ref_lse = torch.logsumexp(logits, 1)
    on = (target >= 0) & (target < V)
    idx = torch.where(on, target, torch.zeros_like(target))
    picked = logits.gather(1, idx[:, None])[:, 0]
    ref = torch.where(on, ref_lse - picked, torch.zeros_like(picked))
    delta = SUM[dtype] * (X.abs().amax(1) * W.abs().sum(1).max()).clamp(max=(X.abs() @ W.abs().t()).amax(1)) \
        if V * x.shape[0] < 1e8 else SUM[dtype] * X.norm(dim=1) * W.norm(dim=1).max()
    bound = 2 * delta + 2.0 ** -20 * (ref_lse.abs() + picked.abs() + 1)
    assert ((lse.double() - ref_lse).abs() <= bound).all()
    assert ((loss.double() - ref).abs() <= bound).all()
    assert (loss[~on] == 0).all()

    p = (logits - ref_lse[:, None]).exp_()
    del logits
    g = torch.where(on, dloss.double(), torch.zeros_like(ref))
    e = (p * g.abs()[:, None]).mul_((2 * delta + 2.0 ** -18)[:, None])
    d = p.mul_(g[:, None])
    d[torch.arange(len(g), device=g.device), idx] -= g
    if dtype != "f32":
        e += ROUND[dtype] * d.abs()
    e += 2.0 ** -37 * g.abs().max() if dtype == "f16" else 2.0 ** -133
    for got, ref, err, mag in ((dx, d @ W, e @ W.abs(), d.abs() @ W.abs()),
                               (dw, d.t() @ X, e.t() @ X.abs(), d.abs().t() @ X.abs())):
        bound = (err + SUM[dtype] * mag) * (1 + ROUND[dtype]) + ROUND[dtype] * ref.abs() + STEP[dtype]
        worst = ((got.double() - ref).abs() - bound).max().item()
        assert worst <= 0, f"beyond the bound by {worst}"
    return loss, dx, dw


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,V,D", [(1, 1, 8), (1, 2, 1), (2, 300, 64), (17, 127, 72), (128, 1000, 256),
                                   (129, 513, 136), (300, 2049, 200), (33, 5000, 1001), (513, 777, 65),
                                   (1, 20000, 512)])
def test_loss_and_gradients(sg, dtype, T, V, D):
    _check(sg, *_problem(T, V, D, dtype, T + V + D), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_several_pieces_of_the_vocabulary(sg, dtype):
    # 4100 x 70000 logits are more than one piece of 512 MB.
    x, w, target, dloss = _problem(4100, 70000, 72, dtype, 5)
    _check(sg, x, w, target, dloss, dtype)


def test_several_pieces_f32(sg):
    x, w, target, dloss = _problem(2000, 40003, 40, "f32", 6)
    _check(sg, x, w, target, dloss, "f32")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_targets_that_are_not_counted(sg, dtype):
    x, w, target, dloss = _problem(70, 400, 96, dtype, 7)
    target[::3] = -100
    target[1] = 400
    target[2] = 2 ** 40
    target[4] = 0
    target[5] = 399
    dloss[7] = 0.0
    loss, dx, _ = _check(sg, x, w, target, dloss, dtype)
    assert (dx[::3] == 0).all() and (dx[1:3] == 0).all() and (dx[7] == 0).all()
    target[:] = -1
    loss, dx, dw = _check(sg, x, w, target, dloss, dtype)
    assert (loss == 0).all() and (dx == 0).all() and (dw == 0).all()


def test_rows_not_counted_may_hold_anything(sg):
    x, w, target, dloss = _problem(20, 300, 64, "bf16", 8)
    loss, lse = sg.linear_cross_entropy(x, w, target)
    x2 = x.clone()
    x2[3], x2[4] = float("inf"), float("nan")
    target[3:5] = -1
    loss2, lse2 = sg.linear_cross_entropy(x2, w, target)
    keep = torch.ones(20, dtype=torch.bool, device="cuda")
    keep[3:5] = False
    assert torch.equal(loss[keep], loss2[keep]) and (loss2[3:5] == 0).all()
    dx, _ = sg.linear_cross_entropy_grad(x2, w, target, lse2, dloss)
    assert (dx[3:5] == 0).all() and not torch.isnan(dx[keep]).any()


@pytest.mark.parametrize("tokens", [20, 200])
@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_rows_without_a_part_reach_no_gradient(sg, dtype, pad, tokens):
    # Whatever they hold: the gradients are the ones of zeros in their place.
    x, w, target, dloss = _problem(tokens, 300, 64, dtype, 12, pad=pad)
    target[5], target[tokens - 1], dloss[9] = -100, 300, 0.0
    out = [5, 9, tokens - 1]
    x[out] = 0
    _, lse = sg.linear_cross_entropy(x, w, target)
    want = sg.linear_cross_entropy_grad(x, w, target, lse, dloss)
    x[5], x[9], x[tokens - 1] = float("nan"), float("inf"), -float("inf")
    _, lse = sg.linear_cross_entropy(x, w, target)
    got = sg.linear_cross_entropy_grad(x, w, target, lse, dloss)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert (got[0][out] == 0).all() and torch.isfinite(got[1]).all()


def test_large_logits_do_not_overflow(sg):
    for dtype in ("bf16", "f32"):
        x, w, target, dloss = _problem(40, 600, 128, dtype, 9, scale=60.0)
        loss, _, _ = _check(sg, x, w, target, dloss, dtype)
        assert torch.isfinite(loss).all() and loss.max() > 100


def test_small_gradients_survive_in_f16(sg):
    # A mean over many tokens: d is far below f16's normal numbers.
    x, w, target, _ = _problem(64, 3000, 64, "f16", 10)
    dloss = torch.full((64,), 1e-3, device="cuda")
    _check(sg, x, w, target, dloss, "f16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_pitches_and_repeated_calls(sg, dtype):
    x, w, target, dloss = _problem(150, 901, 130, dtype, 11, pad=3)
    a = _check(sg, x, w, target, dloss, dtype)
    b = _check(sg, x, w, target, dloss, dtype)
    assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_gradient_against_differences(sg):
    # (L(x + s u) - L(x - s u)) / 2s = <dx, u> up to s^2 / 6 times the third
    # derivative, at most 6 c^3 per token with c = max |u . w|, and the error
    # of the two losses, 2^-19 of their size each, over 2s.
    T, V, D, s = 9, 70, 48, 2.0 ** -7
    x, w, target, _ = _problem(T, V, D, "f32", 12)
    one = torch.ones(T, device="cuda")
    _, lse = sg.linear_cross_entropy(x, w, target)
    dx, dw = sg.linear_cross_entropy_grad(x, w, target, lse, one)
    g = torch.Generator(device="cuda").manual_seed(13)
    u = torch.randn(T, D, generator=g, device="cuda") * D ** -0.5
    v = torch.randn(V, D, generator=g, device="cuda") * D ** -0.5

    def total(a, b):
        return sg.linear_cross_entropy(a, b, target)[0].double().sum().item()
    for dn, grad, direction, c in (
            (total(x + s * u, w) - total(x - s * u, w), dx, u, (u @ w.t()).abs().max().item()),
            (total(x, w + s * v) - total(x, w - s * v), dw, v, (x @ v.t()).abs().max().item())):
        want = (grad.double() * direction.double()).sum().item()
        bound = T * (s * s * c ** 3 + 2.0 ** -19 * 20 / s)
        assert abs(dn / (2 * s) - want) <= bound


def test_empty_batch(sg):
    x = torch.zeros(0, 16, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(30, 16, dtype=torch.bfloat16, device="cuda")
    t = torch.zeros(0, dtype=torch.int64, device="cuda")
    loss, lse = sg.linear_cross_entropy(x, w, t)
    assert loss.shape == (0,)
    dx, dw = sg.linear_cross_entropy_grad(x, w, t, lse, lse)
    assert dx.shape == (0, 16) and (dw == 0).all()


def test_refusals(sg):
    x, w, target, dloss = _problem(8, 20, 16, "bf16", 1)
    with pytest.raises(TypeError):
        sg.linear_cross_entropy(x, w.float(), target)
    with pytest.raises(TypeError):
        sg.linear_cross_entropy(x, w, target.int())
    with pytest.raises(ValueError):
        sg.linear_cross_entropy(x, w[:, :8], target)
    with pytest.raises(ValueError):
        sg.linear_cross_entropy(x, w, target[:4])
    with pytest.raises(sg.SgemmError):
        sg.linear_cross_entropy(x, w[:0], target)
    with pytest.raises(TypeError):
        sg.linear_cross_entropy_grad(x, w, target, dloss.double(), dloss)
    with pytest.raises(ValueError):
        sg.linear_cross_entropy_grad(x, w, target, dloss, dloss[:3])
