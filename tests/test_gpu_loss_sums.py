"""The gradient of the loss takes its probabilities from the logits that the
loss itself summed: over the vocabulary they add up to one.

With a column of ones in w, the rows' gradient of that column is the sum of
d = p - [v = target], zero but for rounding.  What is left:
  lse in FP32: its own rounding, that of the maximum taken out of each tile's
    sum and that of the joined one, 4 |lse| 2^-24 at most;
  the exponentials, 2^-16 (arguments up to 32 with 2^-23, the function itself
    2^-21);
  d held in 16 bits: sum |d| <= 2 times 2^-17 in two planes (up to 128 rows),
    half a unit in the last place in one;
  the sum over the vocabulary, a truncating one in steps of 16 entries (of both
    planes): 2 (2 V / 16) 2^-23.
Logits summed otherwise than the loss's are off by 1.7e-6 of themselves here,
0.4% to 2% of every probability, in one direction.
"""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(scope="module")
def sg():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import fp32_sgemm_gb300 as m
    m.build()
    m.load_library()
    return m


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,V,D", [(100, 3000, 4096), (128, 3000, 8200), (300, 3000, 4096), (300, 2049, 1030)])
def test_probabilities_add_up_to_one(sg, dtype, T, V, D):
    # Terms of one sign, so that what a sum truncates adds up.
    g = torch.Generator(device="cuda").manual_seed(D)
    x = (0.5 + 0.5 * torch.rand(T, D, generator=g, device="cuda")).to(DTYPES[dtype])
    w = (0.5 + 0.5 * torch.rand(V, D, generator=g, device="cuda")).to(DTYPES[dtype])
    w[:, 7] = 1.0
    target = torch.randint(0, V, (T,), generator=g, device="cuda")
    _, lse = sg.linear_cross_entropy(x, w, target)
    dx, _ = sg.linear_cross_entropy_grad(x, w, target, lse, torch.ones(T, device="cuda"))
    eps = torch.finfo(DTYPES[dtype]).eps / 2
    held = 2.0 ** -17 if T <= 128 or dtype == "f32" else eps
    bound = 4 * lse.double().abs() * 2.0 ** -24 + 2.0 ** -16 + 2 * held + V / 4 * 2.0 ** -23
    off = dx[:, 7].double().abs()
    assert (off <= bound * (1 + eps)).all(), f"off by {off.max().item()}, bound {bound.min().item()}"


@pytest.mark.parametrize("T", [60, 300])
def test_logits_have_no_bias_beyond_fp32(sg, T):
    # Sums of 4096 terms of one sign: what truncation takes from lse in the
    # mean stays within two units in the last place of an FP32 number, 2^-22 at
    # most.  (Runs of 1024 terms lose 2^-20.5.  bf16: products of 16 bits, of
    # which the sum truncates little; f16's of 22 bits lose 2^-18.5 here.)
    V, D = 3000, 4096
    g = torch.Generator(device="cuda").manual_seed(T)
    x = (0.5 + 0.5 * torch.rand(T, D, generator=g, device="cuda")).bfloat16()
    w = (0.5 + 0.5 * torch.rand(V, D, generator=g, device="cuda")).bfloat16()
    _, lse = sg.linear_cross_entropy(x, w, torch.zeros(T, dtype=torch.int64, device="cuda"))
    ref = torch.logsumexp(x.double() @ w.double().t(), 1)
    assert abs(((lse.double() - ref) / ref).mean().item()) <= 2.0 ** -22
