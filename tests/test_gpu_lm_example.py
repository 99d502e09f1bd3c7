"""The example model: its gradients against torch's on the same weights in
64 bits, and that it learns and then predicts with a 4-bit head."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import fp32_sgemm_gb300 as m
    m.build()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_lm.py")
    spec = importlib.util.spec_from_file_location("moe_lm", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def _reference(model, tokens, target):
    p = {k: v.detach().double().requires_grad_() for k, v in model.named_parameters()}
    x = p["embed"][tokens]
    scores = torch.softmax(x @ p["router"].t(), dim=1)
    gate, expert = scores.max(dim=1)
    h = torch.nn.functional.silu(torch.einsum("td,thd->th", x, p["up"][expert]))
    y = torch.einsum("th,tdh->td", h, p["down"][expert]) * gate[:, None]
    loss = torch.nn.functional.cross_entropy((x + y) @ p["head"].t(), target, ignore_index=-100)
    loss.backward()
    return loss.detach(), {k: v.grad for k, v in p.items()}


def test_gradients_match_torch(example):
    # FP32 throughout: every product is right to about 2^-20 of its terms, a
    # handful of them follow one another.
    model = example.ExpertModel(vocab=301, dim=72, hidden=136, experts=5, dtype=torch.float32, seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    tokens = torch.randint(0, 301, (97,), generator=g, device="cuda")
    target = torch.randint(0, 301, (97,), generator=g, device="cuda")
    target[::9] = -100
    loss = model.loss(tokens, target)
    loss.backward()
    ref, grads = _reference(model, tokens, target)
    assert abs(loss.item() - ref.item()) <= 2.0 ** -16 * ref.item()
    for name, p in model.named_parameters():
        want = grads[name]
        assert (p.grad.double() - want).norm() <= 2.0 ** -15 * want.norm(), name


def test_learns_and_predicts_with_four_bits(example):
    losses, share = example.main(steps=30)
    assert losses[-1] < 0.25 * losses[0]
    assert share >= 0.9
