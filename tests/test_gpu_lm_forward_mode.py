"""The language-model operators have no forward mode: an operand with a tangent is
refused, never left out."""
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


def _calls(sg):
    """Each call by the operands of which one may carry a tangent, and the others."""
    def rand(*shape):
        return torch.randn(*shape, device="cuda")
    ends = torch.tensor([3, 6], dtype=torch.int32, device="cuda")
    target = torch.arange(6, device="cuda")
    nibbles = torch.zeros(16, 32, dtype=torch.uint8, device="cuda")
    experts = torch.arange(12, device="cuda").view(6, 2) % 4
    _, slots, _ = sg.expert_dispatch(rand(6, 8), experts, 4)
    w, ws = sg.int8_quantize(rand(16, 64))
    w2, ws2 = torch.stack((w, w)), torch.stack((ws, ws))
    q, s = sg.int8_quantize(rand(6, 64))
    return {
        "grouped_gemm": (lambda x, v: sg.grouped_gemm(x, v, ends), rand(6, 64), rand(2, 64, 16)),
        "linear_cross_entropy": (lambda x, v: sg.linear_cross_entropy(x, v, target), rand(6, 64), rand(40, 64)),
        "w4_gemm": (lambda x, v: sg.w4_gemm(x, nibbles, v), rand(6, 64), rand(16, 2)),
        "route_topk": (lambda x: sg.route_topk(x, 2), rand(6, 40)),
        "expert_dispatch": (lambda x: sg.expert_dispatch(x, experts, 4), rand(6, 8)),
        "expert_combine": (lambda x, v: sg.expert_combine(x, slots, v), rand(12, 8), rand(6, 2)),
        "expert_combine, no weights": (lambda x: sg.expert_combine(x, slots), rand(12, 8)),
        "int8_quantize": (lambda x: sg.int8_quantize(x), rand(6, 64)),
        "int8_gemm": (lambda x, v: sg.int8_gemm(x, w, v), rand(6, 64), ws),
        "int8_gemm of integers": (lambda v, u: sg.int8_gemm(q, w, v, x_scales=u, dtype=torch.float32), ws, s),
        "int8_grouped_gemm": (lambda x, v: sg.int8_grouped_gemm(x, w2, v, ends), rand(6, 64), ws2),
    }


NAMES = ["grouped_gemm", "linear_cross_entropy", "w4_gemm", "route_topk", "expert_dispatch", "expert_combine",
         "expert_combine, no weights", "int8_quantize", "int8_gemm", "int8_gemm of integers", "int8_grouped_gemm"]


@pytest.mark.parametrize("name", NAMES)
def test_forward_mode_is_refused(sg, name):
    import torch.autograd.forward_ad as forward_ad
    call, *operands = _calls(sg)[name]

    def parts(result):
        return result if isinstance(result, tuple) else (result,)
    want = parts(call(*operands))
    for i, v in enumerate(operands):
        with forward_ad.dual_level():
            dual = list(operands)
            dual[i] = forward_ad.make_dual(v, torch.ones_like(v))
            with pytest.raises(NotImplementedError):
                call(*dual)
            with torch.no_grad(), pytest.raises(NotImplementedError):
                call(*dual)                             # (tangents go on without recording)
            with forward_ad._set_fwd_grad_enabled(False):
                assert all(torch.equal(a, b) for a, b in zip(parts(call(*dual)), want))
            with torch.inference_mode():
                assert all(torch.equal(a, b) for a, b in zip(parts(call(*dual)), want))
            # Another operand's tangent is none of these operands'.
            assert all(torch.equal(a, b) for a, b in zip(parts(call(*operands)), want))
        # Once the level is left there is no tangent.
        assert all(torch.equal(a, b) for a, b in zip(parts(call(*operands)), want))
