"""A language model's expert layer and vocabulary head on this library, trained
and then served.

Training: a router picks experts (route_topk), the tokens are sorted by expert
(expert_dispatch), each expert multiplies its rows (grouped_gemm; the counts
stay on the device), the rows come back with their weights (expert_combine), and
the loss over the vocabulary is taken without its logits (linear_cross_entropy);
torch's backward pass goes through all of it.  Serving: the experts' matrices are
quantised to 8 bits (int8_quantize) and the head's to 4, and one token at a time
goes through int8_grouped_gemm and w4_gemm.

    python examples/moe_lm.py            # on a GB300
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp32_sgemm_gb300 as sg  # noqa: E402


class ExpertModel(torch.nn.Module):
    """Embedding, one layer of experts (one per token), vocabulary head."""

    def __init__(self, vocab, dim, hidden, experts, dtype, seed=0):
        super().__init__()
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(*shape):
            t = torch.randn(*shape, generator=g, device="cuda") * shape[-1] ** -0.5
            return torch.nn.Parameter(t.to(dtype))
        self.embed = weight(vocab, dim)
        self.router = weight(experts, dim)
        self.up = weight(experts, hidden, dim)
        self.down = weight(experts, dim, hidden)
        self.head = weight(vocab, dim)

    def experts(self, x, served=None):
        """One expert for each token; `served` the experts' matrices in 8 bits."""
        weights, experts = sg.route_topk(x.float() @ self.router.float().t(), 1, normalize=False)
        rows, slots, ends = sg.expert_dispatch(x, experts, self.up.shape[0])
        if served is None:
            h = torch.nn.functional.silu(sg.grouped_gemm(rows, self.up, ends, trans_w=True))
            y = sg.grouped_gemm(h, self.down, ends, trans_w=True)
        else:
            (up, up_scales), (down, down_scales) = served
            h = torch.nn.functional.silu(sg.int8_grouped_gemm(rows, up, up_scales, ends))
            y = sg.int8_grouped_gemm(h, down, down_scales, ends)
        return x + sg.expert_combine(y, slots, weights)

    def eight_bits(self):
        """The experts' matrices in 8 bits, a scale for each output column."""
        def of(w):
            q, scales = sg.int8_quantize(w.detach().flatten(0, 1))
            return q.view(w.shape), scales.view(w.shape[:2])
        return of(self.up), of(self.down)

    def hidden(self, tokens, served=None):
        return self.experts(self.embed[tokens], served)

    def loss(self, tokens, target):
        losses, _ = sg.linear_cross_entropy(self.hidden(tokens), self.head, target)
        return losses.sum() / (target >= 0).sum()


def quantise(w, group=64):
    """4-bit weights of w [N, K] for w4_gemm: (q, scales, zeros)."""
    n, k = w.shape
    v = w.float().view(n, k // group, group)
    low, high = v.amin(2), v.amax(2)
    scale = ((high - low) / 15).clamp(min=1e-8).to(w.dtype)
    zero = (-low / scale.float()).round().clamp(0, 15)
    q = (v / scale.float()[:, :, None] + zero[:, :, None]).round().clamp(0, 15).to(torch.uint8).view(n, k)
    return q[:, 0::2] | (q[:, 1::2] << 4), scale, zero.to(torch.uint8)


def main(steps=30, vocab=1000, dim=256, hidden=512, experts=8, tokens=512, dtype=torch.bfloat16):
    model = ExpertModel(vocab, dim, hidden, experts, dtype)
    g = torch.Generator(device="cuda").manual_seed(1)
    text = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
    follows = torch.randperm(vocab, generator=g, device="cuda")       # what the model has to learn
    target = follows[text]
    target[:16] = -100                                                # a prompt: not predicted
    losses = []
    for _ in range(steps):
        loss = model.loss(text, target)
        loss.backward()
        with torch.no_grad():
            for p in model.parameters():
                if p.grad is not None:
                    p -= (20.0 * p.grad.float()).to(dtype)
                    p.grad = None
        losses.append(loss.item())
    # Serving: a token at a time, the experts in 8 bits and the head in 4.
    with torch.no_grad():
        q, scales, zeros = quantise(model.head)
        served = model.eight_bits()
        right = 0
        for t in range(16, 48):
            x = model.hidden(text[t:t + 1], served)
            right += int(sg.w4_gemm(x, q, scales, zeros).argmax().item() == target[t].item())
    return losses, right / 32


if __name__ == "__main__":
    curve, share = main()
    print("loss: " + " ".join(f"{v:.3f}" for v in curve[::5] + curve[-1:]))
    print(f"8-bit experts and 4-bit head predict {share:.0%} of 32 tokens")
