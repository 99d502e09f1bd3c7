"""A language model's expert layer and vocabulary head on this library, trained
and then served.

Training: tokens are sorted by the expert a router picked, each expert
multiplies its rows (grouped_gemm; the counts stay on the device), and the
loss over the vocabulary is taken without its logits (linear_cross_entropy);
torch's backward pass goes through both.  Serving: the
head's matrix is quantised to 4 bits and one token at a time goes through
w4_gemm.

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

    def experts(self, x):
        scores = torch.softmax(x.float() @ self.router.float().t(), dim=1)
        gate, expert = scores.max(dim=1)
        order = torch.argsort(expert, stable=True)
        # Ends of the experts' rows: computed and used on the device.
        ends = torch.searchsorted(expert[order], torch.arange(self.up.shape[0], device=x.device),
                                  right=True).to(torch.int32)
        rows = x[order]
        h = torch.nn.functional.silu(sg.grouped_gemm(rows, self.up, ends, trans_w=True))
        y = sg.grouped_gemm(h, self.down, ends, trans_w=True)
        y = y * gate[order, None].to(y.dtype)
        return x + torch.zeros_like(y).index_copy(0, order, y)

    def hidden(self, tokens):
        return self.experts(self.embed[tokens])

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
    # Serving: a token at a time, the head in 4 bits.
    with torch.no_grad():
        q, scales, zeros = quantise(model.head)
        right = 0
        for t in range(16, 48):
            x = model.hidden(text[t:t + 1])
            right += int(sg.w4_gemm(x, q, scales, zeros).argmax().item() == target[t].item())
    return losses, right / 32


if __name__ == "__main__":
    curve, share = main()
    print("loss: " + " ".join(f"{v:.3f}" for v in curve[::5] + curve[-1:]))
    print(f"4-bit head predicts {share:.0%} of 32 tokens")
