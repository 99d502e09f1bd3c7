"""Measured cases of the language-model operators: products grouped by expert,
softmax cross entropy over a vocabulary, and products with 4-bit weights.

With ``own`` false, ``run`` computes an operator in its plain form (elementary
torch operations in 32 bits, rounded once at the end); with ``own`` true it
makes the calls a user of fp32_sgemm_gb300 makes.  ``exact`` gives the same
results from the definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # One decoding step of a batch of 16 sequences, each token sent to 2
        # of 64 experts: 32 rows over 64 matrices, most groups empty or of
        # one row.  Latency, then the reading of the touched weights.
        dict(name="experts_decode", op="grouped", dtype="bf16", rows=32, k=1024, n=2048, groups=64,
             trans=False, way="forward", skew=1.0),
        # The same layer on a short prompt: some tens of rows for an expert.
        dict(name="experts_prompt", op="grouped", dtype="bf16", rows=1024, k=2048, n=1408, groups=16,
             trans=True, way="forward", skew=0.7),
        # A training batch, forward.
        dict(name="experts_train", op="grouped", dtype="bf16", rows=32768, k=4096, n=2048, groups=32,
             trans=False, way="forward", skew=0.5),
        # Its backward pass at a middle size: gradients of the rows and of
        # every expert's matrix.
        dict(name="experts_grads", op="grouped", dtype="f16", rows=8192, k=2048, n=5632, groups=8,
             trans=False, way="backward", skew=0.5),
        # FP32, odd sizes: rows and pitches that are no multiple of anything.
        dict(name="experts_f32_odd", op="grouped", dtype="f32", rows=2001, k=1023, n=777, groups=7,
             trans=False, way="forward", skew=0.7),
        # FP32 training step of a small expert layer.
        dict(name="experts_f32_grads", op="grouped", dtype="f32", rows=4096, k=1024, n=2048, groups=8,
             trans=False, way="backward", skew=0.5),
        # Scoring of a few tokens: the loss alone, bound by reading the
        # vocabulary matrix.
        dict(name="loss_score", op="loss", dtype="bf16", rows=16, vocab=32000, dim=1024, grads=False),
        # Loss and gradients, odd sizes throughout (odd row pitches too).
        dict(name="loss_odd", op="loss", dtype="f16", rows=1023, vocab=50001, dim=1001, grads=True),
        # A training step's loss and gradients over a large vocabulary.
        dict(name="loss_train", op="loss", dtype="bf16", rows=8192, vocab=131072, dim=4096, grads=True),
        # One token through a layer with 4-bit weights: latency.
        dict(name="w4_token", op="w4", dtype="bf16", rows=1, k=4096, n=4096, group=128, zeros=False),
        # One token through a large matrix: the stream of the weights.
        dict(name="w4_stream", op="w4", dtype="f16", rows=1, k=8192, n=28672, group=128, zeros=False),
        # A few tokens at once, odd numbers of rows and columns, small groups
        # with zero points.
        dict(name="w4_few", op="w4", dtype="bf16", rows=7, k=4096, n=14335, group=32, zeros=True),
    ]


def _spread(rng, low, high):
    """An integer spread over [low, high] by its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _even(rng, v, step):
    """Most sizes are multiples of `step`, as in real models; some are not."""
    return v if rng.random() < 0.25 else max(step, v // step * step)


def draw(rng):
    op = rng.choice(["grouped", "grouped", "loss", "w4"])
    if op == "grouped":
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        most = 8192 if dtype == "f32" else 32768
        side = 2048 if dtype == "f32" else 5632
        return dict(op=op, dtype=dtype, rows=_spread(rng, 1, most), k=_even(rng, _spread(rng, 256, side), 64),
                    n=_even(rng, _spread(rng, 256, side), 64), groups=_spread(rng, 1, 64),
                    trans=rng.random() < 0.5, way=rng.choice(["forward", "backward"]),
                    skew=round(rng.uniform(0.0, 1.5), 2))
    if op == "loss":
        return dict(op=op, dtype=rng.choice(["bf16", "f16"]), rows=_spread(rng, 1, 8192),
                    vocab=_even(rng, _spread(rng, 1000, 131072), 64), dim=_even(rng, _spread(rng, 256, 4096), 64),
                    grads=rng.random() < 0.6)
    group = rng.choice([32, 64, 128])
    return dict(op=op, dtype=rng.choice(["bf16", "f16", "f32"]), rows=_spread(rng, 1, 32),
                k=group * max(1, _spread(rng, 1024, 16384) // group), n=_even(rng, _spread(rng, 1000, 28672), 64),
                group=group, zeros=rng.random() < 0.5)


def work(case):
    b = BYTES[case["dtype"]]
    if case["op"] == "grouped":
        t, k, n, g = case["rows"], case["k"], case["n"], case["groups"]
        # Matrices that some row needs: at most one for each row.
        w = min(g, t) * k * n
        if case["way"] == "forward":
            return {"bytes": b * (t * k + w + t * n), "flops": 2.0 * t * k * n}
        # Rows, their output gradients and the matrices in; the rows'
        # gradients and every matrix's gradient out.
        return {"bytes": b * (2 * t * k + t * n + w + g * k * n), "flops": 4.0 * t * k * n}
    if case["op"] == "loss":
        t, v, d = case["rows"], case["vocab"], case["dim"]
        if not case["grads"]:
            return {"bytes": b * (t + v) * d + 12 * t, "flops": 2.0 * t * v * d}
        return {"bytes": 2 * b * (t + v) * d + 16 * t, "flops": 6.0 * t * v * d}
    m, k, n, s = case["rows"], case["k"], case["n"], case["group"]
    scales = n * (k // s) * (b + (1 if case["zeros"] else 0))
    return {"bytes": n * k // 2 + scales + b * m * (k + n), "flops": 2.0 * m * k * n}


# ----------------------------------------------------------------- the inputs

def _ends(case, seed):
    """Ends of the experts' row ranges: sizes as a skewed router gives them,
    one expert in eight without a row."""
    r = np.random.RandomState((seed * 7919 + 17) % (1 << 31))
    p = np.exp(case["skew"] * r.standard_normal(case["groups"]))
    idle = r.random_sample(case["groups"]) < 0.125
    if not idle.all():
        p[idle] = 0.0
    return np.cumsum(r.multinomial(case["rows"], p / p.sum()))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dtype = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device="cuda", dtype=dtype).mul_(scale)

    state = dict(case=case)
    if case["op"] == "grouped":
        t, k, n, groups = case["rows"], case["k"], case["n"], case["groups"]
        ends = _ends(case, seed)
        state["ends"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
        # The longest group: the plain form pads every group to it.
        state["most"] = int(np.diff(ends, prepend=0).max())
        state["x"] = normal(t, k)
        shape = (groups, n, k) if case["trans"] else (groups, k, n)
        state["w"] = normal(*shape, scale=k ** -0.5)
        if case["way"] == "backward":
            state["dy"] = normal(t, n, scale=0.01)
    elif case["op"] == "loss":
        t, v, d = case["rows"], case["vocab"], case["dim"]
        state["x"] = normal(t, d)
        state["w"] = normal(v, d, scale=2.0 * d ** -0.5)
        target = torch.randint(0, v, (t,), generator=g, device="cuda")
        # Some tokens are not to be predicted (padding, prompts).
        target[torch.rand(t, generator=g, device="cuda") < 0.05] = -100
        state["target"] = target
        # The gradient of a mean over the tokens, scaled as for half types.
        state["dloss"] = torch.full((t,), 64.0 / t, device="cuda")
    else:
        m, k, n, s = case["rows"], case["k"], case["n"], case["group"]
        state["x"] = normal(m, k)
        state["q"] = torch.randint(0, 256, (n, k // 2), generator=g, device="cuda", dtype=torch.uint8)
        state["scales"] = (torch.rand(n, k // s, generator=g, device="cuda") * 0.01 + 0.005).to(dtype)
        state["zeros"] = (torch.randint(4, 12, (n, k // s), generator=g, device="cuda", dtype=torch.uint8)
                          if case["zeros"] else None)
    return state


# ------------------------------------------------------------- the operators

def run(state):
    case = state["case"]
    if own:
        return _own(state, case)
    return {"grouped": _plain_grouped, "loss": _plain_loss, "w4": _plain_w4}[case["op"]](state, case)


def _own(state, case):
    import fp32_sgemm_gb300 as sg
    if case["op"] == "grouped":
        x, w, ends, trans = state["x"], state["w"], state["ends"], case["trans"]
        if case["way"] == "forward":
            return sg.grouped_gemm(x, w, ends, trans_w=trans)
        dy = state["dy"]
        return {"dx": sg.grouped_gemm(dy, w, ends, trans_w=not trans),
                "dw": sg.grouped_gemm_weight_grad(x, dy, ends, trans_w=trans)}
    if case["op"] == "loss":
        x, w, target = state["x"], state["w"], state["target"]
        loss, lse = sg.linear_cross_entropy(x, w, target)
        if not case["grads"]:
            return loss
        dx, dw = sg.linear_cross_entropy_grad(x, w, target, lse, state["dloss"])
        return {"loss": loss, "dx": dx, "dw": dw}
    return sg.w4_gemm(state["x"], state["q"], state["scales"], state["zeros"])


def _plain_grouped(state, case):
    x, w, ends = state["x"].float(), state["w"].float(), state["ends"].long()
    dtype = state["x"].dtype
    if case["trans"]:
        w = w.transpose(1, 2)
    row = torch.arange(case["rows"], device=x.device)
    group = torch.searchsorted(ends, row, right=True)
    place = row - torch.cat((ends.new_zeros(1), ends[:-1]))[group]
    xp = x.new_zeros(case["groups"], state["most"], case["k"])
    xp[group, place] = x
    if case["way"] == "forward":
        return torch.bmm(xp, w)[group, place].to(dtype)
    dyp = x.new_zeros(case["groups"], state["most"], case["n"])
    dyp[group, place] = state["dy"].float()
    dx = torch.bmm(dyp, w.transpose(1, 2))[group, place]
    dw = torch.bmm(dyp.transpose(1, 2), xp) if case["trans"] else torch.bmm(xp.transpose(1, 2), dyp)
    return {"dx": dx.to(dtype), "dw": dw.to(dtype)}


def _plain_loss(state, case):
    x, w, target = state["x"].float(), state["w"].float(), state["target"]
    logits = x @ w.t()
    top = logits.amax(1, keepdim=True)
    lse = (logits - top).exp().sum(1).log() + top[:, 0]
    counted = target >= 0
    index = target.clamp(min=0)[:, None]
    zero = torch.zeros_like(lse)
    loss = torch.where(counted, lse - logits.gather(1, index)[:, 0], zero)
    if not case["grads"]:
        return loss
    scale = torch.where(counted, state["dloss"], zero)[:, None]
    d = (logits - lse[:, None]).exp() * scale
    d.scatter_add_(1, index, -scale)
    dtype = state["x"].dtype
    return {"loss": loss, "dx": (d @ w).to(dtype), "dw": (d.t() @ x).to(dtype)}


def _plain_w4(state, case):
    x, q, scales = state["x"].float(), state["q"], state["scales"].float()
    n, k, s = case["n"], case["k"], case["group"]
    # Low four bits: even columns; high four bits: odd columns.
    v = torch.stack((q & 15, q >> 4), dim=2).view(n, k // s, s).float()
    z = state["zeros"].float()[:, :, None] if state["zeros"] is not None else 8.0
    w = ((v - z) * scales[:, :, None]).view(n, k)
    return (x @ w.t()).to(state["x"].dtype)


# ------------------------------------------------------------ in 64 bits

def exact(case, seed):
    # 64-bit products run near 1 TFLOP/s here.
    if work(case)["flops"] > 1.5e13:
        return None
    state = prepare(case, seed)
    if case["op"] == "grouped":
        x = state["x"].double()
        bounds = [0] + state["ends"].tolist()
        forward = case["way"] == "forward"
        w = state["w"]
        y = x.new_empty(case["rows"], case["n"] if forward else case["k"])
        dw = None if forward else torch.zeros(w.shape, dtype=torch.float64, device=w.device)
        for e in range(case["groups"]):
            a, b = bounds[e], bounds[e + 1]
            if a == b:
                continue
            we = w[e].double().t() if case["trans"] else w[e].double()
            if forward:
                y[a:b] = x[a:b].mm(we)
            else:
                dy = state["dy"][a:b].double()
                y[a:b] = dy.mm(we.t())
                dw[e] = dy.t().mm(x[a:b]) if case["trans"] else x[a:b].t().mm(dy)
        return y if forward else {"dx": y, "dw": dw}
    if case["op"] == "loss":
        x, w, target = state["x"].double(), state["w"].double(), state["target"]
        loss = torch.zeros(case["rows"], dtype=torch.float64, device=x.device)
        dx, dw = torch.zeros_like(x), torch.zeros_like(w)
        for a in range(0, case["rows"], 1024):      # blocks of rows
            xa, ta = x[a:a + 1024], target[a:a + 1024]
            logp = torch.log_softmax(xa.mm(w.t()), dim=1)
            on = (ta >= 0).nonzero()[:, 0]
            loss[a + on] = -logp[on, ta[on]]
            if case["grads"]:
                d = logp.exp_()
                d[on, ta[on]] -= 1.0
                d *= torch.where(ta >= 0, state["dloss"][a:a + 1024].double(), 0.0)[:, None]
                dx[a:a + 1024] = d.mm(w)
                dw += d.t().mm(xa)
        return {"loss": loss, "dx": dx, "dw": dw} if case["grads"] else loss
    x, scales = state["x"].double(), state["scales"].double()
    q = state["q"].long()
    w = x.new_empty(case["n"], case["k"])
    w[:, 0::2] = (q % 16).double()
    w[:, 1::2] = (q // 16).double()
    z = state["zeros"].double() if state["zeros"] is not None else torch.full_like(scales, 8.0)
    w = (w - z.repeat_interleave(case["group"], 1)) * scales.repeat_interleave(case["group"], 1)
    return x.mm(w.t())
