"""Measured cases of the expert layer's routing and of products in 8-bit
integers: the choice of experts by a router (and its gradient), tokens sorted
by expert and brought back with their weights (and the gradients), and
products of quantised rows with 8-bit weights, by group or not.

With ``own`` false, ``run`` computes an operator in its plain form (elementary
torch operations, rounded once at the end); with ``own`` true it makes the
calls a user of fp32_sgemm_gb300 makes.  ``exact`` gives the same results from
the definition in 64 bits.
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
        # The router of one decoding step: 16 tokens, 2 of 64 experts.  Latency.
        dict(name="route_decode", op="route", dtype="f32", tokens=16, experts=64, k=2, normalize=True, grads=False,
             masked=0.0),
        # A training batch, forward and backward, many experts of which some
        # are masked (dropped, or of another shard).
        dict(name="route_train", op="route", dtype="bf16", tokens=32768, experts=256, k=8, normalize=True, grads=True,
             masked=0.1),
        # Rows of one decoding step brought to their experts.
        dict(name="dispatch_decode", op="dispatch", dtype="bf16", tokens=16, experts=64, k=2, dim=1024, skew=1.0,
             padded=0.0, grads=False),
        # A training batch of 32768 rows, with the gradient by the tokens.
        dict(name="dispatch_train", op="dispatch", dtype="bf16", tokens=16384, experts=32, k=2, dim=4096, skew=0.5,
             padded=0.02, grads=True),
        # The way back of the decoding step.
        dict(name="combine_decode", op="combine", dtype="bf16", tokens=16, experts=64, k=2, dim=1024, skew=1.0,
             padded=0.0, grads=False),
        # Odd sizes in FP32, with gradients: rows that no vector load reaches.
        dict(name="combine_odd", op="combine", dtype="f32", tokens=1001, experts=7, k=3, dim=1023, skew=0.7,
             padded=0.1, grads=True),
        # The training batch's way back, with the gradients by rows and weights.
        dict(name="combine_train", op="combine", dtype="bf16", tokens=8192, experts=64, k=8, dim=2048, skew=0.5,
             padded=0.0, grads=True),
        # One token through a layer with 8-bit weights: latency.
        dict(name="int8_token", op="int8", dtype="bf16", rows=1, k=4096, n=4096, groups=0, skew=0.0, products=1),
        # One token through a large matrix: the stream of the weights.
        dict(name="int8_stream", op="int8", dtype="f16", rows=1, k=8192, n=28672, groups=0, skew=0.0, products=1),
        # A few tokens, quantised once for two products (gate and up
        # projection), an odd number of rows and columns.
        dict(name="int8_pair", op="int8", dtype="f16", rows=7, k=4096, n=14335, groups=0, skew=0.0, products=2),
        # An expert layer on a prompt: some tens of rows for an expert.
        dict(name="int8_experts", op="int8", dtype="bf16", rows=1024, k=2048, n=1408, groups=16, skew=0.7, products=1),
        # A long prompt through one layer.
        dict(name="int8_prefill", op="int8", dtype="bf16", rows=8192, k=4096, n=14336, groups=0, skew=0.0, products=1),
    ]


def _spread(rng, low, high):
    """An integer spread over [low, high] by its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _even(rng, v, step):
    """Most sizes are multiples of `step`, as in real models; some are not."""
    return v if rng.random() < 0.25 else max(step, v // step * step)


def draw(rng):
    op = rng.choice(["route", "dispatch", "combine", "int8", "int8"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "route":
        experts = _spread(rng, 4, 512)
        return dict(op=op, dtype=dtype, tokens=_spread(rng, 1, 32768), experts=experts,
                    k=rng.randint(1, min(8, experts)), normalize=rng.random() < 0.5, grads=rng.random() < 0.5,
                    masked=rng.choice([0.0, 0.1, 0.5]))
    if op in ("dispatch", "combine"):
        k = rng.randint(1, 8)
        dim = _even(rng, _spread(rng, 128, 8192), 64)
        return dict(op=op, dtype=dtype, tokens=_spread(rng, 1, max(1, min(32768, (1 << 28) // (dim * k * BYTES[dtype])))),
                    experts=_spread(rng, k, 256), k=k, dim=dim, skew=round(rng.uniform(0.0, 1.5), 2),
                    padded=rng.choice([0.0, 0.02, 0.3]), grads=rng.random() < 0.6)
    rows, k, n = _spread(rng, 1, 8192), _even(rng, _spread(rng, 256, 16384), 64), _even(rng, _spread(rng, 256, 28672), 64)
    if rng.random() < 0.5:
        k, n = min(k, 4096), min(n, 5632)
        groups = _spread(rng, 1, 64)
    else:
        groups = 0
        while 2.0 * rows * k * n > 4e11:        # (two products cost what one long prompt does)
            rows = (rows + 1) // 2
    return dict(op=op, dtype=dtype, rows=rows, k=k, n=n, groups=groups, skew=round(rng.uniform(0.0, 1.5), 2),
                products=rng.choice([1, 1, 2]))


def work(case):
    b = BYTES[case["dtype"]]
    if case["op"] == "route":
        t, e, k = case["tokens"], case["experts"], case["k"]
        # Logits in, weights (32 bits) and experts (64 bits) out; a pass over
        # the logits: the maximum, the sum and k choices.
        if not case["grads"]:
            return {"bytes": t * e * b + t * k * 12, "flops": 3.0 * t * e}
        return {"bytes": 2 * t * e * b + t * k * 16, "flops": 6.0 * t * e}
    if case["op"] == "dispatch":
        t, k, d = case["tokens"], case["k"], case["dim"]
        n = t * k
        # Tokens and their experts in, rows and places out.
        forward = t * d * b + n * 8 + n * d * b + n * 4
        if not case["grads"]:
            return {"bytes": forward, "flops": 0.0}
        return {"bytes": forward + n * d * b + t * d * b, "flops": 1.0 * n * d}
    if case["op"] == "combine":
        t, k, d = case["tokens"], case["k"], case["dim"]
        n = t * k
        forward = n * d * b + n * 8 + t * d * b
        if not case["grads"]:
            return {"bytes": forward, "flops": 2.0 * n * d}
        return {"bytes": forward + t * d * b + n * d * b + n * 4, "flops": 5.0 * n * d}
    m, k, n, p = case["rows"], case["k"], case["n"], case["products"]
    # Matrices that some row needs: at most one for each row.
    w = min(case["groups"], m) if case["groups"] else 1
    return {"bytes": b * m * k + p * (w * n * (k + 4) + b * m * n), "flops": 2.0 * p * m * k * n}


# ----------------------------------------------------------------- the inputs

def _choices(case, g):
    """Experts of each token as a skewed router picks them (all different), -1
    for padding."""
    t, e, k = case["tokens"], case["experts"], case["k"]
    lean = case["skew"] * torch.randn(e, generator=g, device="cuda")
    noise = torch.rand(t, e, generator=g, device="cuda").clamp_(1e-30, 1.0)
    experts = (lean - (-noise.log()).log()).topk(k, dim=1).indices
    experts[torch.rand(t, generator=g, device="cuda") < case["padded"]] = -1
    return experts


def _places(experts, count):
    """(group_ends, slots): rows sorted by expert, stable; what has no expert
    lies behind the last end, its place r written as -1 - r."""
    flat = experts.reshape(-1)
    key = torch.where((flat >= 0) & (flat < count), flat, torch.full_like(flat, count))
    order = torch.argsort(key, stable=True)
    slots = torch.empty_like(order)
    slots[order] = torch.arange(flat.numel(), device=flat.device)
    slots = torch.where(key < count, slots, -1 - slots)
    ends = torch.bincount(key, minlength=count + 1)[:count].cumsum(0)
    return ends.to(torch.int32), slots.to(torch.int32).view(experts.shape)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dtype = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device="cuda", dtype=dtype).mul_(scale)

    state = dict(case=case)
    if case["op"] == "route":
        t, e, k = case["tokens"], case["experts"], case["k"]
        logits = normal(t, e, scale=2.0)
        if case["masked"]:
            # Some experts for everyone, and a few tokens that have none.
            logits[:, torch.rand(e, generator=g, device="cuda") < case["masked"]] = -math.inf
            logits[torch.rand(t, generator=g, device="cuda") < 0.01] = -math.inf
        state["logits"] = logits
        state["dweights"] = torch.randn(t, k, generator=g, device="cuda") * 0.01
    elif case["op"] == "dispatch":
        state["x"] = normal(case["tokens"], case["dim"])
        state["experts"] = _choices(case, g)
        if case["grads"]:
            state["drows"] = normal(case["tokens"] * case["k"], case["dim"], scale=0.01)
    elif case["op"] == "combine":
        t, k, d = case["tokens"], case["k"], case["dim"]
        state["slots"] = _places(_choices(case, g), case["experts"])[1]
        state["rows"] = normal(t * k, d)
        state["weights"] = torch.rand(t, k, generator=g, device="cuda").softmax(1)
        if case["grads"]:
            state["dy"] = normal(t, d, scale=0.01)
    else:
        m, k, n, groups = case["rows"], case["k"], case["n"], case["groups"]
        x = normal(m, k)
        # Some channels are much larger than the rest, as in real activations.
        state["x"] = x.mul_((1.0 + 8.0 * (torch.rand(k, generator=g, device="cuda") < 0.01)).to(dtype))
        shape = (groups, n, k) if groups else (n, k)
        state["w"] = [torch.randint(-127, 128, shape, generator=g, device="cuda", dtype=torch.int8)
                      for _ in range(case["products"])]
        state["scales"] = [(torch.rand(shape[:-1], generator=g, device="cuda") + 0.5) * (k ** -0.5 / 73.0)
                           for _ in range(case["products"])]
        if groups:
            # Sizes as a skewed router gives them, one expert in eight idle.
            r = np.random.RandomState((seed * 7919 + 17) % (1 << 31))
            p = np.exp(case["skew"] * r.standard_normal(groups))
            idle = r.random_sample(groups) < 0.125
            if not idle.all():
                p[idle] = 0.0
            ends = np.cumsum(r.multinomial(m, p / p.sum()))
            state["ends"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
            # On the host too, for the plain form's loop over the groups.
            state["bounds"] = [0] + ends.tolist()
    return state


# ------------------------------------------------------------- the operators

def run(state):
    case = state["case"]
    if own:
        return _own(state, case)
    return {"route": _plain_route, "dispatch": _plain_dispatch, "combine": _plain_combine,
            "int8": _plain_int8}[case["op"]](state, case)


def _own(state, case):
    import fp32_sgemm_gb300 as sg
    if case["op"] == "route":
        logits, norm = state["logits"], case["normalize"]
        weights, experts = sg.route_topk(logits, case["k"], normalize=norm)
        if not case["grads"]:
            return {"weights": weights, "experts": experts}
        return {"weights": weights, "experts": experts,
                "dlogits": sg.route_topk_grad(logits, experts, state["dweights"], normalize=norm)}
    if case["op"] == "dispatch":
        rows, slots, ends = sg.expert_dispatch(state["x"], state["experts"], case["experts"])
        out = {"rows": rows, "slots": slots, "ends": ends}
        if case["grads"]:
            out["dx"] = sg.expert_combine(state["drows"], slots)
        return out
    if case["op"] == "combine":
        rows, slots, weights = state["rows"], state["slots"], state["weights"]
        y = sg.expert_combine(rows, slots, weights)
        if not case["grads"]:
            return y
        drows, dweights = sg.expert_combine_grad(state["dy"], rows, slots, weights)
        return {"y": y, "drows": drows, "dweights": dweights}
    x, w, scales = state["x"], state["w"], state["scales"]
    grouped = {"group_ends": state["ends"]} if case["groups"] else {}
    gemm = sg.int8_grouped_gemm if case["groups"] else sg.int8_gemm
    if case["products"] == 1:
        return gemm(x, w[0], scales[0], **grouped)
    q, s = sg.int8_quantize(x)
    return [gemm(q, w[i], scales[i], x_scales=s, dtype=x.dtype, **grouped) for i in range(2)]


def _plain_route(state, case):
    logits = state["logits"].float()
    t, e = logits.shape
    order = torch.sort(logits, dim=1, descending=True, stable=True)
    top = order.values[:, :case["k"]]
    chosen = top > -math.inf
    experts = torch.where(chosen, order.indices[:, :case["k"]], -1)
    largest = logits.amax(1, keepdim=True)
    largest = torch.where(largest > -math.inf, largest, torch.zeros_like(largest))
    p = (top - largest).exp()
    total = p.sum(1, keepdim=True) if case["normalize"] else (logits - largest).exp().sum(1, keepdim=True)
    total = torch.where(total > 0, total, torch.ones_like(total))
    weights = p / total
    if not case["grads"]:
        return {"weights": weights, "experts": experts}
    moved = weights * state["dweights"]
    mean = moved.sum(1, keepdim=True)
    if case["normalize"]:
        d = torch.zeros_like(logits)
        moved = moved - weights * mean
    else:
        d = -(logits - largest).exp() / total * mean
    # (What has no expert has weight 0 and adds nothing.)
    d.scatter_add_(1, experts.clamp(min=0), torch.where(chosen, moved, torch.zeros_like(moved)))
    return {"weights": weights, "experts": experts, "dlogits": d.to(state["logits"].dtype)}


def _plain_dispatch(state, case):
    x, experts = state["x"], state["experts"]
    ends, slots = _places(experts, case["experts"])
    has = slots.reshape(-1) >= 0
    place = torch.where(slots >= 0, slots, -1 - slots).long().reshape(-1)
    token = torch.arange(case["tokens"], device=x.device).repeat_interleave(case["k"])
    rows = torch.empty(token.numel(), case["dim"], dtype=x.dtype, device=x.device)
    rows[place] = torch.where(has[:, None], x[token], torch.zeros_like(x[:1]))
    out = {"rows": rows, "slots": slots, "ends": ends}
    if case["grads"]:
        got = state["drows"].float()[place]
        got = torch.where(has[:, None], got, torch.zeros_like(got[:1]))
        out["dx"] = got.view(case["tokens"], case["k"], case["dim"]).sum(1).to(x.dtype)
    return out


def _plain_combine(state, case):
    rows, slots, weights = state["rows"], state["slots"], state["weights"]
    has = (slots >= 0)[:, :, None]
    place = torch.where(slots >= 0, slots, -1 - slots).long()
    got = rows.float()[place]
    got = torch.where(has, got, torch.zeros_like(got[:1, :1]))
    y = (got * weights[:, :, None]).sum(1).to(rows.dtype)
    if not case["grads"]:
        return y
    dy = state["dy"].float()[:, None, :]
    dweights = (got * dy).sum(2)
    moved = torch.where(has, weights[:, :, None] * dy, torch.zeros_like(got[:1, :1]))
    drows = torch.empty_like(rows)
    drows[place.reshape(-1)] = moved.reshape(-1, case["dim"]).to(rows.dtype)
    return {"y": y, "drows": drows, "dweights": dweights}


def _plain_int8(state, case):
    x = state["x"].float()
    scale = x.abs().amax(1, keepdim=True) / 127.0
    scale = torch.where(scale > 0, scale.clamp(min=2.0 ** -126), scale)
    # The quotient in 64 bits: it decides which of two neighbours is nearer.
    over = torch.where(scale > 0, scale, torch.ones_like(scale)).double()
    q = (x.double() / over).round().float()
    rows, n, groups = case["rows"], case["n"], case["groups"]
    bounds = state["bounds"] if groups else [0, rows]
    most = max(b - a for a, b in zip(bounds, bounds[1:]))
    # Groups of like sizes: padded to the longest, all products at once.
    padded = groups and groups * most <= 4 * rows + 256
    if groups:
        ends = state["ends"].long()
        row = torch.arange(rows, device=x.device)
        group = torch.searchsorted(ends, row, right=True)
        place = row - torch.cat((ends.new_zeros(1), ends[:-1]))[group]
    out = []
    for w, ws in zip(state["w"], state["scales"]):
        total = torch.zeros(rows, n, dtype=torch.int32, device=x.device)
        for c in range(0, case["k"], 1024):         # sums below 2^24: exact in 32 bits
            part = q[:, c:c + 1024]
            if padded:
                wide = x.new_zeros(groups, most, part.shape[1])
                wide[group, place] = part
                wide = torch.bmm(wide, w[:, :, c:c + 1024].float().transpose(1, 2))
                total += wide[group, place].to(torch.int32)
                continue
            for e, (a, b) in enumerate(zip(bounds, bounds[1:])):
                if a < b:
                    we = w[e] if groups else w
                    total[a:b] += (part[a:b] @ we[:, c:c + 1024].float().t()).to(torch.int32)
        out.append((total.float() * scale * (ws[group] if groups else ws)).to(state["x"].dtype))
    return out if case["products"] > 1 else out[0]


# ------------------------------------------------------------ in 64 bits

def exact(case, seed):
    # 64-bit products run near 1 TFLOP/s here.
    if work(case)["flops"] > 1.5e13:
        return None
    state = prepare(case, seed)
    return {"route": _exact_route, "dispatch": _exact_dispatch, "combine": _exact_combine,
            "int8": _exact_int8}[case["op"]](state, case)


def _exact_route(state, case):
    logits = state["logits"].cpu().double().numpy()
    t, e = logits.shape
    k = case["k"]
    # Largest first, the lower index among equals.
    order = np.lexsort((np.broadcast_to(np.arange(e), (t, e)), -logits), axis=1)[:, :k]
    rows = np.arange(t)[:, None]
    live = np.isfinite(logits[rows, order])
    experts = np.where(live, order, -1)
    taken = np.zeros((t, e), dtype=bool)
    taken[rows, order] = live
    with np.errstate(invalid="ignore", divide="ignore"):
        powers = np.exp(logits - logits.max(1, keepdims=True))
        powers[~np.isfinite(logits)] = 0.0
        base = (powers * taken if case["normalize"] else powers).sum(1, keepdims=True)
        p = np.where(base > 0, powers / base, 0.0)
    out = {"weights": torch.from_numpy(np.where(live, p[rows, order], 0.0)), "experts": torch.from_numpy(experts)}
    if case["grads"]:
        # As a softmax whose outputs that were not taken have gradient 0.
        g = np.zeros((t, e))
        g[rows, order] = np.where(live, state["dweights"].cpu().double().numpy(), 0.0)
        p = p * taken if case["normalize"] else p
        out["dlogits"] = torch.from_numpy(p * (g - (p * g).sum(1, keepdims=True)))
    return {name: v.cuda() for name, v in out.items()}


def _exact_dispatch(state, case):
    experts = state["experts"].cpu().numpy().reshape(-1)
    count, n = case["experts"], experts.size
    # Expert by expert, the choices in their order; then what has none.
    at = [np.flatnonzero(experts == e) for e in range(count)]
    ends = np.cumsum([len(a) for a in at])
    rest = np.flatnonzero((experts < 0) | (experts >= count))
    listed_rows = np.concatenate(at + [rest])
    slots = np.empty(n, dtype=np.int64)
    slots[listed_rows] = np.arange(n)
    slots[rest] = -1 - slots[rest]
    source = torch.from_numpy(listed_rows).cuda() // case["k"]
    rows = state["x"].double()[source]
    rows[ends[-1]:] = 0.0
    out = {"rows": rows, "slots": torch.from_numpy(slots).to(torch.int32).view(case["tokens"], case["k"]).cuda(),
           "ends": torch.from_numpy(ends).to(torch.int32).cuda()}
    if case["grads"]:
        dx = torch.zeros(case["tokens"], case["dim"], dtype=torch.float64, device="cuda")
        out["dx"] = dx.index_add_(0, source[:ends[-1]], state["drows"].double()[:ends[-1]])
    return out


def _exact_combine(state, case):
    slots, k = state["slots"].long(), case["k"]
    rows, weights = state["rows"].double(), state["weights"].double()
    y = torch.zeros(case["tokens"], case["dim"], dtype=torch.float64, device="cuda")
    drows, dweights = torch.zeros_like(rows), torch.zeros_like(weights)
    for j in range(k):
        t = (slots[:, j] >= 0).nonzero()[:, 0]
        r, w = slots[t, j], weights[t, j]
        y[t] += w[:, None] * rows[r]
        if case["grads"]:
            dy = state["dy"][t].double()
            drows[r] = w[:, None] * dy
            dweights[t, j] = torch.einsum("td,td->t", rows[r], dy)
    return {"y": y, "drows": drows, "dweights": dweights} if case["grads"] else y


def _exact_int8(state, case):
    x = state["x"].double()
    # The scale is a 32-bit number; the rest follows from it.
    scale = (x.abs().max(dim=1).values / 127.0).float().double()
    q = torch.zeros_like(x)
    on = scale > 0
    q[on] = torch.round(x[on] / scale[on, None])
    out = []
    for w, ws in zip(state["w"], state["scales"]):
        y = torch.zeros(case["rows"], case["n"], dtype=torch.float64, device="cuda")
        bounds = [0] + state["ends"].tolist() if case["groups"] else [0, case["rows"]]
        for e in range(len(bounds) - 1):
            a, b = bounds[e], bounds[e + 1]
            if a < b:
                we, se = (w[e], ws[e]) if case["groups"] else (w, ws)
                y[a:b] = q[a:b].mm(we.double().t()) * scale[a:b, None] * se.double()
        out.append(y)
    return out if case["products"] > 1 else out[0]
