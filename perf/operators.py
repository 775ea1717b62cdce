"""Cases that time the expert operators of this package against plain forms.

The operators are those of a layer of experts behind a router: the choice of k experts per token and their weights
(``route``), the exchange between tokens and rows ordered by expert (``plan``, ``dispatch``, ``combine``), the product of
each expert's rows with its own weights (``linear``), and the layer that chains them (``mlp``).

``own`` says which side ``run`` computes: the plain form in elementary torch operations, or this package's entry points.
"""
import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
INF = float("inf")


# ----------------------------------------------------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------------------------------------------------
def _route(tokens, experts, k, dtype, score, renormalize, **more):
    c = dict(op="route", tokens=tokens, experts=experts, k=k, dtype=dtype, score=score, renormalize=renormalize,
             bias=False, groups=1, kept=1, top=1, scale=1.0, masked=0.0, backward=False)
    return {**c, **more}


def _exchange(tokens, experts, k, dim, dtype, **more):
    return {**dict(op="exchange", tokens=tokens, experts=experts, k=k, dim=dim, dtype=dtype, dropped=0.0, residual=False,
                   backward=False), **more}


def _linear(rows, experts, din, dout, dtype, **more):
    """experts = 0: one matrix for all rows."""
    return {**dict(op="linear", rows=rows, experts=experts, din=din, dout=dout, dtype=dtype, activation="none",
                   bias=False, residual=False, unused=0.0, backward=False), **more}


def _layer(tokens, experts, k, dim, hidden, dtype, **more):
    return {**dict(op="layer", tokens=tokens, experts=experts, k=k, dim=dim, hidden=hidden, dtype=dtype,
                   activation="swiglu", bias=False, backward=False), **more}


def listed():
    return [
        # one new token of one sequence: nothing but latency
        dict(_route(1, 64, 6, "fp32", "softmax", False), name="route_one_token"),
        # a long prompt: sigmoid scores, a balance bias, 4 of 8 groups kept, a few padded tokens
        dict(_route(16384, 256, 8, "fp32", "sigmoid", True, bias=True, groups=8, kept=4, top=2, scale=2.5, masked=0.03),
             name="route_prompt_groups"),
        # a training batch, weights not renormalised, so that every score has a gradient
        dict(_route(8190, 96, 4, "bf16", "softmax", False, backward=True), name="route_train"),
        # a batch of sequences that decode one token each
        dict(_exchange(24, 64, 8, 2048, "bf16"), name="exchange_decode"),
        # a training batch with padded tokens, the residual stream added on the way back
        dict(_exchange(4096, 64, 8, 2048, "bf16", dropped=0.05, residual=True, backward=True), name="exchange_train"),
        # one new token through the first product of eight experts: the weights' bytes
        dict(_linear(8, 64, 2048, 2048, "bf16", activation="swiglu"), name="linear_one_token"),
        # a long prompt through the first product of all experts
        dict(_linear(32768, 64, 2048, 2816, "bf16", activation="swiglu"), name="linear_prompt"),
        # a training step of the first product, biased
        dict(_linear(16384, 32, 1024, 4096, "fp16", activation="gelu", bias=True, backward=True), name="linear_train"),
        # the shared matrix that every token passes, added to the residual stream
        dict(_linear(8192, 0, 4096, 4096, "bf16", activation="relu", bias=True, residual=True), name="linear_shared"),
        # a small ragged training step at odd sizes with rows that no expert owns
        dict(_linear(1003, 7, 520, 264, "bf16", activation="silu", bias=True, residual=True, unused=0.1, backward=True),
             name="linear_ragged"),
        # the whole layer for a batch of sequences that decode
        dict(_layer(32, 64, 6, 1024, 512, "bf16"), name="layer_decode"),
        # the whole layer in a training step
        dict(_layer(2048, 32, 4, 1024, 1024, "bf16", bias=True, backward=True), name="layer_train"),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["route", "exchange", "linear", "linear", "layer"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    backward = rng.random() < 0.5
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        experts = groups * _log(rng, 4, 512 // groups)
        kept = rng.randint(1, groups)
        k = min(_log(rng, 1, 16), experts // groups * kept)
        score = rng.choice(["softmax", "sigmoid", "identity"])
        return _route(_log(rng, 1, 16384), experts, k, rng.choice(["fp32", "bf16", "fp16"]), score, rng.random() < 0.5,
                      bias=rng.random() < 0.5, groups=groups, kept=kept, top=rng.choice([1, 2]),
                      scale=rng.choice([1.0, 2.5]), masked=rng.choice([0.0, 0.1]), backward=backward)
    if op == "exchange":
        experts = _log(rng, 2, 256)
        return _exchange(_log(rng, 1, 4096), experts, min(experts, rng.randint(1, 8)), 8 * _log(rng, 8, 256),
                         rng.choice(["fp32", "bf16", "fp16"]), dropped=rng.choice([0.0, 0.1]),
                         residual=rng.random() < 0.5, backward=backward)
    act = rng.choice(["none", "relu", "silu", "gelu", "swiglu"])
    if op == "linear":
        experts = rng.choice([0, _log(rng, 1, 64)])
        return _linear(_log(rng, 1, 16384), experts, 8 * _log(rng, 8, 256), 16 * _log(rng, 4, 128), dtype,
                       activation=act, bias=rng.random() < 0.5, residual=rng.random() < 0.5,
                       unused=rng.choice([0.0, 0.1]) if experts else 0.0, backward=backward)
    experts = _log(rng, 2, 64)
    return _layer(_log(rng, 1, 2048), experts, rng.randint(1, min(8, experts)), 8 * _log(rng, 8, 128),
                  8 * _log(rng, 8, 128), dtype, activation=act, bias=rng.random() < 0.5, backward=backward)


# ----------------------------------------------------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------------------------------------------------
def _leaf(c, t):
    return t.requires_grad_() if c["backward"] else t


def prepare(c, seed):
    g = torch.Generator("cuda").manual_seed(seed * 7919 + 17)
    dt = DTYPES[c["dtype"]]

    def normal(*shape, by=1.0, to=None):
        return (torch.randn(*shape, generator=g, device="cuda") * by).to(to or dt)

    def chance(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    s = {"case": c}
    if c["op"] == "route":
        t, e = c["tokens"], c["experts"]
        scores = normal(t, e, by=1.5, to=torch.float32)
        if c["score"] == "identity":  # memberships in (0, 1)
            scores = scores.sigmoid()
        if c["masked"]:  # padded tokens have no expert left, others lose a few
            scores = scores.masked_fill(chance(t, 1) < c["masked"], -INF)
            scores = scores.masked_fill(chance(t, e) < c["masked"] / 4, -INF)
        s["scores"] = _leaf(c, scores.to(dt))
        s["bias"] = normal(e, by=0.02, to=torch.float32) if c["bias"] else None
        if c["backward"]:
            s["dweights"] = normal(t, c["k"], to=torch.float32)
    elif c["op"] == "exchange":
        t, e, k, d = c["tokens"], c["experts"], c["k"], c["dim"]
        # distinct experts of a token, the low ones more often
        liked = chance(t, e).log() / torch.linspace(1.5, 0.5, e, device="cuda")
        experts = liked.topk(k, dim=1).indices.int()
        if c["dropped"]:
            experts = experts.masked_fill(chance(t, 1) < c["dropped"], -1)
        s["experts"] = experts.contiguous()
        s["x"] = _leaf(c, normal(t, d))
        s["y"] = _leaf(c, normal(t * k, d))
        s["weights"] = _leaf(c, chance(t, k))
        s["residual"] = _leaf(c, normal(t, d)) if c["residual"] else None
        if c["backward"]:
            s["drows"], s["dout"] = normal(t * k, d), normal(t, d)
    elif c["op"] == "linear":
        r, e, n = c["rows"], c["experts"], c["dout"]
        wide = n // 2 if c["activation"] == "swiglu" else n
        s["x"] = _leaf(c, normal(r, c["din"]))
        s["weight"] = _leaf(c, normal(*([e] if e else []), n, c["din"], by=c["din"] ** -0.5))
        s["bias"] = _leaf(c, normal(*([e] if e else []), n, by=0.1)) if c["bias"] else None
        s["residual"] = _leaf(c, normal(r, wide)) if c["residual"] else None
        if c["backward"]:
            s["dout"] = normal(r, wide)
        s["offsets"], s["most"] = None, r
        if e:
            used = r - int(r * c["unused"])
            if used <= e:  # a token or two: distinct experts with a row each
                counts = torch.zeros(e, dtype=torch.int64)
                counts[torch.randperm(e, generator=torch.Generator().manual_seed(seed))[:used]] = 1
            else:
                share = torch.rand(e, generator=torch.Generator().manual_seed(seed)) + 0.5
                counts = (share / share.sum() * used).long()
                counts[seed % e] += used - int(counts.sum())
            s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)]).int().cuda()
            s["most"] = max(1, int(counts.max()))
    else:
        t, e, d, h = c["tokens"], c["experts"], c["dim"], c["hidden"]
        up = 2 * h if c["activation"] == "swiglu" else h
        s["x"] = _leaf(c, normal(t, d))
        s["scores"] = _leaf(c, normal(t, e, by=1.5))
        s["w_in"] = _leaf(c, normal(e, up, d, by=d ** -0.5))
        s["w_out"] = _leaf(c, normal(e, d, h, by=h ** -0.5))
        s["b_in"] = _leaf(c, normal(e, up, by=0.1)) if c["bias"] else None
        s["b_out"] = _leaf(c, normal(e, d, by=0.1)) if c["bias"] else None
        if c["backward"]:
            s["dout"] = normal(t, d)
    return s


def _grads(names, outs, douts, state):
    """Gradients of the leaves that `names` lists, as {"d" + name: ...}."""
    names = [n for n in names if state[n] is not None]
    got = torch.autograd.grad(outs, [state[n] for n in names], douts)
    return {"d" + n: g for n, g in zip(names, got)}


# ----------------------------------------------------------------------------------------------------------------------
# plain forms: elementary operations in 32 bits, rounded once
# ----------------------------------------------------------------------------------------------------------------------
def _first(keys, k):
    """Indices of the k highest keys of each row, the lowest index first among equal ones."""
    return torch.sort(keys, dim=-1, descending=True, stable=True).indices[..., :k]


def _plain_route(scores, bias, c):
    t, e = scores.shape
    masked = scores.detach() == -INF
    with torch.no_grad():  # the choice in 64 bits: two keys may lie closer than 32 bits tell
        s = scores.double().masked_fill(masked, -INF)
        if c["score"] == "softmax":
            s = torch.exp(s - s.amax(1, keepdim=True).nan_to_num(neginf=0.0))
            s = s / s.sum(1, keepdim=True).clamp_min(1e-300)
        elif c["score"] == "sigmoid":
            s = torch.sigmoid(s)
        keys = (s if bias is None else s + bias.double()).masked_fill(masked, -INF)
        if c["groups"] > 1:
            by = keys.view(t, c["groups"], -1)
            best = by.sort(dim=-1, descending=True).values[..., :c["top"]]
            value = torch.where(best[..., 0] == -INF, -INF, best.masked_fill(best == -INF, 0.0).sum(-1))
            stays = torch.zeros_like(value, dtype=torch.bool).scatter_(1, _first(value, c["kept"]), True)
            keys = by.masked_fill(~stays[..., None], -INF).view(t, e)
        experts = _first(keys, c["k"])
        none = keys.gather(1, experts) == -INF
    x = scores.float()
    if c["score"] == "softmax":
        x = torch.softmax(x.masked_fill(masked.all(1, keepdim=True), 0.0), 1)
    elif c["score"] == "sigmoid":
        x = torch.sigmoid(x)
    w = x.gather(1, experts).masked_fill(none, 0.0)
    if c["renormalize"]:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total > 0, total, 1.0)
    return w * c["scale"], experts.int().masked_fill(none, -1)


def _plain_plan(experts, n):
    flat = experts.flatten().long()
    order = torch.sort(torch.where(flat < 0, n, flat), stable=True).indices  # row -> slot, the dropped slots last
    counts = (flat[:, None] == torch.arange(n, device=flat.device)).sum(0)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    rows = torch.empty_like(order)
    rows[order] = torch.arange(order.numel(), device=order.device)
    used = torch.arange(order.numel(), device=order.device) < offsets[-1]
    return offsets.int(), rows.masked_fill(flat < 0, -1).view(experts.shape).int(), order.masked_fill(~used, -1).int()


def _plain_dispatch(x, slots, k):
    at = slots.long()
    return x.float()[at.clamp_min(0) // k].masked_fill((at < 0)[:, None], 0.0)


def _plain_combine(y, weights, rows, residual):
    at = rows.long()
    picked = y.float()[at.clamp_min(0)].masked_fill((at < 0)[..., None], 0.0)
    out = (weights.float()[..., None] * picked).sum(1)
    return out if residual is None else out + residual.float()


def _act(h, name):
    if name == "relu":
        return torch.relu(h)
    if name == "silu":
        return h * torch.sigmoid(h)
    if name == "gelu":
        return 0.5 * h * (1.0 + torch.erf(h * 0.5 ** 0.5))
    if name == "swiglu":
        gate, up = h.chunk(2, dim=-1)
        return gate * torch.sigmoid(gate) * up
    return h


def _plain_linear(x, weight, offsets, most, bias, activation, residual):
    x, weight = x.float(), weight.float()
    if offsets is None:
        h = x @ weight.t()
        y = _act(h if bias is None else h + bias.float(), activation)
    else:  # every expert's rows, padded to the most that one has
        o = offsets.long()
        row = torch.arange(x.shape[0], device=x.device)
        expert = torch.searchsorted(o[1:].contiguous(), row, right=True).clamp_max(o.numel() - 2)
        at = o[:-1, None] + torch.arange(most, device=x.device)
        h = torch.bmm(x[at.clamp_max(x.shape[0] - 1)], weight.transpose(1, 2))
        y = _act(h if bias is None else h + bias.float()[:, None], activation)
        y = y[expert, (row - o[expert]).clamp(0, most - 1)].masked_fill((row >= o[-1])[:, None], 0.0)
    return y if residual is None else y + residual.float()


def _plain(s, c):
    dt = DTYPES[c["dtype"]]
    if c["op"] == "route":
        w, e = _plain_route(s["scores"], s["bias"], c)
        return {"weights": w, "experts": e} | (_grads(["scores"], [w], [s["dweights"]], s) if c["backward"] else {})
    if c["op"] == "exchange":
        offsets, rows, slots = _plain_plan(s["experts"], c["experts"])
        x_rows = _plain_dispatch(s["x"], slots, c["k"]).to(dt)
        out = _plain_combine(s["y"], s["weights"], rows, s["residual"]).to(dt)
        got = {"offsets": offsets, "rows": rows, "slots": slots, "x_rows": x_rows, "out": out}
        if c["backward"]:
            got |= _grads(["x", "y", "weights", "residual"], [x_rows, out], [s["drows"], s["dout"]], s)
        return got
    if c["op"] == "linear":
        y = _plain_linear(s["x"], s["weight"], s["offsets"], s["most"], s["bias"], c["activation"], s["residual"]).to(dt)
        return {"y": y} | (_grads(["x", "weight", "bias", "residual"], [y], [s["dout"]], s) if c["backward"] else {})
    r = dict(score="softmax", groups=1, renormalize=True, k=c["k"], scale=1.0)
    w, e = _plain_route(s["scores"], None, r)
    offsets, rows, slots = _plain_plan(e, c["experts"])
    most = int((offsets[1:] - offsets[:-1]).max())
    x = _plain_dispatch(s["x"], slots, c["k"])
    h = _plain_linear(x, s["w_in"], offsets, most, s["b_in"], c["activation"], None)
    y = _plain_linear(h, s["w_out"], offsets, most, s["b_out"], "none", None)
    out = _plain_combine(y, w, rows, s["x"]).to(dt)
    got = {"experts": e, "out": out}
    if c["backward"]:
        got |= _grads(["x", "scores", "w_in", "w_out", "b_in", "b_out"], [out], [s["dout"]], s)
    return got


# ----------------------------------------------------------------------------------------------------------------------
# this package's entry points
# ----------------------------------------------------------------------------------------------------------------------
def _own(s, c):
    from differentiable_soft_top_b200 import experts as ex
    if c["op"] == "route":
        w, e = ex.route(s["scores"], c["k"], score=c["score"], bias=s["bias"], groups=c["groups"],
                        groups_kept=c["kept"], group_top=c["top"], renormalize=c["renormalize"], scale=c["scale"])
        return {"weights": w, "experts": e} | (_grads(["scores"], [w], [s["dweights"]], s) if c["backward"] else {})
    act = None if c.get("activation") == "none" else c.get("activation")
    if c["op"] == "exchange":
        p = ex.plan(s["experts"], c["experts"])
        x_rows = ex.dispatch(s["x"], p)
        out = ex.combine(s["y"], s["weights"], p, residual=s["residual"])
        got = {"offsets": p.offsets, "rows": p.rows, "slots": p.slots, "x_rows": x_rows, "out": out}
        if c["backward"]:
            got |= _grads(["x", "y", "weights", "residual"], [x_rows, out], [s["drows"], s["dout"]], s)
        return got
    if c["op"] == "linear":
        y = ex.linear(s["x"], s["weight"], s["offsets"], bias=s["bias"], activation=act, residual=s["residual"])
        return {"y": y} | (_grads(["x", "weight", "bias", "residual"], [y], [s["dout"]], s) if c["backward"] else {})
    w, e = ex.route(s["scores"], c["k"], score="softmax")
    out = ex.mlp(s["x"], w, e, s["w_in"], s["w_out"], b_in=s["b_in"], b_out=s["b_out"], activation=act, residual=s["x"])
    got = {"experts": e, "out": out}
    if c["backward"]:
        got |= _grads(["x", "scores", "w_in", "w_out", "b_in", "b_out"], [out], [s["dout"]], s)
    return got


def run(state):
    return (_own if own else _plain)(state, state["case"])


# ----------------------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------------------------------------------------
def work(c):
    z = 4 if c["dtype"] == "fp32" else 2
    if c["op"] == "route":
        t, e, k = c["tokens"], c["experts"], c["k"]
        n = t * e * z + 8 * t * k + 4 * e * c["bias"]
        if c["backward"]:
            n += t * e * z + 4 * t * k  # the scores' gradient and the weights' one
        return {"bytes": n, "flops": t * e * (10 + 6 * c["backward"])}
    if c["op"] == "exchange":
        t, k, d = c["tokens"], c["k"], c["dim"]
        n = 3 * 4 * t * k + z * d * (2 * t * (1 + k) + t * c["residual"]) + 4 * t * k
        if c["backward"]:  # rows' gradients in, tokens' out; the output's gradient in, rows' and weights' out
            n += z * d * (t * k + t + t + t * k + t * c["residual"]) + 4 * t * k
        return {"bytes": n, "flops": t * k * d * (2 + 5 * c["backward"])}
    if c["op"] == "linear":
        r, e, i, o = c["rows"], c["experts"], c["din"], c["dout"]
        wide = o // 2 if c["activation"] == "swiglu" else o
        used = r - int(r * c["unused"])
        most = min(e, used) if e else 1  # experts that can have a row
        n = z * (used * i + most * o * (i + c["bias"]) + r * wide * (1 + c["residual"]))
        if c["backward"]:
            n += z * (r * wide * (1 + c["residual"]) + r * i + max(1, e) * o * (i + c["bias"]))
        return {"bytes": n, "flops": 2 * used * i * o * (3 if c["backward"] else 1)}
    t, e, k, d, h = c["tokens"], c["experts"], c["k"], c["dim"], c["hidden"]
    up = 2 * h if c["activation"] == "swiglu" else h
    most = min(e, t * k)
    n = z * (t * e + 2 * t * d + most * d * (up + h)) + 4 * t * k
    if c["backward"]:
        n += z * (t * d + t * d + t * e + e * d * (up + h) + c["bias"] * e * (d + up))
    return {"bytes": n, "flops": 2 * t * k * d * (up + h) * (3 if c["backward"] else 1)}


# ----------------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits, with gradients written out
# ----------------------------------------------------------------------------------------------------------------------
def _exact_route(scores, bias, dweights, c):
    """The weights as a matrix over all experts: w = scale * chosen * s [/ sum over the chosen]."""
    t, e = scores.shape
    l = scores.detach().double()
    here = l > -INF
    if c["score"] == "softmax":
        top = torch.where(here, l, -1e300).max(1, keepdim=True).values
        s = torch.where(here, torch.exp(torch.where(here, l - top, 0.0)), 0.0)
        s = s / torch.where(s.sum(1, keepdim=True) > 0, s.sum(1, keepdim=True), 1.0)
    elif c["score"] == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-l))
    else:
        s = torch.where(here, l, 0.0)
    key = s + (0.0 if bias is None else bias.double())
    open_ = here.clone()
    if c["groups"] > 1:
        size, left = e // c["groups"], here.clone()
        value = torch.zeros(t, c["groups"], dtype=torch.float64, device=l.device)
        for j in range(c["top"]):
            masked = torch.where(left, key, -INF).view(t, c["groups"], size)
            best, at = masked.max(-1)
            value = value + torch.where(best > -INF, best, -INF if j == 0 else 0.0)
            left.view(t, c["groups"], size).scatter_(2, at[..., None], False)
        stay = torch.zeros(t, c["groups"], dtype=torch.bool, device=l.device)
        for _ in range(c["kept"]):
            free = torch.where(stay, -INF, value.clamp_min(-1e308))
            number = torch.arange(c["groups"], device=l.device).expand(t, -1)
            at = torch.where(free == free.max(1, keepdim=True).values, number, e).min(1, keepdim=True).values
            stay.scatter_(1, at, True)
        open_ &= stay.repeat_interleave(size, 1)
    experts, chosen = [], torch.zeros_like(open_)
    for _ in range(c["k"]):
        best = torch.where(open_, key, -INF)
        top = best.max(1, keepdim=True).values
        number = torch.arange(e, device=l.device).expand(t, e)
        at = torch.where((best == top) & open_, number, e).min(1, keepdim=True).values
        some = at < e
        at = at.clamp_max(e - 1)
        experts.append(torch.where(some, at, -1))
        chosen |= torch.zeros_like(chosen).scatter_(1, at, some)
        open_ = open_.scatter(1, at, False)
    experts = torch.cat(experts, 1)
    at = experts.clamp_min(0)
    picked = torch.where(experts >= 0, s.gather(1, at), 0.0)
    total = picked.sum(1, keepdim=True)
    total = torch.where(total > 0, total, 1.0) if c["renormalize"] else torch.ones_like(total)
    w = c["scale"] * picked / total
    got = {"weights": w, "experts": experts.int()}
    if dweights is not None:
        gk = torch.where(experts >= 0, dweights.double(), 0.0)
        ds = c["scale"] / total * (gk - ((gk * picked).sum(1, keepdim=True) / total if c["renormalize"] else 0.0))
        ds = torch.zeros_like(l).scatter_add(1, at, torch.where(experts >= 0, ds, 0.0))
        if c["score"] == "softmax":
            ds = s * (ds - (s * ds).sum(1, keepdim=True))
        elif c["score"] == "sigmoid":
            ds = ds * s * (1.0 - s)
        got["dscores"] = ds
    return got


def _exact_plan(experts, n):
    slots = [(experts.flatten() == e).nonzero()[:, 0] for e in range(n)]
    ends = torch.tensor([0] + [len(x) for x in slots]).cumsum(0)
    order = torch.cat(slots)
    rows = torch.full((experts.numel(),), -1, device=experts.device)
    rows[order] = torch.arange(len(order), device=experts.device)
    slot = torch.full_like(rows, -1)
    slot[:len(order)] = order
    return ends.tolist(), order, rows.view(experts.shape), slot


def _exact_act(h, name, dy=None):
    """act(h), or dy * act'(h) where dy is given."""
    if name == "swiglu":
        gate, up = h[:, :h.shape[1] // 2], h[:, h.shape[1] // 2:]
        s = 1.0 / (1.0 + torch.exp(-gate))
        if dy is None:
            return gate * s * up
        return torch.cat([dy * up * s * (1.0 + gate * (1.0 - s)), dy * gate * s], 1)
    if name == "relu":
        y, d = h.clamp_min(0.0), (h > 0).double()
    elif name == "silu":
        s = 1.0 / (1.0 + torch.exp(-h))
        y, d = h * s, s * (1.0 + h * (1.0 - s))
    elif name == "gelu":
        cdf = 0.5 * torch.erfc(-h / 2.0 ** 0.5)
        y, d = h * cdf, cdf + h * torch.exp(-0.5 * h * h) / (2.0 * torch.pi) ** 0.5
    else:
        y, d = h, torch.ones_like(h)
    return y if dy is None else dy * d


def _exact_linear(x, weight, ends, bias, name, dy=None):
    """y, or (dx, dweight, dbias) where dy is given, for 64-bit inputs; expert e has rows ends[e]..ends[e + 1]."""
    if dy is not None:
        dx, dw = torch.zeros_like(x), torch.zeros_like(weight)
        db = torch.zeros(weight.shape[:2], dtype=x.dtype, device=x.device)
    out = []
    for e in range(len(ends) - 1):
        a, b = ends[e], ends[e + 1]
        h = x[a:b] @ weight[e].T + (0.0 if bias is None else bias[e])
        if dy is None:
            out.append(_exact_act(h, name))
        else:
            dh = _exact_act(h, name, dy[a:b])
            dx[a:b], dw[e], db[e] = dh @ weight[e], dh.T @ x[a:b], dh.sum(0)
    if dy is not None:
        return dx, dw, db
    y = torch.cat(out)
    return torch.cat([y, y.new_zeros(x.shape[0] - len(y), y.shape[1])])


def exact(c, seed):
    s = {n: v.detach() if isinstance(v, torch.Tensor) else v for n, v in prepare(c, seed).items()}
    d = {n: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for n, v in s.items()}
    back = c["backward"]
    if c["op"] == "route":
        return _exact_route(s["scores"], s["bias"], s.get("dweights"), c)
    if c["op"] == "exchange":
        ends, order, rows, slot = _exact_plan(s["experts"], c["experts"])
        k, n = c["k"], len(order)
        x_rows, out = torch.zeros_like(d["y"]), torch.zeros_like(d["x"]) if d["residual"] is None else d["residual"].clone()
        x_rows[:n] = d["x"][order // k]
        w = d["weights"].flatten()[order]
        out.index_add_(0, order // k, w[:, None] * d["y"][:n])
        got = {"offsets": torch.tensor(ends, dtype=torch.int32, device="cuda"), "rows": rows.int(), "slots": slot.int(),
               "x_rows": x_rows, "out": out}
        if back:
            dx, dy, dw = torch.zeros_like(d["x"]), torch.zeros_like(d["y"]), torch.zeros_like(d["weights"])
            dx.index_add_(0, order // k, d["drows"][:n])
            dy[:n] = w[:, None] * d["dout"][order // k]
            dw.view(-1)[order] = (d["dout"][order // k] * d["y"][:n]).sum(1)
            got |= {"dx": dx, "dy": dy, "dweights": dw} | ({"dresidual": d["dout"]} if c["residual"] else {})
        return got
    if c["op"] == "linear":
        w, b = d["weight"], d["bias"]
        if not c["experts"]:
            w, b, ends = w[None], None if b is None else b[None], [0, c["rows"]]
        else:
            ends = s["offsets"].tolist()
        y = _exact_linear(d["x"], w, ends, b, c["activation"])
        got = {"y": y if d["residual"] is None else y + d["residual"]}
        if back:
            dx, dw, db = _exact_linear(d["x"], w, ends, b, c["activation"], d["dout"])
            got |= {"dx": dx, "dweight": dw.view(d["weight"].shape)}
            got |= {"dbias": db.view(d["bias"].shape)} if c["bias"] else {}
            got |= {"dresidual": d["dout"]} if c["residual"] else {}
        return got
    r = dict(score="softmax", groups=1, renormalize=True, k=c["k"], scale=1.0)
    first = _exact_route(s["scores"], None, None, r)
    k, act = c["k"], c["activation"]
    ends, order, _, _ = _exact_plan(first["experts"], c["experts"])
    x, w = d["x"][order // k], first["weights"].flatten()[order]
    h = _exact_linear(x, d["w_in"], ends, d["b_in"], act)
    y = _exact_linear(h, d["w_out"], ends, d["b_out"], "none")
    out = d["x"].clone().index_add_(0, order // k, w[:, None] * y)
    got = {"experts": first["experts"], "out": out}
    if back:
        do = d["dout"][order // k]
        dw = torch.zeros_like(first["weights"])
        dw.view(-1)[order] = (do * y).sum(1)
        dh, dw_out, db_out = _exact_linear(h, d["w_out"], ends, d["b_out"], "none", w[:, None] * do)
        dr, dw_in, db_in = _exact_linear(x, d["w_in"], ends, d["b_in"], act, dh)
        got["dx"] = d["dout"].clone().index_add_(0, order // k, dr)
        got["dscores"] = _exact_route(s["scores"], None, dw, r)["dscores"]
        got |= {"dw_in": dw_in, "dw_out": dw_out} | ({"db_in": db_in, "db_out": db_out} if c["bias"] else {})
    return got
