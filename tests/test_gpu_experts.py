"""The expert operators against plain definitions in 64 bits (B200).

Tolerances count roundings: u = finfo(type).eps / 2 relative per rounding to a
type, and n * 2^-24 times the sum of the terms' magnitudes for an fp32 sum of n
terms.
"""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="no CUDA device")]

import differentiable_soft_top_b200 as lt  # noqa: E402
from differentiable_soft_top_b200 import experts as ex  # noqa: E402

INF, NAN = float("inf"), float("nan")
F32, BF16, FP16 = torch.float32, torch.bfloat16, torch.float16
E32 = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def randn(*shape, seed=0, dtype=F32, by=1.0):
    g = torch.Generator("cuda").manual_seed(seed * 1009 + sum(shape))
    return (torch.randn(*shape, generator=g, device="cuda") * by).to(dtype)


# ---------------------------------------------------------------------------
# routing
# ---------------------------------------------------------------------------
def route64(scores, k, score, bias, groups, kept, top, renorm, scale):
    """(weights, chosen) token by token in Python floats (fp64)."""
    rows, b = scores.double().cpu().tolist(), None if bias is None else bias.double().cpu().tolist()
    n = len(rows[0]) if rows else 0
    out_w, out_e = [], []
    for l in rows:
        live = [i for i in range(n) if l[i] != -INF and not (b and b[i] == -INF)]
        if any(not l[i] < INF or (b and not b[i] < INF) for i in live):
            out_w.append([NAN] * k)
            out_e.append([-1] * k)
            continue
        if score == "softmax" and live:
            m = max(l[i] for i in live)
            z = math.fsum(math.exp(l[i] - m) for i in live)
            s = {i: math.exp(l[i] - m) / z for i in live}
        elif score == "sigmoid":
            s = {i: 1.0 / (1.0 + math.exp(-l[i])) if l[i] > -700 else 0.0 for i in live}
        else:
            s = {i: l[i] for i in live}
        key = {i: s[i] + (b[i] if b else 0.0) for i in live}
        if groups > 1:
            size = n // groups
            value = {}
            for g in range(groups):
                ks = sorted((key[i] for i in live if i // size == g), reverse=True)[:top]
                if ks:
                    value[g] = sum(ks)
            stay = sorted(value, key=lambda g: (-value[g], g))[:kept]
            live = [i for i in live if i // size in stay]
        pick = sorted(live, key=lambda i: (-key[i], i))[:k]
        total = math.fsum(s[i] for i in pick)
        w = [scale * s[i] / (total if renorm and total else 1.0) for i in pick]
        out_w.append(w + [0.0] * (k - len(pick)))
        out_e.append(pick + [-1] * (k - len(pick)))
    return (torch.tensor(out_w, dtype=torch.float64).view(len(rows), k),
            torch.tensor(out_e, dtype=torch.int32).view(len(rows), k))


def check_route(scores, k, score="softmax", bias=None, groups=1, kept=None, top=1, renorm=True, scale=1.0):
    kept = groups if kept is None else kept
    w, e = ex.route(scores, k, score=score, bias=bias, groups=groups, groups_kept=kept, group_top=top,
                    renormalize=renorm, scale=scale)
    w0, e0 = route64(scores, k, score, bias, groups, kept, top, renorm, scale)
    assert w.dtype == F32 and e.dtype == torch.int32
    assert torch.equal(e.cpu(), e0)
    # exp, its argument (|l| roundings), a sum of E terms in a tree, a quotient, a product
    big = scores.double().masked_fill(scores.isinf() | scores.isnan(), 0.0).abs().max().item() if scores.numel() else 0
    rel = (48 + 4 * big) * E32
    torch.testing.assert_close(w.double().cpu(), w0, rtol=rel, atol=2.0 ** -120, equal_nan=True)
    return w, e


@pytest.mark.parametrize("dtype", [F32, BF16, FP16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid", "identity"])
@pytest.mark.parametrize("t,e,k,groups,kept,top,bias,renorm", [
    (1, 1, 1, 1, 1, 1, False, True),
    (1, 64, 6, 1, 1, 1, False, False),
    (7, 33, 32, 1, 1, 1, False, True),
    (65, 96, 4, 1, 1, 1, True, False),
    (130, 256, 8, 8, 4, 2, True, True),
    (33, 250, 5, 5, 2, 1, False, True),
    (19, 512, 16, 32, 9, 2, False, False),
    (9, 1024, 32, 4, 1, 2, True, True),
    (40, 12, 3, 4, 1, 2, True, True),
])
def test_route_matches_the_definition(dtype, score, t, e, k, groups, kept, top, bias, renorm):
    x = randn(t, e, seed=1, by=1.5)
    if score == "identity":
        x = x.sigmoid()
    b = randn(e, seed=2, by=0.05) if bias else None
    check_route(x.to(dtype), k, score, b, groups, kept, top, renorm, scale=2.5 if bias else 1.0)


def test_route_without_tokens():
    w, e = ex.route(torch.empty(0, 16, device="cuda"), 4)
    assert w.shape == (0, 4) and e.shape == (0, 4)


@pytest.mark.parametrize("score", ["softmax", "sigmoid", "identity"])
@pytest.mark.parametrize("bias", [False, True])
def test_route_ties_go_to_the_lowest_index(score, bias):
    """All equal, and coarse values with many ties, with a zero bias as at the start of training."""
    b = torch.zeros(128, device="cuda") if bias else None
    check_route(torch.full((3, 128), 0.5, device="cuda", dtype=BF16), 8, score, b, 8, 3, 2)
    x = (randn(200, 128, seed=5).abs() * 3).round() / 4
    check_route(x.to(BF16), 8, score, b)
    check_route(x.to(BF16), 6, score, b, 4, 2, 2)


def test_route_keys_closer_than_fp32():
    """Keys whose fp32 values tie or swap: the order is that of the exact keys."""
    g = torch.Generator().manual_seed(3)
    base = torch.randn(64, 1, generator=g).double()
    x = (base + torch.randn(64, 64, generator=g).double() * 1e-7).float().cuda()
    b = (torch.randn(64, generator=g) * 1e-8).cuda()
    for score in ("softmax", "sigmoid", "identity"):
        e = ex.route(x.abs() if score == "identity" else x, 8, score=score, bias=b)[1]
        e0 = route64(x.abs() if score == "identity" else x, 8, score, b, 1, 1, 1, True, 1.0)[1]
        assert torch.equal(e.cpu(), e0), score


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_masks(score, renorm):
    low = torch.finfo(BF16).min
    x = randn(8, 40, seed=7, dtype=BF16)
    x[0] = -INF                     # nothing left
    x[1, 3:] = -INF                 # fewer than k
    x[2] = -INF
    x[2, 39] = 0.0                  # one, in the last place
    x[3, 5] = NAN                   # a NaN that counts
    x[4, 6] = INF
    x[5, ::2] = -INF
    x[6, 8:] = low                  # the type's lowest value is a score, not a mask
    check_route(x[:6].float(), 5, score, None, 1, 1, 1, renorm)
    check_route(x[:6], 5, score, None, 4, 2, 2, renorm)
    if score == "softmax":
        check_route(x[6:], 5, score, None, 1, 1, 1, renorm)
    b = torch.zeros(40, device="cuda")
    b[5] = -INF                     # masks the NaN of token 3
    b[6] = -INF                     # and the inf of token 4
    check_route(x[:6], 5, score, b, 1, 1, 1, renorm)
    b[7] = NAN
    assert (ex.route(x, 5, score=score, bias=b)[1][1:2] >= 0).any()  # masked there: token 1 has only 0..2
    assert (ex.route(x, 5, score=score, bias=b)[1][5] >= 0).any() == bool(x[5, 7] == -INF)


@pytest.mark.parametrize("dtype", [F32, BF16, FP16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid", "identity"])
@pytest.mark.parametrize("groups,bias", [(1, False), (4, False), (4, True)])
def test_route_lowest_values_are_scores(dtype, score, groups, bias):
    """The type's lowest value, often used as a mask, is the lowest score: chosen last, in order of the index, with
    weight 0 beside others and, where all have it, as the definition in 64 bits says."""
    low = torch.finfo(dtype).min
    x = torch.full((4, 24), low, device="cuda", dtype=dtype)
    x[1, 20] = 0.5
    x[2, ::2] = randn(12, seed=5).abs().to(dtype)
    x[3, 7] = -INF
    if score == "identity":
        x[3, 9] = -torch.tensor(torch.finfo(dtype).max * 0.75, device="cuda")
    b = torch.zeros(24, device="cuda") if bias else None
    rule = (9, score, b, groups, groups // 2 + 1, 1, score != "identity", 1.0)
    w, e = ex.route(x, 9, score=score, bias=b, groups=groups, groups_kept=groups // 2 + 1, renormalize=score != "identity")
    w0, e0 = route64(x, *rule)
    assert torch.equal(e.cpu(), e0)
    # exp of arguments below 4 and a sum, as in check_route
    torch.testing.assert_close(w.double().cpu(), w0, rtol=(48 + 4 * 4) * E32, atol=2.0 ** -120)


def test_route_strided_scores():
    wide = randn(50, 100, seed=9)
    check_route(wide[:, 3:67], 4)
    check_route(wide.t()[:64, :32], 4)
    check_route(wide[::3, :10], 4)
    check_route(wide[:1].expand(6, -1), 4)


def route_grad64(scores, chosen, score, renorm, scale, g):
    x = scores.detach().double().cpu().requires_grad_()
    l = x.masked_fill(x == -INF, -1e300)
    s = {"softmax": lambda: torch.softmax(l, 1), "sigmoid": lambda: torch.sigmoid(l), "identity": lambda: l}[score]()
    c = chosen.cpu().long()
    p = s.gather(1, c.clamp_min(0)).masked_fill(c < 0, 0.0)
    if renorm:
        total = p.sum(1, keepdim=True)
        p = p / torch.where(total == 0, 1.0, total)
    return torch.autograd.grad(scale * p, x, g.double().cpu().masked_fill(c < 0, 0.0))[0].nan_to_num(0.0)


@pytest.mark.parametrize("dtype", [F32, BF16, FP16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid", "identity"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("t,e,k", [(1, 1, 1), (5, 33, 8), (64, 256, 8), (3, 1000, 32)])
def test_route_gradient(dtype, score, renorm, t, e, k):
    x = randn(t, e, seed=11)
    x = (x.sigmoid() if score == "identity" else x).to(dtype)
    if t > 3:
        x[1] = -INF
        x[2, 2:] = -INF
    x.requires_grad_()
    w, c = ex.route(x, k, score=score, renormalize=renorm, scale=1.5)
    g = randn(t, k, seed=12)
    (dx,) = torch.autograd.grad(w, x, g)
    want = route_grad64(x, c, score, renorm, 1.5, g)
    assert dx.dtype == dtype and dx.shape == x.shape
    # w, g w summed over k, the difference, a product: relative to the row's largest term
    size = 1.5 * g.abs().amax(1, keepdim=True).double().cpu() * (1.0 if score != "identity" or not renorm else 4.0)
    tol = half_step(dtype) * want.abs() + 64 * E32 * size + 2.0 ** -24
    assert ((dx.double().cpu() - want).abs() <= tol).all()


def test_route_gradient_of_a_bad_token_is_nan_and_of_others_is_not():
    x = randn(4, 16, seed=13)
    x[2, 3] = NAN
    x.requires_grad_()
    w, c = ex.route(x, 4, renormalize=False)
    (dx,) = torch.autograd.grad(w[:, :2].sum(), x)
    assert dx[2].isnan().all() and not dx[[0, 1, 3]].isnan().any()


# ---------------------------------------------------------------------------
# exchange
# ---------------------------------------------------------------------------
def plan64(chosen, n):
    flat = chosen.flatten().cpu().tolist()
    by = [[s for s, e in enumerate(flat) if e == x] for x in range(n)] if n <= 64 else None
    if by is None:
        by = [[] for _ in range(n)]
        for s, e in enumerate(flat):
            if 0 <= e < n:
                by[e].append(s)
    offsets, order = [0], []
    for x in by:
        order += x
        offsets.append(len(order))
    rows = [-1] * len(flat)
    for r, s in enumerate(order):
        rows[s] = r
    return offsets, rows, order + [-1] * (len(flat) - len(order))


def some_choice(t, k, e, seed=0, dropped=0.1):
    g = torch.Generator().manual_seed(seed + t * 31 + e)
    c = torch.rand(t, max(e, k), generator=g).argsort(1)[:, :k].int()
    c[c >= e] = -1
    c[torch.rand(t, generator=g) < dropped] = -1
    return c.cuda()


@pytest.mark.parametrize("t,k,e", [(1, 1, 1), (1, 8, 64), (3, 2, 1024), (512, 8, 16), (4096, 1, 7), (4097, 1, 7),
                                 (1000, 9, 256), (20000, 6, 33), (70001, 8, 1000)])
def test_plan(t, k, e):
    c = some_choice(t, k, e)
    p = ex.plan(c, e)
    offsets, rows, slots = plan64(c, e)
    assert p.offsets.tolist() == offsets
    assert p.rows.flatten().tolist() == rows
    assert p.slots.tolist() == slots


def test_plan_drops_numbers_out_of_range_and_keeps_repeats():
    c = torch.tensor([[0, 5], [2, 2], [-7, 1], [2**31 - 1, -2**31], [2, 0]], dtype=torch.int32, device="cuda")
    p = ex.plan(c, 3)
    offsets, rows, slots = plan64(c, 3)
    assert (p.offsets.tolist(), p.rows.flatten().tolist(), p.slots.tolist()) == (offsets, rows, slots)
    p = ex.plan(torch.full((9, 2), -1, dtype=torch.int32, device="cuda"), 4)  # nobody is chosen
    assert p.offsets.tolist() == [0] * 5 and (p.slots == -1).all() and (p.rows == -1).all()
    p = ex.plan(torch.empty(0, 2, dtype=torch.int32, device="cuda"), 4)
    assert p.offsets.tolist() == [0] * 5 and p.rows.shape == (0, 2)


@pytest.mark.parametrize("dtype", [F32, BF16, FP16])
@pytest.mark.parametrize("t,k,e,dim", [(1, 1, 1, 1), (1, 8, 64, 2048), (24, 6, 16, 72), (5, 32, 40, 7), (300, 4, 8, 1025),
                                     (37, 9, 12, 640)])
@pytest.mark.parametrize("strided", [False, True])
def test_dispatch_and_combine(dtype, t, k, e, dim, strided):
    c = some_choice(t, k, e, seed=2)
    p = ex.plan(c, e)
    pad = 3 if strided else 0

    def rows_like(n, seed):
        return randn(n, dim + pad, seed=seed, dtype=dtype)[:, pad:].requires_grad_()

    x, y, res = rows_like(t, 1), rows_like(t * k, 2), rows_like(t, 3)
    w = torch.rand(t, k, generator=torch.Generator("cuda").manual_seed(4), device="cuda").requires_grad_()
    xr = ex.dispatch(x, p)
    slot = p.slots.long()
    want = x.detach()[slot.clamp_min(0) // k].masked_fill((slot < 0)[:, None], 0.0)
    assert torch.equal(xr, want)
    out = ex.combine(y, w, p, residual=res)
    u = half_step(dtype)
    at = p.rows.long()
    terms = w.detach().double()[..., None] * y.detach().double()[at.clamp_min(0)].masked_fill((at < 0)[..., None], 0.0)
    ref = res.detach().double() + terms.sum(1)
    size = res.detach().double().abs() + terms.abs().sum(1)
    assert ((out.double() - ref).abs() <= u * ref.abs() + (k + 1) * E32 * size + 2.0 ** -24).all()
    # gradients
    gx, go = randn(t * k, dim, seed=5, dtype=dtype), randn(t, dim, seed=6, dtype=dtype)
    dx, dy, dw, dres = torch.autograd.grad([xr, out], [x, y, w, res], [gx, go])
    assert torch.equal(dres, go)
    picked = gx.double()[at.clamp_min(0)].masked_fill((at < 0)[..., None], 0.0)
    ref, size = picked.sum(1), picked.abs().sum(1)
    assert ((dx.double() - ref).abs() <= u * ref.abs() + k * E32 * size + 2.0 ** -24).all()
    used = slot >= 0
    ref = torch.zeros_like(dy, dtype=torch.float64)
    ref[used] = w.detach().double().flatten()[slot[used]][:, None] * go.double()[slot[used] // k]
    assert ((dy.double() - ref).abs() <= (u + E32) * ref.abs() + 2.0 ** -24).all()
    dots = go.double()[:, None] * y.detach().double()[at.clamp_min(0)].masked_fill((at < 0)[..., None], 0.0)
    assert ((dw.double() - dots.sum(2)).abs() <= dim * E32 * dots.abs().sum(2) + 2.0 ** -60).all()


def test_combine_shows_a_nan_weight_and_ignores_rows_of_others():
    c = torch.tensor([[0, 1], [-1, -1], [1, 0]], dtype=torch.int32, device="cuda")
    p = ex.plan(c, 2)
    y = randn(6, 16)
    y[4:] = NAN  # rows that nobody owns
    w = torch.ones(3, 2, device="cuda")
    assert not ex.combine(y, w, p).isnan().any()
    w[1] = NAN
    out = ex.combine(y, w, p)
    assert out[1].isnan().all() and not out[[0, 2]].isnan().any()


def test_indices_out_of_range_are_none():
    rows = torch.tensor([[0, 9], [-3, 1]], dtype=torch.int32, device="cuda")
    slots = torch.tensor([0, 3, 77, -1], dtype=torch.int32, device="cuda")
    p = ex.Plan(torch.zeros(3, dtype=torch.int32, device="cuda"), rows, slots)
    x = randn(2, 8)
    assert torch.equal(ex.dispatch(x, p), torch.stack([x[0], x[1], x[0] * 0, x[0] * 0]))
    y = randn(4, 8)
    assert torch.equal(ex.combine(y, torch.ones(2, 2, device="cuda"), p), torch.stack([y[0], y[1]]))


# ---------------------------------------------------------------------------
# products
# ---------------------------------------------------------------------------
def act64(h, act):
    if act == "relu":
        return h.clamp_min(0.0)
    if act == "silu":
        return h * torch.sigmoid(h)
    if act == "gelu":
        return 0.5 * h * torch.erfc(-h * 0.5 ** 0.5)
    if act == "swiglu":
        a, b = h.chunk(2, 1)
        return a * torch.sigmoid(a) * b
    return h


def some_offsets(r, e, seed, unused):
    """Ragged row counts: some experts have none, the last `unused` rows belong to nobody."""
    g = torch.Generator().manual_seed(seed)
    cuts = torch.randint(0, r - unused + 1, (e - 1,), generator=g).sort().values
    return torch.cat([torch.zeros(1, dtype=torch.int64), cuts, torch.tensor([r - unused])]).int()


def linear_case(r, e, k, n, act, bias, residual, unused, dtype, seed=0, skew=False):
    x, w = randn(r, k, seed=seed, dtype=dtype), randn(max(e, 1), n, k, seed=seed + 1, dtype=dtype, by=k ** -0.5)
    width = n // 2 if act == "swiglu" else n
    b = randn(max(e, 1), n, seed=seed + 2, dtype=dtype, by=0.3) if bias else None
    res = randn(r, width, seed=seed + 3, dtype=dtype) if residual else None
    off = some_offsets(r, e, seed, unused) if e else None
    if skew and e > 1:
        off[1:-1] = off[-1]  # the first expert has everything
    ends = off.tolist() if e else [0, r]
    if not e:
        w, b = w[0], None if b is None else b[0]
    return x, w, None if off is None else off.cuda(), b, res, ends


def check_linear(r, e, k, n, act, bias, residual, unused, dtype, seed=0, skew=False, backward=True):
    x, w, off, b, res, ends = linear_case(r, e, k, n, act, bias, residual, unused, dtype, seed, skew)
    leaves = [t for t in (x, w, b, res) if t is not None]
    for t in leaves:
        t.requires_grad_(backward)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = ex.linear(x, w, off, bias=b, activation=act, residual=res, status=status)
    assert int(status) == 0
    u = half_step(dtype)
    d = lambda t: t.detach().double()  # noqa: E731
    w3 = d(w).view(-1, n, k)
    b2 = None if b is None else d(b).view(-1, n)
    h, size = torch.zeros(r, n, dtype=torch.float64, device="cuda"), torch.zeros(r, n, dtype=torch.float64, device="cuda")
    for i in range(len(ends) - 1):
        s = slice(ends[i], ends[i + 1])
        h[s] = d(x)[s] @ w3[i].T + (0.0 if b2 is None else b2[i])
        size[s] = d(x)[s].abs() @ w3[i].abs().T + (0.0 if b2 is None else b2[i].abs())
    used = torch.arange(r, device="cuda")[:, None] < ends[-1]
    dh = (k + 2) * E32 * size  # error of the sums
    a = act64(h, act)
    if act == "swiglu":  # |silu'| <= 1.1, |silu(x)| <= |x|
        g0, up = h.chunk(2, 1)
        e0, e1 = dh.chunk(2, 1)
        da = 1.1 * e0 * up.abs() + g0.abs() * e1 + 1.1 * e0 * e1
    else:
        da = 1.13 * dh  # |gelu'| <= 1.13
    ref = torch.where(used, a, 0.0) + (0.0 if res is None else d(res))
    # the activation's own functions: a few units of fp32
    tol = u * ref.abs() + torch.where(used, da + 2.0 ** -20 * a.abs(), 0.0) + 4 * E32 * ref.abs() + 2.0 ** -25
    bad = ~((d(y) - ref).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:3].tolist())
    if not backward:
        return
    gy = randn(*y.shape, seed=seed + 9, dtype=dtype)
    got = dict(zip(["x", "w"] + ["b"] * bias + ["res"] * residual, torch.autograd.grad(y, leaves, gy)))
    # dH and its error: h's rounding to the type and its sums moves act' (|silu''|, |gelu''| <= 0.8), dH is rounded
    G = torch.where(used, d(gy), 0.0)
    # (fp16 below 2^-14 has a fixed spacing of 2^-24, so a rounding there is off by up to 2^-25 whatever the value)
    least = 2.0 ** -25 if dtype == FP16 else 0.0
    eh = u * h.abs() + dh + least
    if act == "swiglu":
        sg = torch.sigmoid(g0)
        d1 = sg * (1 + g0 * (1 - sg))
        E0, E1 = eh.chunk(2, 1)
        gh = torch.cat([G * up * d1, G * g0 * sg], 1)
        egh = torch.cat([G.abs() * (E1 * d1.abs() + 0.8 * E0 * (up.abs() + E1)), G.abs() * 1.1 * E0], 1)
    elif act is None:
        gh, egh = G, torch.zeros_like(G)
    elif act == "relu":
        gh, egh = G * (h > 0), G.abs() * (h.abs() <= dh)
    else:
        hh = h.clone().requires_grad_()
        (d1,) = torch.autograd.grad(act64(hh, act).sum(), hh)
        gh, egh = G * d1, G.abs() * 0.8 * eh
    # before its rounding: act' is a sum of terms of order 1, each within a few 2^-22 (exp, erf, quotient)
    outer = torch.cat([G * up, G * g0], 1) if act == "swiglu" else G
    egh_sum = egh + 2.0 ** -20 * (gh.abs() + (outer.abs() if act else 0.0))
    egh = egh_sum + (u * (gh.abs() + egh_sum) + least if act else 0.0)
    gh, egh, egh_sum = [torch.where(used, t, 0.0) for t in (gh, egh, egh_sum)]
    for i in range(len(ends) - 1):
        s = slice(ends[i], ends[i + 1])
        m = ends[i + 1] - ends[i]
        ref = gh[s] @ w3[i]
        tol = u * ref.abs() + (1 + u) * (egh[s] @ w3[i].abs() + (n + 2) * E32 * (gh[s].abs() @ w3[i].abs())) + 2.0 ** -25
        assert ((d(got["x"])[s] - ref).abs() <= tol).all(), i
        ref = gh[s].T @ d(x)[s]
        tol = u * ref.abs() + (1 + u) * (egh[s].T @ d(x)[s].abs() + (m + 2) * E32 * (gh[s].abs().T @ d(x)[s].abs())) + 2.0 ** -25
        assert ((d(got["w"]).view(-1, n, k)[i] - ref).abs() <= tol).all(), i
        if bias:
            ref = gh[s].sum(0)
            tol = u * ref.abs() + (1 + u) * (egh_sum[s].sum(0) + (m + 2) * E32 * gh[s].abs().sum(0)) + 2.0 ** -25
            assert ((d(got["b"]).view(-1, n)[i] - ref).abs() <= tol).all(), i
    assert (got["x"][ends[-1]:] == 0).all()
    if residual:
        assert torch.equal(got["res"], gy)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("r,e,k,n,act,bias,residual,unused", [
    (1, 0, 8, 8, None, False, False, 0),            # the smallest
    (1, 0, 2048, 256, "relu", True, True, 0),       # one token, a long sum split over blocks
    (8, 64, 512, 272, "swiglu", True, False, 0),    # one token of eight experts
    (33, 5, 72, 136, "silu", True, True, 4),
    (100, 3, 64, 128, None, False, False, 100),     # nobody owns a row
    (257, 2, 264, 520, "gelu", True, True, 1),
    (700, 4, 200, 400, "swiglu", True, True, 30),
    (1003, 7, 520, 264, "silu", True, True, 100),
    (2000, 3, 328, 648, None, True, False, 0),
    (515, 1, 1032, 1048, "relu", False, True, 3),
    (1500, 0, 256, 512, "gelu", True, False, 0),
])
def test_linear(dtype, r, e, k, n, act, bias, residual, unused):
    check_linear(r, e, k, n, act, bias, residual, unused, dtype, seed=r)


@pytest.mark.parametrize("act", [None, "swiglu"])
def test_linear_many_experts_and_skew(act):
    check_linear(600, 1024, 64, 64, act, True, False, 10, BF16, seed=3)
    check_linear(3000, 16, 128, 256, act, True, True, 0, BF16, seed=4, skew=True)
    check_linear(40, 300, 136, 272, act, False, True, 5, FP16, seed=5)


def test_linear_without_rows():
    w = randn(3, 16, 8, dtype=BF16).requires_grad_()
    x = torch.empty(0, 8, dtype=BF16, device="cuda", requires_grad=True)
    y = ex.linear(x, w, torch.zeros(4, dtype=torch.int32, device="cuda"))
    dx, dw = torch.autograd.grad(y, [x, w], torch.empty_like(y))
    assert y.shape == (0, 16) and dx.shape == (0, 8) and (dw == 0).all()


def test_linear_rows_of_others_do_not_reach_a_gradient():
    """NaN in rows that no expert owns stays out of everything."""
    x, w, off, b, _, ends = linear_case(300, 3, 128, 256, "gelu", True, False, 77, BF16, seed=6)
    x[ends[-1]:] = NAN
    for t in (x, w, b):
        t.requires_grad_()
    y = ex.linear(x, w, off, bias=b, activation="gelu")
    g = torch.ones_like(y)
    g[ends[-1]:] = NAN
    for t in (y, *torch.autograd.grad(y, [x, w, b], g)):
        assert not t.isnan().any()


def test_linear_strides_and_alignment():
    """Column slices, odd row strides and unaligned starts give the contiguous result."""
    x, w, off, b, res, _ = linear_case(70, 4, 64, 128, "relu", True, True, 3, BF16, seed=8)
    want = ex.linear(x, w, off, bias=b, activation="relu", residual=res)
    wide = randn(70, 200, dtype=BF16)
    for at in (0, 8, 3):
        wide[:, at:at + 64] = x
        assert torch.equal(ex.linear(wide[:, at:at + 64], w, off, bias=b, activation="relu", residual=res), want)
    rw = randn(70, 131, dtype=BF16)
    rw[:, 3:] = res
    assert torch.equal(ex.linear(x, w, off, bias=b, activation="relu", residual=rw[:, 3:]), want)
    flat = torch.empty(w.numel() + 1, dtype=BF16, device="cuda")
    flat[1:] = w.flatten()
    assert torch.equal(ex.linear(x, flat[1:].view(w.shape), off, bias=b, activation="relu", residual=res), want)
    wt = w.transpose(1, 2).contiguous().transpose(1, 2)
    assert torch.equal(ex.linear(x, wt, off, bias=b, activation="relu", residual=res), want)


def test_linear_infinities_and_nan_stay_in_their_rows():
    x, w, off, b, _, ends = linear_case(200, 3, 64, 64, None, False, False, 0, BF16, seed=9)
    x[17, 5], x[150, 60] = INF, NAN
    y = ex.linear(x, w, off)
    rows = (~y.isfinite()).any(1).nonzero().flatten().tolist()
    assert rows == [17, 150]


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
def layer64(logits, x, w_in, w_out, b_in, b_out, chosen, act, score):
    s = torch.softmax(logits, 1) if score == "softmax" else logits
    c = chosen.long()
    p = s.gather(1, c)
    p = p / p.sum(1, keepdim=True)
    out = x.clone()
    for e in range(w_in.shape[0]):
        t, j = (c == e).nonzero(as_tuple=True)
        h = act64(x[t] @ w_in[e].T + b_in[e], act)
        out = out.index_add(0, t, p[t, j][:, None] * (h @ w_out[e].T + b_out[e]))
    return out


@pytest.mark.parametrize("t,e,k,dim,hidden,act", [(1, 8, 2, 64, 32, "swiglu"), (50, 16, 4, 128, 64, "gelu"),
                                                (400, 8, 2, 64, 72, "swiglu")])
@pytest.mark.parametrize("score", ["softmax", "identity"])
def test_layer_forward_and_backward(t, e, k, dim, hidden, act, score):
    """Scores -> choice -> layer -> gradients of everything, also behind soft_topk."""
    up = 2 * hidden if act == "swiglu" else hidden
    logits = randn(t, e, seed=21).requires_grad_()
    leaves = [logits, randn(t, dim, seed=22, dtype=BF16), randn(e, up, dim, seed=23, dtype=BF16, by=dim ** -0.5),
              randn(e, dim, hidden, seed=24, dtype=BF16, by=hidden ** -0.5), randn(e, up, seed=25, dtype=BF16, by=0.1),
              randn(e, dim, seed=26, dtype=BF16, by=0.1)]
    _, x, w_in, w_out, b_in, b_out = [z.requires_grad_() for z in leaves]
    soft = lt.soft_topk(logits, float(k), 0.5) if score == "identity" else logits
    w, c = ex.route(soft, k, score=score)
    out = ex.mlp(x, w, c, w_in, w_out, b_in=b_in, b_out=b_out, activation=act, residual=x)
    g = randn(t, dim, seed=27, dtype=BF16)
    got = torch.autograd.grad(out, leaves, g, retain_graph=True)
    wide = [z.detach().double().requires_grad_() for z in leaves]
    if score == "identity":  # soft_topk's own gradient carries on from the memberships' one
        mem = soft.detach().double().requires_grad_()
        ref = layer64(mem, *wide[1:], c, act, score)
        (gm, *rest) = torch.autograd.grad(ref, [mem, *wide[1:]], g.double())
        (gl,) = torch.autograd.grad(soft, logits, gm.float())
        want = [gl.double(), *rest]
    else:
        ref = layer64(*wide, c, act, score)
        want = torch.autograd.grad(ref, wide, g.double())
    # five roundings to bf16 in a row on the way forward, as many back (h, y, out; dy, dh, ..): each half a step in
    # norm, the weights' gradient a difference of k of them
    u = half_step(BF16)
    assert (out.double() - ref).norm() <= 5 * u * ref.norm()
    for a, b in zip(got, want):
        assert (a.double() - b).norm() <= 12 * u * b.norm() + 1e-12


def test_runs_are_repeatable_bit_for_bit():
    x, w, off, b, res, _ = linear_case(900, 9, 256, 512, "silu", True, True, 11, BF16, seed=31)
    leaves = [t.requires_grad_() for t in (x, w, b, res)]

    def once():
        y = ex.linear(x, w, off, bias=b, activation="silu", residual=res)
        return [y, *torch.autograd.grad(y, leaves, torch.ones_like(y))]

    for a, b2 in zip(once(), once()):
        assert torch.equal(a, b2)


def small_layer(seed=41):
    t, e, k, dim, hidden = 96, 12, 3, 64, 48
    return (randn(t, e, seed=seed), randn(t, dim, seed=seed + 1, dtype=BF16),
            randn(e, 2 * hidden, dim, seed=seed + 2, dtype=BF16, by=0.1),
            randn(e, dim, hidden, seed=seed + 3, dtype=BF16, by=0.1), k)


def test_captured_layer_replays_on_new_inputs():
    logits, x, w_in, w_out, k = small_layer()

    def layer():
        w, c = ex.route(logits, k, bias=None)
        return ex.mlp(x, w, c, w_in, w_out, residual=x)

    layer()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer()
    other = small_layer(seed=51)
    logits.copy_(other[0])
    x.copy_(other[1])
    graph.replay()
    torch.cuda.synchronize()
    want = layer()
    assert torch.equal(out, want)


def test_captured_training_step_replays():
    logits, x, w_in, w_out, k = small_layer(seed=61)
    leaves = [z.requires_grad_() for z in (logits, x, w_in, w_out)]

    def step():
        w, c = ex.route(logits, k, score="sigmoid")
        out = ex.mlp(x, w, c, w_in, w_out)
        return torch.autograd.grad(out, leaves, torch.ones_like(out))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    with torch.no_grad():
        x.copy_(small_layer(seed=71)[1])
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, step()):
        assert torch.equal(a, b)


def test_two_streams_at_once():
    layers = [small_layer(seed=s) for s in (81, 91)]

    def run(l):
        w, c = ex.route(l[0], l[4])
        return ex.mlp(l[1], w, c, l[2], l[3])

    want = [run(l) for l in layers]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(run(layers[i]))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(w, o) for o in g)


def test_launches_are_counted_and_traced():
    logits, x, w_in, w_out, k = small_layer(seed=95)
    before = lt.launch_count()
    lt.trace_enable(True)
    w, c = ex.route(logits, k)
    ex.mlp(x, w, c, w_in, w_out)
    lt.trace_enable(False)
    names = lt.trace_collect()
    assert lt.launch_count() - before == 6
    assert set(names) == {"k_route_fwd", "k_plan_place", "k_dispatch", "k_product_fwd", "k_combine"}
    assert names["k_product_fwd"][0] == 2


# ---------------------------------------------------------------------------
# what users do around the operators
# ---------------------------------------------------------------------------
def test_one_call_layer_equals_its_steps():
    logits, x, w_in, w_out, k = small_layer(seed=101)
    b_in, b_out = randn(12, 96, seed=1, dtype=BF16), randn(12, 64, seed=2, dtype=BF16)
    logits[3] = -INF  # a token without experts keeps its residual
    w, c = ex.route(logits, k)
    p = ex.plan(c, 12)
    h = ex.linear(ex.dispatch(x, p), w_in, p.offsets, bias=b_in, activation="swiglu")
    y = ex.combine(ex.linear(h, w_out, p.offsets, bias=b_out), w, p, residual=x)
    out = ex.mlp(x, w, c, w_in, w_out, b_in=b_in, b_out=b_out, residual=x)
    assert torch.equal(out, y) and torch.equal(out[3], x[3])
    with torch.enable_grad():
        tracked = ex.mlp(x.detach().requires_grad_(), w, c, w_in, w_out, b_in=b_in, b_out=b_out, residual=x)
    assert torch.equal(tracked, out)
    # strided x and residual, a wider output buffer's neighbour left alone
    wide = randn(96, 70, dtype=BF16)
    wide[:, 3:67] = x
    assert torch.equal(ex.mlp(wide[:, 3:67], w, c, w_in, w_out, b_in=b_in, b_out=b_out, residual=wide[:, 3:67]), out)
    empty = ex.mlp(x[:0], w[:0], c[:0], w_in, w_out)
    assert empty.shape == (0, 64)


def test_layer_gradients_equal_those_of_its_steps():
    """The one-call layer's gradients are, bit for bit, those of the chained operators; every subset of them too."""
    logits, x, w_in, w_out, k = small_layer(seed=105)
    b_in, b_out = randn(12, 96, seed=1, dtype=BF16), randn(12, 64, seed=2, dtype=BF16)
    logits[5] = -INF
    w, c = ex.route(logits, k)
    g = randn(96, 64, seed=3, dtype=BF16)
    base = [x, w, w_in, w_out, b_in, b_out]

    def steps(x, w, w_in, w_out, b_in, b_out, res):
        p = ex.plan(c, 12)
        h = ex.linear(ex.dispatch(x, p), w_in, p.offsets, bias=b_in, activation="swiglu")
        return ex.combine(ex.linear(h, w_out, p.offsets, bias=b_out), w, p, residual=res)

    res = randn(96, 64, seed=4, dtype=BF16).requires_grad_()
    leaves = [t.detach().requires_grad_() for t in base]
    want = torch.autograd.grad(steps(*leaves, res), leaves + [res], g)
    got = torch.autograd.grad(ex.mlp(*leaves[:2], c, *leaves[2:4], b_in=leaves[4], b_out=leaves[5], residual=res), leaves + [res], g)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    for mask in (1, 2, 4, 8, 16, 32, 10, 21):
        some = [t.detach().requires_grad_(bool(mask >> i & 1)) for i, t in enumerate(base)]
        out = ex.mlp(*some[:2], c, *some[2:4], b_in=some[4], b_out=some[5])
        part = torch.autograd.grad(out, [t for t in some if t.requires_grad], g)
        assert all(torch.equal(a, want[i]) for a, i in zip(part, [i for i in range(6) if mask >> i & 1])), mask
    # x as its own residual: one rounding of the sum of both gradients
    (both,) = torch.autograd.grad(ex.mlp(leaves[0], w, c, w_in, w_out, b_in=b_in, b_out=b_out, residual=leaves[0]), leaves[0], g)
    exact = want[0].double() + g.double()
    assert ((both.double() - exact).abs() <= half_step(BF16) * (exact.abs() + want[0].double().abs()) + 2.0 ** -24).all()


def test_every_subset_of_gradients():
    """A leaf that wants no gradient changes nothing for the others."""
    x, w, off, b, res, _ = linear_case(150, 4, 64, 128, "silu", True, True, 9, BF16, seed=111)
    g = randn(150, 128, seed=112, dtype=BF16)
    full = None
    for mask in (15, 1, 2, 4, 8, 6, 9):
        leaves = [t.detach().requires_grad_(bool(mask >> i & 1)) for i, t in enumerate((x, w, b, res))]
        y = ex.linear(leaves[0], leaves[1], off, bias=leaves[2], activation="silu", residual=leaves[3])
        got = torch.autograd.grad(y, [t for t in leaves if t.requires_grad], g)
        full = full or got
        want = [full[i] for i in range(4) if mask >> i & 1]
        assert all(torch.equal(a, c) for a, c in zip(got, want))


def test_expanded_gradients_and_inputs():
    """Gradients of broadcast inputs are summed, stride-0 gradients are read as they are meant."""
    x, w, off, _, _, _ = linear_case(60, 3, 64, 64, None, False, False, 0, BF16, seed=121)
    row = randn(1, 64, seed=122, dtype=BF16).requires_grad_()
    y = ex.linear(x, w, off, residual=row.expand(60, 64))
    y.sum().backward()
    assert torch.equal(row.grad, torch.full_like(row, 60.0))
    p = ex.plan(some_choice(60, 2, 3, dropped=0.0), 3)
    weights = torch.full((60, 1), 0.5, device="cuda", requires_grad=True)
    yy = randn(120, 64, seed=123)
    ex.combine(yy, weights.expand(60, 2), p).sum().backward()
    want = yy[p.rows.long()].double().sum((1, 2)).view(60, 1)
    size = yy[p.rows.long()].double().abs().sum((1, 2)).view(60, 1)
    assert ((weights.grad.double() - want).abs() <= 130 * E32 * size).all()


def test_differentiating_twice_is_refused():
    x = randn(4, 8, seed=131).requires_grad_()
    w, _ = ex.route(x, 2)
    with pytest.raises(RuntimeError, match="twice"):
        torch.autograd.grad(w.sum(), x, create_graph=True)


def test_route_gradient_against_differences():
    """Central differences of the operator itself: step h, truncation h^2 / 6 times a third derivative below 1, fp32
    noise of a few 2^-23 over 2 h."""
    h = 2.0 ** -6
    for score in ("softmax", "sigmoid", "identity"):
        for renorm in (False, True):
            x = randn(6, 10, seed=141)
            x = (x.sigmoid() + torch.arange(10, device="cuda") if score == "identity" else x + 0.5 * torch.arange(10, device="cuda"))
            x.requires_grad_()
            g = randn(6, 4, seed=142)
            w, c = ex.route(x, 4, score=score, renormalize=renorm)
            (dx,) = torch.autograd.grad(w, x, g)
            for i in range(10):
                step = torch.zeros_like(x)
                step[:, i] = h
                up, cu = ex.route((x + step).detach(), 4, score=score, renormalize=renorm)
                dn, cd = ex.route((x - step).detach(), 4, score=score, renormalize=renorm)
                same = (cu == c).all(1) & (cd == c).all(1)  # at fixed choice
                diff = ((up - dn) * g).sum(1) / (2 * h)
                tol = g.abs().sum(1) * (h * h / 6 + 16 * E32 * 10 / h)
                assert ((diff - dx[:, i]).abs() <= tol)[same].all(), (score, renorm, i)


def test_tests_own_derivatives_against_differences():
    h = torch.linspace(-4, 4, 257, dtype=torch.float64)
    for act in ("silu", "gelu"):
        x = h.clone().requires_grad_()
        (d,) = torch.autograd.grad(act64(x, act).sum(), x)
        e = 1e-5
        assert ((act64(h + e, act) - act64(h - e, act)) / (2 * e) - d).abs().max() < 1e-9


def test_a_waiting_product_gives_up_and_says_so():
    """Copies that never come (a test knob): status, NaN in the rows of experts, and the next call works."""
    lib = ex._load()
    for case in ((40, 4, 256, 512, None), (400, 4, 256, 512, "swiglu"), (2000, 2, 256, 512, "gelu"), (8, 0, 2048, 256, None)):
        r, e, k, n, act = case
        x, w, off, _, _, ends = linear_case(r, e, k, n, act, False, False, 3 if e else 0, BF16, seed=r)
        want = ex.linear(x, w, off, activation=act)
        w3 = w.view(-1, n, k)
        gh, gx, gw = randn(r, n, seed=5, dtype=BF16), torch.zeros_like(x), torch.zeros_like(w)
        grads = lambda st: (ex._call("linear_dx", 0, gh.data_ptr(), 1, r, n, n, w.data_ptr(), w3.shape[0], k,  # noqa: E731
                                     ex._ptr(off), gx.data_ptr(), k, st.data_ptr()),
                            ex._call("linear_dweight", 0, gh.data_ptr(), 1, r, n, n, x.data_ptr(), k, k, w3.shape[0],
                                     ex._ptr(off), gw.data_ptr(), st.data_ptr()))
        status, status2 = torch.zeros(2, dtype=torch.int32, device="cuda").chunk(2)
        lib.lapsum_experts_test_timeout(500)
        try:
            y = ex.linear(x, w, off, activation=act, status=status)
            grads(status2)
            torch.cuda.synchronize()
        finally:
            lib.lapsum_experts_test_timeout(0)
        assert int(status) == int(status2) == ex.STATUS_TIMEOUT
        used = ends[-1]
        assert y[:used].isnan().all() and (y[used:] == 0).all()
        assert gx[:used].isnan().all() and (gx[used:] == 0).all()
        for i in range(len(ends) - 1):
            g = gw.view(-1, n, k)[i]
            assert g.isnan().all() if ends[i + 1] > ends[i] else (g == 0).all()
        status.zero_()
        assert torch.equal(ex.linear(x, w, off, activation=act, status=status), want) and int(status) == 0
        grads(status)
        assert int(status) == 0 and not gx.isnan().any() and not gw.isnan().any()


def test_offsets_out_of_range_are_never_followed():
    """Nonsense offsets give nonsense rows, but nothing outside the arrays is touched."""
    x, w, _, b, _, _ = linear_case(300, 5, 64, 128, "silu", True, False, 0, BF16, seed=151)
    for bad in ([-5, 10**9, 3, 250, -2**31, 2**31 - 1], [300, 200, 100, 50, 20, 0], [7, 7, 7, 7, 7, 7], [0, 400, 400, 400, 400, 400]):
        off = torch.tensor(bad, dtype=torch.int64).to(torch.int32).cuda()
        leaves = [t.detach().requires_grad_() for t in (x, w, b)]
        y = ex.linear(leaves[0], leaves[1], off, bias=leaves[2], activation="silu")
        torch.autograd.grad(y, leaves, torch.ones_like(y))
        torch.cuda.synchronize()
    # and the next good call is right
    check_linear(300, 5, 64, 128, "silu", True, False, 7, BF16, seed=151)


def test_outputs_stay_inside_their_rows():
    """Neighbours of a strided output, and what lies behind it, keep their values."""
    r, n, k = 70, 40, 64
    x, w, off, _, _, ends = linear_case(r, 3, k, n, None, False, False, 5, BF16, seed=161)
    want = ex.linear(x, w, off)
    buf = torch.full((r + 4, 64), 7.0, dtype=BF16, device="cuda")
    ex._call("linear_fwd", 0, x.data_ptr(), 1, r, k, k, w.data_ptr(), 3, n, off.data_ptr(), None, 0, None, 0, buf.data_ptr(),
             64, None, 0, None)
    assert torch.equal(buf[:r, :n], want)
    assert (buf[:, n:] == 7).all() and (buf[r:] == 7).all()
    pre = torch.full((r, n), 7.0, dtype=BF16, device="cuda")
    ex._call("linear_fwd", 0, x.data_ptr(), 1, r, k, k, w.data_ptr(), 3, n, off.data_ptr(), None, 1, None, 0, buf.data_ptr(),
             64, pre.data_ptr(), n, None)
    assert torch.equal(pre[:ends[-1]], want[:ends[-1]]) and (pre[ends[-1]:] == 7).all()


@pytest.mark.slow
def test_arrays_longer_than_32_bits_count():
    """Rows beyond the 2^31st element of x, y and the exchanged rows."""
    r, n = 140_000, 16_384  # 2.3e9 values
    x, w = randn(r, 64, seed=171, dtype=BF16), randn(n, 64, seed=172, dtype=BF16)
    y = ex.linear(x, w)
    for s in (slice(0, 3), slice(131_070, 131_074), slice(r - 3, r)):
        ref = x[s].double() @ w.double().T
        size = x[s].double().abs() @ w.double().abs().T
        assert ((y[s].double() - ref).abs() <= half_step(BF16) * ref.abs() + 66 * E32 * size).all()
    c = torch.arange(r, device="cuda", dtype=torch.int32).remainder(7).view(r, 1)
    p = ex.plan(c, 7)
    rows = ex.dispatch(y, p)
    for t in (0, 131_072, r - 1):
        assert torch.equal(rows[int(p.rows[t, 0])], y[t])
    back = ex.combine(rows, torch.ones(r, 1, device="cuda"), p)
    assert torch.equal(back[-1000:], y[-1000:])
    (gx,) = torch.autograd.grad(ex.linear(x.requires_grad_(), w), x, y)
    ref, size = y[-4:].double() @ w.double(), y[-4:].double().abs() @ w.double().abs()
    assert ((gx[-4:].double() - ref).abs() <= half_step(BF16) * ref.abs() + (n + 2) * E32 * size).all()


@pytest.mark.parametrize("call,error,match", [
    (lambda t: ex.route(t.x, 0), ValueError, "k must"),
    (lambda t: ex.route(t.x, 65), ValueError, "k must"),
    (lambda t: ex.route(t.x, 2, score="tanh"), ValueError, "score"),
    (lambda t: ex.route(t.x, 2, groups=5), ValueError, "groups"),
    (lambda t: ex.route(t.x, 2, groups=4, groups_kept=5), ValueError, "groups"),
    (lambda t: ex.route(t.x, 2, group_top=3), ValueError, "groups"),
    (lambda t: ex.route(t.x, 2, scale=0.0), ValueError, "scale"),
    (lambda t: ex.route(t.x, 2, bias=t.x[0].double()), ValueError, "bias"),
    (lambda t: ex.route(t.x.double(), 2), TypeError, "scores"),
    (lambda t: ex.route(t.x[0], 2), ValueError, "2-D"),
    (lambda t: ex.plan(t.c.long(), 4), TypeError, "int32"),
    (lambda t: ex.plan(t.c, 0), ValueError, "experts"),
    (lambda t: ex.plan(t.c.repeat(1, 20), 4), ValueError, "places"),
    (lambda t: ex.dispatch(t.x[:5], t.p), ValueError, "tokens"),
    (lambda t: ex.combine(t.x, t.w, t.p), ValueError, "rows"),
    (lambda t: ex.combine(t.rows, t.w.half(), t.p), ValueError, "weights"),
    (lambda t: ex.combine(t.rows, t.w, t.p, residual=t.x.half()), ValueError, "residual"),
    (lambda t: ex.linear(t.x, t.m[0]), TypeError, "bfloat16"),
    (lambda t: ex.linear(t.h, t.m[0].half()), TypeError, "weight"),
    (lambda t: ex.linear(t.h, t.m), ValueError, "2-D"),
    (lambda t: ex.linear(t.h, t.m, t.off[:3]), ValueError, "offsets"),
    (lambda t: ex.linear(t.h, t.m, t.off.long()), TypeError, "int32"),
    (lambda t: ex.linear(t.h, t.m[:, :20], t.off), ValueError, "multiples"),
    (lambda t: ex.linear(t.h[:, :60], t.m[..., :60], t.off), ValueError, "multiples"),
    (lambda t: ex.linear(t.h, t.m[:, :24], t.off, activation="swiglu"), ValueError, "multiples"),
    (lambda t: ex.linear(t.h, t.m, t.off, activation="tanh"), ValueError, "activation"),
    (lambda t: ex.linear(t.h, t.m, t.off, bias=t.m[0, 0]), ValueError, "bias"),
    (lambda t: ex.linear(t.h, t.m, t.off, residual=t.h[:, :8]), ValueError, "residual"),
    (lambda t: ex.mlp(t.h, t.w, t.c, t.m, t.m[:, :, :8]), ValueError, "w_out"),
    (lambda t: ex.mlp(t.h, t.w, t.c[:3], t.m, t.m, activation=None), ValueError, "chosen"),
    (lambda t: ex.mlp(t.h, t.w[:, :1], t.c, t.m, t.m, activation=None), ValueError, "weights"),
])
def test_binding_refuses(call, error, match):
    class T:
        x = randn(6, 64)
        c = torch.zeros(6, 2, dtype=torch.int32, device="cuda")
        w = torch.ones(6, 2, device="cuda")
        p = ex.plan(c, 4)
        rows = randn(12, 64)
        h = x.to(BF16)
        m = randn(4, 64, 64, dtype=BF16)
        off = torch.tensor([0, 2, 2, 4, 6], dtype=torch.int32, device="cuda")
    before = lt.launch_count()
    with pytest.raises(error, match=match):
        call(T)
    assert lt.launch_count() == before
