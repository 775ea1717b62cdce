"""Corners of the expert operators' range against the definitions in 64 bits (B200)."""
import threading

import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="no CUDA device")]

from differentiable_soft_top_b200 import experts as ex  # noqa: E402
from tests.test_gpu_experts import INF, randn, route64, small_layer, some_choice  # noqa: E402

F32, BF16, FP16 = torch.float32, torch.bfloat16, torch.float16


# ---------------------------------------------------------------------------
# routing
# ---------------------------------------------------------------------------
def same_choice(x, k, score, bias, groups=1, kept=1, top=1):
    e = ex.route(x, k, score=score, bias=bias, groups=groups, groups_kept=kept, group_top=top)[1]
    want = route64(x, k, score, bias, groups, kept, top, True, 1.0)[1]
    wrong = (e.cpu() != want).any(1)
    assert not wrong.any(), (int(wrong.sum()), wrong.nonzero().flatten()[:5].tolist())


def test_route_where_a_bias_takes_a_large_score_away():
    """The answer is expert 2, whose key of 7.333e-5 is a score of 0.94 less nearly all of it."""
    x = torch.tensor([[-9.521313667, -9.521381378, 2.819267035]], device="cuda")
    b = torch.tensor([0.0, 0.0, -0.9436348081], device="cuda")
    same_choice(x, 1, "sigmoid", b)
    assert ex.route(x, 1, score="sigmoid", bias=b)[1].item() == 2


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e,k,groups,kept,top", [(3, 1, 1, 1, 1), (40, 1, 1, 1, 1), (40, 5, 1, 1, 1), (64, 8, 8, 3, 2),
                                                 (300, 30, 1, 1, 1), (300, 32, 1, 1, 1)])
def test_route_keys_of_small_and_cancelled_scores(score, e, k, groups, kept, top):
    """Every other expert has a small score and no bias, the rest a larger score and a bias of nearly minus that: all
    keys lie within a few 1e-8 of one another, the errors of an fp32 score reach from 1e-12 to 1e-7."""
    g = torch.Generator().manual_seed(e * 7 + k)
    t = 300
    l0 = torch.full((e,), -9.5213, dtype=torch.float64)
    large = torch.arange(e) % 2 == 0 if e > 3 else torch.tensor([False, False, True])
    l0[large] = torch.randn(int(large.sum()), generator=g, dtype=torch.float64) + 2.0
    x = l0 + torch.where(large, 1e-6, 1e-4) * torch.randn(t, e, generator=g, dtype=torch.float64)
    x = x.float()
    s = torch.sigmoid(l0) if score == "sigmoid" else torch.softmax(l0, 0)
    aim = float(s[~large][0])
    bias = torch.where(large, aim - s, 0.0).float()
    same_choice(x.cuda(), k, score, bias.cuda(), groups, kept, top)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("top", [1, 2])
def test_route_near_ties_of_very_small_scores(score, top):
    """Scores of 1e-20 to 1e-37 one or two fp32 steps apart, where exp's relative error is largest; a zero bias, as at the
    start of training, keeps the comparison of the keys themselves."""
    g = torch.Generator().manual_seed(5)
    x = -(45.0 + 40.0 * torch.rand(200, 1, generator=g)) * (1 + 2.0 ** -23 * torch.randint(0, 6, (200, 64), generator=g))
    if score == "softmax":
        x[:, 0] = 0.0
    b = torch.zeros(64, device="cuda")
    same_choice(x.cuda(), 8, score, b)
    same_choice(x.cuda(), 8, score, b, 8, 3, top)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("groups", [4, 3])
@pytest.mark.parametrize("kept", [1, 2])
def test_route_groups_whose_sum_leaves_fp32(dtype, groups, kept):
    """Two keys of the lowest (or highest) value add up to more than fp32 holds: such a group still comes before one
    without experts, and two such groups are told apart."""
    low, most = torch.finfo(dtype).min, torch.finfo(dtype).max
    x = torch.zeros(6, 24, device="cuda", dtype=dtype)
    n = 24 // groups
    x[0] = low
    x[0, :n] = -INF                           # group 0 has nobody, the sums of the others are beyond fp32
    x[1] = low
    x[1, :n] = low / 2 * 1.5                  # all beyond, the first and the last higher
    x[1, -n:] = low / 2 * 1.25
    x[2] = most
    x[2, -n:] = -INF
    x[2, n:2 * n] = most / 2
    x[3, :n] = most                           # +max and 0, a group of lows between
    x[3, n:2 * n] = low
    x[4] = low
    x[4, 1::2] = -INF
    x[4, :n] = -INF
    x[5] = low
    for bias in (None, torch.zeros(24, device="cuda"), torch.full((24,), torch.finfo(F32).min / 2, device="cuda")):
        for top in (1, 2):
            if bias is not None and bias.any():
                same_choice(x[[0, 4, 5]], 3, "identity", bias, groups, kept, top)
            else:
                same_choice(x, 3, "identity", bias, groups, kept, top)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("e,k,groups,kept", [(40, 6, 1, 1), (40, 6, 4, 2), (300, 32, 1, 1), (33, 5, 3, 2)])
def test_route_subnormal_memberships(dtype, e, k, groups, kept):
    """Memberships below 2^-126, as a sharp soft choice gives to all but a few experts, are told apart."""
    g = torch.Generator().manual_seed(e)
    x = torch.rand(60, e, generator=g, dtype=torch.float64) * 1e-39
    x[:, ::7] *= -1.0
    x[::4, 3] = 0.25
    x = x.to(dtype).cuda()
    b = (torch.randn(e, generator=g, dtype=torch.float64) * 1e-39).float().cuda()
    for bias in (None, b):
        for top in (1, 2):
            same_choice(x, k, "identity", bias, groups, kept, top)


@pytest.mark.parametrize("dtype", [F32, BF16, FP16])
@pytest.mark.parametrize("k", [2, 7, 32])
def test_route_renormalised_memberships_of_the_highest_values(dtype, k):
    """Weights are shares of a sum that fp32 need not hold."""
    low, most = torch.finfo(dtype).min, torch.finfo(dtype).max
    x = torch.zeros(5, 40, device="cuda", dtype=dtype)
    x[0] = most
    x[1] = low
    x[2] = low                                # two scores, the places after them hold the lowest value
    x[2, 5], x[2, 30] = 0.5, 0.25
    x[3, ::3] = most / 2
    x[4] = 0.5
    w, e = ex.route(x, k, score="identity")
    w0, e0 = route64(x, k, "identity", None, 1, 1, 1, True, 1.0)
    assert torch.equal(e.cpu(), e0)
    # a sum of k terms in a tree (5 roundings) and a quotient
    torch.testing.assert_close(w.double().cpu(), w0, rtol=8 * 2.0 ** -24, atol=2.0 ** -126)


# ---------------------------------------------------------------------------
# exchange
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dim", [64, 7])
def test_rows_without_a_slot_get_no_gradient(dim):
    """Rows whose place was taken away after the plan was made, or whose slot is out of range, get 0, whatever stood
    in the gradient's memory."""
    t, k = 50, 3
    c = some_choice(t, k, 8, seed=3)
    p = ex.plan(c, 8)
    taken = torch.rand(t, k, generator=torch.Generator().manual_seed(1)).cuda() < 0.3
    p.rows[taken] = -1
    y, w, g = randn(t * k, dim, seed=1), randn(t, k, seed=2).abs(), randn(t, dim, seed=3)
    at = p.rows.long()
    want = torch.zeros(t * k, dim, device="cuda")
    want[at[at >= 0]] = (w[..., None] * g[:, None])[at >= 0]
    gy, gw = torch.full_like(y, 7.0), torch.full_like(w, 7.0)
    ex._call("combine_bwd", 0, g.data_ptr(), 0, t, k, dim, dim, y.data_ptr(), dim, w.data_ptr(), p.rows.data_ptr(),
             p.slots.data_ptr(), gy.data_ptr(), dim, gw.data_ptr())
    assert torch.equal(gy, want) and (gw[at < 0] == 0).all()
    y.requires_grad_(), w.requires_grad_()
    out = ex.combine(y, w, p)
    dy, dw = torch.autograd.grad(out, [y, w], g)
    assert torch.equal(dy, want) and torch.equal(dw, gw)
    # slots out of range are none
    rows = torch.tensor([[0, 9], [-3, 1]], dtype=torch.int32, device="cuda")
    slots = torch.tensor([0, 3, 77, -1], dtype=torch.int32, device="cuda")
    gy = torch.full((4, dim), 7.0, device="cuda")
    ex._call("combine_bwd", 0, g.data_ptr(), 0, 2, 2, dim, dim, y.data_ptr(), dim, None, rows.data_ptr(), slots.data_ptr(),
             gy.data_ptr(), dim, None)
    assert torch.equal(gy, torch.stack([g[0], g[1], g[0] * 0, g[0] * 0]))


# ---------------------------------------------------------------------------
# autograd
# ---------------------------------------------------------------------------
def test_forward_mode_tangents_are_refused():
    """No operator returns a result without its tangent."""
    import torch.autograd.forward_ad as fwd
    logits, x, w_in, w_out, k = small_layer(seed=5)
    w, c = ex.route(logits, k)
    p = ex.plan(c, 12)
    rows = ex.dispatch(x, p)
    y = ex.linear(rows, w_out.transpose(1, 2).contiguous(), p.offsets)
    with fwd.dual_level():
        def dual(t):
            return fwd.make_dual(t, torch.ones_like(t))
        for call in (lambda: ex.route(dual(logits), k), lambda: ex.dispatch(dual(x), p), lambda: ex.combine(y, dual(w), p),
                     lambda: ex.combine(dual(y), w, p), lambda: ex.linear(dual(rows), w_in, p.offsets),
                     lambda: ex.linear(rows, dual(w_in), p.offsets), lambda: ex.mlp(dual(x), w, c, w_in, w_out),
                     lambda: ex.mlp(x, w, c, w_in, w_out, residual=dual(x))):
            with torch.no_grad(), pytest.raises(NotImplementedError, match="jvp"):
                call()
            with pytest.raises(NotImplementedError, match="jvp"):
                call()
        assert torch.equal(ex.route(logits, k)[0], w)  # others in a level as usual


# ---------------------------------------------------------------------------
# products
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("r", [4, 70, 600])
def test_keeping_gradients_does_not_change_relu(dtype, r):
    """Pre-activations from 2^-40 to 2^-20: with and without gradients the result is the same, rounded once, and the
    gradient passes wherever they are positive."""
    g = torch.Generator("cuda").manual_seed(r)
    x = torch.zeros(r, 64, device="cuda")
    x[:, 0] = 2.0 ** torch.randint(-24, -14, (r,), generator=g, device="cuda")  # exact in both types: one product each
    w = torch.zeros(128, 64, device="cuda")
    w[:, 0] = torch.randn(128, generator=g, device="cuda").sign() * 2.0 ** torch.randint(-14, -5, (128,), generator=g, device="cuda")
    x, w = x.to(dtype), w.to(dtype)
    h = x[:, :1].double() * w[:, 0].double()
    plain = ex.linear(x, w, activation="relu")
    tracked = ex.linear(x.requires_grad_(), w.requires_grad_(), activation="relu")
    assert torch.equal(plain, h.clamp_min(0).to(dtype)) and torch.equal(tracked, plain)
    (dx,) = torch.autograd.grad(tracked, x, torch.ones_like(tracked))
    want = (h > 0).double() @ w.double()
    u = torch.finfo(dtype).eps / 2
    # the sum of at most 128 terms in fp32 and a rounding
    assert ((dx.double() - want).abs() <= u * want.abs() + 128 * 2.0 ** -24 * (w.double().abs().sum(0)) + 2.0 ** -25).all()


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "swiglu"])
@pytest.mark.parametrize("r", [12, 300])
def test_gradients_where_a_pre_activation_leaves_the_type(dtype, act, r):
    """|h| up to 2^18, beyond fp16: gradients are finite and those of the definition, of h clamped to the type's range
    (which changes only swiglu's, by its factor).  All values are powers of two, exact in the type where they fit."""
    f, most = 64, torch.finfo(dtype).max
    g = torch.Generator("cuda").manual_seed(r)

    def powers(n, lo, hi):
        sign = torch.randint(0, 2, (n,), generator=g, device="cuda") * 2.0 - 1.0
        return sign * 2.0 ** torch.randint(lo, hi + 1, (n,), generator=g, device="cuda")

    n = 2 * f if act == "swiglu" else f
    x, w = torch.zeros(r, 8, device="cuda"), torch.zeros(n, 8, device="cuda")
    x[:, 0], w[:, 0] = powers(r, 4, 10), powers(n, -12, 8)
    x, w = x.to(dtype).requires_grad_(), w.to(dtype).requires_grad_()
    b = torch.zeros(n, dtype=dtype, device="cuda", requires_grad=True)
    y = ex.linear(x, w, bias=b, activation=act)
    dy = powers(r * f, -12, -6).view(r, f).to(dtype)
    got = torch.autograd.grad(y, [x, w, b], dy)
    h = (x[:, :1].detach().double() * w[:, 0].detach().double()).clamp(-most, most)
    d = dy.double()

    def silu1(v):
        s = torch.sigmoid(v)
        return s * (1 + v * (1 - s))

    if act == "swiglu":
        a, up = h.chunk(2, 1)
        dh = torch.cat([d * up * silu1(a), d * a * torch.sigmoid(a)], 1)
        scale = torch.cat([d * up, d * a], 1).abs()
    else:
        d1 = {"relu": lambda: (h > 0).double(), "silu": lambda: silu1(h),
              "gelu": lambda: 0.5 * torch.erfc(-h * 0.5 ** 0.5) + h * torch.exp(-0.5 * h * h) / (2 * torch.pi) ** 0.5}[act]()
        dh, scale = d * d1, d.abs()
    # the derivative within 2^-20 of terms of order 1 (where h is small; beyond it vanishes or is 1), dH rounded, sums
    u = torch.finfo(dtype).eps / 2
    e = 2.0 ** -20 * scale.clamp_max(2.0 ** 6) + 2.0 ** -20 * dh.abs()
    edge = u * dh.abs() + (2.0 ** -25 if dtype == FP16 else 0.0) + e
    fits = dh.abs().amax() <= most  # else dH itself overflows, as it should
    assert fits
    for name, a, ref, tol in (("x", got[0][:, 0], dh @ w[:, 0].detach().double(), edge @ w[:, 0].detach().double().abs()),
                              ("w", got[1][:, 0], dh.T @ x[:, 0].detach().double(), edge.T @ x[:, 0].detach().double().abs()),
                              ("b", got[2], dh.sum(0), e.sum(0))):
        size = {"x": dh.abs() @ w[:, 0].detach().double().abs(), "w": dh.abs().T @ x[:, 0].detach().double().abs(),
                "b": dh.abs().sum(0)}[name]
        ok = ref.abs() <= most * (1 - 2 * u)
        err = (a.double() - ref).abs() - (1.01 * tol + u * ref.abs() + (n + r) * 2.0 ** -24 * size + 2.0 ** -25)
        assert a[ok].isfinite().all(), name
        assert (err[ok] <= 0).all(), (name, float(err[ok].max()))


@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_gelu_and_its_derivative_over_the_type(dtype):
    """Every value of the type with 2^-100 <= |h| <= 13.5 (and 0): the error is relative, in the lower tail too."""
    h = torch.arange(-2 ** 15, 2 ** 15, device="cuda").to(torch.int16).view(dtype)
    d = h.double()
    h = h[((d.abs() <= 13.5) & (d.abs() >= 2.0 ** -100)) | (d == 0)].contiguous()
    d = h.double()
    n = len(h)
    cdf = 0.5 * torch.special.erfcx(d.abs() * 0.5 ** 0.5) * torch.exp(-0.5 * d * d)  # lower tail
    cdf = torch.where(d < 0, cdf, 1.0 - cdf)
    phi = torch.exp(-0.5 * d * d) / (2 * torch.pi) ** 0.5
    # half a step of the type (in the range where its step is fixed, half of that); the exponential: two roundings of an
    # argument of up to 132 in base 2 and its constant's, 3 * 132 * 2^-24 * log 2 = 1.6e-5, the tail's factor 1e-6, others 1e-6
    u, rel = torch.finfo(dtype).eps / 2, 2e-5
    least = torch.finfo(dtype).tiny * u + 2.0 ** -126
    x, w = torch.zeros(n, 8, dtype=dtype, device="cuda"), torch.zeros(8, 8, dtype=dtype, device="cuda")
    x[:, 0], w[:, 0] = h, 1.0
    y = ex.linear(x, w, activation="gelu")
    ref = d * cdf
    err = (y[:, 3].double() - ref).abs() - ((u + rel) * ref.abs() + least)
    assert (err <= 0).all(), (float(h[err.argmax()]), float(y[err.argmax(), 3]), float(ref[err.argmax()]))
    pre, gy, gh = h[:, None].expand(n, 8).contiguous(), torch.ones(n, 8, dtype=dtype, device="cuda"), torch.empty(n, 8, dtype=dtype, device="cuda")
    ex._call("linear_act_bwd", 0, gy.data_ptr(), 1 if dtype == BF16 else 2, n, 8, 8, pre.data_ptr(), 8, 1, None, 3, gh.data_ptr(), 8,
             None, None, 0)
    ref, size = cdf + d * phi, cdf + d.abs() * phi
    # an exponential below 2^-126 counts as 0 (the code flushes subnormals): there the derivative is at most 2^-126 times
    # 0.3990 |h| + 0.5 erfcx(|h| / sqrt 2) <= 0.3990 * 13.5 + 0.04 < 6 (|h| > 13.2)
    err = (gh[:, 5].double() - ref).abs() - (u * ref.abs() + (1 + u) * rel * size + least + 5 * 2.0 ** -126)
    assert (err <= 0).all(), (float(h[err.argmax()]), float(gh[err.argmax(), 5]), float(ref[err.argmax()]))


@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_gelu_at_infinity_and_nan(dtype):
    """The limits of gelu at infinite pre-activations, NaN where they are NaN, and its derivative at the ends of what is
    finite."""
    h = torch.tensor([INF, -INF, float("nan"), torch.finfo(dtype).max, torch.finfo(dtype).min, 0.0, -0.0, 1.0], device="cuda").to(dtype)
    x, w = torch.zeros(8, 8, dtype=dtype, device="cuda"), torch.zeros(8, 8, dtype=dtype, device="cuda")
    b = h.clone()  # by the bias, so that no infinity meets another input's 0
    y = ex.linear(x, w, bias=b, activation="gelu")[0]
    assert y[0] == INF and y[1] == 0 and y[2].isnan() and y[3] == torch.finfo(dtype).max and (y[4:7] == 0).all()
    pre, gy, gh = h[:, None].expand(8, 8).contiguous(), torch.ones(8, 8, dtype=dtype, device="cuda"), torch.empty(8, 8, dtype=dtype, device="cuda")
    ex._call("linear_act_bwd", 0, gy.data_ptr(), 1 if dtype == BF16 else 2, 8, 8, 8, pre.data_ptr(), 8, 1, None, 3, gh.data_ptr(), 8,
             None, None, 0)
    d = gh[:, 0].tolist()
    assert d[2] != d[2] and d[3:7] == [1.0, 0.0, 0.5, 0.5]


def test_the_test_knob_is_the_threads_own():
    """While one host thread makes its products give up, those of another are right."""
    x, w = randn(40, 64, seed=1, dtype=BF16), randn(128, 64, seed=2, dtype=BF16)
    want, lib, got = ex.linear(x, w), ex._load(), []
    lib.lapsum_experts_test_timeout(500)
    try:
        other = threading.Thread(target=lambda: got.append(ex.linear(x, w)))
        other.start()
        other.join()
        own = ex.linear(x, w)
        torch.cuda.synchronize()
    finally:
        lib.lapsum_experts_test_timeout(0)
    assert torch.equal(got[0], want) and own.isnan().all()
    assert torch.equal(ex.linear(x, w), want)
