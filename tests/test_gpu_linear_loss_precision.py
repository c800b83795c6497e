"""What keeps the output-layer losses' gradients and log-sum-exps accurate, each pinned
so that its loss shows: the second term of 16-bit derivatives for up to 32 tokens, the
factor that derivatives carry, and log-sum-exps kept in 64 bits.

A gradient is compared with the two numbers of its type that its exact value, less and
plus a tolerance for everything but its last rounding, rounds to.
"""
import math

import pytest
import torch

import dense_gemm_16_amd as mg
from gpu_helpers import say

pytestmark = pytest.mark.gpu

TORCH = {"f16": torch.float16, "bf16": torch.bfloat16}


def between(got, exact, tol):
    """Elements outside [round(exact - tol), round(exact + tol)]: rounding is monotone, so
    there are none if got is the rounding of a number within tol of exact."""
    low, high = (exact - tol).to(got.dtype), (exact + tol).to(got.dtype)
    return int(((got < low) | (got > high)).sum())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("distil", [False, True])
@pytest.mark.parametrize("T", [1, 5, 31, 32])
def test_few_tokens_hold_derivatives_to_two_terms(T, distil, dtype):
    """x and w lie in different columns, so all logits are 0 over V = 128 columns, and dz =
    c / 128, less c p at the targets (p = 1; distillation: two entries of 1/2): known but
    for its rounding, which is off by u |dz| for one term (u: half a step of the type) and
    u^2 |dz| for two, FP16's smallest steps aside (c 2^-37: the factor puts the largest c
    above 2^13).  q, the coefficient and the difference round in FP32: 2^-22 c (q + p).
    Sums of n products: n 2^-23 sum |dz w|, and one product by the factor's inverse."""
    V, D = 128, 144
    g = torch.Generator(device="cuda").manual_seed(T)
    u = torch.finfo(TORCH[dtype]).eps / 2
    x, w = torch.zeros(T, D, device="cuda"), torch.zeros(V, D, device="cuda")
    x[:, :72] = torch.randn(T, 72, generator=g, device="cuda")
    w[:, 72:] = torch.randn(V, 72, generator=g, device="cuda")
    x, w = x.to(TORCH[dtype]), w.to(TORCH[dtype])
    grad = torch.rand(T, generator=g, device="cuda") + 0.25
    tau = 2.0 if distil else 1.0
    index = torch.rand(T, V, generator=g, device="cuda").argsort(1)[:, :1 + distil].contiguous()
    say(f"two terms {T} distil={distil} {dtype}")
    if distil:
        logits = torch.full((T, 2), 1.5, device="cuda")
        _, lse, student = mg.linear_distillation(x, w, logits, index, temperature=tau)
        dx, dw = mg.linear_distillation_backward(x, w, logits, index, lse, student, grad,
                                                 temperature=tau)
    else:
        _, lse = mg.linear_cross_entropy(x, w, index[:, 0].contiguous())
        dx, dw = mg.linear_cross_entropy_backward(x, w, index[:, 0].contiguous(), lse, grad)
    X, W = x.double(), w.double()
    c = (tau * grad.double())[:, None]
    p = torch.zeros(T, V, device="cuda", dtype=torch.double)
    p.scatter_(1, index, 1.0 / (1 + distil))
    dz = c * (1.0 / V - p)
    e = u * u * dz.abs() + 2.0 ** -22 * c * (1.0 / V + p)
    if dtype == "f16":
        e = e + float(c.max()) * 2.0 ** -37
    one = dz.to(TORCH[dtype]).double()
    for name, got, exact, tol, less in (
            ("dx", dx, dz @ W, (e + (V + 2) * 2.0 ** -23 * dz.abs()) @ W.abs(), one @ W),
            ("dw", dw, dz.t() @ X, (e + (T + 2) * 2.0 ** -23 * dz.abs()).t() @ X.abs(), one.t() @ X)):
        assert between(got, exact, tol) == 0, name
        # with derivatives of one term this would not hold (a lone token has but two or
        # three values of them, which may round well)
        assert T == 1 or between(less.to(got.dtype), exact, tol) > got.numel() // 20, name


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_equal_weights_are_held_exactly(dtype):
    """Logits that are all 0 over V = 128 columns: dz = g / 128, and g / 128 - g at the
    target.  With equal g, whatever its bits, the factor makes both whole multiples of a
    power of two that the type holds: dw is dz's sums in FP32 and one rounding.  (g = 1 /
    90, as from a mean, is not a number of either type.)"""
    T, V, D = 100, 128, 136
    g = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn(T, D, generator=g, device="cuda").to(TORCH[dtype])
    w = torch.zeros(V, D, device="cuda", dtype=TORCH[dtype])
    target = torch.randint(0, V, (T,), generator=g, device="cuda")
    target[::10] = -100
    live = target != -100
    weight = torch.tensor(1.0 / 90, device="cuda")
    say(f"equal weights {dtype}")
    _, lse = mg.linear_cross_entropy(x, w, target)
    dx, dw = mg.linear_cross_entropy_backward(x, w, target, lse, weight)
    dz = torch.full((T, V), 2.0 ** -7, dtype=torch.double, device="cuda")
    dz[live, target[live]] -= 1.0
    dz = dz * live[:, None] * weight.double()
    assert not dx.any()
    # sums of T products and the factor's product: (T + 2) 2^-23 (T of them FP32 additions,
    # whichever way the matrix unit rounds), FP16's subnormals aside
    tol = (T + 2) * 2.0 ** -23 * (dz.abs().t() @ x.double().abs())
    assert between(dw, dz.t() @ x.double(), tol) == 0
    one = dz.to(TORCH[dtype]).double()   # rounded without the factor it does not hold
    assert between((one.t() @ x.double()).to(dw.dtype), dz.t() @ x.double(), tol) > dw.numel() // 20


def test_log_sum_exps_are_kept_in_64_bits():
    g = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn(300, 64, generator=g, device="cuda")
    w = torch.randn(5000, 64, generator=g, device="cuda") / 8
    target = torch.randint(0, 5000, (300,), generator=g, device="cuda")
    say("lse in 64 bits")
    _, lse = mg.linear_cross_entropy(x, w, target)
    _, klse, _ = mg.linear_distillation(x, w, torch.zeros(300, 1, device="cuda"), target[:, None],
                                        temperature=2.0)
    for got, tau in ((lse, 1.0), (klse, 2.0)):
        z = x.double() @ w.double().t() / tau
        want = torch.logsumexp(z, 1)
        tol = (64 * 2.0 ** -23 * (x.double().abs() @ w.double().abs().t()) / tau).amax(1)
        tol = tol + 2.0 ** -20 * (1 + z.abs().amax(1) + math.log(5000))
        assert ((got - want).abs() <= tol).all()
        # most are no FP32 numbers: nothing rounds them to 32 bits on the way
        assert int((got.float().double() != got).sum()) > 250


# ------------------------------------------------------- rows that are nearly certain

def certain(T, V, D, dtype, size, seed):
    """x along each row's target (a logit of about `size`, the others of a few), the
    targets, and the logits in 64 bits."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = (torch.randn(V, D, generator=g, device="cuda") * (2 / math.sqrt(D))).to(dtype)
    target = torch.randint(0, V, (T,), generator=g, device="cuda")
    at = w[target].float()
    x = at * (size / (at * at).sum(1, keepdim=True))
    x += 0.5 * torch.randn(T, D, generator=g, device="cuda")
    x = x.to(dtype)
    return x, w, target, x.double() @ w.double().t(), g


def spread_of(z, p, ez):
    """What logits off by up to ez, the same ones in all of a loss, change in lse - sum p z
    and in its derivative q - p.  With q the softmax, the first order is sum (q - p) dz,
    the second half the variance of dz under q, at most 2 ez^2 (1 - max q); q itself is off
    by q times the difference of its own dz and their mean under q."""
    q = torch.softmax(z, 1)
    rest = 1 - q.amax(1)
    most = ez.amax(1)
    loss = ((q - p).abs() * ez).sum(1) * (1 + 4 * most) + 4 * rest * most ** 2
    own = torch.where(q == q.amax(1, keepdim=True), rest[:, None] * 2 * most[:, None],
                      q * 2 * most[:, None])
    return loss, own * (1 + 4 * most[:, None])


SIZES = [(64, 1000, 256, "f32", 200.0), (20, 3000, 512, "f32", 40.0), (300, 5000, 1024, "f32", 20.0),
         (16, 1000, 256, "bf16", 200.0), (64, 1000, 520, "f16", 60.0),
         (100, 20000, 1000, "bf16", 40.0), (300, 17000, 1032, "f16", 40.0),
         (300, 17001, 200, "bf16", 200.0), (512, 16384, 128, "bf16", 20.0),
         (1000, 33003, 2112, "bf16", 40.0), (70, 500, 65, "bf16", 100.0),
         (8192, 40001, 72, "bf16", 100.0), (200, 9000, 256, "f16", 20.0)]


# misaligned: w is copied into whole k-tiles first (as where D is no whole number of chunks)
CASES = [(*c, False) for c in SIZES] + [(*c, True) for c in SIZES
                                        if c[0] * c[1] <= 1 << 24 and c[2] % 8 == 0]


@pytest.mark.parametrize("T,V,D,dtype,size,misaligned", CASES)
def test_nearly_certain_rows_keep_their_small_losses(T, V, D, dtype, size, misaligned):
    """A loss far below its logits: lse and the named logit have to come from the same
    sums, whose errors (of up to D 2^-23 sum |x w|, 1e-4 and more here) then cancel.  What
    is left of them is spread_of's, and the evaluation in FP32: exponentials and some 30
    roundings of sums near 1, below 2^-19 in all.  As a distillation of one entry too."""
    dt = torch.float32 if dtype == "f32" else TORCH[dtype]
    x, w, target, z, g = certain(T, V, D, dt, size, T + V)
    if misaligned:
        room = torch.empty(V * D + 1, dtype=dt, device="cuda")[1:].view(V, D)
        w = room.copy_(w)
    say(f"certain {T}x{V}x{D} {dtype} {size} misaligned={misaligned}")
    at = target[:, None]
    # log(1 + sum of the others): exact however small
    others = (z - z.gather(1, at)).scatter_(1, at, -math.inf)
    want = torch.log1p(torch.exp(others).sum(1))
    p = torch.zeros_like(z).scatter_(1, at, 1.0)
    ez = D * 2.0 ** -23 * (x.double().abs() @ w.double().abs().t())
    tol, e = spread_of(z, p, ez)
    del others
    grad = torch.rand(T, generator=g, device="cuda") + 0.25
    loss, lse = mg.linear_cross_entropy(x, w, target)
    kloss, klse, student = mg.linear_distillation(x, w, torch.zeros(T, 1, device="cuda"), at)
    for name, got in (("ce", loss), ("kd", kloss)):
        assert (got >= 0).all(), (name, float(got.min()))
        err = (got.double() - want).abs()
        worst = (err - tol - 2.0 ** -19 - 2.0 ** -23 * want).max()
        assert worst <= 0, (name, float(worst), float(err.max()))
    # the derivative: c (q - 1) at the target, c q elsewhere; a q below FP32's normal range
    # is 0 or off by as much, 2^-126 at most (e^-200 = 2^-289 lies far below it), and so may
    # a gradient of the narrower types be
    c = grad.double()[:, None]
    q = torch.softmax(z, 1)
    dz = q.scatter(1, at, -(-torch.expm1(-want))[:, None]) * c
    u = torch.finfo(dt).eps / 2
    e = c * (e + 2.0 ** -19 * torch.maximum(q, p) + 2.0 ** -126)
    if dtype != "f32":
        e = e + u * dz.abs() + (float(c.max()) * 2.0 ** -37 if dtype == "f16" else 0.0)
    X, W = x.double(), w.double()
    dx, dw = dz @ W, dz.t() @ X
    tol_x = (e + V * 2.0 ** -23 * (dz.abs() + e)) @ W.abs()
    tol_w = (e + T * 2.0 ** -23 * (dz.abs() + e)).t() @ X.abs()
    sub = 2.0 ** -25 if dtype == "f16" else 2.0 ** -126
    for name, got in (("ce", mg.linear_cross_entropy_backward(x, w, target, lse, grad)),
                      ("kd", mg.linear_distillation_backward(x, w, torch.zeros(T, 1, device="cuda"),
                                                             at, klse, student, grad))):
        for which, g_, want_, tol_ in (("dx", got[0], dx, tol_x), ("dw", got[1], dw, tol_w)):
            bound = tol_ + u * (want_.abs() + tol_) + sub
            worst = ((g_.double() - want_).abs() / bound).max()
            assert worst <= 1, (name, which, float(worst))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_student_that_matches_its_teacher_has_almost_no_loss(dtype):
    """Logits of about 100 at twenty entries of weights 2^-1, 2^-2, ... and the student's
    own logits as the teacher's: q is p but for the rest of the vocabulary, and the loss
    nearly 0, whatever the errors that the logits share."""
    T, V, D, top, tau = 40, 2000, 512, 20, 2.0
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    x, w, target, z, g = certain(T, V, D, dt, 120.0, 5)
    teacher, index = z.topk(top, 1)
    teacher = teacher.float().contiguous()
    say(f"matched student {dtype}")
    loss, lse, student = mg.linear_distillation(x, w, teacher, index.contiguous(), temperature=tau)
    p = torch.softmax(teacher.double() / tau, 1)
    log_q = torch.log_softmax(z / tau, 1).gather(1, index)
    want = tau * tau * (p * (torch.log_softmax(teacher.double() / tau, 1) - log_q)).sum(1)
    P = torch.zeros_like(z).scatter_(1, index, p)
    ez = D * 2.0 ** -23 * (x.double().abs() @ w.double().abs().t()) / tau
    tol, _ = spread_of(z / tau, P, ez)
    # teacher and student logs: FP32 exponents and sums, each below 2^-19 as above
    assert (loss >= 0).all()
    assert ((loss.double() - want).abs() <= tau * tau * (tol + 2 * 2.0 ** -19)).all()


# entries per wavefront 1, 2, 4, 8 and 16 (at once, and more than once); x in LDS up to 16
# KiB a row and from memory past it; k ending inside a slab; the partial first k-tile
@pytest.mark.parametrize("top", [1, 3, 7, 13, 30, 60, 150])
@pytest.mark.parametrize("T,D,dtype", [(5, 72, "f32"), (9, 4104, "f32"), (40, 520, "f16"),
                                       (7, 8200, "bf16"), (3, 8192, "f16"), (130, 1096, "bf16")])
def test_named_logits_are_those_behind_the_log_sum_exp(T, D, dtype, top):
    """With every entry of a vocabulary named, lse is the log-sum-exp of the student's
    logits as returned, however far their own errors (of up to 1e-4) go: off by the
    evaluation's 2^-19 and by the rounding of log2(e) / tau, 2^-24 of the largest."""
    dt = torch.float32 if dtype == "f32" else TORCH[dtype]
    x, w, _, z, g = certain(T, top, D, dt, 150.0, T + D + top)
    index = torch.rand(T, top, generator=g, device="cuda").argsort(1).contiguous()
    say(f"named {T}x{top}x{D} {dtype}")
    _, lse, student = mg.linear_distillation(x, w, torch.zeros(T, top, device="cuda"), index,
                                             temperature=2.0)
    at = z.gather(1, index)
    ez = D * 2.0 ** -23 * (x.double().abs() @ w.double().abs().t()).gather(1, index)
    assert ((student.double() - at).abs() <= ez).all()
    want = torch.logsumexp(student.double() / 2, 1)
    assert ((lse - want).abs() <= 2.0 ** -19 + 2.0 ** -24 * student.double().abs().amax(1)).all()


@pytest.mark.parametrize("T,V,D,dtype", [(300, 17000, 1032, "f16"), (300, 17001, 136, "bf16"),
                                         (512, 16640, 256, "bf16"), (200, 30000, 72, "f16")])
def test_named_logits_of_large_tiles(T, V, D, dtype):
    """The same on 256x256 tiles, a single entry against the softmax's value at it: with
    logits of about 150 that is 1 less the small rest, as the student's own logit gives it."""
    x, w, target, z, g = certain(T, V, D, TORCH[dtype], 150.0, V + D)
    say(f"named {T}x{V}x{D} {dtype}")
    _, lse, student = mg.linear_distillation(x, w, torch.zeros(T, 1, device="cuda"),
                                             target[:, None])
    others = (z - z.gather(1, target[:, None])).scatter_(1, target[:, None], -math.inf)
    rest = torch.log1p(torch.exp(others).sum(1))
    sure = rest < 2.0 ** -30
    assert sure.sum() > T // 2
    gap = lse - student[:, 0].double()
    assert (gap[sure].abs() <= 2.0 ** -19 + 2.0 ** -24 * student[sure, 0].double().abs()).all()
