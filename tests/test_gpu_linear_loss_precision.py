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
