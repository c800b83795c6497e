"""The output-layer losses (softmax cross entropy, distillation from a teacher's
top logits) and their gradients against the definitions in float64.

Tolerances, element by element (u: half a step of the dtype, 2^-8 BF16, 2^-11 FP16,
2^-24 FP32; the inputs are exact in it):
* a logit is a sum of D products in FP32: off by ez = D 2^-23 sum |x w|;
* exponents are s z - l in FP32 with |s z|, |l| at most a row's largest logit
  magnitude Z / tau times log2 e, exp2 and log2 are good to a few units, the sums
  over a row are trees and short chains: lse and log q are off by
  d = max_row(ez) / tau + 2^-20 (1 + Z / tau + log V);
* a loss is two or, for distillation, at most 1 + sum p such terms, times tau^2,
  plus the teacher's log p with the same kind of error in its own logits;
* dz = c (q P - p) is off by c q d 4 (the exponential of an error below 1/4, lse and
  logit both), by c p 2^-20 (1 + the row's teacher range / tau) for the teacher's p,
  by u |dz| for its rounding, and by c_max 2^-37 where FP16 underflows (the factor
  puts c_max above 2^13 and the smallest step is 2^-24);
* dx and dw sum n = V or T products in FP32, n 2^-23 sum |dz w|, and round once
  more (u |dx|; FP16 below its normal range 2^-25).
"""
import math

import pytest
import torch

import dense_gemm_16_amd as mg
from gpu_helpers import say

pytestmark = pytest.mark.gpu

TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
IGNORE = -100


def layer(T, V, D, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = torch.randn(V, D, generator=g, device="cuda") * (2.0 / math.sqrt(D))
    x = torch.randn(T, D, generator=g, device="cuda")
    return x.to(TORCH[dtype]), w.to(TORCH[dtype]), g


def reference(x, w, index, logits, tau, grad, ce):
    """float64 (loss, dx, dw) and their tolerances.  index: T x n (negative: absent);
    logits: the teacher's (None for cross entropy, whose one entry has weight 1)."""
    u = 2.0 ** -24 if x.dtype == torch.float32 else torch.finfo(x.dtype).eps / 2
    half = x.dtype == torch.float16
    X, W = x.double(), w.double()
    T, V, D = X.shape[0], W.shape[0], X.shape[1]
    held = index >= 0
    live = held.any(1)
    if not ce:
        t = torch.where(held, logits.double() / tau, -math.inf)
        live &= t.amax(1) > -math.inf
        t = torch.where(live[:, None], t, 0.0)
        p = torch.softmax(t, 1) * held * live[:, None]
    else:
        p = held.double()
    X = torch.where(live[:, None], X, 0.0)
    at = index.clamp(min=0)
    z = X @ W.t() / tau
    log_q = torch.log_softmax(z, 1)
    q = log_q.exp()
    picked = log_q.gather(1, at)
    loss = tau * tau * (torch.xlogy(p, p) - torch.where(p > 0, p * picked, 0.0)).sum(1)
    loss = torch.where(live, loss, 0.0)
    ez = D * 2.0 ** -23 * (X.abs() @ W.abs().t()) / tau
    Z = z.abs().amax(1)
    d = ez.amax(1) + 2.0 ** -20 * (1 + Z + math.log(V))
    spread = torch.zeros_like(Z) if ce else torch.where(
        p > 0, (t - t.amax(1, keepdim=True)).abs(), 0.0).amax(1) + math.log(index.shape[1] + 1)
    tol_loss = tau * tau * (2 * d + 2.0 ** -20 * (1 + spread) * (1 + Z))
    tol_loss += 2.0 ** -22 * loss.abs() + index.shape[1] * 2.0 ** -23 * tau * tau * (Z + 1)
    c = torch.where(live, tau * grad.double(), 0.0)[:, None]
    dz = q.clone().scatter_add_(1, at, -p) * c
    target = torch.zeros_like(q).scatter_add_(1, at, p)
    e = c.abs() * (4 * q * d[:, None] + 2.0 ** -20 * (1 + spread[:, None]) * target)
    e += u * dz.abs() + (float(c.abs().max()) * 2.0 ** -37 if half else 0.0)
    e = e * (1 + u)
    dx, dw = dz @ W, dz.t() @ X
    sub = 2.0 ** -25 if half else 0.0
    tol_dx = (e + V * 2.0 ** -23 * (dz.abs() + e)) @ W.abs()
    tol_dw = (e + T * 2.0 ** -23 * (dz.abs() + e)).t() @ X.abs()
    tol_dx += u * (dx.abs() + tol_dx) + sub
    tol_dw += u * (dw.abs() + tol_dw) + sub
    return (loss, dx, dw), (tol_loss, tol_dx, tol_dw)


def check(got, want, tol):
    for name, g, r, t in zip(("loss", "dx", "dw"), got, want, tol):
        if g is None:
            continue
        g = g.double()
        assert torch.isfinite(g).all(), name
        worst = ((g - r).abs() - t).max() if g.numel() else torch.tensor(-1.0)
        assert worst <= 0, (name, float(worst), float((g - r).abs().max()), float(t.max()))


def ce_case(T, V, D, dtype, seed, mask=True):
    x, w, g = layer(T, V, D, dtype, seed)
    target = torch.randint(0, V, (T,), generator=g, device="cuda")
    if mask and T > 2:
        target[torch.rand(T, generator=g, device="cuda") < 0.2] = IGNORE
    grad = torch.rand(T, generator=g, device="cuda") + 0.25
    if dtype == "bf16":
        grad /= T
    return x, w, target, grad


def run_ce(x, w, target, grad, **kw):
    loss, lse = mg.linear_cross_entropy(x, w, target, ignore_index=IGNORE)
    dx, dw = mg.linear_cross_entropy_backward(x, w, target, lse, grad, ignore_index=IGNORE, **kw)
    torch.cuda.synchronize()
    return loss, dx, dw


SIZES = [(1, 1, 8), (1, 1000, 64), (3, 17, 24), (16, 512, 256), (64, 1000, 256), (65, 257, 72),
         (130, 300, 520), (200, 4099, 136), (1, 33000, 128), (257, 2050, 320), (1003, 3001, 200)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,V,D", SIZES)
def test_cross_entropy(T, V, D, dtype):
    x, w, target, grad = ce_case(T, V, D, dtype, T + V + D)
    say(f"ce {T}x{V}x{D} {dtype}")
    got = run_ce(x, w, target, grad)
    index = torch.where(target == IGNORE, -1, target)[:, None]
    check(got, *reference(x, w, index, None, 1.0, grad, True))
    assert not got[1][target == IGNORE].any() and not got[0][target == IGNORE].any()


# dx summed over slices of the vocabulary: 64x64 tiles (more slices than 16), 128x128,
# 256x256 with the vocabulary ending inside a k-tile; each ending anywhere
@pytest.mark.parametrize("T,V,D,dtype", [(1, 20011, 264, "f32"), (3, 20011, 264, "f16"),
                                         (40, 9999, 72, "bf16"), (200, 8003, 1032, "bf16"),
                                         (300, 5001, 768, "f32"), (1500, 16392, 1496, "bf16")])
def test_cross_entropy_over_slices_of_the_vocabulary(T, V, D, dtype):
    x, w, target, grad = ce_case(T, V, D, dtype, T + V + D)
    say(f"ce {T}x{V}x{D} {dtype}")
    got = run_ce(x, w, target, grad)
    index = torch.where(target == IGNORE, -1, target)[:, None]
    check(got, *reference(x, w, index, None, 1.0, grad, True))


# whole 256x256 tiles, ragged ones, K ending inside a k-tile, 128x128 tiles of FP32;
# dw's last eight columns, past whole 256-wide tiles; sizes that are brought to whole
# tiles (2^36 multiply-adds on), dx over slices and as one product, a last step whose
# tiles T and its whole-tile rows would choose differently
@pytest.mark.parametrize("T,V,D,dtype", [(512, 16384, 128, "bf16"), (500, 16391, 72, "bf16"),
                                         (512, 16384, 192, "f16"), (130, 16500, 264, "f16"),
                                         (65, 17001, 520, "bf16"),
                                         (1000, 33003, 2112, "f16"), (4000, 5000, 4096, "bf16"),
                                         (8000, 8648, 1024, "bf16"),
                                         (700, 12001, 88, "f16"),
                                         (1024, 4096, 100, "f32"), (1025, 4097, 64, "f32")])
def test_cross_entropy_on_large_tiles(T, V, D, dtype):
    x, w, target, grad = ce_case(T, V, D, dtype, T + V + D)
    say(f"ce {T}x{V}x{D} {dtype}")
    got = run_ce(x, w, target, grad)
    index = torch.where(target == IGNORE, -1, target)[:, None]
    check(got, *reference(x, w, index, None, 1.0, grad, True))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,V,D", [(33, 513, 65), (5, 40, 1), (129, 700, 131), (64, 8200, 7)])
def test_cross_entropy_with_rows_ending_inside_a_chunk(T, V, D, dtype):
    x, w, target, grad = ce_case(T, V, D, dtype, T + V + D)
    say(f"ce {T}x{V}x{D} {dtype}")
    got = run_ce(x, w, target, grad)
    index = torch.where(target == IGNORE, -1, target)[:, None]
    check(got, *reference(x, w, index, None, 1.0, grad, True))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_cross_entropy_strided_operands_and_outputs(dtype):
    T, V, D = 70, 300, 64
    x, w, target, grad = ce_case(T, V, D, dtype, 11)

    def inside(t, offset, extra):
        buf = torch.full((offset + t.shape[0] * (t.shape[1] + extra),), float("nan"),
                         dtype=t.dtype, device="cuda")
        v = buf[offset:].view(t.shape[0], -1)[:, :t.shape[1]]
        v.copy_(t)
        return v, buf[offset:].view(t.shape[0], -1)[:, t.shape[1]:]

    index = torch.where(target == IGNORE, -1, target)[:, None]
    want, tol = reference(x, w, index, None, 1.0, grad, True)
    for ox, oe, wo, we in ((0, 8, 0, 16), (1, 0, 0, 0), (0, 0, 1, 0), (3, 5, 2, 3)):
        say(f"ce strided {dtype} {ox} {oe} {wo} {we}")
        xv, _ = inside(x, ox, oe)
        wv, _ = inside(w, wo, we)
        dx, dx_pad = inside(torch.zeros_like(x), ox, 3)
        dw, dw_pad = inside(torch.zeros_like(w), wo, 1)
        got = run_ce(xv, wv, target, grad, dx=dx, dw=dw)
        assert got[1] is dx and got[2] is dw
        check(got, want, tol)
        assert dx_pad.isnan().all() and dw_pad.isnan().all()


def test_cross_entropy_in_several_pieces_of_the_vocabulary():
    T, V, D = 8192, 40001, 64   # pieces of 32768 entries
    for dtype in ("bf16", "f16", "f32"):
        x, w, target, grad = ce_case(T, V, D, dtype, 5)
        say(f"ce pieces {dtype}")
        got = run_ce(x, w, target, grad)
        index = torch.where(target == IGNORE, -1, target)[:, None]
        want, tol = reference(x, w, index, None, 1.0, grad, True)
        check(got, want, tol)
        del got, want, tol


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_rows_without_a_loss_may_hold_anything(dtype):
    T, V, D = 100, 520, 128
    x, w, target, grad = ce_case(T, V, D, dtype, 3)
    target[7] = target[50] = target[99] = IGNORE
    index = torch.where(target == IGNORE, -1, target)[:, None]
    want, tol = reference(x, w, index, None, 1.0, grad, True)
    x[7] = float("nan")
    x[50] = float("inf")
    grad[99] = float("nan")
    say(f"ce masked garbage {dtype}")
    check(run_ce(x, w, target, grad), want, tol)
    say(f"ce no row counts {dtype}")
    loss, dx, dw = run_ce(x, w, torch.full_like(target, IGNORE), grad)
    assert not loss.any() and not dx.any() and not dw.any()
    assert not dx.isnan().any() and not dw.isnan().any()


def test_a_target_outside_the_vocabulary_shows():
    x, w, target, grad = ce_case(40, 100, 64, "bf16", 9, mask=False)
    target[3], target[20] = 100, -1
    say("ce bad target")
    loss, dx, dw = run_ce(x, w, target, grad)
    bad = torch.zeros(40, dtype=torch.bool, device="cuda")
    bad[3] = bad[20] = True
    assert torch.equal(loss.isnan(), bad) and torch.equal(dx.isnan().all(1), bad)
    assert torch.equal(dx.isnan().any(1), bad) and dw.isnan().all()


def test_ignore_index_inside_the_vocabulary_and_zero_gradients():
    x, w, target, grad = ce_case(64, 50, 32, "f32", 9, mask=False)
    grad[5:20] = 0.0
    target[30:40] = 0
    say("ce ignore_index 0")
    loss, lse = mg.linear_cross_entropy(x, w, target, ignore_index=0)
    dx, dw = mg.linear_cross_entropy_backward(x, w, target, lse, grad, ignore_index=0)
    index = torch.where(target == 0, -1, target)[:, None]
    check((loss, dx, dw), *reference(x, w, index, None, 1.0, grad, True))
    want = torch.logsumexp(x.double() @ w.double().t(), 1)
    assert ((lse.double() - want).abs() <= 1e-5 * (1 + want.abs())).all()


def test_extreme_logits():
    # rows of logits near +-1e4 and +-infinity
    x = torch.zeros(6, 8, device="cuda")
    w = torch.zeros(300, 8, device="cuda")
    w[:, 0] = torch.linspace(-1, 1, 300, device="cuda")
    w[7, 1] = 1.0
    x[0, 0], x[1, 0], x[2, 0], x[3, 0] = 1e4, -1e4, 3e4, 1e-3
    x[4, 1] = float("-inf")                 # z[4, 7] = -inf, the others NaN (0 x inf)
    x[5, 0], x[5, 1] = 1.0, 80.0
    target = torch.tensor([0, 0, 299, 5, 7, 7], device="cuda")
    say("ce extreme logits")
    loss, _ = mg.linear_cross_entropy(x, w, target)
    want = torch.logsumexp(x.double() @ w.double().t(), 1)
    want = want - (x.double() @ w.double().t()).gather(1, target[:, None])[:, 0]
    fine = [0, 1, 2, 3, 5]
    assert ((loss.double() - want).abs()[fine] <= 2.0 ** -20 * (1 + 3e4)).all()
    assert loss[4].isnan()
    # a +infinite logit, alone infinite in its row: lse is +infinity, not NaN
    x = torch.ones(2, 8, device="cuda")
    w = torch.rand(300, 8, device="cuda")
    w[17, 2] = float("inf")
    _, lse = mg.linear_cross_entropy(x, w, torch.zeros(2, dtype=torch.long, device="cuda"))
    assert torch.equal(lse.float(), torch.full((2,), float("inf"), device="cuda"))
    # every logit -infinity
    w = torch.rand(300, 8, device="cuda")
    w[:, 2] = float("-inf")
    _, lse = mg.linear_cross_entropy(x, w, torch.zeros(2, dtype=torch.long, device="cuda"))
    assert torch.equal(lse.float(), torch.full((2,), float("-inf"), device="cuda"))


# ------------------------------------------------------------------ distillation

def kd_case(T, V, D, top, dtype, seed, teacher=torch.float32):
    x, w, g = layer(T, V, D, dtype, seed)
    logits = (3 * torch.randn(T, top, generator=g, device="cuda")).to(teacher)
    keys = torch.rand(T, V, generator=g, device="cuda") if V <= 5000 else None
    index = keys.argsort(1)[:, :top] if keys is not None else torch.randint(
        0, V, (T, top), generator=g, device="cuda")
    if index.shape[1] < top:   # fewer vocabulary entries than `top`: the rest is absent
        index = torch.nn.functional.pad(index, (0, top - index.shape[1]), value=-1)
    index = index.contiguous()
    if T > 2:
        index[torch.rand(T, top, generator=g, device="cuda") < 0.2] = -1
        index[torch.rand(T, generator=g, device="cuda") < 0.1] = -1
    grad = torch.rand(T, generator=g, device="cuda") + 0.25
    if dtype == "bf16":
        grad /= T
    return x, w, logits, index, grad


def run_kd(x, w, logits, index, tau, grad, **kw):
    loss, lse, student = mg.linear_distillation(x, w, logits, index, temperature=tau)
    dx, dw = mg.linear_distillation_backward(x, w, logits, index, lse, student, grad,
                                             temperature=tau, **kw)
    torch.cuda.synchronize()
    return loss, dx, dw


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,V,D,top,tau", [
    (1, 1, 8, 1, 1.0), (1, 1000, 64, 5, 2.0), (3, 17, 24, 17, 1.0), (33, 4099, 520, 8, 1.0),
    (65, 257, 72, 64, 1.5), (130, 300, 136, 100, 4.0), (40, 2000, 100, 1024, 2.0),
    (257, 2050, 320, 32, 0.5), (50, 30, 65, 40, 1.0)])
def test_distillation(T, V, D, top, tau, dtype):
    x, w, logits, index, grad = kd_case(T, V, D, top, dtype, T + V + D)
    say(f"kd {T}x{V}x{D} top {top} tau {tau} {dtype}")
    got = run_kd(x, w, logits, index, tau, grad)
    check(got, *reference(x, w, index, logits, tau, grad, False))


@pytest.mark.parametrize("T,V,D,top,dtype", [(512, 16384, 128, 64, "bf16"),
                                             (500, 16391, 72, 16, "f16"),
                                             (8192, 40001, 64, 4, "bf16")])
def test_distillation_on_large_tiles_and_pieces(T, V, D, top, dtype):
    x, w, logits, index, grad = kd_case(T, V, D, top, dtype, T + V + D)
    say(f"kd {T}x{V}x{D} top {top} {dtype}")
    got = run_kd(x, w, logits, index, 2.0, grad)
    check(got, *reference(x, w, index, logits, 2.0, grad, False))


@pytest.mark.parametrize("teacher", [torch.float16, torch.bfloat16])
def test_distillation_teacher_types_and_strides(teacher):
    T, V, D, top, tau = 60, 400, 64, 12, 2.0
    x, w, logits, index, grad = kd_case(T, V, D, top, "bf16", 2, teacher)
    wide_l = torch.full((T, top + 3), float("nan"), dtype=teacher, device="cuda")
    wide_i = torch.full((T, top + 5), 1 << 40, device="cuda")
    wide_l[:, :top], wide_i[:, :top] = logits, index
    say(f"kd teacher {teacher}")
    got = run_kd(x, w, wide_l[:, :top], wide_i[:, :top], tau, grad)
    check(got, *reference(x, w, index, logits, tau, grad, False))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_distillation_special_rows(dtype):
    T, V, D, top, tau = 20, 300, 64, 6, 1.5
    x, w, logits, index, grad = kd_case(T, V, D, top, dtype, 4)
    index = torch.randint(0, V, (T, top), device="cuda",
                          generator=torch.Generator(device="cuda").manual_seed(1))
    logits[0, 2] = -math.inf                      # an entry without weight
    logits[1] = -math.inf                         # no entry has weight: no loss
    logits[2] = torch.finfo(torch.float32).min    # all equal: uniform
    logits[3, 1:] = torch.finfo(torch.float32).min
    index[4] = index[4, 0]                        # one index six times
    index[5, 3] = index[5, 1]
    index[6] = -1                                 # nothing held
    logits[7], index[7, 1:] = math.nan, -1
    logits[7, 0] = 2.0                            # garbage where nothing is held
    want, tol = reference(x, w, torch.where(torch.isnan(logits), -1, index),
                          torch.nan_to_num(logits, nan=0.0, neginf=-math.inf), tau, grad, False)
    x[1] = math.nan                               # rows without a loss may hold anything
    x[6] = math.inf
    say(f"kd special rows {dtype}")
    check(run_kd(x, w, logits, index, tau, grad), want, tol)
    index[8, 0] = V                               # outside the vocabulary: shows
    index[9, 0], logits[9, 0] = 3, math.nan
    loss, dx, dw = run_kd(x, w, logits, index, tau, grad)
    bad = torch.zeros(T, dtype=torch.bool, device="cuda")
    bad[8] = bad[9] = True
    assert torch.equal(loss.isnan(), bad) and torch.equal(dx.isnan().any(1), bad)
    assert dw.isnan().any()


def test_one_entry_of_weight_one_is_cross_entropy():
    x, w, target, grad = ce_case(100, 700, 96, "bf16", 21)
    index = torch.where(target == IGNORE, -1, target)[:, None].contiguous()
    say("kd as ce")
    a = run_ce(x, w, target, grad)
    b = run_kd(x, w, torch.zeros(100, 1, device="cuda"), index, 1.0, grad)
    want, tol = reference(x, w, index, None, 1.0, grad, True)
    check(a, want, tol)
    check(b, want, tol)


# ------------------------------------------------------------ gradients, calls

def test_gradients_against_differences():
    """Central differences of the FP32 losses along random directions.  With a the
    largest |logit| change per unit of the direction, a row's third derivative is at
    most (2 a)^3 / (6 sqrt 3) times tau^2 / tau^3, so the truncation is h^2 / 6 of
    that; each loss is off by 2^-19 (see the tolerances above)."""
    T, V, D, top, tau, h = 24, 200, 48, 5, 2.0, 2.0 ** -6
    x, w, target, grad = ce_case(T, V, D, "f32", 31)
    _, _, logits, index, _ = kd_case(T, V, D, top, "f32", 32)
    g = torch.Generator(device="cuda").manual_seed(8)

    def ce(x, w):
        return mg.linear_cross_entropy(x, w, target, ignore_index=IGNORE)[0]

    def kd(x, w):
        return mg.linear_distillation(x, w, logits, index, temperature=tau)[0]

    say("differences")
    for f, run, t in ((ce, lambda: run_ce(x, w, target, grad)[1:], 1.0),
                      (kd, lambda: run_kd(x, w, logits, index, tau, grad)[1:], tau)):
        dx, dw = run()
        for _ in range(4):
            ex = torch.randn(T, D, generator=g, device="cuda") / math.sqrt(D)
            ew = torch.randn(V, D, generator=g, device="cuda") / math.sqrt(D)
            for bx, bw in ((ex, 0 * ew), (0 * ex, ew)):
                up, down = f(x + h * bx, w + h * bw), f(x - h * bx, w - h * bw)
                slope = ((up - down).double() * grad).sum() / (2 * h)
                want = (dx.double() * bx).sum() + (dw.double() * bw).sum()
                a = (bx.double() @ w.double().t() + x.double() @ bw.double().t()).abs().max()
                cut = h * h / 6 * (2 * a) ** 3 / (6 * math.sqrt(3)) / t
                tol = grad.double().sum() * (cut + 2 * 2.0 ** -19 * t * t / (2 * h))
                assert (slope - want).abs() <= tol, (float(slope), float(want), float(tol))


def test_repeatable_and_one_gradient_at_a_time():
    x, w, target, grad = ce_case(300, 5000, 256, "bf16", 17)
    say("ce twice")
    a, b = run_ce(x, w, target, grad), run_ce(x, w, target, grad)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    only = run_ce(x, w, target, grad, need_dw=False)
    assert only[2] is None and torch.equal(only[1], a[1])
    only = run_ce(x, w, target, grad, need_dx=False)
    assert only[1] is None and torch.equal(only[2], a[2])
    # a number and a vector as the upstream gradient
    c = run_ce(x, w, target, 0.5)
    d = run_ce(x, w, target, torch.full_like(grad, 0.5))
    assert all(torch.equal(p, q) for p, q in zip(c, d))


def test_no_rows():
    x, w = torch.empty(0, 64, device="cuda"), torch.randn(100, 64, device="cuda")
    none = torch.empty(0, dtype=torch.long, device="cuda")
    say("ce of no rows")
    loss, lse = mg.linear_cross_entropy(x, w, none)
    dx, dw = mg.linear_cross_entropy_backward(x, w, none, lse, 1.0)
    assert loss.shape == (0,) and dx.shape == (0, 64) and not dw.any()
    nothing = torch.empty(0, 3, device="cuda")
    loss, lse, student = mg.linear_distillation(x, w, nothing, nothing.long())
    dx, dw = mg.linear_distillation_backward(x, w, nothing, nothing.long(), lse, student, 1.0)
    assert loss.shape == (0,) and not dw.any()


def test_workspace_too_small_is_refused():
    x, w, target, grad = ce_case(64, 300, 64, "bf16", 1)
    T, V, D = 64, 300, 64
    ptr = (x.data_ptr(), D, w.data_ptr(), D)
    s = torch.cuda.current_stream().cuda_stream
    out = torch.zeros(4, T, device="cuda")
    for backward in (0, 1):
        st, n = mg.migemm_linear_loss_workspace_size(backward, T, V, D, 0, mg.BF16, *ptr)
        assert st == mg.OK and n > 0
        ws = torch.empty(n + 256, dtype=torch.uint8, device="cuda")
        for p, b in ((None, n), (ws.data_ptr(), n - 1), (ws.data_ptr() + 128, n)):
            if backward:
                st = mg.migemm_linear_ce_backward(T, V, D, mg.BF16, *ptr, target.data_ptr(), -100,
                                                  out[0].data_ptr(), out[1].data_ptr(), None, 1,
                                                  None, 1, p, b, s)
            else:
                st = mg.migemm_linear_ce_forward(T, V, D, mg.BF16, *ptr, target.data_ptr(), -100,
                                                 out[0].data_ptr(), out[1].data_ptr(), p, b, s)
            assert st == mg.ERR_WORKSPACE


def test_side_stream_and_graph_replay():
    x, w, target, grad = ce_case(128, 3000, 128, "bf16", 77)
    kx, kw, logits, index, kgrad = kd_case(100, 1000, 64, 8, "f16", 78)
    eager = run_ce(x, w, target, grad)
    keager = run_kd(kx, kw, logits, index, 2.0, kgrad)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    say("losses on a side stream by handle")
    loss, lse = mg.linear_cross_entropy(x, w, target, ignore_index=IGNORE,
                                        stream=side.cuda_stream)
    dx, dw = mg.linear_cross_entropy_backward(x, w, target, lse, grad, ignore_index=IGNORE,
                                              stream=side.cuda_stream)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip((loss, dx, dw), eager))
    torch.cuda.synchronize()
    say("losses in a graph")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        loss, lse = mg.linear_cross_entropy(x, w, target, ignore_index=IGNORE)
        dx, dw = mg.linear_cross_entropy_backward(x, w, target, lse, grad, ignore_index=IGNORE)
        kl, klse, st = mg.linear_distillation(kx, kw, logits, index, temperature=2.0)
        kdx, kdw = mg.linear_distillation_backward(kx, kw, logits, index, klse, st, kgrad,
                                                   temperature=2.0)
    for i in range(3):
        if i:
            x.mul_(1.25)
            kx.mul_(0.75)
        eager, keager = run_ce(x, w, target, grad), run_kd(kx, kw, logits, index, 2.0, kgrad)
        for t in (loss, dx, dw, kl, kdx, kdw):
            t.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip((loss, dx, dw), eager))
        assert all(torch.equal(p, q) for p, q in zip((kl, kdx, kdw), keager))


def test_a_layer_quantised_distilled_and_served():
    """The operators as they would be used together: an output layer is quantised to
    MXFP4, distilled against its own full-precision logits, and served by the 4-bit
    product, whose logits the losses of the decoded weight agree with."""
    T, V, D, top, tau = 32, 900, 128, 16, 2.0
    x, w, target, grad = ce_case(T, V, D, "bf16", 55)
    say("quantise, distil, serve")
    teacher = mg.gemm(x, w.t()).float().topk(top, dim=1)
    qw, qx = mg.quantize_mx(w), mg.quantize_mx(x)
    wd, xd = mg.dequantize_mx(qw, torch.bfloat16), mg.dequantize_mx(qx, torch.bfloat16)
    got = run_kd(x, wd, teacher.values.contiguous(), teacher.indices.contiguous(), tau, grad)
    check(got, *reference(x, wd, teacher.indices, teacher.values, tau, grad, False))
    served = mg.gemm_mx(qx, qw)
    # decoded operands are exact in bfloat16, so both products sum the same terms
    tol = 2 * D * 2.0 ** -23 * (xd.double().abs() @ wd.double().abs().t())
    assert ((served.double() - mg.gemm(xd, wd.t()).double()).abs() <= tol).all()
    loss, lse = mg.linear_cross_entropy(xd, wd, target, ignore_index=IGNORE)
    want = torch.logsumexp(served.double(), 1)
    assert ((lse.double() - want).abs() <= 2.0 ** -18 * (1 + want.abs())).all()


def test_fp32_logits_past_what_small_tiles_can_launch():
    """More than 2^35 logits: 64x64 tiles of them would be 2^23 or more, whose 512
    threads each one launch does not hold.  The rows that are compared lie in the
    first, the last (ragged) and random tiles."""
    T, V, D = 600001, 64001, 4
    x, w, target, _ = ce_case(T, V, D, "f32", 3)
    say(f"ce {T}x{V}x{D} f32 forward")
    loss, _ = mg.linear_cross_entropy(x, w, target, ignore_index=IGNORE)
    assert torch.isfinite(loss).all() and not loss[target == IGNORE].any()
    g = torch.Generator(device="cuda").manual_seed(4)
    rows = torch.cat((torch.arange(20, device="cuda"), T - 1 - torch.arange(80, device="cuda"),
                      torch.randint(0, T, (100,), generator=g, device="cuda")))
    index = torch.where(target == IGNORE, -1, target)[rows, None]
    want, tol = reference(x[rows], w, index, None, 1.0, torch.ones(200, device="cuda"), True)
    check((loss[rows], None, None), want, tol)


# Pieces of 32768, 7168 and 65 columns: the vocabulary past whole tiles is a step of its
# own in a product of several pieces, whose k ends inside a chunk; dx is the library's
# product added up over the steps, the first of them on slices of k (configuration 17)
@pytest.mark.parametrize("T,V,D,dtype", [(8192, 40001, 512, "bf16"), (8192, 40001, 512, "f16"),
                                         (8100, 73729, 264, "bf16"), (8000, 33003, 328, "f16")])
def test_whole_tiles_and_pieces_together(T, V, D, dtype):
    x, w, target, grad = ce_case(T, V, D, dtype, T + V + D)
    target[:40] = torch.arange(V - 40, V, device="cuda")   # targets in every step
    target[40:60] = torch.arange(32760, 32780, device="cuda")
    index = torch.where(target == IGNORE, -1, target)[:, None]
    say(f"ce {T}x{V}x{D} {dtype}")
    got = run_ce(x, w, target, grad)
    want, tol = reference(x, w, index, None, 1.0, grad, True)
    check(got, want, tol)
    again = run_ce(x, w, target, grad)
    assert all(torch.equal(p, q) for p, q in zip(got, again))
    say(f"kd {T}x{V}x{D} {dtype}")
    check(run_kd(x, w, torch.zeros(T, 1, device="cuda"), index.contiguous(), 1.0, grad), want, tol)


# --------------------------------------------------- offsets of more than 32 bits

def test_inputs_and_gradients_of_more_than_2_31_elements_by_tokens():
    """x, dx, dz and their copies pass 2^31 elements: rows of dx at both ends and around
    the borders, and dw, the sum over all rows, added up over six parts (each of whose
    tolerances, six times over, covers sums of six times as many terms)."""
    T, V, D = 600000, 520, 4096
    x = torch.empty(T, D, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(2)
    for s in range(0, T, 100000):
        x[s:s + 100000] = torch.randn(100000, D, generator=g, device="cuda").bfloat16()
    w = (torch.randn(V, D, generator=g, device="cuda") / 32).bfloat16()
    target = torch.randint(0, V, (T,), generator=g, device="cuda")
    target[::7] = IGNORE
    grad = (torch.rand(T, generator=g, device="cuda") + 0.25) / T
    assert T * D > 1 << 31
    say(f"ce {T}x{V}x{D} bf16")
    loss, dx, dw = run_ce(x, w, target, grad)
    index = torch.where(target == IGNORE, -1, target)[:, None]
    border = (1 << 31) // D
    rows = torch.cat([torch.arange(a, a + 60, device="cuda")
                      for a in (0, border // 2 - 30, border - 30, T - 60)])
    (l, d, _), (tl, td, _) = reference(x[rows], w, index[rows], None, 1.0, grad[rows], True)
    check((loss[rows], dx[rows], None), (l, d, None), (tl, td, None))
    want, tol = torch.zeros(V, D, device="cuda"), torch.zeros(V, D, device="cuda")
    want, tol = want.double(), tol.double()
    for s in range(0, T, 100000):
        p = slice(s, s + 100000)
        r, t = reference(x[p], w, index[p], None, 1.0, grad[p], True)
        want += r[2]
        tol += t[2]
        del r, t
    check((None, None, dw), (None, None, want), (None, None, 6 * tol))


def test_weights_and_gradients_of_more_than_2_31_elements_by_the_vocabulary():
    """w, its gradient and the offsets into them pass 2^31 elements, in two pieces of the
    vocabulary; rows of dw at both ends and around the borders, and all of dx."""
    T, V, D = 40, 1100000, 2048
    g = torch.Generator(device="cuda").manual_seed(3)
    w = torch.empty(V, D, dtype=torch.bfloat16, device="cuda")
    for s in range(0, V, 100000):
        w[s:s + 100000] = (torch.randn(100000, D, generator=g, device="cuda") / 32).bfloat16()
    x = torch.randn(T, D, generator=g, device="cuda").bfloat16()
    border = (1 << 31) // D
    target = torch.randint(0, V, (T,), generator=g, device="cuda")
    target[:4] = torch.tensor([0, V - 1, border, border - 1], device="cuda")
    grad = torch.rand(T, generator=g, device="cuda") + 0.25
    say(f"ce {T}x{V}x{D} bf16")
    loss, dx, dw = run_ce(x, w, target, grad)
    u, X = 2.0 ** -8, x.double()
    z, ez = (torch.empty(T, V, dtype=torch.double, device="cuda") for _ in range(2))
    for s in range(0, V, 100000):
        W = w[s:s + 100000].double()
        z[:, s:s + 100000], ez[:, s:s + 100000] = X @ W.t(), X.abs() @ W.abs().t()
    ez *= D * 2.0 ** -23
    log_q = torch.log_softmax(z, 1)
    d = ez.amax(1) + 2.0 ** -20 * (1 + z.abs().amax(1) + math.log(V))
    at = target[:, None]
    want = -log_q.gather(1, at)[:, 0]
    assert ((loss.double() - want).abs() <= 2 * d + 2.0 ** -22 * want).all()
    q, c = log_q.exp(), grad.double()[:, None]
    p = torch.zeros_like(q).scatter_(1, at, 1.0)
    dz = c * (q - p)
    e = (c * (4 * q * d[:, None] + 2.0 ** -20 * p) + u * dz.abs()) * (1 + u)
    want, tol = (torch.zeros(T, D, dtype=torch.double, device="cuda") for _ in range(2))
    n = e + V * 2.0 ** -23 * (dz.abs() + e)
    for s in range(0, V, 100000):
        W = w[s:s + 100000].double()
        want += dz[:, s:s + 100000] @ W
        tol += n[:, s:s + 100000] @ W.abs()
    check((None, dx, None), (None, want, None), (None, tol + u * (want.abs() + tol), None))
    rows = torch.cat([torch.arange(a, a + 400, device="cuda")
                      for a in (0, border // 2 - 200, border - 200, V - 400)])
    rows = torch.cat((rows, target))
    want, n = dz[:, rows].t() @ X, (e + T * 2.0 ** -23 * (dz.abs() + e))[:, rows].t() @ X.abs()
    check((None, None, dw[rows]), (None, None, want), (None, None, n + u * (want.abs() + n)))
