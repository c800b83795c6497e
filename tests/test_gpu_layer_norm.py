"""Layer norm and its gradients against the definitions in float64.

Tolerances, element by element (u: half a step of the result's dtype, f = 2^-24; the inputs
are exact in their dtype):
* a lane adds at most 16 elements of a row in turn (rows past 16384: D / 1024 + 16), 6
  steps join a wavefront and at most 16 values the wavefronts, so a mean is off by
  em = n f mean |x| with n = 40 + D / 1024, products adding one f;
* the squares are of x - mean, off by em + f |x - mean| each; a shift of em adds em^2 to
  the variance (the distances sum to 0), so it is off by (n + 4) f var + 2 em^2;
* rstd is off by er = half of that over var + eps, and 3 f more (sum, root, quotient);
* h = (x - mean) rstd by eh = |h| (er + 3 f) + em rstd, y by |w| eh + 3 f (|h w| + |b|) and
  its last rounding u |y| (FP16 below its normal range 2^-25);
* backwards, g = dy w is off by f |g|, the row's two sums by (n + 2) f sum |g| and
  (n + 3) f sum |g h| + sum |g| eh, dx by rstd times those over D, eh |s2| / D, and
  (er + 6 f) of the sum of its terms' magnitudes;
* dw and db add a lane's rows in turn, at most 4 + T / 512 of them (long rows: T / 64 + 32),
  then at most 100 values: off by (104 + T / 64) f of the sum of magnitudes, and
  sum |dy| eh.
"""
import math

import pytest
import torch

import dense_gemm_16_amd as mg
from gpu_helpers import say

pytestmark = pytest.mark.gpu

TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
F = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def case(T, D, dtype, weight, seed, spread=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    dt, wt = TORCH[dtype], TORCH[weight]
    x = (randn(T, D) * torch.exp(0.5 * randn(T, 1)) + spread * randn(T, 1)).to(dt)
    return x, (1 + 0.3 * randn(D)).to(wt), (0.3 * randn(D)).to(wt), randn(T, D).to(dt)


def reference(x, w, b, dy, eps, vector=None):
    """float64 {name: (value, tolerance)}; vector: the dtype of dw and db."""
    u, T, D = half_step(x.dtype), *x.shape
    sub = 2.0 ** -25 if x.dtype == torch.float16 else 0.0
    vector = vector or (x.dtype if w is None else w.dtype)
    X, DY = x.double(), dy.double()
    W = torch.ones(D, device=x.device).double() if w is None else w.double()
    B = torch.zeros(D, device=x.device).double() if b is None else b.double()
    n = 40 + D / 1024
    mean = X.mean(1, keepdim=True)
    em = n * F * X.abs().mean(1, keepdim=True)
    d = X - mean
    var = (d * d).mean(1, keepdim=True)
    r = 1 / (var + eps).sqrt()
    er = ((n + 4) * F * var + 2 * em * em) / (2 * (var + eps)) + 3 * F
    h = d * r
    eh = h.abs() * (er + 3 * F) + em * r
    y = h * W + B
    g = DY * W
    s1, s2 = g.sum(1, keepdim=True), (g * h).sum(1, keepdim=True)
    e1 = (n + 2) * F * g.abs().sum(1, keepdim=True)
    e2 = (n + 3) * F * (g * h).abs().sum(1, keepdim=True) + (g.abs() * eh).sum(1, keepdim=True)
    dx = r * (g - s1 / D - h * s2 / D)
    size = r * (g.abs() + s1.abs() / D + (h * s2).abs() / D)
    edx = r * (e1 / D + h.abs() * e2 / D + eh * s2.abs() / D) + (er + 6 * F) * size
    dw, db = (DY * h).sum(0), DY.sum(0)
    edw = (104 + T / 64) * F * (DY * h).abs().sum(0) + (DY.abs() * eh).sum(0)
    edb = (104 + T / 64) * F * DY.abs().sum(0)
    uv, subv = half_step(vector), 2.0 ** -25 if vector == torch.float16 else 0.0
    ey = W.abs() * eh + 3 * F * ((h * W).abs() + B.abs())
    return {"y": (y, ey + u * (y.abs() + ey) + sub),
            "mean": (mean[:, 0], (em + F * mean.abs())[:, 0]),
            "rstd": (r[:, 0], (r * er)[:, 0]),
            "dx": (dx, edx + u * (dx.abs() + edx) + sub),
            "dw": (dw, edw + uv * (dw.abs() + edw) + subv),
            "db": (db, edb + uv * (db.abs() + edb) + subv)}


def check(got, want):
    for name, t in got.items():
        value, tol = want[name]
        t = t.double()
        assert torch.isfinite(t).all(), name
        worst = ((t - value).abs() - tol).max() if t.numel() else torch.tensor(-1.0)
        assert worst <= 0, (name, float(worst), float((t - value).abs().max()))


def both(x, w, b, dy, eps=1e-5, **kw):
    y, mean, rstd = mg.layer_norm(x, w, b, eps=eps)
    dx, dw, db = mg.layer_norm_backward(dy, x, w, mean, rstd, **kw)
    torch.cuda.synchronize()
    got = {"y": y, "mean": mean, "rstd": rstd, "dx": dx, "dw": dw, "db": db}
    return {k: v for k, v in got.items() if v is not None}


# each form of a row (16 to 1024 lanes, longer rows), whole and ending inside a chunk, and
# fewer and more rows than workgroups
SIZES = [(1, 1), (3, 8), (70, 127), (5000, 128), (33, 129), (1, 512), (2100, 300), (9, 513),
         (130, 1024), (3, 1025), (65, 2048), (700, 1537), (5, 2049), (2500, 4096), (2, 4097),
         (40, 8192), (3, 8200), (9, 16384), (2, 16385), (70, 20001), (1, 70000)]


@pytest.mark.parametrize("dtype,weight", [("f32", "f32"), ("f16", "f16"), ("f16", "f32"),
                                          ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("T,D", SIZES)
def test_layer_norm(T, D, dtype, weight):
    x, w, b, dy = case(T, D, dtype, weight, T + D)
    say(f"layer norm {T}x{D} {dtype} {weight}")
    check(both(x, w, b, dy), reference(x, w, b, dy, 1e-5))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D", [100, 1000, 4000, 17000])
def test_strided_and_misaligned(dtype, D):
    T = 21
    x, w, b, dy = case(T, D, dtype, dtype, D)
    want = reference(x, w, b, dy, 1e-5)

    def inside(t, offset, extra):
        buf = torch.full((offset + t.shape[0] * (t.shape[1] + extra),), float("nan"),
                         dtype=t.dtype, device="cuda")
        view = buf[offset:].view(t.shape[0], -1)[:, :t.shape[1]]
        return buf, view.copy_(t)

    say(f"layer norm inside buffers {T}x{D} {dtype}")
    _, xs = inside(x, 1, 3)
    _, dys = inside(dy, 3, 5)
    ybuf, y = inside(torch.zeros_like(x), 5, 1)
    dxbuf, dx = inside(torch.zeros_like(x), 7, 9)
    vec = torch.empty(2 * D + 3, dtype=x.dtype, device="cuda")
    w1 = vec[1:D + 1].copy_(w)
    b1 = vec[D + 1:2 * D + 1].copy_(b)
    grads = torch.full((2 * D + 3,), float("nan"), dtype=x.dtype, device="cuda")
    dw, db = grads[1:D + 1], grads[D + 2:2 * D + 2]
    out, mean, rstd = mg.layer_norm(xs, w1, b1, out=y)
    got = mg.layer_norm_backward(dys, xs, w1, mean, rstd, dx=dx, dw=dw, db=db)
    torch.cuda.synchronize()
    assert out is y and got[0] is dx and got[1] is dw and got[2] is db
    check({"y": y, "mean": mean, "rstd": rstd, "dx": dx, "dw": dw, "db": db}, want)
    # what lies between and around is as it was
    for buf, view in ((ybuf, y), (dxbuf, dx)):
        view.zero_()
        assert int(torch.isnan(buf).sum()) == buf.numel() - view.numel()
    assert torch.isnan(grads[[0, D + 1, 2 * D + 2]]).all()


def test_optional_operands_and_results():
    x, w, b, dy = case(50, 600, "bf16", "f32", 1)
    for weight, bias in ((None, None), (w, None), (None, b)):
        say(f"layer norm weight {weight is not None} bias {bias is not None}")
        got = both(x, weight, bias, dy)
        assert ("dw" in got) == (weight is not None)
        check(got, reference(x, weight, bias, dy, 1e-5))
    full = both(x, w, b, dy)
    for kw in ({"need_dx": False}, {"need_dw": False}, {"need_db": False},
               {"need_dw": False, "need_db": False}, {"need_dx": False, "need_dw": False}):
        got = both(x, w, b, dy, **kw)
        assert set(full) - set(got) == {k[5:] for k in kw}
        assert all(torch.equal(v, full[k]) for k, v in got.items())
    y, mean, rstd = mg.layer_norm(x, w, b, stats=False)
    assert mean is None and rstd is None and torch.equal(y, full["y"])
    long, w, b, dy = case(3, 30000, "bf16", "bf16", 2)
    full = both(long, w, b, dy)
    for kw in ({"need_dx": False}, {"need_dw": False, "need_db": False}):
        got = both(long, w, b, dy, **kw)
        assert all(torch.equal(v, full[k]) for k, v in got.items())


@pytest.mark.parametrize("D", [40, 700, 5000, 20000])
def test_special_rows(D):
    x, w, b, dy = case(12, D, "f32", "f32", D)
    x[1] = 3.25                     # equal elements: y = b
    x[3, D // 2] = float("inf")
    x[5, D - 1] = float("nan")
    x[7] *= 1e-30                   # the variance vanishes against eps
    x[9] = 10000.0 + x[9]           # far from zero
    say(f"special rows of {D}")
    y, mean, rstd = mg.layer_norm(x, w, b)
    torch.cuda.synchronize()
    assert torch.isnan(y[3]).all() and torch.isnan(y[5]).all()
    assert torch.equal(y[1], b) and float(mean[1]) == 3.25
    keep = [i for i in range(12) if i not in (3, 5)]
    dx, dw, db = mg.layer_norm_backward(dy[keep].contiguous(), x[keep].contiguous(), w,
                                        mean[keep].contiguous(), rstd[keep].contiguous())
    torch.cuda.synchronize()
    want = reference(x[keep], w, b, dy[keep], 1e-5)
    check({"y": y[keep], "mean": mean[keep], "rstd": rstd[keep], "dx": dx, "dw": dw, "db": db}, want)
    # a bad row spoils its own dx and the sums, not its neighbours' dx
    dx2, dw2, _ = mg.layer_norm_backward(dy, x, w, mean, rstd)
    torch.cuda.synchronize()
    assert torch.equal(dx2[keep], dx) and torch.isnan(dx2[[3, 5]]).all() and torch.isnan(dw2).any()
    # eps = 0: a row of equal elements is NaN, the others follow the formula
    y, mean, rstd = mg.layer_norm(x, w, b, eps=0.0)
    torch.cuda.synchronize()
    assert torch.isnan(y[1]).all() and torch.isinf(rstd[1])
    # row 7's squares are at most 1e-60 x 100, below FP32's smallest number (2^-149, 1.4e-45):
    # its variance is 0, its elements +-infinity (or NaN)
    assert torch.isinf(rstd[7]) and not torch.isfinite(y[7]).any()
    keep.remove(1)
    keep.remove(7)
    check({"y": y[keep]}, reference(x[keep], w, b, dy[keep], 0.0))


def test_gradients_against_differences():
    """dx, dw and db against central differences of the forward pass in float64 (of the
    definition), and the forward pass's own in float32 steps."""
    T, D = 4, 37
    x, w, b, dy = case(T, D, "f32", "f32", 9)

    def value(x, w, b):
        d = x - x.mean(1, keepdim=True)
        return ((d / ((d * d).mean(1, keepdim=True) + 1e-5).sqrt() * w + b) * dy.double()).sum()

    got = both(x, w, b, dy)
    args = [x.double(), w.double(), b.double()]
    for i, name in enumerate(("dx", "dw", "db")):
        flat = args[i].reshape(-1)
        for k in range(0, flat.numel(), 5):
            def moved(s):
                a = [t.clone() for t in args]
                a[i].view(-1)[k] += s
                return float(value(*a))
            step = 1e-5
            diff = (moved(step) - moved(-step)) / (2 * step)
            one = float(got[name].reshape(-1)[k])
            # the difference's own error: step^2 / 6 of a third derivative of order 1 / sigma^3
            assert abs(diff - one) <= 1e-4 * (1 + abs(diff)), (name, k, diff, one)


def test_no_rows():
    x, w, b, dy = case(0, 64, "f16", "f16", 1)
    got = both(x, w, b, dy)
    assert got["y"].shape == (0, 64) and got["dx"].shape == (0, 64)
    assert not got["dw"].any() and not got["db"].any()


def test_refusals():
    x, w, b, dy = case(4, 64, "bf16", "bf16", 1)
    y, mean, rstd = mg.layer_norm(x, w, b)
    for call in (lambda: mg.layer_norm(x, w[:-1], b), lambda: mg.layer_norm(x, w.half(), b),
                 lambda: mg.layer_norm(x, w, b.float()), lambda: mg.layer_norm(x.t(), None, None),
                 lambda: mg.layer_norm(x, w.cpu(), b), lambda: mg.layer_norm(x[0], w, b),
                 lambda: mg.layer_norm(x, w, b, out=torch.empty_like(x, dtype=torch.float32)),
                 lambda: mg.layer_norm(x[:1].expand(4, 64), w, b),
                 lambda: mg.layer_norm_backward(dy.float(), x, w, mean, rstd),
                 lambda: mg.layer_norm_backward(dy, x, w, mean.double(), rstd),
                 lambda: mg.layer_norm_backward(dy, x, w, mean, rstd[:3]),
                 lambda: mg.layer_norm_backward(dy, x, None, mean, rstd, dw=w.clone()),
                 lambda: mg.layer_norm_backward(dy, x, w, mean, rstd, db=w.float())):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(mg.MigemmError):
        mg.layer_norm(x, w, b, out=x)
    with pytest.raises(mg.MigemmError):
        mg.layer_norm(x, w, b, eps=-1.0)
    with pytest.raises(mg.MigemmError):
        mg.layer_norm_backward(dy, x, w, mean, rstd, dx=dy)


def test_repeatable_side_stream_and_graph_replay():
    x, w, b, dy = case(900, 1032, "bf16", "f32", 5)
    x2, w2, b2, dy2 = case(40, 20000, "f16", "f16", 6)
    eager, long = both(x, w, b, dy), both(x2, w2, b2, dy2)
    for _ in range(3):
        again = both(x, w, b, dy)
        assert all(torch.equal(v, eager[k]) for k, v in again.items())
    side = torch.cuda.Stream()
    say("layer norm on a side stream by handle")
    y, mean, rstd = mg.layer_norm(x, w, b, stream=side.cuda_stream)
    dx, dw, db = mg.layer_norm_backward(dy, x, w, mean, rstd, stream=side.cuda_stream)
    side.synchronize()
    for t, k in ((y, "y"), (dx, "dx"), (dw, "dw"), (db, "db")):
        assert torch.equal(t, eager[k])
    torch.cuda.synchronize()
    say("layer norm in a graph")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a = {}
        for tag, (x_, w_, b_, dy_) in (("", (x, w, b, dy)), ("long", (x2, w2, b2, dy2))):
            y, mean, rstd = mg.layer_norm(x_, w_, b_)
            dx, dw, db = mg.layer_norm_backward(dy_, x_, w_, mean, rstd)
            a |= {tag + "y": y, tag + "dx": dx, tag + "dw": dw, tag + "db": db}
    for i in range(3):
        if i:
            x.mul_(1.25)
            dy2.mul_(0.5)
        eager, long = both(x, w, b, dy), both(x2, w2, b2, dy2)
        for t in a.values():
            t.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a[k], eager[k]) for k in ("y", "dx", "dw", "db"))
        assert all(torch.equal(a["long" + k], long[k]) for k in ("y", "dx", "dw", "db"))


@pytest.mark.parametrize("T,D", [(4, 2), (37, 3), (20, 5), (9, 7)])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_rows_shorter_than_a_chunk(T, D, dtype):
    x, w, b, dy = case(T, D, dtype, "f32", T * D)
    say(f"layer norm {T}x{D} {dtype}")
    check(both(x, w, b, dy, 0.1), reference(x, w, b, dy, 0.1))


@pytest.mark.parametrize("T,D,dtype", [(24000, 2001, "bf16"), (90000, 515, "f16"), (9000, 4099, "f32"),
                                       (400000, 120, "bf16"), (1500, 16383, "f32")])
def test_rows_read_past_the_caches(T, D, dtype):
    """Past 256 MiB of x, dy and dx: rows off 16-byte boundaries, each form of a row."""
    x, w, b, dy = case(T, D, dtype, "f32", T)
    assert 3 * x.numel() * x.element_size() > 256 << 20
    say(f"layer norm {T}x{D} {dtype}, long")
    check(both(x, w, b, dy), reference(x, w, b, dy, 1e-5))


def test_the_longest_row():
    x, w, b, dy = case(2, 1 << 24, "bf16", "f32", 1)
    say("layer norm 2x2^24")
    check(both(x, w, b, dy), reference(x, w, b, dy, 1e-5))


def test_more_than_2_31_elements():
    T, D = (1 << 31) // 4096 + 700, 4096
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.empty(T, D, dtype=torch.bfloat16, device="cuda")
    for t in range(0, T, 1 << 16):
        x[t:t + (1 << 16)] = torch.randn(min(1 << 16, T - t), D, generator=g, device="cuda")
    w = (1 + 0.3 * torch.randn(D, generator=g, device="cuda")).bfloat16()
    say(f"layer norm {T}x{D}")
    y, mean, rstd = mg.layer_norm(x, w, w)
    # dy = y's first rows over again, zero elsewhere: the sums over rows stay small enough to check
    rows = torch.tensor([0, 1, 511, 512, T // 2, (1 << 31) // D - 1, (1 << 31) // D, T - 1],
                        device="cuda")
    dy = torch.zeros_like(x)
    dy[rows] = torch.randn(len(rows), D, generator=g, device="cuda").bfloat16()
    dx, dw, db = mg.layer_norm_backward(dy, x, w, mean, rstd)
    torch.cuda.synchronize()
    want = reference(x[rows], w, w, dy[rows], 1e-5)
    # rows of zeros add nothing to the sums or to their bounds
    check({"y": y[rows], "mean": mean[rows], "rstd": rstd[rows], "dx": dx[rows], "dw": dw,
           "db": db}, want)
    dx[rows] = 0
    assert not dx.any()
    assert math.isfinite(float(y[::4097].float().sum()))


# either side of the rows that one launch takes backwards: 1024, and 8 MiB of x
FEW = [(1, 16384), (127, 16384), (128, 16384), (129, 16384), (256, 16380), (1023, 40), (1024, 2048),
       (1024, 4096), (1025, 40), (64, 5), (65, 9), (257, 129), (1000, 2049), (500, 8192), (513, 700)]
# and rows of every form past them
MANY = [(1025, 1), (1030, 8), (1100, 127), (1400, 129), (1029, 512), (1025, 513), (1031, 1024),
        (1027, 1025), (1040, 2048), (1050, 1537), (1026, 2049), (1030, 8192), (1025, 8200),
        (1025, 16384)]


@pytest.mark.parametrize("dtype,weight", [("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"),
                                          ("bf16", "f32")])
@pytest.mark.parametrize("T,D", FEW + MANY)
def test_rows_of_one_launch_and_more(T, D, dtype, weight):
    x, w, b, dy = case(T, D, dtype, weight, T + D)
    say(f"layer norm {T}x{D} {dtype} {weight}")
    check(both(x, w, b, dy), reference(x, w, b, dy, 1e-5))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,D", [(90, 77), (300, 1001), (1500, 77), (1200, 1001), (1100, 4003)])
def test_strided_rows_of_one_launch_and_more(T, D, dtype):
    """Rows off 16-byte boundaries with NaN between them, and results inside larger buffers."""
    x, w, b, dy = case(T, D, dtype, dtype, D + T)
    want = reference(x, w, b, dy, 1e-5)

    def inside(t, offset, extra):
        buf = torch.full((t.shape[0], t.shape[1] + extra), float("nan"), dtype=t.dtype, device="cuda")
        buf[:, offset:offset + t.shape[1]] = t
        return buf, buf[:, offset:offset + t.shape[1]]

    say(f"layer norm {T}x{D} inside buffers {dtype}")
    xs, dys = inside(x, 3, 8)[1], inside(dy, 1, 5)[1]
    y, mean, rstd = mg.layer_norm(xs, w, b)
    xbuf, dx = inside(torch.zeros_like(x), 5, 7)
    vectors = torch.full((2 * D + 3,), float("nan"), dtype=w.dtype, device="cuda")
    dw, db = vectors[1:1 + D], vectors[2 + D:2 + 2 * D]
    mg.layer_norm_backward(dys, xs, w, mean, rstd, dx=dx, dw=dw, db=db)
    torch.cuda.synchronize()
    check({"y": y, "mean": mean, "rstd": rstd, "dx": dx, "dw": dw, "db": db}, want)
    assert torch.isnan(vectors[[0, 1 + D, -1]]).all()
    dx.zero_()
    assert int(torch.isnan(xbuf).sum()) == xbuf.numel() - dx.numel()
    # each result alone
    for name in ("dx", "dw", "db"):
        need = {f"need_{n}": n == name for n in ("dx", "dw", "db")}
        got = dict(zip(("dx", "dw", "db"), mg.layer_norm_backward(dys, xs, w, mean, rstd, **need)))
        torch.cuda.synchronize()
        assert all(got[n] is None for n in got if n != name)
        check({name: got[name]}, want)


@pytest.mark.parametrize("T,D", [(200, 1032), (1100, 1032), (30, 16000)])
def test_backward_captured_and_on_a_side_stream(T, D):
    x, w, b, dy = case(T, D, "bf16", "f32", 7)
    y, mean, rstd = mg.layer_norm(x, w, b)
    say(f"layer norm {T}x{D} captured")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = mg.layer_norm_backward(dy, x, w, mean, rstd)
    side = torch.cuda.Stream()
    for i in range(3):
        dy.copy_(dy.roll(i, 0))
        want = mg.layer_norm_backward(dy, x, w, mean, rstd)
        for t in held:
            t.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        got = mg.layer_norm_backward(dy, x, w, mean, rstd, stream=side.cuda_stream)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want))
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("T", [60, 1500])
def test_infinities_stay_in_their_rows_and_columns(T):
    x, w, b, dy = case(T, 300, "f32", "f32", T)
    y, mean, rstd = mg.layer_norm(x, w, b)
    dy[T // 2, 7] = float("inf")
    say(f"layer norm {T}x300 with an infinity in dy")
    dx, dw, db = mg.layer_norm_backward(dy, x, w, mean, rstd)
    torch.cuda.synchronize()
    rows, columns = ~torch.isfinite(dx).all(1), ~torch.isfinite(dw)
    assert rows.nonzero().tolist() == [[T // 2]] and columns.nonzero().tolist() == [[7]]
    assert (~torch.isfinite(db)).nonzero().tolist() == [[7]]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,D", [(6, 40), (6, 700), (6, 5000), (6, 20000), (1100, 700)])
def test_squares_past_the_range(T, D, dtype):
    """Distances of 1e20, whose squares FP32 does not hold: an infinite variance, so y is the
    bias and dx 0, and the row adds nothing to dw; the rows beside it are as without it."""
    x, w, b, dy = case(T, D, dtype, dtype, D)
    x[3] = 1e20 * torch.where(torch.arange(D, device="cuda") % 2 == 0, 1.0, -1.0)
    say(f"layer norm {T}x{D} {dtype} with a row past the squares' range")
    got = both(x, w, b, dy)
    assert torch.equal(got["y"][3], b) and not got["rstd"][3] and not got["dx"][3].any()
    keep = [i for i in range(T) if i != 3]
    want = reference(x[keep], w, b, dy[keep], 1e-5)
    check({k: got[k][keep] for k in ("y", "mean", "rstd", "dx")} | {"dw": got["dw"]}, want)
