"""The AdamW step against its formulas in float64, and against the same formulas one
float32 operation at a time.

Tolerances (u: half a step of the parameter's dtype, f = 2^-24): the factors are off by f
each, so m = b1 m + r1 g is off by em = 3 f (|b1 m| + |r1 g|), g by another f where it is
scaled, v likewise by 4 f and 5 f of its (positive) terms, its root by 4 f; the quotient of
the step adds its denominator's three roundings, its own, and the factor's two: the step
is off by 12 f |step| + rate em / denominator, p by that, 3 f |p| and u |p|.

8-bit codes: a value is off by half a step of E4M3, 2^-4 of its magnitude or 2^-10 of its
scale, whichever is more, a positive root by 2^-9 of the scale at most (it never becomes 0).
"""
import math

import pytest
import torch

import dense_gemm_16_amd as mg
from gpu_helpers import say

pytestmark = pytest.mark.gpu

TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
F = 2.0 ** -24
HYPER = dict(lr=2e-3, betas=(0.9, 0.99), eps=1e-8, weight_decay=0.1)


def tensors(sizes, param, grad, bits, master, seed, steps=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(n):
        return torch.randn(n, generator=g, device="cuda")

    params = [(0.05 * randn(n)).to(TORCH[param]) for n in sizes]
    grads = [(1e-2 * randn(n) * torch.exp(randn(n))).to(TORCH[grad]) for n in sizes]
    states = [mg.adamw_state(p, bits=bits, master=master) for p in params]
    if master:  # copies hold more than the parameters
        for p, s in zip(params, states):
            s.master.add_(1e-5 * randn(p.numel()))
    if steps:
        for s in states:
            n = s.avg.numel()
            m, r = 1e-2 * randn(n), 1e-2 * randn(n).abs()
            if bits == 32:
                s.avg.copy_(m)
                s.sq.copy_(r * r)
            else:
                for value, codes, scales in ((m, s.avg, s.avg_scales), (r, s.sq, s.sq_scales)):
                    blocks = torch.nn.functional.pad(value, (0, -n % 256)).view(-1, 256)
                    scales.copy_(blocks.abs().amax(1) / 448)
                    codes.copy_((blocks / scales[:, None]).view(-1)[:n].to(codes.dtype))
    return params, grads, states


def copied(params, grads, states):
    return ([p.clone() for p in params], [g.clone() for g in grads],
            [mg.AdamState(*(None if t is None else t.clone() for t in s)) for s in states])


def spread(scales, n):
    return scales.repeat_interleave(256)[:n]


def moments(s):
    """The state's m and v in float64."""
    if s.avg_scales is None:
        return s.avg.double(), s.sq.double()
    n = s.avg.numel()
    # the decoded float32 product is what the step starts from
    m = (s.avg.view(torch.float8_e4m3fn).float() * spread(s.avg_scales, n)).double()
    r = (s.sq.view(torch.float8_e4m3fn).float() * spread(s.sq_scales, n)).double()
    return m, r * r


def check_step(before, after, step, scale=1.0, hyper=HYPER):
    lr, (b1, b2), eps, wd = (hyper[k] for k in ("lr", "betas", "eps", "weight_decay"))
    for (p0, g, s0), (p1, _, s1) in zip(zip(*before), zip(*after)):
        n = p0.numel()
        if n == 0:
            continue
        u = torch.finfo(p0.dtype).eps / 2
        m0, v0 = moments(s0)
        G = g.double() * scale
        extra = 0 if scale == 1.0 else F
        m = b1 * m0 + (1 - b1) * G
        em = (3 * F + extra) * ((b1 * m0).abs() + ((1 - b1) * G).abs())
        v = b2 * v0 + (1 - b2) * G * G
        ev = (5 * F + 2 * extra) * v
        r = v.sqrt()
        er = r * (4 * F + extra)
        old = p0.double() if s0.master is None else s0.master.double()
        rate = lr / (1 - b1 ** step)
        den = r / math.sqrt(1 - b2 ** step) + eps
        move = rate * m / den
        emove = 12 * F * move.abs() + rate * em / den
        p = old * (1 - lr * wd) - move
        ep = emove + 3 * F * (old.abs() + p.abs())
        if s0.master is not None:
            assert ((s1.master.double() - p).abs() <= ep).all()
            assert torch.equal(p1, s1.master.to(p1.dtype))
        sub = 2.0 ** -25 if p0.dtype == torch.float16 else 0.0
        assert ((p1.double() - p).abs() <= ep + u * (p.abs() + ep) + sub).all()
        if s1.avg_scales is None:
            assert ((s1.avg.double() - m).abs() <= em).all()
            assert ((s1.sq.double() - v).abs() <= ev).all()
            continue
        for value, err, codes, scales, root in ((m, em, s1.avg, s1.avg_scales, False),
                                                (r, er, s1.sq, s1.sq_scales, True)):
            blocks = torch.nn.functional.pad(value.abs(), (0, -n % 256)).view(-1, 256).amax(1)
            worst = torch.nn.functional.pad(err, (0, -n % 256)).view(-1, 256).amax(1)
            assert ((scales.double() - blocks / 448).abs() <= worst / 448 + 2 * F * blocks).all()
            unit = spread(scales, n).double()
            held = codes.view(torch.float8_e4m3fn).double()
            least = 2.0 ** -9 if root else 2.0 ** -10
            tol = torch.maximum(2.0 ** -4 * value.abs(), least * unit) * (1 + 2.0 ** -20) + err
            assert ((held * unit - value).abs() <= tol).all()
            if root:
                assert (held[(value > 0) & (unit > 0)] >= 2.0 ** -9).all()


def plain_step(params, grads, states, step, hyper=HYPER):
    """The formulas one float32 operation at a time, in place."""
    lr, (b1, b2), eps, wd = (hyper[k] for k in ("lr", "betas", "eps", "weight_decay"))
    for p, g, s in zip(params, grads, states):
        n, eight = p.numel(), s.avg_scales is not None
        if eight:
            m = s.avg.float() * spread(s.avg_scales, n)
            r = s.sq.float() * spread(s.sq_scales, n)
            v = r * r
        else:
            m, v = s.avg, s.sq
        m = m * b1 + g.float() * (1 - b1)
        v = v * b2 + (g.float() * g.float()) * (1 - b2)
        r = torch.sqrt(v)
        if eight:
            for value, codes, scales, root in ((m, s.avg, s.avg_scales, False),
                                               (r, s.sq, s.sq_scales, True)):
                blocks = torch.nn.functional.pad(value, (0, -n % 256)).view(-1, 256)
                top = blocks.abs().amax(1)
                scales.copy_(torch.where(top < 2.0 ** -100, 0.0, top * (1 / 448)))
                x = blocks * torch.where(scales > 0, 1.0 / scales, 0.0)[:, None]
                if root:
                    x = torch.where((blocks > 0) & (scales > 0)[:, None], x.clamp(min=2.0 ** -9), x)
                codes.copy_(x.view(-1)[:n].to(torch.float8_e4m3fn))
        else:
            s.avg.copy_(m)
            s.sq.copy_(v)
        old = p.float() if s.master is None else s.master
        new = old * (1 - lr * wd) - (m / (r * (1 / math.sqrt(1 - b2 ** step)) + eps)) * (
            lr / (1 - b1 ** step))
        if s.master is not None:
            s.master.copy_(new)
        p.copy_(new)


SIZES = [1, 255, 256, 257, 4095, 4096, 4097, 0, 3, 8192 + 16, 70001, 15, 16, 17]
TYPES = [("f32", "f32", False), ("f16", "f16", False), ("f16", "f32", True), ("bf16", "bf16", False),
         ("bf16", "bf16", True), ("bf16", "f32", False), ("bf16", "f32", True),
         ("f16", "f32", False), ("f16", "f16", True)]


@pytest.mark.parametrize("param,grad,master", TYPES)
@pytest.mark.parametrize("bits", [32, 8])
def test_step(param, grad, master, bits):
    for steps in (0, 5):
        case = tensors(SIZES, param, grad, bits, master, bits, steps)
        before = copied(*case)
        say(f"adamw {param} {grad} master {master} {bits} bits after {steps}")
        mg.adamw_(*case, step=steps + 1, **HYPER)
        torch.cuda.synchronize()
        check_step(before, case, steps + 1)
        assert all(torch.equal(a, b) for a, b in zip(before[1], case[1]))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("param,master", [("f32", False), ("bf16", True)])
def test_states_are_the_formulas_bits(bits, param, master):
    """Over several steps, each from the last one's states: the same bits, codes too."""
    case = tensors([70000, 300, 5], param, param, bits, master, 3)
    plain = copied(*case)
    say(f"adamw in step with the formulas, {param} {bits} bits")
    for step in range(1, 6):
        mg.adamw_(*case, step=step, **HYPER)
        plain_step(*plain, step)
        torch.cuda.synchronize()
        for a, b in zip(case[2], plain[2]):
            for x, y in zip(a[:4], b[:4]):
                if x is not None:
                    assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
        for a, b in zip(case[1], plain[1]):
            a.add_(0.1 * a.roll(1))
            b.copy_(a)


def test_every_code_and_scale():
    """All 256 codes of both states and scales over FP32's range decode and come back."""
    n = 256 * 40
    codes = torch.arange(256, dtype=torch.uint8, device="cuda").repeat(40)
    codes[(codes & 127) == 127] = 0  # NaN codes
    scales = torch.exp2(torch.arange(40, device="cuda") * 3.0 - 60)
    p, g = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    state = mg.AdamState(codes.clone(), (codes & 127).clone(), scales.clone(), scales.clone())
    say("adamw every code")
    # betas next to 1 leave the moments as they are, but for the decay in FP32
    mg.adamw_([p], [g], [state], step=1, lr=0.0, betas=(1 - 2.0 ** -30, 1 - 2.0 ** -30),
              weight_decay=0.0)
    torch.cuda.synchronize()
    f8 = torch.float8_e4m3fn
    assert torch.equal(state.avg.view(f8).float(), codes.view(f8).float())
    # v, the square, is FP32: that of a root of 2^-63 or more is normal, and exact for four
    # digits; smaller squares are off by half of 2^-149 in each of two products and a sum, so
    # by 2^-147, and the root by its root, 2^-73, at most
    old = (codes & 127).view(f8).double() * scales.repeat_interleave(256).double()
    new = state.sq.view(f8).double() * state.sq_scales.repeat_interleave(256).double()
    # and that of a root of 2^64 is past FP32's largest, which spoils its block
    past = (448 * scales.double() >= 2.0 ** 64).repeat_interleave(256)
    assert torch.isnan(new[past]).all() and past.float().mean() < 0.1
    exact = ((old >= 2.0 ** -63) | (old == 0)) & ~past
    assert exact.float().mean() > 0.8
    assert torch.equal(state.sq[exact], (codes & 127)[exact])
    step = torch.maximum(2.0 ** -4 * old, 2.0 ** -9 * scales.repeat_interleave(256).double())
    assert ((new - old).abs() <= 2.0 ** -73 + step * 1.001)[~exact & ~past].all()
    assert torch.allclose(state.avg_scales, scales, rtol=1e-6, atol=0)
    assert torch.allclose(state.sq_scales[~past[::256]], scales[~past[::256]], rtol=1e-6, atol=0)


def test_special_blocks():
    n = 256 * 6 + 100
    p, g, s = (x[0] for x in tensors([n], "f32", "f32", 8, False, 1, 5))
    g[300] = float("nan")
    g[700] = float("inf")
    g[256 * 3:256 * 4] = 0
    s.avg_scales[3] = s.sq_scales[3] = 0           # a block without gradients so far
    g[256 * 4:256 * 5] = 1e-35                      # too small to be held
    s.avg_scales[4] = s.sq_scales[4] = 0
    before = copied([p], [g], [s])
    say("adamw special blocks")
    mg.adamw_([p], [g], [s], step=6, **HYPER)
    torch.cuda.synchronize()
    assert torch.isnan(s.avg_scales[[1, 2]]).all() and torch.isnan(s.sq_scales[[1, 2]]).all()
    bad = torch.zeros(n, dtype=torch.bool, device="cuda")
    bad[[300, 700]] = True
    assert torch.equal(~torch.isfinite(p), bad)  # the step itself spoils the elements alone
    assert not s.avg_scales[[3, 4]].any() and not s.sq_scales[[3, 4]].any()
    assert not s.avg[256 * 3:256 * 5].view(torch.uint8).any()
    m, _ = moments(s)
    assert torch.isnan(m[256:768]).all() and torch.isfinite(m[768:]).all()
    keep = [0, 5, 6]
    for k in keep:
        cut = slice(256 * k, min(n, 256 * (k + 1)))

        def part(c):
            (q,), (h,), (t,) = c
            return [q[cut]], [h[cut]], [mg.AdamState(t.avg[cut], t.sq[cut], t.avg_scales[k:k + 1],
                                                     t.sq_scales[k:k + 1])]

        check_step(part(before), part(([p], [g], [s])), 6)
    # a gradient of zero without a state leaves the decay alone
    assert torch.equal(p[256 * 3:256 * 4], before[0][0][256 * 3:256 * 4] * (1 - 2e-3 * 0.1))


def test_eps_zero_and_no_gradient():
    p, g, s = (x[0] for x in tensors([600], "f32", "f32", 32, False, 1))
    g.zero_()
    g[5] = 1.0
    mg.adamw_([p], [g], [s], step=1, lr=1e-2, eps=0.0, weight_decay=0.0)
    torch.cuda.synchronize()
    # 0 / 0 shows, and m / sqrt(v) is the sign
    assert torch.isnan(p[:5]).all() and torch.isnan(p[6:]).all() and torch.isfinite(p[5])


@pytest.mark.parametrize("bits", [32, 8])
def test_many_tensors_and_views(bits):
    """More tensors than one launch takes, of odd sizes, in the middle of buffers, at every
    offset to 16 bytes; what lies between them is as it was."""
    sizes = [(37 * i) % 700 + (i % 5 == 0) * 5000 for i in range(150)]
    case = tensors(sizes, "bf16", "f32", bits, True, 2, 4)

    def packed(list_, align=1):
        at, starts = 1, []
        for t in list_:
            starts.append(at)
            at += t.numel() + 3
        buf = torch.full((at + 8,), 77, dtype=torch.float32, device="cuda").to(list_[0].dtype)
        views = [buf[a:a + t.numel()].copy_(t) for a, t in zip(starts, list_)]
        return buf, views

    bufs, lists = [], []
    fields = [case[0], case[1]] + [[s[i] for s in case[2]] for i in range(5) if case[2][0][i] is not None]
    for f in fields:
        b, v = packed(f)
        bufs.append((b, [t.numel() for t in v]))
        lists.append(v)
    none = [None] * 150
    if bits == 32:
        params, grads, avg, sq, master = lists
        states = list(map(mg.AdamState, avg, sq, none, none, master))
    else:
        params, grads, avg, sq, ms, ss, master = lists
        states = list(map(mg.AdamState, avg, sq, ms, ss, master))
    say(f"adamw 150 views {bits} bits")
    mg.adamw_(params, grads, states, step=5, **HYPER)
    torch.cuda.synchronize()
    check_step(case, (params, grads, states), 5)
    for (buf, counts), views in zip(bufs, lists):
        held = torch.ones(buf.numel(), dtype=torch.bool, device="cuda")
        at = 1
        for n in counts:
            held[at:at + n] = False
            at += n + 3
        assert (buf.float()[held] == buf.float()[0]).all()


def test_numbers_on_the_device():
    """lr, step and grad_scale read on the device give what the same numbers give from the
    host; a grad_scale that is not finite changes nothing."""
    for bits in (32, 8):
        case = tensors([5000, 300], "bf16", "bf16", bits, True, 3, 4)
        host, dev, skip = copied(*case), copied(*case), copied(*case)
        say(f"adamw numbers on the device {bits} bits")
        scale = 2.0 ** -6
        kw = HYPER | {"lr": float(torch.tensor(2e-3))}
        mg.adamw_(*host, step=7, grad_scale=scale, **kw)
        lr = torch.tensor([2e-3], device="cuda")
        step = torch.tensor(7, device="cuda")
        gs = torch.tensor(scale, device="cuda")
        mg.adamw_(*dev, step=step, grad_scale=gs, **(HYPER | {"lr": lr}))
        torch.cuda.synchronize()
        check_step(case, host, 7, scale=scale, hyper=kw)
        for a, b in zip(host[2], dev[2]):
            assert all(x is None or torch.equal(x.view(torch.uint8), y.view(torch.uint8))
                       for x, y in zip(a[:4], b[:4]))
            # pow on the device may differ from the host's in its last bits: one rounding of
            # each factor, so 4 f of the step
            assert torch.allclose(a.master, b.master, rtol=2.0 ** -22, atol=2.0 ** -21 * 2e-3)
        for bad in (float("inf"), float("nan"), -float("inf")):
            mg.adamw_(*skip, step=7, grad_scale=torch.tensor(bad, device="cuda"), **kw)
        torch.cuda.synchronize()
        for a, b in zip(case[2] + [case[0]], skip[2] + [skip[0]]):
            assert all(x is None or torch.equal(x.view(torch.uint8), y.view(torch.uint8))
                       for x, y in zip(a, b))


def test_graph_replay_side_stream_and_repeats():
    case = tensors([40000, 300, 17], "bf16", "bf16", 8, False, 3, 4)
    eager, side_case, graph_case = copied(*case), copied(*case), copied(*case)
    side = torch.cuda.Stream()
    say("adamw on a side stream by handle")
    torch.cuda.synchronize()
    step = torch.tensor(5, device="cuda")
    for i in range(3):
        mg.adamw_(*eager, step=torch.tensor(5 + i, device="cuda"), **HYPER)
        mg.adamw_(*side_case, step=torch.tensor(5 + i, device="cuda"), **HYPER,
                  stream=side.cuda_stream)
    torch.cuda.synchronize()

    def same(a, b):
        flat = lambda c: c[0] + [t for s in c[2] for t in s if t is not None]  # noqa: E731
        return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8))
                   for x, y in zip(flat(a), flat(b)))

    assert same(eager, side_case)
    say("adamw in a graph that counts its steps")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mg.adamw_(*graph_case, step=step, **HYPER)
        step.add_(1)
    fresh = copied(*case)
    for i in range(3):
        g.replay()
        mg.adamw_(*fresh, step=torch.tensor(5 + i, device="cuda"), **HYPER)
        torch.cuda.synchronize()
        assert same(graph_case, fresh) and int(step) == 6 + i


def test_refusals():
    (p,), (g,), (s,) = tensors([512], "bf16", "bf16", 8, False, 1)
    s32 = mg.adamw_state(p)
    wide = mg.adamw_state(p, master=True)
    for call in (lambda: mg.adamw_([p], [g], [s, s], step=1),
                 lambda: mg.adamw_([p], [g.half()], [s], step=1),
                 lambda: mg.adamw_([p], [g[:-1]], [s], step=1),
                 lambda: mg.adamw_([p, p], [g, g], [s, s32], step=1),
                 lambda: mg.adamw_([p, p], [g, g], [s32, wide], step=1),
                 lambda: mg.adamw_([p], [g], [s._replace(avg_scales=None)], step=1),
                 lambda: mg.adamw_([p], [g], [s._replace(sq_scales=s.sq_scales[:1])], step=1),
                 lambda: mg.adamw_([p], [g], [s32._replace(avg_scales=s.avg_scales)], step=1),
                 lambda: mg.adamw_([p], [g], [s._replace(avg=s.avg.float())], step=1),
                 lambda: mg.adamw_([p[::2]], [g[::2]], [mg.adamw_state(p[:256])], step=1),
                 lambda: mg.adamw_([p], [g.cpu()], [s], step=1),
                 lambda: mg.adamw_([p.int()], [g], [s], step=1),
                 lambda: mg.adamw_([p], [g], [s], step=torch.tensor(1)),
                 lambda: mg.adamw_([p], [g], [s], step=torch.tensor([1, 2], device="cuda")),
                 lambda: mg.adamw_([p], [g], [s], step=1, lr=torch.tensor(1.0, device="cuda").double()),
                 lambda: mg.adamw_([p.float()], [g.float()], [mg.adamw_state(p, master=True)], step=1)):
        with pytest.raises(ValueError):
            call()
    for kw in ({"step": 0}, {"step": 1, "betas": (1.0, 0.9)}, {"step": 1, "eps": -1.0},
               {"step": 1, "lr": float("inf")}):
        with pytest.raises(mg.MigemmError):
            mg.adamw_([p], [g], [s], **kw)
    with pytest.raises(mg.MigemmError):
        mg.adamw_([p, p], [g, g], [s, mg.adamw_state(p, bits=8)], step=1)
    with pytest.raises(mg.MigemmError):
        mg.adamw_([p], [p], [s], step=1)
    # one gradient may serve two parameters
    q = p.clone()
    mg.adamw_([p, q], [g, g], [s, mg.adamw_state(q, bits=8)], step=1)
    torch.cuda.synchronize()
    assert torch.equal(p, q)


@pytest.mark.parametrize("bits,param,grad,master", [(32, "f32", "f32", False), (32, "bf16", "bf16", True),
                                                    (8, "f16", "f32", True), (8, "bf16", "bf16", False)])
def test_steps_past_the_caches(bits, param, grad, master):
    """Past 512 MiB read and written, two tensors, the second off 16-byte boundaries in every
    array: the bits of the same tensors in steps of their own, which go through the caches."""
    n = 31_000_003
    (p, q), (g, h), states = tensors([n, n], param, grad, bits, master, 7, 3)

    def moved(t):
        return None if t is None else torch.cat((t[:1], t))[1:]

    def moved_codes(t):
        return torch.cat((t[:1].view(torch.uint8), t.view(torch.uint8)))[1:].view(t.dtype)

    s = states[1]
    codes = moved if bits == 32 else moved_codes
    second = (moved(q), moved(h), mg.AdamState(codes(s.avg), codes(s.sq), moved(s.avg_scales),
                                               moved(s.sq_scales), moved(s.master)))
    whole = [p, second[0]], [g, second[1]], [states[0], second[2]]
    written = whole[0] + [t for s in whole[2] for t in s if t is not None]
    size = sum(t.numel() * t.element_size() for t in whole[1] + 2 * written)  # read and written
    assert size > 512 << 20
    parts = [copied([p], [g], [states[0]]), copied([q], [h], [states[1]])]
    cut = 16 * 4096 * 50
    say(f"adamw {n} twice {param} {bits} bits")
    mg.adamw_(*whole, step=4, **HYPER)
    for (a,), (b,), (t,) in parts:
        for c in range(0, n, cut):
            e, k = slice(c, min(n, c + cut)), slice(c // 256, (min(n, c + cut) + 255) // 256)
            piece = mg.AdamState(t.avg[e], t.sq[e], None if bits == 32 else t.avg_scales[k],
                                 None if bits == 32 else t.sq_scales[k],
                                 None if t.master is None else t.master[e])
            mg.adamw_([a[e]], [b[e]], [piece], step=4, **HYPER)
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(whole[0][i], parts[i][0][0])
        for x, y in zip(whole[2][i], parts[i][2][0]):
            if x is not None:
                assert torch.equal(x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x,
                                   y.view(torch.uint8) if y.dtype == torch.float8_e4m3fn else y)


@pytest.mark.parametrize("bits", [32, 8])
def test_more_than_2_31_elements(bits):
    n = (1 << 31) + 4096 * 3 + 77
    p = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    s = mg.adamw_state(p, bits=bits)
    gen = torch.Generator(device="cuda").manual_seed(1)
    cuts = [slice(0, 512), slice((1 << 31) - 512, (1 << 31) + 512), slice(n - 77 - 256, n)]
    for c in cuts:
        p[c] = torch.randn(p[c].numel(), generator=gen, device="cuda").bfloat16()
        g[c] = torch.randn(p[c].numel(), generator=gen, device="cuda").bfloat16()
    before = [(p[c].clone(), g[c].clone()) for c in cuts]
    say(f"adamw {n} elements {bits} bits")
    mg.adamw_([p], [g], [s], step=1, **HYPER)
    torch.cuda.synchronize()
    for c, (p0, g0) in zip(cuts, before):
        if bits == 8:
            b = slice(c.start // 256, (c.stop + 255) // 256)
            after = mg.AdamState(s.avg[c], s.sq[c], s.avg_scales[b], s.sq_scales[b])
        else:
            after = mg.AdamState(s.avg[c], s.sq[c])
        check_step(([p0], [g0], [mg.adamw_state(p0, bits=bits)]), ([p[c]], [g0], [after]), 1)
        p[c] = 0
        s.avg[c] = 0
    assert not p.any() and not s.avg.view(torch.uint8).any()
