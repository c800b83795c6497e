"""Embedding lookup and its gradient against the definitions.

Forwards each element is one FP32 product rounded once: compared bit for bit.  Backwards
(u: half a step of the gradient's dtype, f = 2^-24) an entry of c tokens is a sum of c
values in FP32, in any order off by at most c f sum |dy|; the product with the scale and
the sum with what was there add 2 f of their magnitudes, the last rounding u |dw| (FP16
below its normal range 2^-25).
"""
import pytest
import torch

import dense_gemm_16_amd as mg
from gpu_helpers import say

pytestmark = pytest.mark.gpu

TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
IGNORE = -100


def draw_index(T, V, g, kind):
    if kind == "one":        # every token the same
        return torch.full((T,), V - 1, dtype=torch.int64, device="cuda")
    if kind == "ignored":    # padding alone
        return torch.full((T,), IGNORE, dtype=torch.int64, device="cuda")
    u = torch.rand(T, generator=g, device="cuda", dtype=torch.float64)
    # a few entries named often, many once
    index = (u ** 6 * V).long().clamp(max=V - 1)
    index = torch.where(torch.rand(T, generator=g, device="cuda") < 0.1, IGNORE, index)
    if kind == "bad":        # outside the table, either side
        far = torch.tensor([V, -1, 1 << 40, -(1 << 62), V + 7], device="cuda")
        bad = torch.rand(T, generator=g, device="cuda") < 0.2
        index = torch.where(bad, far[torch.randint(0, 5, (T,), generator=g, device="cuda")], index)
    return index


def case(T, V, D, dtype, seed, kind="mixed"):
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = torch.randn(V, D, generator=g, device="cuda").to(TORCH[dtype])
    dy = torch.randn(T, D, generator=g, device="cuda").to(TORCH[dtype])
    return w, draw_index(T, V, g, kind), dy


def forward_reference(w, index, scale, ignore=IGNORE):
    V = w.shape[0]
    inside = (index >= 0) & (index < V) & (index != ignore)
    y = (w[torch.where(inside, index, 0)].float() * scale).to(w.dtype)
    y = torch.where(inside[:, None], y, float("nan"))
    return torch.where((index == ignore)[:, None], 0.0, y)


def gradient_reference(dy, index, V, scale, dtype, old=None, ignore=IGNORE):
    inside = (index >= 0) & (index < V) & (index != ignore)
    # on the host: float64 atomics on a few rows take a minute there
    at, rows = index[inside].cpu(), dy[inside].cpu().double()
    total = torch.zeros(V, dy.shape[1], dtype=torch.float64)
    size = total.clone()
    total.index_add_(0, at, rows)
    size.index_add_(0, at, rows.abs())
    total, size = total.cuda(), size.cuda()
    count = torch.bincount(at, minlength=V).double()[:, None].cuda()
    f, u = 2.0 ** -24, torch.finfo(dtype).eps / 2
    tol = abs(scale) * size * (count + 2) * f
    value = scale * total
    if old is not None:
        value = value + old.double()
        tol += 2 * f * (old.double().abs() + abs(scale) * total.abs())
    sub = 2.0 ** -25 if dtype == torch.float16 else 0.0
    tol += u * (value.abs() + tol) + sub * (count > 0)
    return value, tol


def check(dw, want):
    value, tol = want
    assert torch.isfinite(dw).all()
    worst = ((dw.double() - value).abs() - tol).max()
    assert worst <= 0, (float(worst), float((dw.double() - value).abs().max()))


def same(a, b):
    return torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(
        torch.nan_to_num(a), torch.nan_to_num(b))


def both(T, V, D, dtype, seed, kind="mixed", scale=3.0):
    w, index, dy = case(T, V, D, dtype, seed, kind)
    say(f"embedding {T} of {V}x{D} {dtype} {kind}")
    y = mg.embedding(w, index, scale=scale)
    dw = mg.embedding_backward(dy, index, V, scale=scale)
    torch.cuda.synchronize()
    assert same(y, forward_reference(w, index, scale))
    check(dw, gradient_reference(dy, index, V, scale, dy.dtype))
    old = w.clone()
    got = mg.embedding_backward(dy, index, V, scale=scale, dw=old, accumulate=True)
    torch.cuda.synchronize()
    assert got is old
    check(old, gradient_reference(dy, index, V, scale, dy.dtype, w))
    # rows that no token names are as they were
    named = torch.zeros(V, dtype=torch.bool, device="cuda")
    named[index[(index >= 0) & (index < V)]] = True
    assert torch.equal(old[~named], w[~named])


# rows below a wavefront's lanes, of several segments, ending inside a chunk; lists shorter
# than a stretch, ending inside one, past the sort by counting (8192)
SIZES = [(1, 1, 1), (1, 1000, 64), (7, 5, 3), (8, 300, 8), (9, 300, 40), (100, 511, 129),
         (100, 512, 520), (1003, 3001, 200), (2048, 50, 1032), (5000, 40000, 72), (8192, 700, 136),
         (16, 131072, 4096), (300, 2000, 8200)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,V,D", SIZES)
def test_embedding(T, V, D, dtype):
    both(T, V, D, dtype, T + V + D)


@pytest.mark.parametrize("T,V,D", [(32768, 50000, 16), (32769, 50000, 16), (40000, 300, 24),
                                   (200000, 131072, 8), (70000, 5, 40), (1 << 20, 1000, 2)])
def test_long_lists(T, V, D):
    both(T, V, D, "f32" if T % 2 else "bf16", T)


@pytest.mark.parametrize("kind", ["mixed", "one"])
def test_a_list_of_2_24(kind):
    """Counts over thousands of tiles, stretches longer than a wavefront, rows of one element."""
    both((1 << 24) + 3, 70000, 1, "f32", 1, kind)


@pytest.mark.parametrize("kind", ["one", "ignored", "bad"])
@pytest.mark.parametrize("T,V,D", [(1, 40, 16), (31, 1, 24), (700, 900, 520), (33000, 700, 64)])
def test_special_lists(T, V, D, kind):
    both(T, V, D, "bf16", T + V, kind)
    both(T, V, D, "f32", T + V, kind)


@pytest.mark.parametrize("V", [(1 << 18) - 1, 1 << 18, (1 << 25) - 1, (1 << 25) + 5, (1 << 27) + 3])
def test_long_tables(V):
    """Entries past two digits of the sort, and past what one workgroup's packs."""
    T, D = 500, 2
    g = torch.Generator(device="cuda").manual_seed(V)
    index = torch.randint(0, V, (T,), generator=g, device="cuda")
    index[:4] = torch.tensor([V - 1, 0, V // 2, V - 1])
    dy = torch.randn(T, D, generator=g, device="cuda")
    say(f"table of {V}")
    dw = mg.embedding_backward(dy, index, V, scale=0.5)
    w = torch.randn(V, D, generator=g, device="cuda")
    y = mg.embedding(w, index, scale=0.5)
    torch.cuda.synchronize()
    check(dw, gradient_reference(dy, index, V, 0.5, torch.float32))
    assert same(y, forward_reference(w, index, 0.5))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_gradient_in_32_bits(dtype):
    w, index, dy = case(3000, 1000, 264, dtype, 4)
    old = torch.randn(1000, 264, device="cuda")
    say(f"{dtype} into f32")
    dw = mg.embedding_backward(dy, index, 1000, scale=0.1, out_dtype=torch.float32)
    more = mg.embedding_backward(dy, index, 1000, scale=0.1, dw=old.clone(), accumulate=True)
    torch.cuda.synchronize()
    assert dw.dtype == torch.float32
    # scale as the library is given it: a float
    scale = float(torch.tensor(0.1))
    check(dw, gradient_reference(dy, index, 1000, scale, torch.float32))
    check(more, gradient_reference(dy, index, 1000, scale, torch.float32, old))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_strided_and_misaligned(dtype):
    T, V, D = 300, 210, 77
    w, index, dy = case(T, V, D, dtype, 8)

    def inside(t, offset, extra):
        buf = torch.full((offset + t.shape[0] * (t.shape[1] + extra),), float("nan"),
                         dtype=t.dtype, device="cuda")
        return buf, buf[offset:].view(t.shape[0], -1)[:, :t.shape[1]].copy_(t)

    say(f"embedding inside buffers {dtype}")
    ybuf, y = inside(torch.zeros_like(dy), 3, 1)
    dbuf, dw = inside(torch.zeros_like(w), 1, 5)
    mg.embedding(inside(w, 1, 3)[1], index, scale=1.5, out=y)
    mg.embedding_backward(inside(dy, 5, 7)[1], index, V, scale=1.5, dw=dw)
    torch.cuda.synchronize()
    assert same(y, forward_reference(w, index, 1.5))
    check(dw, gradient_reference(dy, index, V, 1.5, dy.dtype))
    for buf, view in ((ybuf, y), (dbuf, dw)):
        view.zero_()
        assert int(torch.isnan(buf).sum()) == buf.numel() - view.numel()


def test_ignore_index_inside_the_table():
    w, index, dy = case(400, 60, 64, "f32", 3)
    index = index.clamp(min=0)
    say("ignored entry of the table")
    y = mg.embedding(w, index, ignore_index=0)
    dw = mg.embedding_backward(dy, index, 60, ignore_index=0)
    torch.cuda.synchronize()
    assert (index == 0).any() and not dw[0].any()
    assert same(y, forward_reference(w, index, 1.0, ignore=0))
    check(dw, gradient_reference(dy, index, 60, 1.0, torch.float32, ignore=0))


def test_gradient_rows_without_an_entry_may_hold_anything():
    w, index, dy = case(500, 90, 72, "f16", 6, "bad")
    inside = (index >= 0) & (index < 90)
    dy[~inside] = float("nan")
    say("rows without an entry")
    dw = mg.embedding_backward(dy, index, 90)
    torch.cuda.synchronize()
    check(dw, gradient_reference(torch.where(inside[:, None], dy, 0.0), index, 90, 1.0, dy.dtype))
    # an infinity shows in its own entry alone
    at = int(inside.nonzero()[0])
    dy[at, 3] = float("inf")
    dw = mg.embedding_backward(dy, index, 90)
    torch.cuda.synchronize()
    bad = ~torch.isfinite(dw)
    assert bad[index[at], 3] and int(bad.sum()) == 1


def test_no_tokens():
    w, index, dy = case(0, 70, 33, "bf16", 1)
    y = mg.embedding(w, index)
    dw = mg.embedding_backward(dy, index, 70)
    kept = mg.embedding_backward(dy, index, 70, dw=w.clone(), accumulate=True)
    torch.cuda.synchronize()
    assert y.shape == (0, 33) and dw.shape == (70, 33) and not dw.any() and torch.equal(kept, w)


def test_gradient_against_differences():
    """The loss sum(y dy) is linear in the table: its differences are the gradient."""
    w, index, dy = case(60, 20, 5, "f32", 2)
    dw = mg.embedding_backward(dy, index, 20, scale=2.0)
    base = (mg.embedding(w, index, scale=2.0).double() * dy.double()).sum()
    for v in range(20):
        for k in range(0, 5, 2):
            moved = w.clone()
            moved[v, k] += 0.5
            diff = ((mg.embedding(moved, index, scale=2.0).double() * dy.double()).sum() - base) / 0.5
            assert abs(float(diff) - float(dw[v, k])) <= 1e-4 * (1 + abs(float(diff)))


def test_refusals():
    w, index, dy = case(20, 30, 16, "bf16", 1)
    for call in (lambda: mg.embedding(w, index.int()), lambda: mg.embedding(w, index[None]),
                 lambda: mg.embedding(w, index[::2]), lambda: mg.embedding(w.t(), index),
                 lambda: mg.embedding(w, index.cpu()), lambda: mg.embedding(w.double(), index),
                 lambda: mg.embedding(w, index, out=dy.float()),
                 lambda: mg.embedding(w, index, out=dy[:3]),
                 lambda: mg.embedding_backward(dy, index, 30, accumulate=True),
                 lambda: mg.embedding_backward(dy, index[:-1], 30),
                 lambda: mg.embedding_backward(dy, index, 30, dw=w[:-1]),
                 lambda: mg.embedding_backward(dy, index, 30, dw=w.half()),
                 lambda: mg.embedding_backward(dy, index, 30, out_dtype=torch.float16),
                 lambda: mg.embedding_backward(dy, index, 30, dw=w, out_dtype=torch.float32)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(mg.MigemmError):
        mg.embedding(w.int(), index)
    with pytest.raises(mg.MigemmError):
        mg.embedding(w, index[:20], out=w[:20])
    with pytest.raises(mg.MigemmError):
        mg.embedding_backward(dy, index, 0, dw=w[:0])


def test_repeatable_side_stream_and_graph_replay():
    w, index, dy = case(3000, 900, 264, "bf16", 5)
    w2, index2, dy2 = case(40000, 3000, 40, "f32", 6)
    say("embedding repeated")

    def run():
        return (mg.embedding(w, index, scale=2.0), mg.embedding_backward(dy, index, 900, scale=2.0),
                mg.embedding_backward(dy2, index2, 3000))

    eager = run()
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(run(), eager))
    side = torch.cuda.Stream()
    say("embedding on a side stream by handle")
    s = side.cuda_stream
    got = (mg.embedding(w, index, scale=2.0, stream=s),
           mg.embedding_backward(dy, index, 900, scale=2.0, stream=s),
           mg.embedding_backward(dy2, index2, 3000, stream=s))
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, eager))
    torch.cuda.synchronize()
    say("embedding in a graph")
    g = torch.cuda.CUDAGraph()
    added = torch.zeros(900, 264, device="cuda")
    with torch.cuda.graph(g):
        held = run()
        mg.embedding_backward(dy, index, 900, scale=2.0, dw=added, accumulate=True)
    added.zero_()
    once = mg.embedding_backward(dy, index, 900, scale=2.0, out_dtype=torch.float32)
    for i in range(3):
        if i:  # other tokens in the same place
            index.copy_(index.roll(17))
            index2.copy_(index2.flip(0))
        eager = run()
        for t in held:
            t.fill_(float("nan"))
        before = added.clone()
        more = mg.embedding_backward(dy, index, 900, scale=2.0, dw=before, accumulate=True)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, eager))
        assert torch.equal(added, more)
        if i == 0:
            assert torch.equal(added, once)


@pytest.mark.parametrize("T,V,D,dtype", [(40000, 900, 2001, "f32"), (3000, 40000, 2001, "f32"),
                                         (70000, 3000, 2003, "bf16")])
def test_rows_past_the_caches(T, V, D, dtype):
    """From 256 MiB of dy and of rows to zero, which lie off 16-byte boundaries."""
    both(T, V, D, dtype, T)


@pytest.mark.parametrize("run", [15, 16, 17, 32, 33, 47, 48, 49, 64, 65, 200])
@pytest.mark.parametrize("T", [5000, 40000])
def test_entries_over_several_stretches(T, run):
    """Entries of `run` tokens each, so that they begin and end everywhere in the stretches
    of 16 and 32 pairs, and one more of the rest."""
    V, D = 4000, 24
    g = torch.Generator(device="cuda").manual_seed(run)
    index = (torch.arange(T, device="cuda") // run).clamp(max=V - 1)
    index = index[torch.randperm(T, generator=g, device="cuda")]
    dy = torch.randn(T, D, generator=g, device="cuda")
    say(f"{T} tokens, {run} to an entry")
    dw = mg.embedding_backward(dy, index, V)
    wide = mg.embedding_backward(dy.repeat(1, 12), index, V)
    torch.cuda.synchronize()
    want = gradient_reference(dy, index, V, 1.0, torch.float32)
    check(dw, want)
    # a wavefront to a segment of columns sums in the same order
    assert torch.equal(wide, dw.repeat(1, 12))


def test_more_than_2_31_elements():
    V, D, T = (1 << 31) // 2048 + 300, 2048, 1500
    g = torch.Generator(device="cuda").manual_seed(3)
    w = torch.empty(V, D, dtype=torch.bfloat16, device="cuda")
    for v in range(0, V, 1 << 17):
        w[v:v + (1 << 17)] = torch.randn(min(1 << 17, V - v), D, generator=g, device="cuda")
    index = torch.randint(0, V, (T,), generator=g, device="cuda")
    index[:5] = torch.tensor([0, V - 1, (1 << 31) // D, (1 << 31) // D - 1, V - 1])
    dy = torch.randn(T, D, generator=g, device="cuda").bfloat16()
    say(f"embedding {T} of {V}x{D}")
    y = mg.embedding(w, index)
    dw = mg.embedding_backward(dy, index, V)
    torch.cuda.synchronize()
    assert torch.equal(y, w[index])
    rows, where = torch.unique(index, return_inverse=True)
    check(dw[rows], gradient_reference(dy, where, len(rows), 1.0, dy.dtype))
    dw[rows] = 0
    assert not dw.any()
    # rows of the tokens past 2^31 elements
    del dw, w
    T, V = (1 << 31) // 2048 + 300, 40
    dy = torch.zeros(T, D, dtype=torch.bfloat16, device="cuda")
    index = torch.randint(0, V, (T,), generator=g, device="cuda")
    some = torch.tensor([0, 5, (1 << 31) // D - 1, (1 << 31) // D, T - 1], device="cuda")
    dy[some] = torch.randn(5, D, generator=g, device="cuda").bfloat16()
    small = torch.randn(V, D, generator=g, device="cuda").bfloat16()
    say(f"embedding {T} of {V}x{D}")
    y = mg.embedding(small, index)
    dw = mg.embedding_backward(dy, index, V)
    torch.cuda.synchronize()
    assert torch.equal(y[some], small[index[some]]) and torch.equal(y[::9973], small[index[::9973]])
    check(dw, gradient_reference(dy[some], index[some], V, 1.0, dy.dtype))


def test_out_of_memory_is_torchs_error():
    """An output that no allocation can hold (64 TiB) raises what torch's allocator raises; the
    next call runs."""
    w = torch.ones(1, 1 << 20, dtype=torch.float32, device="cuda")
    index = torch.zeros(1 << 24, dtype=torch.int64, device="cuda")
    with pytest.raises(torch.OutOfMemoryError):
        mg.embedding(w, index)
    assert torch.equal(mg.embedding(w, index[:1]), w)


# lists of one launch (up to 2048 tokens; a lane holds one, two, four or eight of them), and
# the shapes of SIZES in lists that are sorted
@pytest.mark.parametrize("kind", ["mixed", "one", "ignored", "bad"])
@pytest.mark.parametrize("T,V,D", [(15, 3, 9), (16, 2, 600), (17, 2, 600), (70, 1, 2056),
                                   (255, 40, 65), (256, 9, 4104), (257, 300, 24), (511, 70, 3),
                                   (512, 4000, 136), (513, 65, 1029), (1000, 7, 2500),
                                   (1024, 16, 264), (1024, 129, 1), (1025, 16, 264)])
def test_lists_of_one_launch(T, V, D, kind):
    both(T, V, D, "f32" if D % 2 else "bf16", T + D, kind)
    both(T, V, D, "f16", T + D, kind)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,V,D", [(1025, 1, 1), (1100, 1000, 64), (1200, 5, 3), (1031, 300, 8),
                                   (2000, 300, 40), (1500, 511, 129), (1027, 512, 520),
                                   (1040, 131072, 4096), (1100, 2000, 8200)])
def test_short_sorted_lists(T, V, D, dtype):
    both(T, V, D, dtype, T + V + D)


@pytest.mark.parametrize("T", [90, 700, 2500])
def test_strided_and_misaligned_lists(T):
    """Rows off 16-byte boundaries, with NaN between them, which no sum takes in and no store
    meets."""
    V, D = 130, 531
    for dtype in ("f32", "f16", "bf16"):
        w, index, dy = case(T, V, D, dtype, T)
        index[T // 2:] = torch.where(index[T // 2:] >= 0, 5, index[T // 2:])
        big = torch.full((T, D + 6), float("nan"), dtype=dy.dtype, device="cuda")
        big[:, 3:3 + D] = dy
        for accumulate in (False, True):
            out = torch.full((V, D + 9), float("nan"), dtype=dy.dtype, device="cuda")
            out[:, 1:1 + D] = w
            say(f"embedding {T} strided {dtype} {accumulate}")
            mg.embedding_backward(big[:, 3:3 + D], index, V, scale=0.75, dw=out[:, 1:1 + D],
                                  accumulate=accumulate)
            torch.cuda.synchronize()
            check(out[:, 1:1 + D], gradient_reference(dy, index, V, 0.75, dy.dtype,
                                                      w if accumulate else None))
            assert torch.isnan(out[:, 0]).all() and torch.isnan(out[:, 1 + D:]).all()


@pytest.mark.parametrize("V", [(1 << 18) - 1, 1 << 18, (1 << 27) - 1, (1 << 27) + 3])
def test_sorted_lists_of_long_tables(V):
    """Entries of two, three and four digits."""
    T, D = 9000, 2
    g = torch.Generator(device="cuda").manual_seed(V)
    index = torch.randint(0, V, (T,), generator=g, device="cuda")
    index[:4] = torch.tensor([V - 1, 0, V // 2, V - 1])
    dy = torch.randn(T, D, generator=g, device="cuda")
    say(f"{T} of a table of {V}")
    for n in (1500, T):  # by counting, by digits
        dw = mg.embedding_backward(dy[:n], index[:n], V)
        torch.cuda.synchronize()
        rows, where = torch.unique(index[:n], return_inverse=True)
        check(dw[rows], gradient_reference(dy[:n], where, len(rows), 1.0, torch.float32))
        dw[rows] = 0
        assert not dw.any()


@pytest.mark.parametrize("T", [40, 800])
def test_one_launch_repeated_and_captured(T):
    w, index, dy = case(T, 90, 1300, "bf16", T)
    index[::3] = 7
    say(f"embedding of {T} captured")
    want = mg.embedding_backward(dy, index, 90, scale=2.0)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = mg.embedding_backward(dy, index, 90, scale=2.0, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(got, want)
    g = torch.cuda.CUDAGraph()
    added = w.clone()
    with torch.cuda.graph(g):
        held = mg.embedding_backward(dy, index, 90, scale=2.0)
        mg.embedding_backward(dy, index, 90, scale=2.0, dw=added, accumulate=True)
    more = w.clone()
    for i in range(3):
        index.copy_(index.roll(i))
        held.fill_(float("nan"))
        added.copy_(more)
        want = mg.embedding_backward(dy, index, 90, scale=2.0)
        mg.embedding_backward(dy, index, 90, scale=2.0, dw=more, accumulate=True)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(held, want) and torch.equal(added, more)


def test_gradient_rows_of_short_sorted_lists_may_hold_anything():
    w, index, dy = case(1500, 90, 72, "f16", 6, "bad")
    inside = (index >= 0) & (index < 90)
    dy[~inside] = float("nan")
    say("rows without an entry, sorted")
    dw = mg.embedding_backward(dy, index, 90)
    torch.cuda.synchronize()
    check(dw, gradient_reference(torch.where(inside[:, None], dy, 0.0), index, 90, 1.0, dy.dtype))


# either side of 2048 tokens, and of 4096 workgroups of 2048 columns
@pytest.mark.parametrize("kind", ["mixed", "one", "bad"])
@pytest.mark.parametrize("T,V,D", [(1500, 70, 33), (2047, 300, 72), (2048, 5, 520), (2048, 900, 4096),
                                   (2049, 300, 72), (1365, 40, 6144), (1366, 40, 6144),
                                   (33, 17, 251903), (2, 3, 1 << 21), (3, 2, (1 << 21) - 5)])
def test_lists_and_rows_of_one_launch(T, V, D, kind):
    both(T, V, D, "f32" if D % 2 else "f16", T + D, kind)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,V,D", [(2049, 1, 1), (2100, 1000, 64), (2200, 5, 3), (2050, 300, 8),
                                   (3000, 300, 40), (2500, 511, 129), (2051, 512, 520),
                                   (2060, 20000, 4096), (1100, 2000, 8200), (2100, 2000, 8200)])
def test_sorted_lists(T, V, D, dtype):
    both(T, V, D, dtype, T + V + D)
    if D < 1000:
        both(T, V, D, dtype, T + V + D, "one")


def test_gradient_rows_of_sorted_lists_may_hold_anything():
    w, index, dy = case(2500, 90, 72, "f16", 6, "bad")
    inside = (index >= 0) & (index < 90)
    dy[~inside] = float("nan")
    say("rows without an entry, sorted")
    dw = mg.embedding_backward(dy, index, 90)
    torch.cuda.synchronize()
    check(dw, gradient_reference(torch.where(inside[:, None], dy, 0.0), index, 90, 1.0, dy.dtype))
    at = int(inside.nonzero()[0])
    dy[at, 3] = float("-inf")
    dw = mg.embedding_backward(dy, index, 90)
    torch.cuda.synchronize()
    bad = ~torch.isfinite(dw)
    assert bad[index[at], 3] and int(bad.sum()) == 1


# one stretch of 8 pairs: so few tokens that there is one, of rows so wide (FP32: a workgroup to
# 1024 columns) that their lists are sorted; and two stretches
@pytest.mark.parametrize("kind", ["mixed", "one", "bad"])
@pytest.mark.parametrize("T,D", [(8, (1 << 20) + 1), (7, 1198081), (6, 1396737), (5, 1677313),
                                 (5, 1 << 21), (8, 1 << 21), (9, (1 << 20) + 1), (4, 1 << 21)])
def test_lists_of_one_stretch(T, D, kind):
    both(T, 3, D, "f32" if D % 2 else "bf16", T, kind)


def whole_case(T, V, D, kind, seed):
    """Gradients of -1, 0 and 1: as long as their magnitudes add up to less than 2^24, FP32
    sums of them are exact in any order, and so a stretch that is left out, added twice or
    joined to another entry shows, however many tokens an entry has."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    if kind == "middle":  # entries of a few tokens on both sides of one of 0.6 T
        index = torch.randint(0, V, (T,), generator=g, device="cuda")
        index = torch.where(torch.rand(T, generator=g, device="cuda") < 0.6, V // 2, index)
    else:
        index = draw_index(T, V, g, kind)
    u = torch.rand(T, D, generator=g, device="cuda")
    dy = (u < 3 / 8).float() - (u > 7 / 8).float()
    old = torch.randint(-100, 100, (V, D), generator=g, device="cuda").float()
    assert float(dy.abs().sum(0).max()) + 100 < 2 ** 24
    inside = ((index >= 0) & (index < V)).cpu()
    total = torch.zeros(V, D, dtype=torch.int64)
    total.index_add_(0, index.cpu()[inside], dy.cpu()[inside].long())
    return index, dy, old, total.cuda()


@pytest.mark.parametrize("kind", ["one", "mixed", "middle"])
@pytest.mark.parametrize("T,V,D", [(12, 3, (1 << 20) + 8), (900, 7, 520), (2048, 300, 72), (2049, 5, 24),
                                   (8192, 40, 40), (8193, 40, 260), (33000, 700, 64), (70000, 5, 264),
                                   (300000, 4000, 24), (1 << 20, 1000, 2), ((1 << 24) + 3, 70000, 1)])
def test_sums_of_whole_numbers_are_exact(T, V, D, kind):
    index, dy, old, total = whole_case(T, V, D, kind, T)
    say(f"whole gradients, {T} of {V}x{D} {kind}")
    dw = mg.embedding_backward(dy, index, V)
    half = mg.embedding_backward(dy.bfloat16(), index, V, scale=0.5, out_dtype=torch.float32)
    added = mg.embedding_backward(dy, index, V, scale=2.0, dw=old.clone(), accumulate=True)
    rounded = mg.embedding_backward(dy.bfloat16(), index, V)
    torch.cuda.synchronize()
    assert torch.equal(dw, total.float()) and torch.equal(half, total.float() * 0.5)
    # (twice a sum and what was there: below 2^25, and a product and a sum of one rounding)
    assert torch.equal(added, (2 * total.double() + old.double()).float())
    assert torch.equal(rounded, total.float().bfloat16())


# lists that are sorted by counting (2049 to 8192 tokens; shorter ones take one launch without
# a sort), and the first one past them
@pytest.mark.parametrize("T", [2100, 8192, 8193])
@pytest.mark.parametrize("V", [(1 << 18) - 1, 1 << 18, (1 << 25) - 1, (1 << 25) + 5, (1 << 27) + 3])
def test_counted_lists_of_long_tables(T, V):
    D = 2
    g = torch.Generator(device="cuda").manual_seed(V)
    index = torch.randint(0, V, (T,), generator=g, device="cuda")
    index[:4] = torch.tensor([V - 1, 0, V // 2, V - 1])
    index[100:150] = V - 2
    dy = torch.randint(-4, 5, (T, D), generator=g, device="cuda").float()
    say(f"{T} of a table of {V}")
    dw = mg.embedding_backward(dy, index, V)
    torch.cuda.synchronize()
    rows, where = torch.unique(index, return_inverse=True)
    total = torch.zeros(len(rows), D, dtype=torch.int64).index_add_(0, where.cpu(), dy.cpu().long())
    assert torch.equal(dw[rows].cpu(), total.float())
    dw[rows] = 0
    assert not dw.any()
