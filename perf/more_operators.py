"""The measured cases of three operators around an output layer's losses: layer
norm, whose result the layer multiplies; the lookup in a table of embeddings, in
tied models the layer's own weight; and the AdamW step that takes the gradients.

``listed()`` gives the cases, ``draw(rng)`` further ones of the same ranges,
``prepare(case, seed)`` the inputs on the GPU, ``run(state)`` one pass,
``work(case)`` the bytes and operations a pass cannot do without, and
``exact(case, seed)`` the outputs from the definitions in 64 bits.  Where
``own`` is false, ``run`` computes the operators with elementary torch
operations in 32 bits; where it is true, with this repository's kernels.

8-bit AdamW states: the first moment and the root of the second are E4M3 codes
(``float8_e4m3fn``), each block of 256 consecutive elements with one float32 scale,
its largest magnitude / 448.  A positive root never becomes code 0.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
IGNORE = -100
EPS = 1e-5
BLOCK = 256
E4M3_MAX = 448.0
E4M3_MIN = 2.0 ** -9
ADAM = {"lr": 1e-3, "betas": (0.9, 0.999), "eps": 1e-8, "weight_decay": 0.1}
STEP = 100


def _norm(name, rows, cols, dtype, weight, backward=True):
    return {"name": name, "op": "norm", "rows": rows, "cols": cols, "dtype": dtype,
            "weight": weight, "backward": backward}


def _embed(name, tokens, vocab, dim, dtype, grad, into=""):
    """grad: "" (forward only), "dense" (a gradient of its own) or "add" (added to
    one that is there); into: the gradient's type."""
    return {"name": name, "op": "embed", "tokens": tokens, "vocab": vocab, "dim": dim,
            "dtype": dtype, "grad": grad, "into": into or dtype}


def _adamw(name, layers, width, vocab, param, grad, bits, master):
    return {"name": name, "op": "adamw", "layers": layers, "width": width, "vocab": vocab,
            "param": param, "grad": grad, "bits": bits, "master": master}


def listed():
    return [
        # one token of a decoding step: latency alone
        _norm("norm-1x4096-bf16", 1, 4096, "bf16", "bf16", False),
        # fine-tuning on one ragged batch, odd sizes
        _norm("norm-1003x1032-f16", 1003, 1032, "f16", "f16"),
        # a small model in full precision, rows off 16-byte boundaries
        _norm("norm-8191x771-f32", 8191, 771, "f32", "f32"),
        # pre-training: the tokens of one GPU, weights kept in 32 bits
        _norm("norm-16384x8192-bf16", 16384, 8192, "bf16", "f32"),
        # the activations of sixteen sequences at one decoding step
        _embed("embed-16x131072x4096-bf16", 16, 131072, 4096, "bf16", ""),
        # fine-tuning on one ragged batch, the gradient of a separate table
        _embed("embed-1003x30001x1032-f16", 1003, 30001, 1032, "f16", "dense"),
        # pre-training with a tied table: added to what the output layer's loss left
        _embed("embed-32768x131072x4096-bf16", 32768, 131072, 4096, "bf16", "add"),
        # many short sequences, full precision
        _embed("embed-65536x50001x2048-f32", 65536, 50001, 2048, "f32", "dense"),
        # a test-sized model: many small tensors
        _adamw("adamw-1x64-f32", 1, 64, 1000, "f32", "f32", 32, False),
        # mixed precision with master copies, some hundred tensors
        _adamw("adamw-8x1024-bf16-master", 8, 1024, 32000, "bf16", "bf16", 32, True),
        # odd sizes, 8-bit states, gradients accumulated in 32 bits
        _adamw("adamw-4x771-f16-8bit", 4, 771, 5001, "f16", "f32", 8, False),
        # the largest tensor of a large model with 8-bit states
        _adamw("adamw-1x4096-bf16-8bit", 1, 4096, 131072, "bf16", "bf16", 8, False),
    ]


def _log_uniform(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _width(rng, low, high):
    """A row length: mostly a multiple of 64 or of 8, sometimes any number."""
    step = rng.choice((64, 64, 8, 8, 1))
    return max(step, _log_uniform(rng, low, high) // step * step)


def draw(rng):
    op = rng.choice(("norm", "embed", "adamw"))
    dtype = rng.choice(("f32", "f16", "bf16", "bf16"))
    if op == "norm":
        cols = _width(rng, 64, 16384)
        rows = _log_uniform(rng, 1, min(65536, (1 << 26) // cols))
        weight = rng.choice((dtype, "f32"))
        case = _norm("", rows, cols, dtype, weight, rng.random() < 0.75)
    elif op == "embed":
        dim = _width(rng, 64, 4096)
        tokens = _log_uniform(rng, 1, min(65536, (1 << 27) // dim))
        vocab = _log_uniform(rng, 500, min(131072, (1 << 28) // dim))
        case = _embed("", tokens, vocab, dim, dtype, rng.choice(("", "dense", "add")),
                      rng.choice((dtype, "f32")))
    else:
        width = _width(rng, 64, 2048)
        layers, vocab = rng.randint(0, 8), _log_uniform(rng, 500, 65536)
        bits = rng.choice((32, 8))
        master = dtype != "f32" and rng.random() < 0.5
        case = _adamw("", layers, width, vocab, dtype, rng.choice((dtype, "f32")), bits, master)
    del case["name"]
    return case


def _tensor_sizes(case):
    """Elements of each tensor of a model with a tied table and `layers` layers."""
    w = case["width"]
    layer = [w, w, 3 * w * w, 3 * w, w * w, w, w, w, 4 * w * w, 4 * w, 4 * w * w, w]
    return [case["vocab"] * w] + layer * case["layers"] + [w, w]


# ------------------------------------------------------------------- inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def prepare(case, seed):
    g = _generator(seed)
    return {"case": case, **_PREPARE[case["op"]](case, g)}


def _prepare_norm(case, g):
    # a residual stream: rows of differing size and offset, a few large columns
    rows, cols, dt = case["rows"], case["cols"], DTYPES[case["dtype"]]
    x = _randn(g, rows, cols) * torch.exp(0.5 * _randn(g, rows, 1))
    x *= 1.0 + 10.0 * (torch.rand(cols, generator=g, device="cuda") < 0.005)
    x += 0.5 * _randn(g, rows, 1)
    weight = (1.0 + 0.2 * _randn(g, cols)).to(DTYPES[case["weight"]])
    bias = (0.2 * _randn(g, cols)).to(DTYPES[case["weight"]])
    state = {"x": x.to(dt), "weight": weight, "bias": bias}
    if case["backward"]:
        state["dy"] = (0.1 * _randn(g, rows, cols)).to(dt)
    return state


def _prepare_embed(case, g):
    tokens, vocab, dim, dt = case["tokens"], case["vocab"], case["dim"], DTYPES[case["dtype"]]
    # the k-th most frequent entry about 1 / k times as often as the first; spread over the table
    u = torch.rand(tokens, generator=g, device="cuda", dtype=torch.float64)
    rank = (torch.exp(u * math.log(vocab + 1)).long() - 1).clamp_(0, vocab - 1)
    index = (rank * 7919 + 13) % vocab
    # a tenth of the tokens are padding
    index = torch.where(torch.rand(tokens, generator=g, device="cuda") < 0.1, IGNORE, index)
    index[-1] = vocab - 1
    state = {"w": (0.02 * _randn(g, vocab, dim)).to(dt), "index": index, "scale": math.sqrt(dim)}
    if case["grad"]:
        state["dy"] = (0.1 * _randn(g, tokens, dim) / math.sqrt(dim)).to(dt)
    if case["grad"] == "add":
        state["dw"] = (0.02 * _randn(g, vocab, dim)).to(DTYPES[case["into"]])
    return state


def _codes(x, scale):
    """E4M3 codes of `x` (whole blocks) under one scale per block."""
    inverse = torch.where(scale > 0, 1.0 / scale, 0.0)
    return (x * inverse.unsqueeze(1)).to(torch.float8_e4m3fn)


def _block_scale(x):
    """largest magnitude / 448 per block, 0 where it is below 2^-100."""
    largest = x.abs().amax(1)
    return torch.where(largest >= 2.0 ** -100, largest * (1.0 / E4M3_MAX), 0.0)


def _root_codes(r, scale):
    """As _codes for roots: a positive one is at least the smallest code."""
    q = _codes(r, scale).float()
    least = (q == 0) & (r > 0) & (scale > 0).unsqueeze(1)
    return torch.where(least, E4M3_MIN, q).to(torch.float8_e4m3fn)


def _prepare_adamw(case, g):
    # every tensor starts at a whole block of one buffer; zeros fill the gaps
    sizes = _tensor_sizes(case)
    starts, total = [], 0
    for n in sizes:
        starts.append(total)
        total += (n + BLOCK - 1) // BLOCK * BLOCK
    held = torch.zeros(total // BLOCK, BLOCK, device="cuda")
    flat = held.view(-1)
    for at, n in zip(starts, sizes):
        flat[at:at + n] = 1.0
    # steps of differing size over the tensors; entries of the table that no token named have none
    size = torch.exp(_randn(g, total // BLOCK, 1)) * 1e-3
    size = torch.where(torch.rand(total // BLOCK, 1, generator=g, device="cuda") < 0.1, 0.0, size)
    grad = _randn(g, total // BLOCK, BLOCK).mul_(size).mul_(held)
    m = _randn(g, total // BLOCK, BLOCK).mul_(0.3 * size).mul_(held)
    root = _randn(g, total // BLOCK, BLOCK).abs_().add_(0.1).mul_(size).mul_(held)
    param = _randn(g, total // BLOCK, BLOCK).mul_(0.02).mul_(held)
    state = {"param": param.to(DTYPES[case["param"]]).view(-1),
             "grad": grad.to(DTYPES[case["grad"]]).view(-1)}
    if case["master"]:
        state["master"] = param.view(-1)
    if case["bits"] == 8:
        ms, rs = _block_scale(m), _block_scale(root)
        state |= {"avg": _codes(m, ms).view(-1), "avg_scales": ms,
                  "sq": _root_codes(root, rs).view(-1), "sq_scales": rs}
    else:
        state |= {"avg": m.view(-1), "sq": root.square_().view(-1)}
    # the tensors themselves, as the model holds them
    held = {k: [v[at // BLOCK:(at + n + BLOCK - 1) // BLOCK] if k.endswith("scales")
                else v[at:at + n] for at, n in zip(starts, sizes)] for k, v in state.items()}
    return {"flat": state, "tensors": held}


_PREPARE = {"norm": _prepare_norm, "embed": _prepare_embed, "adamw": _prepare_adamw}


# ------------------------------------------------------------------ one pass

def run(state):
    return _RUN[state["case"]["op"]](state)


def _run_norm(s):
    x, weight, bias = s["x"], s["weight"], s["bias"]
    backward = s["case"]["backward"]
    if own:
        import dense_gemm_16_amd as mg
        y, mean, rstd = mg.layer_norm(x, weight, bias, eps=EPS, stats=backward)
        if not backward:
            return {"y": y}
        dx, dw, db = mg.layer_norm_backward(s["dy"], x, weight, mean, rstd)
        return {"y": y, "mean": mean, "rstd": rstd, "dx": dx, "dw": dw, "db": db}
    xf, wf = x.float(), weight.float()
    mean = xf.mean(1, keepdim=True)
    d = xf - mean
    rstd = 1.0 / torch.sqrt((d * d).mean(1, keepdim=True) + EPS)
    h = d * rstd
    y = (h * wf + bias.float()).to(x.dtype)
    if not backward:
        return {"y": y}
    dy = s["dy"].float()
    g = dy * wf
    gh = g * h
    dx = rstd * (g - g.mean(1, keepdim=True) - h * gh.mean(1, keepdim=True))
    return {"y": y, "mean": mean[:, 0], "rstd": rstd[:, 0], "dx": dx.to(x.dtype),
            "dw": (dy * h).sum(0).to(weight.dtype), "db": dy.sum(0).to(weight.dtype)}


def _run_embed(s):
    case, w, index, scale = s["case"], s["w"], s["index"], s["scale"]
    if own:
        import dense_gemm_16_amd as mg
        y = mg.embedding(w, index, scale=scale, ignore_index=IGNORE)
        if not case["grad"]:
            return {"y": y}
        dw = mg.embedding_backward(s["dy"], index, case["vocab"], scale=scale, ignore_index=IGNORE,
                                   dw=s.get("dw"), accumulate=case["grad"] == "add",
                                   out_dtype=DTYPES[case["into"]])
        return {"y": y, "dw": dw}
    held = (index != IGNORE).unsqueeze(1)
    at = index.clamp(min=0)
    y = torch.where(held, w[at].float() * scale, 0.0).to(w.dtype)
    if not case["grad"]:
        return {"y": y}
    rows = torch.where(held, s["dy"].float() * scale, 0.0)
    if case["grad"] == "add" and case["into"] == "f32":
        return {"y": y, "dw": s["dw"].index_add_(0, at, rows)}
    dw = torch.zeros((case["vocab"], case["dim"]), device="cuda").index_add_(0, at, rows)
    if case["grad"] == "add":
        return {"y": y, "dw": s["dw"].copy_(dw.add_(s["dw"]))}
    return {"y": y, "dw": dw.to(DTYPES[case["into"]])}


def _run_adamw(s):
    case, f = s["case"], s["flat"]
    if own:
        import dense_gemm_16_amd as mg
        t = s["tensors"]
        none = [None] * len(t["param"])
        states = list(map(mg.AdamState, t["avg"], t["sq"], t.get("avg_scales", none),
                          t.get("sq_scales", none), t.get("master", none)))
        mg.adamw_(t["param"], t["grad"], states, step=STEP, **ADAM)
        return _without_grad(f)
    # every operation goes by the element or by the block, so all tensors are taken as one
    b1, b2 = ADAM["betas"]
    lr = ADAM["lr"]
    g = f["grad"].float()
    eight = case["bits"] == 8
    if eight:
        m = (f["avg"].float().view(-1, BLOCK) * f["avg_scales"].unsqueeze(1)).view(-1)
        r = (f["sq"].float().view(-1, BLOCK) * f["sq_scales"].unsqueeze(1)).view(-1)
        v = r * r
    else:
        m, v = f["avg"], f["sq"]
    m = m * b1 + g * (1 - b1)
    v = v * b2 + (g * g) * (1 - b2)
    r = torch.sqrt(v)
    p = f["master"] if case["master"] else f["param"].float()
    p = p * (1 - lr * ADAM["weight_decay"]) - (m / (r * (1 / math.sqrt(1 - b2 ** STEP))
                                                    + ADAM["eps"])) * (lr / (1 - b1 ** STEP))
    if case["master"]:
        f["master"].copy_(p)
    f["param"].copy_(p)
    if eight:
        m, r = m.view(-1, BLOCK), r.view(-1, BLOCK)
        f["avg_scales"].copy_(_block_scale(m))
        f["sq_scales"].copy_(_block_scale(r))
        f["avg"].copy_(_codes(m, f["avg_scales"]).view(-1))
        f["sq"].copy_(_root_codes(r, f["sq_scales"]).view(-1))
    else:
        f["avg"].copy_(m)
        f["sq"].copy_(v)
    return _without_grad(f)


def _without_grad(flat):
    return {k: v for k, v in flat.items() if k != "grad"}


_RUN = {"norm": _run_norm, "embed": _run_embed, "adamw": _run_adamw}


# ---------------------------------------------------------------- its work

def _distinct(case):
    """The expected number of table rows that the tokens name."""
    v = case["vocab"]
    k = torch.arange(1, v + 1, dtype=torch.float64)
    share = torch.log((k + 1) / k) / math.log(v + 1)
    return float((1 - torch.exp(0.9 * case["tokens"] * torch.log1p(-share))).sum())


def work(case):
    if case["op"] == "norm":
        n, b = case["rows"] * case["cols"], SIZE[case["dtype"]]
        vectors = case["cols"] * SIZE[case["weight"]]
        if not case["backward"]:
            return {"bytes": 2 * n * b + 2 * vectors, "flops": 8 * n}
        # x and dy read, y and dx written
        return {"bytes": 4 * n * b + 4 * vectors + 8 * case["rows"], "flops": 22 * n}
    if case["op"] == "embed":
        t, d, b, into = case["tokens"], case["dim"], SIZE[case["dtype"]], SIZE[case["into"]]
        rows = _distinct(case)
        total = 8 * t + (rows + t) * d * b
        if case["grad"] == "dense":
            total += t * d * b + case["vocab"] * d * into
        elif case["grad"] == "add":
            total += t * d * b + 2 * rows * d * into
        return {"bytes": total, "flops": t * d * (3 if case["grad"] else 1)}
    n = sum(_tensor_sizes(case))
    param, grad = SIZE[case["param"]], SIZE[case["grad"]]
    each = grad + (param + 8 if case["master"] else 2 * param)
    each += 16 if case["bits"] == 32 else 4 + 16 / BLOCK
    return {"bytes": int(n * each), "flops": 16 * n}


# ------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    return _EXACT[case["op"]](case, prepare(case, seed))


def _exact_norm(case, s):
    x = s["x"].double()
    var, mean = torch.var_mean(x, 1, unbiased=False, keepdim=True)
    rstd = (var + EPS).rsqrt()
    h = (x - mean) * rstd
    y = torch.addcmul(s["bias"].double(), h, s["weight"].double())
    if not case["backward"]:
        return {"y": y}
    dy = s["dy"].double()
    g = dy * s["weight"].double()
    c = case["cols"]
    along = (g * h).sum(1, keepdim=True) / c
    return {"y": y, "mean": mean[:, 0], "rstd": rstd[:, 0],
            "dx": (g - g.sum(1, keepdim=True) / c - along * h) * rstd,
            "dw": torch.einsum("td,td->d", dy, h), "db": dy.sum(0)}


def _exact_embed(case, s):
    w, index, dim = s["w"], s["index"], case["dim"]
    counted = index >= 0
    y = torch.zeros(case["tokens"], dim, device="cuda", dtype=torch.float64)
    y[counted] = w[index[counted]].double() * s["scale"]
    if not case["grad"]:
        return {"y": y}
    # the tokens of each entry side by side, summed between the borders of a running sum
    order = torch.argsort(torch.where(counted, index, case["vocab"]), stable=True)
    order = order[:int(counted.sum())]
    entries, count = torch.unique_consecutive(index[order], return_counts=True)
    end = count.cumsum(0)
    total = torch.zeros(case["vocab"], dim, device="cuda", dtype=torch.float64)
    for c in range(0, dim, 256):
        run_sum = s["dy"][order, c:c + 256].double().cumsum(0)[end - 1]
        run_sum[1:] -= run_sum[:-1].clone()
        total[entries, c:c + 256] = run_sum * s["scale"]
    if case["grad"] == "add":
        total += s["dw"].double()
    return {"y": y, "dw": total}


def _exact_adamw(case, s):
    f = s["flat"]
    b1, b2 = ADAM["betas"]
    g = f["grad"].double()
    m, v = f["avg"].double(), f["sq"].double()
    if case["bits"] == 8:
        m *= f["avg_scales"].double().repeat_interleave(BLOCK)
        v *= f["sq_scales"].double().repeat_interleave(BLOCK)
        v = v.square_()
    m += (1 - b1) * (g - m)
    v += (1 - b2) * (g.square_() - v)
    p = f["master" if case["master"] else "param"].double()
    p -= ADAM["lr"] * ADAM["weight_decay"] * p
    p -= ADAM["lr"] * (m / (1 - b1 ** STEP)) / ((v / (1 - b2 ** STEP)).sqrt_() + ADAM["eps"])
    out = {"param": p}
    if case["master"]:
        out["master"] = p
    if case["bits"] == 8:
        # codes next to a border have no one value
        return out | {"avg": None, "sq": None,
                      "avg_scales": m.abs_().view(-1, BLOCK).amax(1) / E4M3_MAX,
                      "sq_scales": v.sqrt_().view(-1, BLOCK).amax(1) / E4M3_MAX}
    return out | {"avg": m, "sq": v}


_EXACT = {"norm": _exact_norm, "embed": _exact_embed, "adamw": _exact_adamw}
