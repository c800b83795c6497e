"""The measured cases of four operators around a matrix product: microscaled
4-bit (MXFP4) quantisation, the product of two MXFP4 matrices, and the two
losses of a linear output layer that never keep its logits, softmax cross
entropy and distillation from a teacher's top logits, with their gradients.

``listed()`` gives the cases, ``draw(rng)`` further ones of the same ranges,
``prepare(case, seed)`` the inputs on the GPU, ``run(state)`` one pass,
``work(case)`` the bytes and operations a pass cannot do without, and
``exact(case, seed)`` the outputs from the definitions in 64 bits.  Where
``own`` is false, ``run`` computes the operators with elementary torch
operations in 32 bits; where it is true, with this repository's kernels.

MXFP4: a row is cut into blocks of 32 elements; each block has one scale byte e
(the value 2^(e - 127), 255 for NaN) and 32 four-bit elements (sign, two
exponent bits, one mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6), two to a byte, the
even element in the low half.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BLOCK = 32
FP4 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
IGNORE = -100


def _quantize(name, rows, cols, dtype, transposed):
    return {"name": name, "op": "quantize", "rows": rows, "cols": cols, "dtype": dtype,
            "transposed": transposed}


def _product(name, m, n, k, out):
    return {"name": name, "op": "product", "m": m, "n": n, "k": k, "out": out}


def _ce(name, tokens, vocab, dim, dtype, backward=True):
    return {"name": name, "op": "ce", "tokens": tokens, "vocab": vocab, "dim": dim,
            "dtype": dtype, "backward": backward}


def _kd(name, tokens, vocab, dim, dtype, top, temperature, backward=True):
    return {"name": name, "op": "kd", "tokens": tokens, "vocab": vocab, "dim": dim,
            "dtype": dtype, "top": top, "temperature": temperature, "backward": backward}


def listed():
    return [
        # the activations of sixteen sequences at one decoding step
        _quantize("quantize-16x4096-bf16", 16, 4096, "bf16", False),
        # a weight stored input-major (k as the row index), quantised along k when a model is loaded
        _quantize("quantize-8192x8192-f32-t", 8192, 8192, "f32", True),
        # one token through a square projection: the weight is read once, nothing is reused
        _product("product-1x8192x8192", 1, 8192, 8192, "bf16"),
        # a short ragged prompt; k ends inside a tile of k, n inside a tile of columns
        _product("product-300x5000x2080", 300, 5000, 2080, "f32"),
        # a long prompt or a batch of them
        _product("product-8192x8192x8192", 8192, 8192, 8192, "bf16"),
        # a test-sized model in full precision
        _ce("ce-64x1000x256-f32", 64, 1000, 256, "f32"),
        # scoring eight candidate tokens against a large vocabulary (no gradient)
        _ce("ce-score-8x131072x4096-bf16", 8, 131072, 4096, "bf16", False),
        # fine-tuning on one ragged batch, odd sizes, loss-scaled half precision
        _ce("ce-1003x30001x1032-f16", 1003, 30001, 1032, "f16"),
        # pre-training: one long sequence per GPU against a large vocabulary
        _ce("ce-8192x131072x4096-bf16", 8192, 131072, 4096, "bf16"),
        # a test-sized student
        _kd("kd-33x4099x520-f32", 33, 4099, 520, "f32", 8, 1.0),
        # a half-precision student, tokens of one batch
        _kd("kd-2048x32000x2048-f16", 2048, 32000, 2048, "f16", 32, 1.5),
        # a student of a large teacher
        _kd("kd-4096x65536x4096-bf16", 4096, 65536, 4096, "bf16", 64, 2.0),
    ]


def _log_uniform(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _width(rng, low, high):
    """A row length: mostly a multiple of 64 or of 8, sometimes any number."""
    step = rng.choice((64, 64, 8, 8, 1))
    return max(step, _log_uniform(rng, low, high) // step * step)


def draw(rng):
    op = rng.choice(("quantize", "product", "product", "ce", "ce", "kd", "kd"))
    if op == "quantize":
        return _without_name(_quantize("", _log_uniform(rng, 1, 8192), _width(rng, 32, 8192),
                                       rng.choice(("f32", "f16", "bf16")), rng.random() < 0.4))
    if op == "product":
        m = _log_uniform(rng, 1, 64) if rng.random() < 0.5 else _log_uniform(rng, 64, 8192)
        return _without_name(_product("", m, _log_uniform(rng, 64, 8192),
                                      BLOCK * _log_uniform(rng, 2, 256),
                                      rng.choice(("f32", "f16", "bf16"))))
    dtype = rng.choice(("f32", "f16", "bf16", "bf16"))
    wide = dtype != "f32"
    tokens = _log_uniform(rng, 1, 8192 if wide else 2048)
    vocab = _log_uniform(rng, 500, 131072 if wide else 32768)
    dim = _width(rng, 128, 4096 if wide else 2048)
    backward = rng.random() < 0.75
    if op == "ce":
        return _without_name(_ce("", tokens, vocab, dim, dtype, backward))
    return _without_name(_kd("", tokens, vocab, dim, dtype, _log_uniform(rng, 1, 64),
                             rng.choice((1.0, 1.5, 2.0, 4.0)), backward))


def _without_name(case):
    del case["name"]
    return case


# ------------------------------------------------------------------- inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def prepare(case, seed):
    g = _generator(seed)
    return {"case": case, **_PREPARE[case["op"]](case, g)}


def _prepare_quantize(case, g):
    # rows of differing size with a few large entries, as activations and weights have
    rows, cols = case["rows"], case["cols"]
    stored = (cols, rows) if case["transposed"] else (rows, cols)
    x = _randn(g, *stored)
    x *= torch.exp(0.5 * _randn(g, stored[0], 1))
    x *= 1.0 + 15.0 * (torch.rand(*stored, generator=g, device="cuda") < 0.005)
    x = x.to(DTYPES[case["dtype"]])
    return {"x": x.t() if case["transposed"] else x}


def _prepare_operand(g, rows, k):
    """Random elements and scales of a rows x k MXFP4 matrix: every four-bit
    code, scales of a few neighbouring powers of two, rows of scales padded to 16 bytes."""
    data = torch.randint(0, 256, (rows, k // 2), generator=g, device="cuda", dtype=torch.uint8)
    blocks = k // BLOCK
    scales = torch.zeros((rows, (blocks + 15) // 16 * 16), device="cuda", dtype=torch.uint8)
    scales[:, :blocks] = torch.randint(118, 124, (rows, blocks), generator=g, device="cuda",
                                       dtype=torch.uint8)
    return data, scales


def _prepare_product(case, g):
    return {"a": _prepare_operand(g, case["m"], case["k"]),
            "b": _prepare_operand(g, case["n"], case["k"])}


def _prepare_layer(case, g, towards):
    """The output layer's input and weight: logits of standard deviation 2, the
    logit of each row's `towards` raised as in a trained model."""
    dt = DTYPES[case["dtype"]]
    w = (_randn(g, case["vocab"], case["dim"]) * (2.0 / math.sqrt(case["dim"]))).to(dt)
    x = _randn(g, case["tokens"], case["dim"])
    x += 1.5 * w[towards].float()
    return x.to(dt), w


def _prepare_grad(case, g, counted):
    """The upstream gradient of each row's loss: the mean over the counted rows,
    times a loss scale in half precision."""
    scale = 16384.0 if case["dtype"] == "f16" else 1.0
    return counted.float() * (scale / max(1, int(counted.sum())))


def _prepare_ce(case, g):
    tokens = case["tokens"]
    target = torch.randint(0, case["vocab"], (tokens,), generator=g, device="cuda")
    x, w = _prepare_layer(case, g, target)
    # a tenth of the rows (prompt tokens) carry no loss, the last one always does
    prompt = torch.rand(tokens, generator=g, device="cuda") < 0.1
    prompt[-1] = False
    target = torch.where(prompt, IGNORE, target)
    return {"x": x, "w": w, "target": target, "grad": _prepare_grad(case, g, ~prompt)}


def _prepare_kd(case, g):
    tokens, vocab, top = case["tokens"], case["vocab"], case["top"]
    # distinct indices: one from each of `top` equal parts of the vocabulary, in random order
    part = torch.arange(top, device="cuda", dtype=torch.float64)
    u = torch.rand((tokens, top), generator=g, device="cuda", dtype=torch.float64)
    index = ((part + u) * (vocab / top)).long().clamp_(max=vocab - 1)
    order = torch.rand((tokens, top), generator=g, device="cuda").argsort(1)
    index = index.gather(1, order)
    x, w = _prepare_layer(case, g, index[:, 0])
    logits = (3.0 * _randn(g, tokens, top) + 10.0).sort(dim=1, descending=True).values
    # some rows hold fewer entries (index -1), a few none at all
    held = torch.randint(1, 4 * top + 1, (tokens, 1), generator=g, device="cuda")
    held = torch.where(torch.rand((tokens, 1), generator=g, device="cuda") < 0.05, 0, held)
    held[-1] = top
    absent = torch.arange(top, device="cuda") >= held
    index = torch.where(absent, -1, index)
    return {"x": x, "w": w, "logits": logits.contiguous(), "index": index.contiguous(),
            "grad": _prepare_grad(case, g, (held > 0)[:, 0])}


_PREPARE = {"quantize": _prepare_quantize, "product": _prepare_product, "ce": _prepare_ce,
            "kd": _prepare_kd}


# ------------------------------------------------------------------ one pass

def run(state):
    return _RUN[state["case"]["op"]](state)


def _table():
    """The two values that each byte of elements stands for."""
    half = torch.tensor(FP4 + tuple(-v for v in FP4), device="cuda")
    byte = torch.arange(256, device="cuda")
    return torch.stack((half[byte & 15], half[byte >> 4]), 1)


def _values(data, scales, k):
    """The float32 values of an MXFP4 matrix."""
    rows = data.shape[0]
    v = _table()[data.int()].view(rows, k // BLOCK, BLOCK)
    s = torch.exp2(scales[:, :k // BLOCK].double() - 127.0).float()
    return (v * s.unsqueeze(2)).view(rows, k)


def _run_quantize(s):
    x, dt = s["x"], s["x"].dtype
    if own:
        import dense_gemm_16_amd as mg
        return {"values": mg.dequantize_mx(mg.quantize_mx(x), dt)}
    rows, cols = x.shape
    blocks = (cols + BLOCK - 1) // BLOCK
    v = torch.zeros((rows, blocks * BLOCK), device="cuda")
    v[:, :cols] = x
    v = v.view(rows, blocks, BLOCK)
    largest = v.abs().amax(2)
    # frexp: largest = m 2^p with 0.5 <= m < 1, so floor(log2) = p - 1; 6 = 1.5 * 2^2 is the largest element
    e = torch.where(largest > 0, torch.frexp(largest).exponent - 3, -127).clamp(-127, 127)
    scale = torch.exp2(e.double()).unsqueeze(2)
    a = (v.double() / scale).abs()
    # elements are whole multiples of 0.5 below 2, of 1 below 4 and of 2 above; round() ties to even
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = ((a / step).round() * step).clamp(max=6.0) * torch.sign(v)
    return {"values": (q * scale).view(rows, -1)[:, :cols].to(dt)}


def _run_product(s):
    case = s["case"]
    k, out = case["k"], DTYPES[case["out"]]
    if own:
        import dense_gemm_16_amd as mg
        return mg.gemm_mx(mg.MxMatrix(*s["a"], k), mg.MxMatrix(*s["b"], k), out_dtype=out)
    return (_values(*s["a"], k) @ _values(*s["b"], k).t()).to(out)


def _softmax_gradients(s, p, counted):
    """dx and dw from p, the derivative of each row's loss to its logits."""
    dt = s["x"].dtype
    p = torch.where(counted.unsqueeze(1), p * s["grad"].unsqueeze(1), 0.0)
    return {"dx": (p @ s["w"].float()).to(dt), "dw": (p.t() @ s["x"].float()).to(dt)}


def _run_ce(s):
    x, w, target = s["x"], s["w"], s["target"]
    if own:
        import dense_gemm_16_amd as mg
        loss, lse = mg.linear_cross_entropy(x, w, target, ignore_index=IGNORE)
        if not s["case"]["backward"]:
            return {"loss": loss}
        dx, dw = mg.linear_cross_entropy_backward(x, w, target, lse, s["grad"],
                                                  ignore_index=IGNORE)
        return {"loss": loss, "dx": dx, "dw": dw}
    counted = target != IGNORE
    at = target.clamp(min=0).unsqueeze(1)
    z = x.float() @ w.float().t()
    top = z.amax(1, keepdim=True)
    e = torch.exp(z - top)
    total = e.sum(1, keepdim=True)
    loss = (top + torch.log(total) - z.gather(1, at))[:, 0]
    loss = torch.where(counted, loss, 0.0)
    if not s["case"]["backward"]:
        return {"loss": loss}
    p = e.div_(total)
    p.scatter_add_(1, at, torch.full_like(at, -1.0, dtype=p.dtype))
    return {"loss": loss, **_softmax_gradients(s, p, counted)}


def _run_kd(s):
    case, x, w = s["case"], s["x"], s["w"]
    tau = case["temperature"]
    if own:
        import dense_gemm_16_amd as mg
        loss, lse, student = mg.linear_distillation(x, w, s["logits"], s["index"],
                                                    temperature=tau)
        if not case["backward"]:
            return {"loss": loss}
        dx, dw = mg.linear_distillation_backward(x, w, s["logits"], s["index"], lse, student,
                                                 s["grad"], temperature=tau)
        return {"loss": loss, "dx": dx, "dw": dw}
    held = s["index"] >= 0
    counted = held.any(1)
    at = s["index"].clamp(min=0)
    t = torch.where(held, s["logits"] / tau, -math.inf)
    t = torch.where(counted.unsqueeze(1), t, 0.0)
    t = t - t.amax(1, keepdim=True)
    log_p = t - torch.log(torch.exp(t).sum(1, keepdim=True))
    teacher = torch.where(held, torch.exp(log_p), 0.0)
    z = x.float() @ w.float().t() / tau
    top = z.amax(1, keepdim=True)
    e = torch.exp(z - top)
    total = e.sum(1, keepdim=True)
    log_q = z.gather(1, at) - top - torch.log(total)
    terms = torch.where(teacher > 0, teacher * (log_p - log_q), 0.0)
    loss = torch.where(counted, tau * tau * terms.sum(1), 0.0)
    if not case["backward"]:
        return {"loss": loss}
    q = e.div_(total)
    q.scatter_add_(1, at, -teacher)
    return {"loss": loss, **_softmax_gradients(s, q.mul_(tau), counted)}


_RUN = {"quantize": _run_quantize, "product": _run_product, "ce": _run_ce, "kd": _run_kd}


# ---------------------------------------------------------------- its work

def work(case):
    size = {"f32": 4, "f16": 2, "bf16": 2}
    if case["op"] == "quantize":
        n, blocks = case["rows"] * case["cols"], (case["cols"] + BLOCK - 1) // BLOCK
        # read once, written as values and scales (the values in the source's type)
        return {"bytes": 2 * n * size[case["dtype"]] + case["rows"] * blocks, "flops": 2 * n}
    if case["op"] == "product":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": (m + n) * (k // 2 + k // BLOCK) + m * n * size[case["out"]],
                "flops": 2 * m * n * k}
    t, v, d, b = case["tokens"], case["vocab"], case["dim"], size[case["dtype"]]
    passes = 2 if case["backward"] else 1
    # x and w read, their gradients written; the logits' product, and the two of the gradients
    entries = 12 * t * case["top"] if case["op"] == "kd" else 8 * t
    return {"bytes": passes * (t + v) * d * b + entries + 8 * t,
            "flops": 2 * t * v * d * (3 if case["backward"] else 1)}


# ------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    return _EXACT[case["op"]](case, prepare(case, seed))


def _exact_quantize(case, s):
    x = s["x"].double()
    rows, cols = x.shape
    blocks = (cols + BLOCK - 1) // BLOCK
    x = torch.nn.functional.pad(x, (0, blocks * BLOCK - cols)).view(rows, blocks, BLOCK)
    scale = torch.ones(rows, blocks, device="cuda", dtype=torch.float64)
    byte = torch.zeros(rows, blocks, device="cuda", dtype=torch.int64)
    largest = x.abs().amax(2)
    # the largest byte e with 4 * 2^(e - 127) <= largest, or 0
    for e in range(255):
        fits = largest >= 4.0 * 2.0 ** (e - 127)
        byte = torch.where(fits, e, byte)
    scale = torch.exp2(byte.double() - 127.0).unsqueeze(2)
    a = x.abs() / scale
    # nearest element, midpoints to the one with an even code
    code = torch.zeros_like(a, dtype=torch.int64)
    for i in range(1, 8):
        middle = (FP4[i - 1] + FP4[i]) / 2
        code += (a > middle) | ((a == middle) & (i % 2 == 0))
    value = torch.tensor(FP4, device="cuda", dtype=torch.float64)[code] * torch.sign(x) * scale
    return {"values": value.view(rows, -1)[:, :cols]}


def _exact_product(case, s):
    k = case["k"]

    def matrix(data, scales):
        code = torch.stack((data & 15, data >> 4), 2).view(data.shape[0], k).long()
        element = torch.tensor(FP4, device="cuda", dtype=torch.float64)[code & 7]
        element = torch.where(code >= 8, -element, element)
        power = scales[:, :k // BLOCK].double() - 127.0
        return element * torch.exp2(power).repeat_interleave(BLOCK, 1)

    return matrix(*s["a"]) @ matrix(*s["b"]).t()


def _exact_loss(s, tau, teacher, entropy, at, counted):
    """loss and gradients for soft targets `teacher` at columns `at` (tokens x
    top), their summed p log p in `entropy`; rows that are not counted have none."""
    x, w = s["x"].double(), s["w"].double()
    log_q = torch.log_softmax(x @ w.t() / tau, 1)
    loss = tau * tau * (entropy - (teacher * log_q.gather(1, at)).sum(1))
    loss = loss * counted
    if not s["case"]["backward"]:
        return {"loss": loss}
    p = log_q.exp_().scatter_add_(1, at, -teacher)
    p *= (tau * counted * s["grad"].double()).unsqueeze(1)
    return {"loss": loss, "dx": p @ w, "dw": p.t() @ x}


def _exact_ce(case, s):
    counted = (s["target"] != IGNORE).double()
    at = (s["target"] * counted.long()).unsqueeze(1)
    return _exact_loss(s, 1.0, torch.ones_like(at).double(), 0.0, at, counted)


def _exact_kd(case, s):
    held = (s["index"] >= 0).double()
    counted = (held.sum(1) > 0).double()
    weight = torch.exp(s["logits"].double() / case["temperature"]) * held
    teacher = weight / weight.sum(1, keepdim=True).clamp(min=1e-300)
    entropy = torch.special.xlogy(teacher, teacher).sum(1)
    at = s["index"] * held.long()
    return _exact_loss(s, case["temperature"], teacher, entropy, at, counted)


_EXACT = {"quantize": _exact_quantize, "product": _exact_product, "ce": _exact_ce,
          "kd": _exact_kd}
