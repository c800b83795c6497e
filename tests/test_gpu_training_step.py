"""A whole training step of a tied model out of the library's calls: embedding, layer norm,
the output layer's cross entropy, their backward passes (the embedding's gradient added to
the output layer's, both being the table's), and the AdamW step; against the same step in
float64.

The gradients' tolerances are relative to each gradient's root mean square over rows: the
intermediates are rounded to the dtype (u = 2^-24 FP32; 2^-8 BF16) at five places, each
of which moves what follows by about u of its size, and FP32 sums of V and D terms add
(V + D) 2^-24 at most.  64 (u + (V + D) 2^-24) covers them with the condition of the norm
(rows of width D with standard deviation near the scale) and of the softmax (logits of a
few units) taken as 8 in all.
"""
import math

import pytest
import torch

import dense_gemm_16_amd as mg
from gpu_helpers import say

pytestmark = pytest.mark.gpu

IGNORE = -100


def forward_backward(w, gamma, beta, index, target, scale):
    x = mg.embedding(w, index, scale=scale, ignore_index=IGNORE)
    y, mean, rstd = mg.layer_norm(x, gamma, beta)
    loss, lse = mg.linear_cross_entropy(y, w, target, ignore_index=IGNORE)
    count = max(1, int((target != IGNORE).sum()))
    dy, dw = mg.linear_cross_entropy_backward(y, w, target, lse, 1.0 / count, ignore_index=IGNORE)
    dx, dgamma, dbeta = mg.layer_norm_backward(dy, x, gamma, mean, rstd)
    mg.embedding_backward(dx, index, w.shape[0], scale=scale, ignore_index=IGNORE, dw=dw,
                          accumulate=True)
    return loss, dw, dgamma, dbeta


def reference(w, gamma, beta, index, target, scale):
    w, gamma, beta = (t.double().cpu().requires_grad_() for t in (w, gamma, beta))
    index, target = index.cpu(), target.cpu()
    held = index != IGNORE
    x = torch.where(held[:, None], w[index.clamp(min=0)] * scale, 0.0)
    d = x - x.mean(1, keepdim=True)
    y = d / ((d * d).mean(1, keepdim=True) + 1e-5).sqrt() * gamma + beta
    loss = torch.nn.functional.cross_entropy(y @ w.t(), target, ignore_index=IGNORE,
                                             reduction="none")
    (loss.sum() / max(1, int((target != IGNORE).sum()))).backward()
    return loss.detach(), w.grad, gamma.grad, beta.grad


@pytest.mark.parametrize("T,V,D", [(1, 50, 64), (77, 300, 128), (300, 1000, 264)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_step_of_a_tied_model(T, V, D, dtype):
    g = torch.Generator(device="cuda").manual_seed(T)
    w = (torch.randn(V, D, generator=g, device="cuda") / math.sqrt(D)).to(dtype)
    gamma = (1 + 0.1 * torch.randn(D, generator=g, device="cuda")).to(dtype)
    beta = (0.1 * torch.randn(D, generator=g, device="cuda")).to(dtype)
    index = torch.randint(0, V, (T,), generator=g, device="cuda")
    target = index.roll(-1)
    if T > 2:  # a padded end
        index[-2:] = IGNORE
        target[-3:] = IGNORE
    scale = math.sqrt(D)
    say(f"training step {T} of {V}x{D} {dtype}")
    got = forward_backward(w, gamma, beta, index, target, scale)
    torch.cuda.synchronize()
    want = reference(w, gamma, beta, index, target, scale)
    u = torch.finfo(dtype).eps / 2
    tol = 64 * (u + (V + D) * 2.0 ** -24)
    for a, b in zip(got, want):
        a, b = a.double().cpu(), b
        assert torch.isfinite(a).all()
        rms = b.square().mean().sqrt()
        assert (a - b).square().mean().sqrt() <= tol * (rms + (a.dim() == 1) * 1e-3)
    # the step: states of 8 bits for the table, 32 for the vectors
    params, grads = [w, gamma, beta], list(got[1:])
    before = [p.clone() for p in params]
    table, vectors = mg.adamw_state(w, bits=8), [mg.adamw_state(p) for p in params[1:]]
    mg.adamw_(params[:1], grads[:1], [table], step=1, lr=1e-2, weight_decay=0.0)
    mg.adamw_(params[1:], grads[1:], vectors, step=1, lr=1e-2, weight_decay=0.0)
    torch.cuda.synchronize()
    for p, q, d in zip(params, before, grads):
        # the first step moves every element by lr against its gradient's sign
        move = -1e-2 * d.double() / (d.double().abs() + 1e-8)
        new = q.double() + move
        assert ((p.double() - new).abs() <= 16 * 2.0 ** -24 * 1e-2 + (u + 2.0 ** -22) * new.abs()).all()


def test_captured_step_beside_an_eager_one():
    """The whole step captured into a graph, its number counted on the device, replayed
    against the same steps run one by one from the same start."""
    T, V, D, dtype = 120, 500, 128, torch.bfloat16

    def start():
        g = torch.Generator(device="cuda").manual_seed(1)
        w = (torch.randn(V, D, generator=g, device="cuda") / math.sqrt(D)).to(dtype)
        gamma = torch.ones(D, dtype=dtype, device="cuda")
        beta = torch.zeros(D, dtype=dtype, device="cuda")
        index = torch.randint(0, V, (T,), generator=g, device="cuda")
        params = [w, gamma, beta]
        return params, [mg.adamw_state(p, bits=8, master=True) for p in params], index

    def one(params, states, index, step):
        w, gamma, beta = params
        x = mg.embedding(w, index, scale=8.0)
        y, mean, rstd = mg.layer_norm(x, gamma, beta)
        loss, lse = mg.linear_cross_entropy(y, w, index)
        dy, dw = mg.linear_cross_entropy_backward(y, w, index, lse, 1.0 / T)
        dx, dgamma, dbeta = mg.layer_norm_backward(dy, x, gamma, mean, rstd)
        mg.embedding_backward(dx, index, V, scale=8.0, dw=dw, accumulate=True)
        mg.adamw_(params, [dw, dgamma, dbeta], states, step=step, lr=1e-2)
        return loss

    eager, captured = start(), start()
    count = torch.ones((), dtype=torch.int64, device="cuda")
    say("training step captured")
    one(*start(), torch.ones((), dtype=torch.int64, device="cuda"))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss = one(*captured, count)
        count.add_(1)
    for i in range(3):
        want = one(*eager, torch.tensor(i + 1, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(loss, want)
        for a, b in zip(eager[0], captured[0]):
            assert torch.equal(a, b)


def test_refusals_on_another_stream():
    """What is not on the GPU is refused as on the current stream."""
    x = torch.ones(6, 16, device="cuda")
    w, index = torch.ones(16, device="cuda"), torch.zeros(6, dtype=torch.int64, device="cuda")
    y, mean, rstd = mg.layer_norm(x, w)
    state = mg.adamw_state(x)
    side = torch.cuda.Stream()
    s = side.cuda_stream
    say("refusals on another stream")
    for call in (lambda: mg.layer_norm(x, w.cpu(), stream=s),
                 lambda: mg.layer_norm_backward(y.cpu(), x, w, mean, rstd, stream=s),
                 lambda: mg.layer_norm_backward(y, x, w, mean, rstd.cpu(), stream=s),
                 lambda: mg.embedding(x, index.cpu(), stream=s),
                 lambda: mg.embedding_backward(y, index.cpu(), 6, stream=s),
                 lambda: mg.adamw_([x], [y.cpu()], [state], step=1, stream=s),
                 lambda: mg.adamw_([x], [y], [state._replace(sq=state.sq.cpu())], step=1, stream=s),
                 lambda: mg.adamw_([x], [None], [state], step=1, stream=s)):
        with pytest.raises(ValueError):
            call()
    torch.cuda.synchronize()


@pytest.mark.parametrize("T,V,D", [(77, 300, 128), (300, 1000, 264), (500, 400, 96)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_step_of_a_tied_model_within_its_roundings(T, V, D, dtype):
    """Targets drawn apart from the tokens, so that the sums over tokens do not cancel (where
    a target is the next token, dbeta's own terms and targets' do).  Seven roundings, of x,
    y, the losses' derivative, dy, dx and twice the gradient, move each element of theirs by
    u at most, so the root mean square of what follows by u of its own: the norm's derivative
    is a projection, and a token's own logit of about sqrt(D) (10 and more here, log V is
    below 7) leaves its softmax's p (1 - p) below 0.1 for most.  8 u covers the seven added
    up, the FP32 sums as above."""
    g = torch.Generator(device="cuda").manual_seed(T + V)
    w = (torch.randn(V, D, generator=g, device="cuda") / math.sqrt(D)).to(dtype)
    gamma = (1 + 0.1 * torch.randn(D, generator=g, device="cuda")).to(dtype)
    beta = (0.1 * torch.randn(D, generator=g, device="cuda")).to(dtype)
    index, target = torch.randint(0, V, (2, T), generator=g, device="cuda")
    index[-2:] = IGNORE
    target[-3:] = IGNORE
    scale = math.sqrt(D)
    say(f"training step {T} of {V}x{D} {dtype}, targets apart")
    got = forward_backward(w, gamma, beta, index, target, scale)
    torch.cuda.synchronize()
    tol = 8 * (torch.finfo(dtype).eps / 2 + (V + D) * 2.0 ** -24)
    for a, b in zip(got, reference(w, gamma, beta, index, target, scale)):
        error = (a.double().cpu() - b).square().mean().sqrt()
        assert float(error) <= tol * float(b.square().mean().sqrt())
