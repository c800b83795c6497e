"""The entry points of layer norm, embeddings and AdamW refuse what their documentation
excludes, before any HIP call, and size their workspaces (CPU only)."""
import ctypes

import pytest
import torch

import dense_gemm_16_amd as mg

MB = 1 << 20
# distinct ranges, never dereferenced
X, Y, DY, DX, W, B, MEAN, RSTD, DW, DB, WS, INDEX = (MB << (4 + i) for i in range(12))
BAD = mg.ERR_INVALID_ARG
INF, NAN = float("inf"), float("nan")
T, V, D = 40, 300, 64


# ----------------------------------------------------------------- layer norm

def norm(**kw):
    a = dict(T=T, D=D, dtype=mg.BF16, X=X, ldx=D, w_dtype=mg.BF16, W=W, B=B, eps=1e-5, Y=Y, ldy=D,
             mean=MEAN, rstd=RSTD) | kw
    return mg.migemm_layer_norm_forward(*a.values())


def norm_backward(**kw):
    a = dict(T=100 * T, D=D, dtype=mg.BF16, dY=DY, lddy=D, X=X, ldx=D, w_dtype=mg.BF16, W=W, mean=MEAN,
             rstd=RSTD, dX=DX, lddx=D, dW=DW, dB=DB, ws=WS, bytes=16 * MB) | kw
    return mg.migemm_layer_norm_backward(*a.values())


@pytest.mark.parametrize("kw", [
    {"T": -1}, {"T": 1 << 31}, {"D": 0}, {"D": -1}, {"D": (1 << 24) + 1, "ldx": 1 << 25, "ldy": 1 << 25},
    {"dtype": mg.I8}, {"dtype": 9}, {"w_dtype": mg.F16}, {"w_dtype": mg.I8},
    {"dtype": mg.F32, "w_dtype": mg.BF16}, {"ldx": D - 1}, {"ldy": D - 1}, {"ldx": 1 << 32},
    {"ldy": 1 << 32}, {"X": None}, {"Y": None}, {"eps": -1e-6}, {"eps": INF}, {"eps": NAN},
    {"Y": X}, {"Y": W}, {"mean": X}, {"mean": RSTD}, {"rstd": Y + 4}, {"B": Y + 2}, {"mean": W + 2}])
def test_layer_norm_refusals(kw):
    assert norm(**kw) == BAD


@pytest.mark.parametrize("kw", [
    {"T": -1}, {"T": 1 << 31}, {"D": 0}, {"D": (1 << 24) + 1, "ldx": 1 << 25, "lddy": 1 << 25, "lddx": 1 << 25},
    {"dtype": mg.I32}, {"w_dtype": mg.F16}, {"ldx": D - 1}, {"lddy": D - 1}, {"lddx": D - 1},
    {"lddx": 1 << 32}, {"dY": None}, {"X": None}, {"mean": None}, {"rstd": None}, {"dX": X},
    {"dX": DY}, {"dW": W}, {"dW": DB}, {"dB": MEAN}, {"dX": WS}, {"ws": X}, {"ws": DW},
    {"bytes": -1}])
def test_layer_norm_backward_refusals(kw):
    assert norm_backward(**kw) == BAD


@pytest.mark.parametrize("kw", [{"ws": None}, {"ws": WS + 64}, {"bytes": 64}, {"bytes": 0}])
def test_layer_norm_workspace_refusals(kw):
    assert norm_backward(**kw) == mg.ERR_WORKSPACE
    assert norm_backward(dB=None, **kw) == mg.ERR_WORKSPACE
    assert norm_backward(dW=None, dX=None, **kw) == mg.ERR_WORKSPACE


def test_layer_norm_workspace_size():
    size = mg.migemm_layer_norm_workspace_size
    st, n = size(100 * T, D, 1)
    assert st == mg.OK and n >= 2 * D * 4
    assert size(100 * T, D, 0) == (mg.OK, 0) and size(0, D, 1) == (mg.OK, 0)
    # few rows take one launch and none
    assert size(T, D, 1) == (mg.OK, 0) and size(T, D, 0) == (mg.OK, 0)
    # rows too long for registers keep two sums each
    assert size(T, 20000, 0)[1] >= 8 * T
    # partial sums stay within half a thousand rows, however many tokens there are
    assert size(1 << 30, 4096, 1)[1] <= 512 * 2 * 4096 * 4
    for args in ((-1, D, 1), (1 << 31, D, 1), (T, 0, 1), (T, (1 << 24) + 1, 1)):
        assert size(*args)[0] == BAD
    assert mg.lib().migemm_layer_norm_workspace_size(T, D, 1, None) == BAD


def test_layer_norm_no_ops():
    assert norm(T=0, X=None, Y=None, W=None, B=None, mean=None, rstd=None) == mg.OK
    assert norm_backward(T=0, dY=None, X=None, W=None, mean=None, rstd=None, dX=None, dW=None,
                         dB=None, ws=None, bytes=0) == mg.OK
    assert norm_backward(dX=None, dW=None, dB=None, ws=None, bytes=0) == mg.OK


# ----------------------------------------------------------------- embeddings

def embed(**kw):
    a = dict(T=T, V=V, D=D, dtype=mg.F16, W=W, ldw=D, index=INDEX, ignore=-100, scale=2.0, Y=Y,
             ldy=D) | kw
    return mg.migemm_embedding_forward(*a.values())


def embed_backward(**kw):
    a = dict(T=100 * T, V=V, D=D, dtype=mg.F16, dY=DY, lddy=D, index=INDEX, ignore=-100, scale=2.0,
             accumulate=0, dw_dtype=mg.F16, dW=DW, lddw=D, ws=WS, bytes=16 * MB) | kw
    return mg.migemm_embedding_backward(*a.values())


SHARED = [{"T": -1}, {"T": 1 << 31}, {"V": 0}, {"V": (1 << 28) + 1}, {"D": 0}, {"dtype": mg.I8},
          {"dtype": 9}, {"index": None}]


@pytest.mark.parametrize("kw", SHARED + [
    {"D": (1 << 21) + 1, "ldw": 1 << 22, "ldy": 1 << 22}, {"ldw": D - 1}, {"ldy": D - 1},
    {"ldw": 1 << 32}, {"W": None}, {"Y": None}, {"Y": W}, {"Y": INDEX}, {"Y": W + 2 * V * D - 2}])
def test_embedding_refusals(kw):
    assert embed(**kw) == BAD


@pytest.mark.parametrize("kw", SHARED + [
    {"D": (1 << 21) + 1, "lddw": 1 << 22, "lddy": 1 << 22}, {"lddy": D - 1}, {"lddw": D - 1},
    {"lddw": 1 << 32}, {"dY": None}, {"dW": None}, {"dW": DY}, {"dW": INDEX}, {"ws": DY},
    {"ws": DW}, {"dW": WS}, {"accumulate": 2}, {"accumulate": -1}, {"dw_dtype": mg.BF16},
    {"dw_dtype": mg.I32}, {"dtype": mg.F32}, {"bytes": -1}])
def test_embedding_backward_refusals(kw):
    assert embed_backward(**kw) == BAD


@pytest.mark.parametrize("kw", [{"ws": None}, {"ws": WS + 64}, {"bytes": 256}, {"bytes": 0}])
def test_embedding_workspace_refusals(kw):
    assert embed_backward(**kw) == mg.ERR_WORKSPACE


def test_embedding_workspace_size():
    size = mg.migemm_embedding_workspace_size
    st, n = size(100 * T, V, D)
    assert st == mg.OK and n >= 8 * 100 * T
    # few tokens take one launch and none
    assert size(0, V, D) == (mg.OK, 0) and size(T, V, D) == (mg.OK, 0)
    # sorted entries and tokens; the rows that stretches share are few for many tokens
    st, n = size(1 << 22, 131072, 1024)
    assert st == mg.OK and 16 << 22 <= n <= (16 << 22) + 4096 * 2 * 1024 * 4 + (8 << 20)
    for args in ((-1, V, D), (1 << 31, V, D), (T, 0, D), (T, V, 0), (T, (1 << 28) + 1, D)):
        assert size(*args)[0] == BAD
    assert mg.lib().migemm_embedding_workspace_size(T, V, D, None) == BAD


def test_embedding_no_ops():
    assert embed(T=0, index=None, Y=None) == mg.OK
    assert embed_backward(T=0, dY=None, index=None, accumulate=1, ws=None, bytes=0) == mg.OK


# --------------------------------------------------------------------- adamw

P, G, M, S, MS, SS, MASTER, LR, STEP, GS = (MB << (4 + i) for i in range(10))


def tensor(count=1000, **kw):
    a = dict(count=count, param=P, grad=G, master=None, avg=M, sq=S, avg_scales=None,
             sq_scales=None) | kw
    return mg.AdamwTensor(*a.values())


def options(**kw):
    a = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, step=1, lr_device=None,
             step_device=None, grad_scale=None) | kw
    return mg.AdamwOptions(*a.values())


def adamw(*tensors, param=mg.F32, grad=mg.F32, bits=32, o=None, count=None, **kw):
    array = (mg.AdamwTensor * max(1, len(tensors)))(*tensors)
    return mg.migemm_adamw(len(tensors) if count is None else count, array, param, grad, bits,
                           o or options(**kw))


EIGHT = dict(avg_scales=MS, sq_scales=SS)


@pytest.mark.parametrize("kw", [
    {"lr": INF}, {"lr": NAN}, {"beta1": 1.0}, {"beta1": -0.1}, {"beta2": 1.0}, {"beta2": NAN},
    {"eps": -1e-9}, {"eps": INF}, {"weight_decay": INF}, {"step": 0}, {"step": -3},
    {"param": mg.I8}, {"grad": mg.BF16}, {"param": mg.F16, "grad": mg.BF16}, {"bits": 16},
    {"bits": 4}, {"count": -1}, {"count": (1 << 24) + 1}, {"lr_device": LR + 2},
    {"step_device": STEP + 4}, {"grad_scale": GS + 1}, {"lr_device": P + 8}, {"grad_scale": S},
    {"step_device": M + 3992}])
def test_adamw_refusals(kw):
    assert adamw(tensor(), **kw) == BAD


@pytest.mark.parametrize("kw", [
    {"count": -1}, {"count": 1 << 40}, {"param": None}, {"grad": None}, {"avg": None},
    {"sq": None}, {"avg_scales": MS}, {"sq_scales": SS}, {"master": MASTER}, {"param": P + 2},
    {"grad": G + 1}, {"avg": M + 2}, {"param": G}, {"avg": S}, {"avg": P + 3996}, {"grad": S + 4}])
def test_adamw_tensor_refusals(kw):
    assert adamw(tensor(**kw)) == BAD


@pytest.mark.parametrize("kw", [
    {"avg_scales": None}, {"sq_scales": None}, {"avg_scales": MS + 2}, {"avg_scales": SS},
    {"avg_scales": M + 996}, {"master": P}, {"master": MASTER + 2}, {"param": P + 1}])
def test_adamw_8_bit_tensor_refusals(kw):
    assert adamw(tensor(**({**EIGHT, "master": MASTER} | kw)), param=mg.BF16, bits=8) == BAD


def test_adamw_lists():
    # a tensor named twice, one whose state is another's parameter, a master copy in one only
    two = dict(param=P + MB, grad=G + MB, avg=M + MB, sq=S + MB)
    for n in (2, 100):  # the ranges on the stack, and not
        far = [tensor(param=P + i * 8192, grad=G + i * 8192, avg=M + i * 8192, sq=S + i * 8192)
               for i in range(n - 1)]
        assert adamw(*far, tensor()) == BAD
        assert adamw(*far, tensor(**two | {"avg": P})) == BAD
        assert adamw(*far, tensor(**two | {"grad": M + 400})) == BAD
        assert adamw(*far, tensor(**two, master=MASTER), param=mg.F16) == BAD
    # two gradients may be one
    assert adamw(tensor(count=0), tensor(count=0)) == mg.OK
    assert adamw() == mg.OK
    assert adamw(tensor(count=0, param=None, grad=None, avg=None, sq=None)) == mg.OK
    assert mg.migemm_adamw(1, None, 0, 0, 32, options()) == BAD
    assert mg.migemm_adamw(0, None, 0, 0, 32, None) == BAD


def test_adamw_structures_match_the_header():
    assert ctypes.sizeof(mg.AdamwTensor) == 64 and ctypes.sizeof(mg.AdamwOptions) == 72


# ------------------------------------------------------------------ wrappers

def test_wrappers_check_their_tensors():
    x, w, t = torch.zeros(4, 8), torch.zeros(5, 8), torch.zeros(4, dtype=torch.long)
    v = torch.zeros(4)
    for call in (lambda: mg.layer_norm(x), lambda: mg.layer_norm_backward(x, x, None, v, v),
                 lambda: mg.embedding(w, t), lambda: mg.embedding_backward(x, t, 5),
                 lambda: mg.adamw_([x], [x], [mg.adamw_state(x)], step=1)):
        with pytest.raises(ValueError, match="must be on the GPU"):
            call()
    with pytest.raises(ValueError, match="1 parameters, 0 gradients"):
        mg.adamw_([x], [], [mg.adamw_state(x)], step=1)
    mg.adamw_([], [], [], step=1)


def test_adamw_states():
    p = torch.randn(3, 300, dtype=torch.bfloat16)
    s = mg.adamw_state(p, bits=8, master=True)
    assert s.avg.dtype == s.sq.dtype == torch.float8_e4m3fn and s.avg.shape == p.shape
    assert s.avg_scales.shape == s.sq_scales.shape == (4,) and torch.equal(s.master, p.float())
    assert not s.avg.float().any() and not s.sq.float().any() and not s.avg_scales.any()
    s = mg.adamw_state(p)
    assert s.avg.dtype == torch.float32 and s.avg_scales is None and s.master is None
    with pytest.raises(ValueError, match="bits must be 32 or 8"):
        mg.adamw_state(p, bits=16)
    with pytest.raises(ValueError, match="needs no master"):
        mg.adamw_state(p.float(), master=True)


def test_states_do_not_follow_the_default_dtype():
    p = torch.zeros(300, dtype=torch.bfloat16)
    kept = torch.get_default_dtype()
    try:
        for default in (torch.float64, torch.bfloat16):
            torch.set_default_dtype(default)
            wide, eight = mg.adamw_state(p), mg.adamw_state(p, bits=8)
            assert all(t.dtype == torch.float32
                       for t in (wide.avg, wide.sq, eight.avg_scales, eight.sq_scales))
    finally:
        torch.set_default_dtype(kept)


def test_operands_that_are_no_tensors():
    x, v, t = torch.zeros(4, 8), torch.zeros(4), torch.zeros(4, dtype=torch.long)
    rows = [[0.0] * 8] * 4
    for call in (lambda: mg.layer_norm(rows), lambda: mg.layer_norm_backward(x, rows, None, v, v),
                 lambda: mg.embedding(rows, t), lambda: mg.embedding_backward(rows, t, 5),
                 lambda: mg.adamw_([rows], [x], [mg.adamw_state(x)], step=1)):
        with pytest.raises(ValueError, match="must be a tensor"):
            call()


@pytest.mark.parametrize("off", [1, 2, 3])
def test_row_statistics_and_tokens_off_their_elements(off):
    """Workgroups read them by scalar loads, which drop an address's lowest bits."""
    assert norm_backward(mean=MEAN + off) == BAD and norm_backward(rstd=RSTD + off) == BAD
    assert norm_backward(T=T, mean=MEAN + off) == BAD
    assert embed_backward(index=INDEX + off) == BAD and embed_backward(T=T, index=INDEX + 4) == BAD
