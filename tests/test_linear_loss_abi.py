"""The output-layer losses' entry points refuse what their documentation excludes,
before any HIP call, and size their workspace (CPU only)."""
import random

import pytest
import torch

import dense_gemm_16_amd as mg

MB = 1 << 20
# distinct ranges, never dereferenced
X, W, TGT, LOSS, LSE, GRAD, DX, DW, WS, TL, TI, ST = (MB << (4 + i) for i in range(12))
BAD = mg.ERR_INVALID_ARG
T, V, D = 40, 300, 64


def ws_bytes(backward, top=0, **kw):
    a = dict(T=T, V=V, D=D, top=top, dtype=mg.BF16, X=X, ldx=D, W=W, ldw=D) | kw
    return mg.migemm_linear_loss_workspace_size(backward, *a.values())


def ce_forward(**kw):
    a = dict(T=T, V=V, D=D, dtype=mg.BF16, X=X, ldx=D, W=W, ldw=D, target=TGT, ignore=-100,
             loss=LOSS, lse=LSE, ws=WS, bytes=MB) | kw
    return mg.migemm_linear_ce_forward(*a.values())


def ce_backward(**kw):
    a = dict(T=T, V=V, D=D, dtype=mg.BF16, X=X, ldx=D, W=W, ldw=D, target=TGT, ignore=-100,
             lse=LSE, grad=GRAD, dX=DX, lddx=D, dW=DW, lddw=D, ws=WS, bytes=16 * MB) | kw
    return mg.migemm_linear_ce_backward(*a.values())


def kd_forward(**kw):
    a = dict(T=T, V=V, D=D, top=8, dtype=mg.F16, X=X, ldx=D, W=W, ldw=D, t_dtype=mg.F32,
             teacher=TL, ldt=8, index=TI, ldi=8, tau=1.0, loss=LOSS, lse=LSE, student=ST, lds=8,
             ws=WS, bytes=MB) | kw
    return mg.migemm_linear_kd_forward(*a.values())


def kd_backward(**kw):
    a = dict(T=T, V=V, D=D, top=8, dtype=mg.F16, X=X, ldx=D, W=W, ldw=D, t_dtype=mg.F32,
             teacher=TL, ldt=8, index=TI, ldi=8, tau=1.0, lse=LSE, student=ST, lds=8, grad=GRAD,
             dX=DX, lddx=D, dW=DW, lddw=D, ws=WS, bytes=16 * MB) | kw
    return mg.migemm_linear_kd_backward(*a.values())


SHARED = [{"T": -1}, {"T": 1 << 31}, {"V": 0}, {"V": 1 << 31}, {"D": 0}, {"D": 1 << 21},
          {"T": (1 << 23) - 255}, {"V": (1 << 28) + 1}, {"T": 1 << 22, "V": (1 << 16) + 1},
          {"dtype": mg.I8}, {"dtype": 9}, {"ldx": D - 1}, {"ldw": D - 1}, {"ldx": 1 << 32},
          {"X": None}, {"W": None}, {"lse": None}, {"bytes": -1}, {"ws": X}, {"ws": W}]


@pytest.mark.parametrize("call", [ce_forward, ce_backward, kd_forward, kd_backward])
@pytest.mark.parametrize("kw", SHARED)
def test_shared_refusals(call, kw):
    assert call(**kw) == BAD


@pytest.mark.parametrize("kw", [{"target": None}, {"loss": None}, {"loss": LSE}, {"lse": X},
                                {"loss": TGT}, {"loss": WS}, {"loss": LSE + 8 * T - 4}])
def test_ce_forward_refusals(kw):
    assert ce_forward(**kw) == BAD


@pytest.mark.parametrize("kw", [{"target": None}, {"grad": None}, {"lddx": D - 1},
                                {"lddw": D - 1}, {"dX": X}, {"dW": W}, {"dX": DW}, {"dX": WS},
                                {"dW": GRAD}, {"lddw": 1 << 32}])
def test_ce_backward_refusals(kw):
    assert ce_backward(**kw) == BAD


KD = [{"top": 0}, {"top": 1025, "ldt": 1025, "ldi": 1025, "lds": 1025}, {"top": -1},
      {"t_dtype": mg.I32}, {"teacher": None}, {"index": None}, {"ldt": 7}, {"ldi": 7},
      {"tau": 0.0}, {"tau": -1.0}, {"tau": 1e-19}, {"tau": 2e18}, {"tau": float("inf")}, {"tau": float("nan")},
      {"student": None}, {"lds": 7}]


@pytest.mark.parametrize("kw", KD + [{"student": LOSS}, {"loss": TI}])
def test_kd_forward_refusals(kw):
    assert kd_forward(**kw) == BAD


@pytest.mark.parametrize("kw", KD + [{"dX": ST}, {"dW": TL}])
def test_kd_backward_refusals(kw):
    assert kd_backward(**kw) == BAD


@pytest.mark.parametrize("call", [ce_forward, ce_backward, kd_forward, kd_backward])
@pytest.mark.parametrize("kw", [{"ws": None}, {"ws": WS + 64}, {"bytes": 1024}, {"bytes": 0}])
def test_workspace_refusals(call, kw):
    assert call(**kw) == mg.ERR_WORKSPACE


def test_no_rows_is_a_no_op():
    assert ce_forward(T=0, X=None, target=None, loss=None, lse=None, ws=None, bytes=0) == mg.OK
    assert ce_backward(T=0, X=None, dW=None, ws=None, bytes=0) == mg.OK
    assert kd_forward(T=0, X=None, ws=None, bytes=0) == mg.OK


def test_workspace_size():
    st, forward = ws_bytes(0)
    assert st == mg.OK and forward > 0
    st, backward = ws_bytes(1)
    # the tokens' copy, the row data and the derivative at least
    assert st == mg.OK and backward >= 64 * 64 * 2 + 256 * 16 + 64 * 320 * 2
    assert ws_bytes(1, top=8)[1] >= backward + T * 8 * 4
    # a misaligned weight is copied: V rounded up to 64 rows more
    assert ws_bytes(0, W=W + 2)[1] >= forward + 320 * 64 * 2
    assert ws_bytes(1, ldw=D + 1)[1] >= backward + 320 * 64 * 2
    assert ws_bytes(0, T=0) == (mg.OK, 0)
    # FP32 at 2^36 logits and one past it
    assert ws_bytes(0, dtype=mg.F32, T=1 << 22, V=1 << 14)[0] == mg.OK
    assert ws_bytes(0, dtype=mg.F32, T=1 << 22, V=(1 << 14) + 1)[0] == BAD
    for kw in ({"T": -1}, {"V": 0}, {"D": 0}, {"dtype": mg.I32}, {"ldx": 1}, {"top": 1025},
               {"top": -1}):
        assert ws_bytes(0, **kw)[0] == BAD
    # the derivative is held in pieces of 2^28 entries at most, whatever V is
    small = ws_bytes(1, T=8192, V=65536, D=1024, ldx=1024, ldw=1024)[1]
    large = ws_bytes(1, T=8192, V=1 << 20, D=1024, ldx=1024, ldw=1024)[1]
    assert large == small < 1 << 30


def test_wrappers_check_their_tensors():
    x, w, t = torch.zeros(4, 8), torch.zeros(5, 8), torch.zeros(4, dtype=torch.long)
    with pytest.raises(ValueError, match="must be on the GPU"):
        mg.linear_cross_entropy(x, w, t)
    with pytest.raises(ValueError, match="must be on the GPU"):
        mg.linear_cross_entropy_backward(x, w, t, torch.zeros(4), 1.0)
    with pytest.raises(ValueError, match="must be on the GPU"):
        mg.linear_distillation(x, w, torch.zeros(4, 2), torch.zeros(4, 2, dtype=torch.long))


def _forward_tile(T, V):
    """(rows, columns) of the FP32 forward product's tiles: its workspace holds 8 bytes
    for each of a row's chunks, 16 columns wide on 64x64 tiles (four to a tile), 32 on
    128x128."""
    st, n = ws_bytes(0, dtype=mg.F32, T=T, V=V, D=64, ldx=64, ldw=64)
    assert st == mg.OK
    for tile, chunk in ((64, 16), (128, 32)):
        if n == -(-8 * T * -(-V // tile) * (tile // chunk) // 256) * 256:
            return tile
    raise AssertionError(f"workspace of {n} bytes matches no tile")


def test_large_fp32_losses_fit_a_launch():
    """A launch holds fewer than 2^32 threads, 512 to a tile: every size up to the
    documented 2^36 logits, ragged ones too, takes tiles that are few enough."""
    rng = random.Random(1)
    sizes = [(600000, 64000), (1000000, 65000), (300000, 128256), (524289, 128256),
             (65, 1 << 28), ((1 << 23) - 256, 8191), (129, (1 << 28) - 1), (8391, 8191777)]
    for _ in range(2000):
        V = int(2 ** rng.uniform(13, 28))
        sizes.append((min((1 << 23) - 256, int(2 ** rng.uniform(34.9, 36)) // V), V))
    for T, V in sizes:
        if T * V > 1 << 36:
            continue
        b = _forward_tile(T, V)
        assert -(-T // b) * -(-V // b) * 512 < 1 << 32, (T, V, b)
    # below it the tile is still chosen by rounds
    assert _forward_tile(723, 5489) == 64 and _forward_tile(1024, 65536) == 128
