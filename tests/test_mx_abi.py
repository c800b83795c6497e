"""The MXFP4 entry points refuse what their documentation excludes, before any
HIP call (CPU only)."""
import numpy as np
import pytest
import torch

import dense_gemm_16_amd as mg
import mx_oracle as mx

P, Q, R = 1 << 20, 1 << 24, 1 << 28   # never dereferenced
BAD = mg.ERR_INVALID_ARG


def quantize(**kw):
    a = dict(src_dtype=mg.BF16, op=mg.OP_N, rows=4, cols=100, src=P, lds=100, data=Q, ldd=64,
             scales=R, ldsc=16) | kw
    return mg.migemm_quantize_mx(*a.values())


@pytest.mark.parametrize("kw", [
    {"src_dtype": mg.I8}, {"src_dtype": 9}, {"op": 2}, {"rows": -1}, {"cols": -1},
    {"rows": 1 << 31}, {"lds": 99}, {"lds": 1 << 32}, {"op": mg.OP_T, "lds": 3}, {"src": None},
    {"data": None}, {"scales": None}, {"data": Q + 8}, {"scales": R + 4}, {"ldd": 48},
    {"ldd": 72}, {"ldsc": 8}, {"ldsc": 20}, {"cols": 520, "lds": 520, "ldd": 272, "ldsc": 16},
    {"data": P}, {"scales": Q}, {"scales": P + 16}, {"ldd": 1 << 32}])
def test_quantize_refusals(kw):
    assert quantize(**kw) == BAD


@pytest.mark.parametrize("kw", [{"rows": 0, "src": None, "data": None, "scales": None},
                                {"cols": 0, "lds": 1, "src": None, "data": None, "scales": None}])
def test_quantize_of_nothing(kw):
    assert quantize(**kw) == mg.OK


def dequantize(**kw):
    a = dict(dst_dtype=mg.F32, rows=4, cols=100, data=Q, ldd=64, scales=R, ldsc=16, dst=P,
             ld=100) | kw
    return mg.migemm_dequantize_mx(*a.values())


@pytest.mark.parametrize("kw", [
    {"dst_dtype": mg.I32}, {"rows": -1}, {"ld": 99}, {"dst": None}, {"data": None},
    {"data": Q + 1}, {"ldd": 60}, {"ldsc": 4}, {"dst": Q}, {"dst": R}])
def test_dequantize_refusals(kw):
    assert dequantize(**kw) == BAD


def gemm(**kw):
    a = dict(config=-1, M=8, N=24, K=96, A=P, lda=48, sa=P + (1 << 16), ldas=16, B=Q, ldb=48,
             sb=Q + (1 << 16), ldbs=16, alpha=1.0, beta=0.0, c_dtype=mg.F32, C=R, ldc=24) | kw
    return mg.migemm_gemm_mx(*a.values())


@pytest.mark.parametrize("kw", [
    {"M": -1}, {"N": 1 << 31}, {"K": 95}, {"K": 100}, {"K": 16}, {"K": -32}, {"lda": 47},
    {"lda": 40}, {"ldb": 32}, {"ldas": 8}, {"ldbs": 24 + 1}, {"A": P + 8}, {"B": None},
    {"sa": None}, {"sb": Q + 5}, {"c_dtype": mg.I32}, {"c_dtype": mg.I8}, {"C": None},
    {"config": -2}, {"config": 6}, {"ldc": 23}, {"C": P}, {"C": Q + (1 << 16)}, {"ldc": 1 << 32}])
def test_gemm_refusals(kw):
    assert gemm(**kw) == BAD


@pytest.mark.parametrize("kw", [{"M": 0, "A": None}, {"N": 0, "ldc": 1, "B": None, "C": None}])
def test_gemm_of_nothing(kw):
    assert gemm(**kw) == mg.OK


def test_wrappers_want_gpu_tensors():
    x = torch.zeros(4, 32)
    m = mg.MxMatrix(torch.zeros(4, 16, dtype=torch.uint8), torch.zeros(4, 16, dtype=torch.uint8), 32)
    for call in (lambda: mg.quantize_mx(x), lambda: mg.dequantize_mx(m, torch.float32),
                 lambda: mg.gemm_mx(m, m)):
        with pytest.raises(ValueError, match="must be on the GPU"):
            call()
    assert m.shape == (4, 32)


def test_oracle_rule_on_hand_worked_blocks():
    x = np.zeros((1, 64))
    x[0, :8] = [4.0, -7.9, 0.25, 0.75, 2.5, 5.0, -0.0, 1.0]   # m = 7.9: e = 0
    x[0, 32:35] = [96.0, 15.0, -10.0]                          # m = 96: e = 4, unit 16
    codes, byte = mx.quantize(x)
    assert byte.tolist() == [[127, 131]]
    assert codes[0, :8].tolist() == [6, 15, 0, 2, 4, 6, 8, 2]
    assert codes[0, 32:35].tolist() == [7, 2, 9]
    back = mx.decode(mx.pack(codes), byte, 64)
    assert back[0, :8].tolist() == [4.0, -6.0, 0.0, 1.0, 2.0, 4.0, 0.0, 1.0]
    assert back[0, 32:35].tolist() == [96.0, 16.0, -8.0]


def test_configurations_have_names():
    n = mg.migemm_mx_config_count()
    names = [mg.migemm_mx_config_name(c) for c in range(n)]
    assert n == 6 and all(names) and len(set(names)) == n
    assert mg.migemm_mx_config_name(n) is None and mg.migemm_mx_config_name(-1) is None
