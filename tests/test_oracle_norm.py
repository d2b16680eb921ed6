"""CPU pins of oracle/norm.py: closed forms, a float64 definition, and the
marking of rows that are not finite."""
import numpy as np
import pytest

from oracle import formats as F, gemm as G, norm as NM, quant as Q

RNG = np.random.Generator(np.random.PCG64(5))


def bits(a):
    return F.f32_to_bf16(np.asarray(a, np.float32))


def test_constant_row_norms_to_ones():
    """r = c everywhere: y = c / sqrt(c^2 + eps), and the transform of a
    constant block b is sqrt(b) in its first place, zero elsewhere."""
    x = bits(np.full((1, 128), 4.0))
    o = NM.rmsnorm_quantize(x, None, None, 1e-6, 64, "int8")
    want = np.zeros((1, 128))
    want[0, [0, 64]] = 8.0
    assert np.allclose(o["y"], want, atol=1e-6)
    assert o["q"][0, 0] == 127 and np.count_nonzero(o["q"]) == 2


def test_zero_row():
    o = NM.rmsnorm_quantize(bits(np.zeros((2, 64))), None, None, 1e-6, 64, "int8")
    assert (o["scales"] == 0).all() and (o["q"] == 0).all()


def test_residual_rounds_once():
    x, r = bits([[256.0] * 16]), bits([[1.0] * 16])        # 257 needs 9 bits: ties to even at 256
    assert np.array_equal(NM.residual_sum(x, r), x)


@pytest.mark.parametrize("fmt", ["int8", "bf16", "mxfp4", "mxfp8"])
def test_against_the_float64_definition(fmt):
    """The fp32 steps stay within K-independent rounding of the definition:
    two products (2^-24 each), inv (2^-24) and log2(b) + 1 butterfly and
    scaling roundings, each at most 2^-24 of the block's absolute sum."""
    x, r = bits(RNG.laplace(size=(4, 256))), bits(RNG.laplace(size=(4, 256)))
    w = (1 + 0.1 * RNG.standard_normal(256)).astype(np.float32)
    o = NM.rmsnorm_quantize(x, r, w, 1e-6, 64, fmt)
    s = F.bf16_to_f32(o["r"]).astype(np.float64)
    n = s / np.sqrt((s * s).mean(1, keepdims=True) + float(np.float32(1e-6))) * w
    i = np.arange(64)
    H = (-1.0) ** np.array([[bin(a & b).count("1") for b in i] for a in i])
    y = (n.reshape(4, 4, 64) @ H / 8).reshape(4, 256)
    tol = 10 * 2.0 ** -24 * np.abs(n).reshape(4, 4, 64).sum(-1) / 8
    assert (np.abs(o["y"] - y).reshape(4, 4, 64) <= tol[..., None]).all()
    if fmt == "int8":
        got = Q.int8_dequantize(o["q"], o["scales"])
        assert (np.abs(got - o["y"]) <= o["scales"][:, None] * 0.5001).all()


def test_rows_that_are_not_finite_are_marked():
    x = bits(RNG.laplace(size=(3, 64)))
    x[1, 5] = 0x7F80
    big = bits(np.full((3, 64), 3e38))
    for fmt in ("int8", "bf16", "mxfp4", "mxfp8"):
        o = NM.rmsnorm_quantize(x, None, None, 1e-6, 64, fmt)
        assert list(o["finite"]) == [True, False, True]
    assert not NM.rmsnorm_quantize(big, big, None, 1e-6, 64, "int8")["finite"].any()   # the sum overflows


def test_grouped_oracle_is_the_plain_product_per_group():
    a = RNG.standard_normal((7, 128)).astype(np.float32)
    w = RNG.standard_normal((3 * 5, 128)).astype(np.float32)
    aq, as_ = Q.mx_quantize(a, "e4m3")
    wq, ws = Q.mx_quantize(w, "e2m1")
    off = [1, 1, 4, 6]
    y, cov = G.qgemm_mx_grouped(aq, as_, "mxfp8", wq, ws, off)
    A, W = Q.mx_dequantize(aq, as_, "e4m3"), Q.mx_dequantize(wq, ws, "e2m1").reshape(3, 5, 128)
    assert list(cov) == [False, True, True, True, True, True, False]
    assert np.allclose(y[1:4], A[1:4] @ W[1].T) and np.allclose(y[4:6], A[4:6] @ W[2].T)
