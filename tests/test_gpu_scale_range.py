"""MX block scales over the range for which the exact products are promised:
scale bytes 3 .. 246 of E4M3 operands and 0 .. 252 of E2M1 ones, so that an
element times its block's scale is a bf16 value: a multiple of 2^-133 below
2^128.  (E4M3 elements are multiples of 2^-9 up to 448 < 2^9, E2M1 multiples
of 2^-1 up to 6 < 2^3.)  At both ends, against operands whose scales bring the
products back to ordinary sizes."""
import numpy as np
import pytest
import torch

import video_diffusion_transformer_block_amd as V
from oracle import gemm as G, quant as Q
from helpers import assert_elementwise, log, need_gpu, terms_mx
from test_gpu_few_rows import dev, rng_of, values, weights

pytestmark = pytest.mark.gpu
RANGE = {"mxfp8": (3, 246), "mxfp4": (0, 252)}


def codes(rng, rows, K, fmt):
    """Every finite code, the smallest and the largest magnitudes among them."""
    if fmt == "mxfp4":
        return rng.integers(0, 256, size=(rows, K // 2), dtype=np.uint8)
    q = rng.integers(0, 127, size=(rows, K), dtype=np.uint8)
    q[:, ::7] = 126                                        # 448
    q[:, 1::7] = 1                                         # 2^-9
    return q | (rng.integers(0, 2, size=q.shape, dtype=np.uint8) << 7)


@pytest.mark.parametrize("fmt", list(RANGE))
@pytest.mark.parametrize("end", [0, 1])
@pytest.mark.parametrize("T,E", [(1, 1), (4, 1), (9, 2), (16, 1), (32, 3), (90, 2)])
def test_ends_of_the_range(fmt, end, T, E):
    need_gpu()
    log(f"scale range {fmt} end={end} T={T} E={E}")
    rng = rng_of(T, E, end)
    N, K = 70, 384
    aq = codes(rng, T, K, fmt)
    wq = codes(rng, E * N, K, "mxfp4")
    a_end, w_end = RANGE[fmt][end], RANGE["mxfp4"][1 - end]
    # the activations at one end and the weights so far at the other as keeps
    # the products in fp32; every third block the other way round
    as_ = np.full((T, K // 32), a_end, np.uint8)
    ws = np.full((E * N, K // 32), min(254 - a_end, 252), np.uint8)
    ws[:, ::3] = w_end
    as_[:, ::3] = min(max(254 - w_end, RANGE[fmt][0]), RANGE[fmt][1])
    # and blocks whose products fall far below the others'
    as_[:, 1::5] = 127
    ws[:, 1::5] = 100
    off = np.linspace(0, T, E + 1).astype(np.int32)
    a, w = V.MXTensor(dev(aq), dev(as_), fmt), V.MXTensor(dev(wq), dev(ws), "mxfp4")
    want, _ = G.qgemm_mx_grouped(aq, as_, fmt, wq, ws, off)
    terms = np.concatenate([terms_mx(aq[lo:hi], as_[lo:hi], fmt, wq[e * N:(e + 1) * N], ws[e * N:(e + 1) * N], None)
                            for e, (lo, hi) in enumerate(zip(off[:-1], off[1:])) if hi > lo])
    assert np.isfinite(want).all() and np.abs(want).max() < 2.0 ** 40
    y = V.qgemm_mx_grouped(a, w, dev(off), None, "f32")
    torch.cuda.synchronize()
    assert_elementwise(values(y), want, terms, K, "f32", f"grouped {fmt}")
    if E == 1:
        y = V.qgemv_mx(a, w, None, "f32")
        torch.cuda.synchronize()
        assert_elementwise(values(y), want, terms, K, "f32", f"gemv {fmt}")
